// attention_line.cuh -- what the tree attentions over the 8-bit and the 4-bit
// cache share: how their work is cut into pieces and joined again, the rows'
// preparation (queries in two e4m3 terms, tree masks), and the wrappers of the
// tensor cores, TMEM and barriers that both kernels use.
//
// The key tiles of all (sequence, KV head, row tile), and kEnd more for each
// one's end, are one line of units, cut into equal pieces, one per CTA (one CTA
// per SM), whatever the lengths are; a piece that covers part of an item leaves
// (O, m, l) in the workspace and k_attn_merge joins them.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "device_info.h"
#include "e4m3.cuh"
#include "tcgen05.cuh"

namespace ssd {
namespace line {

constexpr int kPage = 16;
constexpr int kMaxNodes = 128;
constexpr int kSub = 128;                  // keys of a sub-tile (MMA M of S^T, K of O^T)
constexpr int kPages = kSub / kPage;       // 8
// P v_scale goes to halves: at most 2^11 where m was taken (the first tile), and
// m moves before it exceeds 2^15 (halves end just below 2^16), to where it is
// 2^12: the first tile's largest of 128 keys is a low guess of the largest of
// thousands, and moving m costs about a tile's time.  l sums P / 2^7: with
// v_scale down to 2^-100, P itself reaches 2^115, and thousands of those pass fp32.
constexpr float kBias = 11.f, kMoved = 12.f, kGrow = 15.f, kSumUnit = 0x1p-7f, kSumBias = kBias - 7.f;
// Keys of the smallest piece, and the longest table whose items are not cut: joining costs 2 to 3 us.  One query, 8
// heads of 128: 2000 keys 12.3 us in pieces of 512, 15.0 of 1024, 17.0 whole; 1000 keys 12.4 either way; 40 sequences
// of 900 keys, 2 KV heads, 14.2 whole, 16.7 cut; 4 of 700 keys 11.0 and 12.3.
constexpr int kMinKeys = 512, kWholeKeys = 1024;
// An item's end costs its CTA a few tiles' time: O leaves TMEM, the next rows come in, the pipeline drains.  3, 4, 6,
// 8: ragged batch of 1 to 16384 keys 98, 95, 96, 100 us; 256 sequences of up to 600 keys 76, 75, 76, 79; 64 of 100 to
// 600 (draft) 73, 76, 77, 80; equal lengths within 1%.
constexpr int kEnd = 4;

// D[tmem] (+)= A B of one step of 16 halves of K; A in TMEM (lane = row, two of K per column), B as above
SSD_DEV void umma_f16(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t bhi, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(bhi), "r"(idesc), "r"(accum)
      : "memory");
}
// Shared-memory matrix descriptor, 128-byte or (D = 64 rows) 64-byte swizzle.
// Low word: address / 16, and the bytes / 16 between column blocks of an
// MN-major operand; high word: bytes / 16 between groups of 8 rows, version, swizzle.
SSD_DEV constexpr uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) {
  return (sbo >> 4) | (1u << 14) | (swizzle << 29);
}
constexpr uint32_t kSw128 = 2, kSw64 = 4;
// Instruction descriptors, fp32 sums, M = 128: e4m3 A and B, both K-major; fp16 A K-major, B MN-major
__host__ __device__ constexpr uint32_t idesc_f8(int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16(int N) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
// byte offset of (row r, byte c) in a block of 128-byte rows, 128-byte swizzled
SSD_DEV uint32_t sw128(int r, int c) {
  return (r >> 3) * 1024 + (r & 7) * 128 + ((((c >> 4) ^ (r & 7)) << 4) | (c & 15));
}
SSD_DEV uint32_t sw64(int r, int c) {  // 64-byte rows
  const uint32_t o = r * 64 + c;
  return o ^ (((o >> 7) & 3) << 4);
}
SSD_DEV void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// One lane of the warp.  What it issues takes its operands from uniform
// registers; under `if (lane == 0)` each operand is moved there first, and an
// MMA cost about 100 clocks of the issuing warp.
SSD_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Bounded wait of a whole warp for one phase.  All lanes wait: the warp is then
// suspended until the phase completes (one poll, about 95 clocks from arrival
// to wake-up); a wait by one lane in divergent code polls every 150 clocks,
// wakes in 220 and, with a CTA of such warps, keeps the barrier unit busy.
// Gives up after 2^20 polls of at most a few microseconds each; a role whose
// wait gives up leaves, and with it, one bounded wait later, all others.
SSD_DEV bool warp_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 1048576;\n"
      "POLL:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra.uni DONE;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra.uni POLL;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return __any_sync(0xffffffffu, ok != 0);
}
// 16 columns of this thread's lane, waited for by tmem_wait16
SSD_DEV void tmem_ld16_async(uint32_t taddr, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
SSD_DEV void tmem_wait16(float *v) {  // orders the uses of v after the wait
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
SSD_DEV void tmem_ld4(uint32_t at, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
      : "r"(at)
      : "memory");
}
// 16 columns of this thread's lane; the stores are waited for by tmem_wait_st
SSD_DEV void tmem_st16_async(uint32_t at, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 16 TMEM lanes x 16 columns: of columns 8 w .. + 7, lane l holds columns 2 (l % 4) and the next of TMEM lane l / 4
// (v[4 w], v[4 w + 1]) and of TMEM lane 8 + l / 4 (v[4 w + 2], v[4 w + 3])
SSD_DEV void tmem_st_16x16(uint32_t at, const uint32_t *v) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
SSD_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Two 16 x 16 byte blocks, transposed: lane l gives the address of row l % 16 of block l / 16 and gets bytes
// 4 (l % 4) .. + 3 of columns l / 4 (c[2 b]) and 8 + l / 4 (c[2 b + 1]) of block b: four rows' bytes of one column
SSD_DEV void load_columns(uint32_t saddr, uint32_t *c) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
               : "r"(saddr)
               : "memory");
}
SSD_DEV void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
SSD_DEV bool bar_or(int id, int n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
SSD_DEV uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

SSD_DEV uint16_t e4m3_of_half2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
SSD_DEV uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// One value per 16 columns and lane -> the columns' sums over the warp's lanes:
// five exchanges that halve the columns held (a fixed order).  Column
// (lane >> 1) & 15 ends in both lanes of a pair.
SSD_DEV float warp_columns(float *v, int lane) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int o = 16 >> s, n = 8 >> s;
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float keep = up ? v[k + n] : v[k], send = up ? v[k] : v[k + n];
      v[k] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}
SSD_DEV float warp_top(float v) {  // maximum over the warp, NaN left out
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// What the kernels of both caches are given.
struct Line {
  const uint16_t *q;
  const int32_t *table;
  int maxb;
  int64_t num_blocks;
  const int32_t *prefix_len, *parent;
  int B, N, Nq, Hq, Hkv, group, nrows, mtiles, per_b;  // per_b: items of a sequence
  uint32_t group_magic;                                // row / group = row * magic >> 16 (row < 4096)
  int split;                                           // pieces may cut items
  int keys;                                            // keys of a tile
  float scale_log2;
  uint16_t *out;
  float *lse;
  float *part_o;   // [CTA][2][rows][d]: a piece's first item (begun elsewhere), then its last (ended elsewhere)
  float2 *part_ml;  // [CTA][2][rows] (m, l)
  int4 *info;      // [CTA] what its last item still needs: {parts, sequence, KV head, row tile}
  uint32_t *status;
};

SSD_DEV int keys_of(const Line &a, int b, int &L) {
  const int prefix = a.prefix_len[b];
  L = max(prefix, 0);
  if (prefix == -1) return 0;  // a slot without a request
  const int64_t n = min(static_cast<int64_t>(L) + a.N, static_cast<int64_t>(a.maxb) * kPage);
  return static_cast<int>(min(n, static_cast<int64_t>(0x7fffffff - 2 * kSub)));
}
SSD_DEV int tiles_of(const Line &a, int nkeys) { return max(1, (nkeys + a.keys - 1) / a.keys); }
SSD_DEV int units_of(const Line &a, int b) {  // of an item
  int L;
  return tiles_of(a, keys_of(a, b, L)) + kEnd;
}

SSD_DEV long long quotient(long long x, int y) {  // x >= 0, y > 0; a 64-bit division takes ten times a 32-bit one's time
  return x >> 32 ? x / y : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}

// A CTA's piece of the line of units.
struct Piece {
  int b, item, t0;  // sequence, item of it and the first unit's number in it
  int left;         // units of the piece
  int chunk;        // units of a full piece
  int tiles;        // tiles that the CTA runs
};

// The segments of a piece: one item (or part of it) after the other.  An item
// has kEnd units behind its tiles, for the time that its end takes (O leaves
// TMEM, the next rows come in), or a CTA of many short items would be the last.
struct Segments {
  int b, hk, mt, nt, nkeys, L, t0, t1, left;
  SSD_DEV void sequence(const Line &a) {
    nkeys = keys_of(a, b, L);
    nt = tiles_of(a, nkeys);
  }
  SSD_DEV bool first(const Line &a, const Piece &p) {
    if (p.left <= 0) return false;
    b = p.b;
    hk = p.item / a.mtiles;
    mt = p.item - hk * a.mtiles;
    t0 = p.t0;
    left = p.left;
    sequence(a);
    if (t0 >= nt || (!a.split && t0 > 0)) {  // the item's end, or begun in the piece before, which takes it whole
      left -= nt + kEnd - t0;
      return step(a);
    }
    return take(a);
  }
  SSD_DEV bool take(const Line &a) {
    t1 = (a.split && left < nt - t0) ? t0 + left : nt;
    left -= t1 < nt ? t1 - t0 : nt + kEnd - t0;
    return true;
  }
  SSD_DEV bool step(const Line &a) {
    if (left <= 0) return false;
    t0 = 0;
    if (++mt == a.mtiles) {
      mt = 0;
      if (++hk == a.Hkv) {
        hk = 0;
        if (++b == a.B) return false;
        sequence(a);
      }
    }
    return take(a);
  }
};

// The line of units: every thread sums some sequences' units, then the sums are scanned; the thread that finds the CTA's
// first unit writes the piece (preset to no tiles).  Ends with the piece not yet visible to the other threads.
template <int THREADS, int KEYS>
SSD_DEV void find_piece(const Line &a, long long *scan, Piece *out) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int per = (a.B + THREADS - 1) / THREADS, b0 = tid * per, b1 = min(a.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += units_of(a, b);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  long long upto = lane < (THREADS / 32) ? scan[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const long long total = __shfl_sync(0xffffffffu, upto, 31);
  const long long before = __shfl_sync(0xffffffffu, upto, max(warp - 1, 0)) * (warp > 0);
  const long long T = total * a.per_b;
  long long chunk = quotient(T + gridDim.x - 1, gridDim.x);
  if (a.split) chunk = max(chunk, static_cast<long long>(kMinKeys / KEYS));
  const long long lo = chunk * blockIdx.x, hi = min(T, lo + chunk);
  long long x = (before + inc - mine) * a.per_b;  // units before this thread's first sequence
  if (lo < hi && lo >= x && lo < x + mine * a.per_b) {
    int b = b0;
    for (;; ++b) {
      const long long n = static_cast<long long>(units_of(a, b)) * a.per_b;
      if (lo < x + n) break;
      x += n;
    }
    Piece p;
    p.b = b;
    const int n = units_of(a, b);
    p.item = static_cast<int>(quotient(lo - x, n));
    p.t0 = static_cast<int>((lo - x) - static_cast<long long>(p.item) * n);
    p.left = static_cast<int>(hi - lo);
    p.chunk = static_cast<int>(chunk);
    p.tiles = 0;
    Segments sg;
    for (bool more = sg.first(a, p); more; more = sg.step(a)) p.tiles += sg.t1 - sg.t0;
    *out = p;
  }
}

// The order of the MMAs, which is the order of the loads: S runs ahead of P V by
// up to NB tiles, but not into the next segment, whose rows may not be ready: its
// first S comes behind the last P V, while the softmax warps write O out.
struct Order {
  int begin, end;  // of the segment that P V is in
  Segments sg;
  bool more;
  SSD_DEV void start(const Line &a, const Piece &p) {
    begin = 0;
    more = sg.first(a, p);
    end = more ? sg.t1 - sg.t0 : 0;
  }
  SSD_DEV void done(const Line &a, int j) {  // P V has done j tiles
    if (j < end) return;
    begin = end;
    more = more && sg.step(a);
    if (more) end += sg.t1 - sg.t0;
  }
};

// A segment's rows: q1, q2 into the operand tiles at qb, the row scales, and
// each query's tree mask, by warp w of the n that share it (barrier `bar`).
// Four lanes share a row, each with its quarter in registers (the next row's
// is fetched meanwhile).
template <class C, int D, int RT>
__device__ __noinline__ void prepare_rows(const Line &a, const Segments sg, uint8_t *qb, int *par,
                                          uint32_t (*anc)[kMaxNodes / 32], float *qs, int w, int n, int bar) {
  const int lane = threadIdx.x & 31;
  constexpr int V = D / 32;  // 16-byte pieces of a quarter row
  const int sub = lane & 3;
  auto fetch = [&](int r, uint4 (&x)[V]) {
    const int row = sg.mt * RT + r;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = make_uint4(0, 0, 0, 0);
    if (r < RT && row < a.nrows) {
      const int qi = static_cast<int>((row * a.group_magic) >> 16), head = sg.hk * a.group + (row - qi * a.group);
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + ((static_cast<int64_t>(sg.b) * a.Nq + qi) * a.Hq + head) * D + sub * (D / 4));
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = __ldg(src + v);
    }
  };
  uint4 x[V], next[V];
  fetch(w * 8 + (lane >> 2), x);
  const bool tree = sg.nkeys > 0 && static_cast<int64_t>(sg.t1) * C::kKeys > sg.L;
  if (tree)
    for (int m = w * 32 + lane; m < a.N; m += n * 32) par[m] = a.parent[static_cast<int64_t>(sg.b) * a.N + m];
  if (w == 0 && lane == 0) {
    const int L = a.prefix_len[sg.b];
    if (L < -1 || (L >= 0 && static_cast<int64_t>(L) + a.N > static_cast<int64_t>(a.maxb) * kPage))
      atomicOr(a.status, kFlagBadPrefix);
  }
  bar_sync(bar, n * 32);
  if (tree) {
    for (int i = w * 32 + lane; i < a.Nq; i += n * 32) {
      uint32_t *const bits = anc[i];
#pragma unroll
      for (int k = 0; k < kMaxNodes / 32; ++k) bits[k] = 0;
      for (int m = a.N - a.Nq + i; m >= 0;) {
        bits[m >> 5] |= 1u << (m & 31);
        const int up = par[m];
        if (up < -1 || up >= m) {
          atomicOr(a.status, kFlagBadTree);
          break;
        }
        m = up;
      }
    }
  }
#pragma unroll 1
  for (int r0 = w * 8; r0 < RT; r0 += n * 8) {
    const int r = r0 + (lane >> 2);
    fetch(r + n * 8, next);
    auto each = [&](auto &&f) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f(v * 2, 0, x[v].x);
        f(v * 2, 16, x[v].y);
        f(v * 2 + 1, 0, x[v].z);
        f(v * 2 + 1, 16, x[v].w);
      }
    };
    uint32_t m2 = 0;  // the row's largest magnitude: bf16 magnitudes order like integers
    each([&](int, int, uint32_t b) { m2 = max_u16x2(m2, b & 0x7FFF7FFFu); });
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    if (__any_sync(0xffffffffu, m >= 0x7F80u)) {  // infinities (which e4m3 would clamp) and NaN: NaN, and not the largest
      m = 0;
#pragma unroll 1
      for (int v = 0; v < V; ++v) {
        uint4 w = x[0];
#pragma unroll
        for (int k = 1; k < V; ++k) w = v == k ? x[k] : w;
        auto clean = [&](uint32_t b) {
          uint32_t lo = b & 0xFFFFu, hi = b >> 16;
          if ((lo & 0x7FFFu) < 0x7F80u) m = max(m, lo & 0x7FFFu);
          else lo = 0x7FC0u;
          if ((hi & 0x7FFFu) < 0x7F80u) m = max(m, hi & 0x7FFFu);
          else hi = 0x7FC0u;
          return lo | hi << 16;
        };
        w = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = v == k ? w : x[k];
      }
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // 2^e brings the largest element into [2^7, 2^8); e in [-120, 120] (smaller rows: fewer bits)
    const int e2 = m == 0 ? 0 : min(max(static_cast<int>(m >> 7) - 127 - 7, -120), 120);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
    uint32_t c1[V * 2], c2[V * 2];
#pragma unroll
    for (int k = 0; k < V * 2; ++k) c1[k] = c2[k] = 0;
    // in halves: a value has 8 bits and both terms lie above their last place, 2^-24 (what is smaller e4m3 cuts)
    each([&](int word, int shift, uint32_t b) {
      const uint32_t h = half2_of(__uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv);
      const uint32_t t1 = e4m3_of_half2(h);
      const uint32_t t2 = e4m3_of_half2(hfma2(e4m3_to_half2(static_cast<uint16_t>(t1)), 0xBC00BC00u, h));
      c1[word] |= t1 << shift;
      c2[word] |= t2 << shift;
    });
    if (r < RT) {
#pragma unroll
      for (int v = 0; v < V; v += 2) {  // 16 codes
        const int at = sub * (D / 4) + v * 8;
        *reinterpret_cast<uint4 *>(qb + sw128(r, at)) = make_uint4(c1[v * 2], c1[v * 2 + 1], c1[v * 2 + 2], c1[v * 2 + 3]);
        *reinterpret_cast<uint4 *>(qb + (D == 128 ? C::kQTile + sw128(r, at) : sw128(r, 64 + at))) =
            make_uint4(c2[v * 2], c2[v * 2 + 1], c2[v * 2 + 2], c2[v * 2 + 3]);
      }
      if (sub == 0) qs[r] = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = next[v];
  }
  fence_proxy_async();  // the operand tiles -> visible to the tensor cores
  __syncwarp();
}

// Joins the parts of the items that were cut: block (x, y) the item that CTA x
// began and did not end, eight of its rows, a warp per row.
template <int D, int RT>
__global__ void __launch_bounds__(256) k_attn_merge(const __grid_constant__ Line a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are done
  const int4 need = a.info[blockIdx.x];
  const int lane = threadIdx.x & 31, j = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int hk = need.z, mt = need.w, row = mt * RT + j;
  if (need.x == 0 || j >= RT || row >= a.nrows) return;
  const float NEG_INF = -__int_as_float(0x7f800000);
  // part 0 is the second slot of CTA x, the others the first slots of the CTAs behind it
  auto slot = [&](int p) { return static_cast<int64_t>(blockIdx.x + p) * 2 + (p == 0 ? 1 : 0); };
  float M = NEG_INF;
  for (int p = lane; p < need.x; p += 32) M = fmaxf(M, a.part_ml[slot(p) * RT + j].x);
  M = warp_max(M);
  constexpr int E = D / 32;
  float acc[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int p = 0; p < need.x; ++p) {
    const float2 ml = a.part_ml[slot(p) * RT + j];
    if (ml.y == 0.f) continue;  // no key there
    const float f = ex2(ml.x - M);
    l = fmaf(ml.y, f, l);
    const float *src = a.part_o + (slot(p) * RT + j) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(src[e], f, acc[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int qi = static_cast<int>((row * a.group_magic) >> 16), head = hk * a.group + (row - qi * a.group);
  const int64_t orow = (static_cast<int64_t>(need.y) * a.Nq + qi) * a.Hq + head;
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + orow * D) + lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    uint32_t b2;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b2) : "f"(acc[e + 1] * inv), "f"(acc[e] * inv));
    dst[e / 2] = b2;
  }
  if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? NEG_INF : (M - kSumBias + log2f(l)) * 0.69314718055994531f;
}

}  // namespace line
}  // namespace ssd

namespace {

// Rows of a tile: up to 64, the tiles of equal size, a multiple of the MMA's step of 16; above, 128 (the MMA's M, a
// lane per row).  With a lane per row 64 rows take 142 us instead of 94 (ragged batch), 48 rows 336 instead of 198
// (verify): half of the lanes have none.
struct Shape {
  int nrows, mtiles, RT;
};
Shape shape_of(int Nq, int Hq, int Hkv) {
  Shape s;
  s.nrows = (Hq / Hkv) * Nq;
  s.mtiles = (s.nrows + 127) / 128;
  const int tile = (s.nrows + s.mtiles - 1) / s.mtiles;
  s.RT = tile <= 64 ? (tile + 15) / 16 * 16 : 128;
  return s;
}
size_t align256(size_t x) { return (x + 255) / 256 * 256; }
struct Workspace {
  size_t o, ml, info, total;
};
Workspace workspace_of(const Shape &s, int d, int ctas) {
  Workspace w;
  const size_t rows = static_cast<size_t>(ctas) * 2 * s.RT;
  w.o = 0;
  w.ml = align256(rows * d * sizeof(float));
  w.info = w.ml + align256(rows * sizeof(float2));
  w.total = w.info + align256(static_cast<size_t>(ctas) * sizeof(int4));
  return w;
}


// The fields that the caches share, from arguments that have been checked; false: a piece would leave 32 bits.
// Items of tables up to kWholeKeys are not cut; without room for the parts none is.
bool make_line(ssd::line::Line &a, const Shape &sh, const void *q, const int32_t *block_table, int maxb,
               int64_t num_blocks, const int32_t *prefix_len, const int32_t *parent, int B, int N, int Nq, int Hq,
               int Hkv, int d, float scale, void *out, float *lse, uint32_t *status, void *ws, size_t ws_bytes,
               unsigned &grid) {
  using namespace ssd::line;
  a.q = static_cast<const uint16_t *>(q);
  a.table = block_table;
  a.maxb = maxb;
  a.num_blocks = num_blocks;
  a.prefix_len = prefix_len;
  a.parent = parent;
  a.B = B;
  a.N = N;
  a.Nq = Nq;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.nrows = sh.nrows;
  a.mtiles = sh.mtiles;
  a.per_b = Hkv * sh.mtiles;
  a.group_magic = (65536u + a.group - 1) / a.group;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.status = status;
  // one CTA per SM, none without a tile of its own
  const int sms = attn_num_sms();
  a.keys = sh.RT <= 64 ? 2 * kSub : kSub;
  const int64_t max_keys = static_cast<int64_t>(maxb) * kPage;
  const int64_t max_tiles = (max_keys + a.keys - 1) / a.keys;
  const int64_t units = max_tiles * B * a.per_b;
  grid = static_cast<unsigned>(units < sms ? units : sms);
  if ((max_tiles + kEnd) * B * a.per_b / grid > 0x3fffffff) return false;  // a piece counts in 32 bits
  const Workspace w = workspace_of(sh, d, sms);
  a.split = max_keys > kWholeKeys && ws && ws_bytes >= w.total && !(reinterpret_cast<uintptr_t>(ws) & 255u);
  if (a.split) {
    char *const p = static_cast<char *>(ws);
    a.part_o = reinterpret_cast<float *>(p + w.o);
    a.part_ml = reinterpret_cast<float2 *>(p + w.ml);
    a.info = reinterpret_cast<int4 *>(p + w.info);
  }
  return true;
}

// Joins the pieces behind the attention kernel: launched with it, started when its grid ends.
template <int D, int RT>
cudaError_t launch_merge(const ssd::line::Line &a, unsigned grid, cudaStream_t cs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (min(RT, a.nrows) + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = cs;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ssd::line::k_attn_merge<D, RT>, a);
}

}  // namespace
