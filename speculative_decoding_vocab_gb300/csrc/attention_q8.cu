// attention_q8.cu -- tree-masked decode attention over a paged K/V cache held
// in 8 bits (e4m3 codes, one scale per block of 16 positions and KV head), on
// the sm_103a tensor cores.
//
// A decode step has few query rows and many keys, so up to 64 rows per KV head
// the keys take the MMA's 128-wide side and the rows its N:
//     S^T [128 keys x rows] = K8 Q^T,      O^T [d x rows] += V^T P^T;
// above, the rows fill that side themselves:
//     S [128 rows x 128 keys] = Q K8^T,    O [128 rows x d] += P V.
// S: the keys' codes go to the tensor cores as they are (kind::f8f6f4, fp32
// sums), and what 8 bits would lose of the bf16 queries is kept in a second term:
//   q = 2^e (q1 + q2): e4m3 holds 4 significant bits, so q1 = e4m3(q) leaves a
//     remainder of at most 4 bits, and q2 = e4m3(q - q1) is exact (bf16 has 8;
//     below 2^-17 of the row's largest element the remainder is cut): two MMAs
//     into the same S.
// P V: in halves (kind::f16, fp32 sums).  A half holds every code of V exactly,
// and a probability to 11 bits, off by at most 2^-11 of itself, or by 2^-25 where it
// is subnormal, 2^-36 of the row's largest or less: a key that takes most of a row (an
// attention sink) does not cost the row the thousands of others.  Two e4m3 terms
// did: they end 2^-19 below the largest, and with 0.99 of a row on one of 8192
// keys, its value 0, the output was off by 0.7 of itself (halves: 0.002).
// The product takes its A from TMEM, so that is where V^T (or P) goes in halves:
// byte columns of a V sub-tile by ldmatrix, two codes per conversion, stored in the
// lanes' fragment order.  With a lane per row P is there and V, as the B, in
// shared memory.
// Block scales enter in fp32: x = s * k_scale * scale * 2^e, P = 2^(x - m + 11),
// and P * v_scale is what is rounded (a lane has one key of 16 rows, or one row of
// 32 keys).  m starts as the largest x + log2(v_scale) of the row's first keys
// and moves (O and l are rescaled) when some P * v_scale exceeds 2^15, so the
// row's largest lies in [2^11, 2^15] and halves end 2^36 to 2^40 below it.  l sums
// the fp32 P.
//
// Work split: the key tiles of all (sequence, KV head, row tile), and kEnd more
// for each one's end, are one line of units, cut into equal pieces, one per CTA
// (one CTA per SM), whatever the lengths are; a piece that covers part of an
// item leaves (O, m, l) in the workspace and k_attn_q8_merge joins them.
//
// CTA: softmax warps (groups of four: 16 rows of the tile each, or with a lane
// per row a quarter of its keys), four helper warps that turn V into halves and
// prepare the next segment's rows (q1, q2, tree masks), one or two producer warps
// and an MMA warp.  A tile is 256 keys up to 64 rows and 128 above (S twice, P or
// V in halves twice and O fill TMEM's 512 columns): what a warp does once per tile costs
// it as much as the arithmetic, so tiles are as large as fits.  K and V sub-tiles come
// in the order in which they are used (S runs up to NB tiles ahead of P V),
// through one ring, so that every slot that is not being read is a copy in flight; V's
// slot goes back when its codes have been read.
//
// Bound: HBM where the rows are few; else the softmax warps' latencies (4 per
// scheduler, half of the issue slots used).  All roles' loops run at once, and what they
// take together does not fit the SM's instruction cache: smaller code is
// faster code here (loops that are not the softmax warps' are rolled).
// 64 sequences of 8192 keys, 8 KV heads of 128 with 6 queries of 8 heads each
// (1.08 GB): 191 us, 5.7 TB/s.  Ragged batch of 48 sequences up to 16384 keys, 64 rows
// (411 MB): 95 us, 4.3 TB/s.  One sequence, 100003 keys, one query (205 MB): 44 us,
// of which the set-up, the first tile and the merge take 12.  16 sequences of
// 2048 keys with 256 rows (d 64): 60 us (66 with P in two e4m3 terms, which
// two conversions and three packed operations a pair took).
//   tried for V in halves: by the softmax warps (verify 227, ragged 114), P V issued by a
//   warp of its own (verify 205, ragged 109), V's buffers by sub-tiles in a ring of
//   three at 64 rows (ragged 98 instead of 97).
//   tried: softmax warps in streams of whole tiles (instruction fetch), four
//   producer warps (verify 214), setmaxnreg (spills), m moved in every tile (each
//   pays a tile's time), next rows prepared by the softmax warps behind short items
//   (no gain), S of the next item before the last P V (verify 198 replayed instead of
//   195), three S and P buffers for the draft (67 instead of 66).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <cmath>

#include "../../include/ssd.h"
#include "common.cuh"
#include "device_info.h"
#include "e4m3.cuh"
#include "tcgen05.cuh"

namespace ssd {
namespace q8 {

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
constexpr int kSmemBudget = 212 * 1024;
constexpr int kBatch = 32 / kPages;        // tiles that a producer warp's lanes hold the blocks of
constexpr int kIds = 4 * kBatch;           // tiles whose block ids are held in shared memory (K runs ahead of V)

// D[tmem] (+)= A B of one 32-byte step of K; A and B by the low words of their
// shared-memory descriptors (the high words are constants)
SSD_DEV void umma_f8(uint32_t d_tmem, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                     uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}\n" ::"r"(d_tmem),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accum)
      : "memory");
}
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
// four codes -> four halves (exact)
SSD_DEV void halves_of(uint32_t codes, uint32_t &h0, uint32_t &h1) {
  h0 = e4m3_to_half2(static_cast<uint16_t>(codes & 0xFFFFu));
  h1 = e4m3_to_half2(static_cast<uint16_t>(codes >> 16));
}
// four codes with NaN ones made 0; `any` collects whether there were some
SSD_DEV uint32_t without_nan(uint32_t codes, uint32_t among, uint32_t &any) {
  const uint32_t nan = ((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u & among;  // bytes 0x7F, 0xFF
  any |= nan;
  return codes & ~((nan >> 7) * 0xFFu);
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

struct Args {
  const uint16_t *q;
  const uint8_t *vc;
  const float *ks, *vs;
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

SSD_DEV int keys_of(const Args &a, int b, int &L) {
  const int prefix = a.prefix_len[b];
  L = max(prefix, 0);
  if (prefix == -1) return 0;  // a slot without a request
  const int64_t n = min(static_cast<int64_t>(L) + a.N, static_cast<int64_t>(a.maxb) * kPage);
  return static_cast<int>(min(n, static_cast<int64_t>(0x7fffffff - 2 * kSub)));
}
SSD_DEV int tiles_of(const Args &a, int nkeys) { return max(1, (nkeys + a.keys - 1) / a.keys); }
SSD_DEV int units_of(const Args &a, int b) {  // of an item
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
  SSD_DEV void sequence(const Args &a) {
    nkeys = keys_of(a, b, L);
    nt = tiles_of(a, nkeys);
  }
  SSD_DEV bool first(const Args &a, const Piece &p) {
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
  SSD_DEV bool take(const Args &a) {
    t1 = (a.split && left < nt - t0) ? t0 + left : nt;
    left -= t1 < nt ? t1 - t0 : nt + kEnd - t0;
    return true;
  }
  SSD_DEV bool step(const Args &a) {
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

// The order of the MMAs, which is the order of the loads: S runs ahead of P V by
// up to NB tiles, but not into the next segment, whose rows may not be ready: its
// first S comes behind the last P V, while the softmax warps write O out.
struct Order {
  int begin, end;  // of the segment that P V is in
  Segments sg;
  bool more;
  SSD_DEV void start(const Args &a, const Piece &p) {
    begin = 0;
    more = sg.first(a, p);
    end = more ? sg.t1 - sg.t0 : 0;
  }
  SSD_DEV void done(const Args &a, int j) {  // P V has done j tiles
    if (j < end) return;
    begin = end;
    more = more && sg.step(a);
    if (more) end += sg.t1 - sg.t0;
  }
};

template <int D, int RT>
struct Cfg {
  static constexpr bool kRowLanes = RT > 64;               // rows, not keys, on the MMA's 128-wide side
  static constexpr int KT = RT <= 64 ? 2 : 1;              // sub-tiles of a tile
  static constexpr int kKeys = KT * kSub;                  // keys of a tile
  static constexpr int kTmaWarps = KT;                     // producer warps: one for every sub-tile of a tile
  static constexpr int CG = kRowLanes ? 32 : 16;           // rows of a softmax warp (keys, with a lane per row)
  static constexpr int kGroups = RT / CG;                  // groups of four warps
  static constexpr int NB = 2;                             // S and P buffers; S runs NB tiles ahead
  static constexpr int kSoftWarps = 4 * kGroups;
  // helper warps: warp w of the four writes TMEM lanes 32 w .. + 31 (those that a warp of its number modulo 4 reaches)
  static constexpr int kHelpWarp = kSoftWarps, kTmaWarp = kHelpWarp + 4, kMmaWarp = kTmaWarp + kTmaWarps;
  static constexpr int kWarps = kMmaWarp + 1;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kQTile = RT * 128;                  // q1 (or q2) at D = 128; [q1 | q2] at D = 64
  static constexpr int kQBuf = D == 128 ? 2 * kQTile : kQTile;
  // P V's operand in shared memory, halves: P^T of a sub-tile in rows of 128 bytes, a key each; with a lane per row V
  // in blocks of 64 elements, rows of 128 bytes, a key each
  static constexpr int kBlock = kSub * 128;
  static constexpr int kHBuf = kRowLanes ? (D / 64) * kBlock : KT * kBlock;  // of a tile
  static constexpr int kSlot = kSub * D;                   // K or V of a sub-tile
  static constexpr int kFixed = 2 * kQBuf + NB * kHBuf;
  static constexpr int kFit = (kSmemBudget - kFixed) / kSlot;
  static constexpr int kSlots = kFit > 16 ? 16 : kFit;
  static constexpr int kQ = 0, kH = 2 * kQBuf, kRing = kFixed;
  static constexpr int kSmem = kFixed + kSlots * kSlot + 1024;
  // TMEM: NB x KT x S, O, and at its end P V's other operand in halves: V^T (as many buffers as fit), or P
  static constexpr int kOCol = NB * KT * RT, kOCols = kRowLanes ? D : RT;
  static constexpr int kACols = KT * (kSub / 2);           // of a tile
  static constexpr int kABufs = kOCol + kOCols + NB * kACols <= 512 ? NB : 1;
  static constexpr int kACol = 512 - kABufs * kACols;
  static constexpr int kMeta = 24 / KT;                    // tiles whose block scales are held
  static_assert(kSmem + 13824 <= 227 * 1024, "shared memory with the static part");
  static_assert(kSlots >= (NB + 1) * KT, "S runs NB tiles ahead");
  // A producer writes the scales of tiles i .. i + kBatch - 1 before the wait of tile i's K; its load before that waited
  // for the use of its slot, kSlots + KT sub-tiles further back.  P V of tile i - NB is the last of a tile before K of
  // tile i.
  static_assert(kMeta >= NB + kBatch + (kSlots + KT + 2 * KT - 1) / (2 * KT), "block scales");
  static_assert(!kRowLanes || (RT == 128 && kGroups == 4), "a lane per row, a quarter of the keys per group");
  static_assert(!kRowLanes || kABufs == NB, "P is written while the product before reads its own");
  static_assert(kRowLanes || (KT == 2 && CG == 16 && RT <= 64), "tiles of two sub-tiles, P in rows of 128 bytes");
  static_assert(kOCol + kOCols <= kACol && RT % CG == 0 && kGroups <= 4, "TMEM and rows");
};

// A segment's rows: q1, q2 into the operand tiles at qb, the row scales, and
// each query's tree mask, by warp w of the n that share it (barrier `bar`).
// Four lanes share a row, each with its quarter in registers (the next row's
// is fetched meanwhile).
template <int D, int RT>
__device__ __noinline__ void prepare_rows(const Args &a, const Segments sg, uint8_t *qb, int *par,
                                          uint32_t (*anc)[kMaxNodes / 32], float *qs, int w, int n, int bar) {
  using C = Cfg<D, RT>;
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

template <int D, int RT>
__global__ void __launch_bounds__(Cfg<D, RT>::kThreads, 1)
    k_branch_attn_q8(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ Args a) {
  using C = Cfg<D, RT>;
  constexpr int CG = C::CG, NB = C::NB, NSLOT = C::kSlots, KT = C::KT, kMeta = C::kMeta;
  constexpr int kSoftThreads = C::kSoftWarps * 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *const smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[NSLOT], empty[NSLOT];
  __shared__ __align__(8) uint64_t sfull[NB], pfull[NB], vfull[NB][KT], pvdone[NB], qfull[2], qempty[2];
  __shared__ uint32_t tmem_base;
  // a block's k_scale * scale * log2 e, v_scale (-1: hidden), log2 v_scale
  __shared__ __align__(16) float4 meta[kMeta][KT * kPages];
  __shared__ __align__(16) int s_ids[C::kTmaWarps][kIds][kPages];  // block ids of a tile's sub-tile, -1 for none
  __shared__ int s_row[C::kTmaWarps][kIds];                        // and its head's first row in a block
  __shared__ int par[2][kMaxNodes];
  __shared__ uint32_t anc[2][kMaxNodes][kMaxNodes / 32];    // per query: the nodes that it sees
  __shared__ float qs[2][RT];                               // row scales 2^e
  __shared__ __align__(16) float4 rowc[RT / 2];             // two rows: 2^e, 2^e, 11 - m, 11 - m
  __shared__ float s_m[RT], s_f[RT], red[4][RT];
  __shared__ int s_nan[4];                                  // a tree node's v held NaN, by segment mod 4 (the helper
                                                            // warps are in the segment behind the softmax warps' at most)
  __shared__ long long scan[32];
  __shared__ Piece s_piece;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes
  const float NEG_INF = -__int_as_float(0x7f800000);

  if (tid == 0) {
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int u = 0; u < NB; ++u) {
      mbar_init(&sfull[u], 1);
      mbar_init(&pfull[u], 4 * C::kGroups);
      for (int h = 0; h < KT; ++h) mbar_init(&vfull[u][h], 4);
      mbar_init(&pvdone[u], 1);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&qfull[u], 4);
      mbar_init(&qempty[u], 1 + C::kSoftWarps);
    }
    fence_mbar_init();
    s_abort = 0;
    s_nan[0] = s_nan[1] = s_nan[2] = s_nan[3] = 0;
    s_piece.left = 0;
    s_piece.tiles = 0;
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  // the line of units: every thread sums some sequences' units, then the sums are scanned
  {
    const int per = (a.B + C::kThreads - 1) / C::kThreads, b0 = tid * per, b1 = min(a.B, b0 + per);
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
    long long upto = lane < C::kWarps ? scan[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const long long total = __shfl_sync(0xffffffffu, upto, 31);
    const long long before = __shfl_sync(0xffffffffu, upto, max(warp - 1, 0)) * (warp > 0);
    const long long T = total * a.per_b;
    long long chunk = quotient(T + gridDim.x - 1, gridDim.x);
    if (a.split) chunk = max(chunk, static_cast<long long>(kMinKeys / C::kKeys));
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
      s_piece = p;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
  const Piece piece = s_piece;
  const int ntiles = piece.tiles;

  // the rows of segment `sg` into buffer `buf`, by warp w of the n that share it (barrier `bar`)
  auto prepare = [&](const Segments &sg, int buf, int w, int n, int bar) {
    prepare_rows<D, RT>(a, sg, smem + C::kQ + buf * C::kQBuf, par[buf], anc[buf], qs[buf], w, n, bar);
  };

  Segments sg;
  if (warp >= C::kTmaWarp && warp < C::kMmaWarp) {
    // ---------------- producers: warp p loads sub-tile p of every tile, K and V.  A copy costs 45 clocks (the TMA unit's
    // own pace for 2 KB).  Block ids and scales are fetched for kBatch tiles at a time, one batch ahead (two dependent
    // trips to memory for a batch): lane l holds block l % 8 of the batch's tile l / 8.
    const int pw = warp - C::kTmaWarp, page = lane % kPages;
    bool more = sg.first(a, piece);
    int t = more ? sg.t0 : 0;
    auto advance = [&](int n) {  // this lane's place in the line of tiles
      t += n;
      while (more && t >= sg.t1) {
        t -= sg.t1;
        more = sg.step(a);
      }
    };
    int hk, blk;
    float ks, vs;
    auto ids = [&] {
      hk = more ? sg.hk : 0;
      blk = -1;
      vs = 0.f;
      ks = -1.f;  // no block there
      const int64_t lp = (static_cast<int64_t>(t) * KT + pw) * kPages + page;
      if (more && lp < a.maxb && lp * kPage < sg.nkeys) {
        blk = a.table[static_cast<int64_t>(sg.b) * a.maxb + lp];
        ks = 0.f;
      }
      advance(kBatch);
    };
    auto scales = [&] {
      if (blk >= 0 && blk < a.num_blocks) {
        const int64_t unit = static_cast<int64_t>(blk) * a.Hkv + hk;
        ks = __ldg(a.ks + unit);
        vs = __ldg(a.vs + unit);
      } else if (ks >= 0.f) {
        atomicOr(a.status, kFlagBadBlock);
        blk = -1;
      }
    };
    advance(lane / kPages);
    ids();
    scales();
    int slot = pw;
    uint32_t phase = 1;  // of empty[slot]; the first round's slots are free
    int c = 0;           // tiles of K and of V loaded so far
    bool ok = true;
    Order order;
    order.start(a, piece);
    for (int i = 0, j = 0; j < ntiles; ++c) {
      const bool is_k = i - j < NB && i < order.end;  // K of tile i, or V of tile j
      if (is_k) {
        const int w = i % kBatch;
        if (w == 0) {
          if (blk >= 0 && !(good_scale(ks) && good_scale(vs))) {  // bad scales hide their block
            atomicOr(a.status, kFlagBadValue);
            blk = -1;
          }
          const float v = vs < kMinBlockScale ? 0.f : vs;
          const int at = i + lane / kPages;
          meta[at % kMeta][pw * kPages + page] =
              blk >= 0 ? make_float4(fminf(ks * a.scale_log2, 3e38f), v, __log2f(fmaxf(v, kMinBlockScale)), 0.f)
                       : make_float4(0.f, -1.f, 0.f, 0.f);
          s_ids[pw][at % kIds][page] = blk;
          if (page == 0) s_row[pw][at % kIds] = hk * kPage;
          __syncwarp();
          ids();
        }
        if (w == kBatch / 2) scales();
      }
      const int x = (is_k ? i : j) % kIds;
      const CUtensorMap *const map = is_k ? &kmap : &vmap;
      const int row = s_row[pw][x];
      const int4 lo = *reinterpret_cast<const int4 *>(s_ids[pw][x]), hi = *reinterpret_cast<const int4 *>(s_ids[pw][x] + 4);
      const int e[kPages] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      ok = c * KT + pw < NSLOT || warp_wait(&empty[slot], phase);
      if (!ok) break;
      uint8_t *const dst = smem + C::kRing + slot * C::kSlot;
      if (elect_one()) {
        if ((lo.x | lo.y | lo.z | lo.w | hi.x | hi.y | hi.z | hi.w) >= 0) {
          mbar_arrive_expect_tx(&full[slot], C::kSlot);
#pragma unroll
          for (int k = 0; k < kPages; ++k) tma_load_3d(dst + k * (kPage * D), map, 0, row, e[k], &full[slot]);
        } else {  // some blocks are missing or bad
          int n = 0;
          for (int k = 0; k < kPages; ++k) n += s_ids[pw][x][k] >= 0;
          mbar_arrive_expect_tx(&full[slot], n * (kPage * D));
#pragma unroll 1
          for (int k = 0; k < kPages; ++k)
            if (s_ids[pw][x][k] >= 0) tma_load_3d(dst + k * (kPage * D), map, 0, row, s_ids[pw][x][k], &full[slot]);
        }
      }
      __syncwarp();
      slot += KT;
      if (slot >= NSLOT) {
        slot -= NSLOT;
        phase ^= 1;
      }
      if (is_k) ++i;
      else order.done(a, ++j);
    }
    if (!ok) {
      s_abort = 1;
      // this warp's copies in flight land before the shared memory is given back
      for (int k = 0; k < (NSLOT + KT - 1) / KT && --c >= 0; ++k) {
        const int load = c * KT + pw;
        (void)warp_wait(&full[load % NSLOT], (load / NSLOT) & 1);
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ---------------- MMA issue (one elected lane): S of up to NB tiles ahead, then P V and S in turn.  This loop
    // is one warp's chain of scalar work per tile, so what can be is kept in running words.
    constexpr uint32_t idesc_s = idesc_f8(C::kRowLanes ? kSub : RT), idesc_o = idesc_f16(C::kRowLanes ? D : RT);
    constexpr uint32_t hi128 = desc_hi(1024, kSw128), hi64 = desc_hi(512, kSw64), hi_kv = D == 128 ? hi128 : hi64;
    const uint32_t base = smem_u32(smem);
    const uint32_t ring_k = desc_lo(base + C::kRing, 16), h_lo = desc_lo(base + C::kH, C::kBlock);
    bool ok = true;
    int slot = 0, seg = 0;
    uint32_t phase = 0;  // of full[slot]
    bool more = sg.first(a, piece);
    int t = more ? sg.t0 : 0;
    auto next_slot = [&] {
      if (++slot == NSLOT) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto umma_s = [&](uint32_t d, uint32_t k, uint32_t q) {
#pragma unroll
      for (int term = 0; term < 2; ++term)
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          const uint32_t qk = q + (term * (D == 128 ? C::kQTile : 64) >> 4) + kk * 2, more = (term > 0 || kk > 0) ? 1u : 0u;
          if (C::kRowLanes)
            umma_f8(d, qk, hi128, k + kk * 2, hi_kv, idesc_s, more);
          else
            umma_f8(d, k + kk * 2, hi_kv, qk, hi128, idesc_s, more);
        }
    };
    auto issue_s = [&](int i) {
      const int buf = seg & 1, u = i % NB;
      if (t == sg.t0) ok = warp_wait(&qfull[buf], (seg >> 1) & 1);
      const uint32_t q = desc_lo(base + C::kQ, 16) + buf * (C::kQBuf >> 4);
      const bool last = ++t == sg.t1;
#pragma unroll
      for (int h = 0; h < KT; ++h) {
        // the S buffer is free: P of tile i - NB, made from it, has been waited for
        ok = ok && warp_wait(&full[slot], phase);
        tc_fence_after();
        if (!ok) return;
        if (elect_one()) {
          umma_s(tmem + (u * KT + h) * RT, ring_k + slot * (C::kSlot >> 4), q);
          umma_commit(&empty[slot]);
          if (h == KT - 1) {
            umma_commit(&sfull[u]);
            if (last) umma_commit(&qempty[buf]);
          }
        }
        __syncwarp();
        next_slot();
      }
      if (last) {
        more = sg.step(a);
        t = sg.t0;
        ++seg;
      }
    };
    Order order;
    order.start(a, piece);
    for (int i = 0, j = 0; j < ntiles && ok;) {
      if (i - j < NB && i < order.end) {
        issue_s(i++);
      } else {  // P V of tile j
        const int u = j % NB;
        const uint32_t o = tmem + C::kOCol;
        const uint32_t later = j > order.begin;  // not the segment's first tile
        ok = warp_wait(&pfull[u], (j / NB) & 1);
        const uint32_t at = tmem + C::kACol + (j % C::kABufs) * C::kACols, b = h_lo + u * (C::kHBuf >> 4);
#pragma unroll 1
        for (int h = 0; h < KT; ++h) {
          ok = ok && warp_wait(&vfull[u][h], (j / NB) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            umma_commit(&empty[slot]);  // the helper warps have read V; given back in the order of the loads (S before)
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk)  // 16 keys: two groups of 8 rows
              umma_f16(o, at + h * (kSub / 2) + kk * 8, b + h * (C::kBlock >> 4) + kk * (2048 >> 4), hi128, idesc_o,
                       kk > 0 || h > 0 ? 1u : later);
            if (h == KT - 1) umma_commit(&pvdone[u]);
          }
          __syncwarp();
          next_slot();
        }
        order.done(a, ++j);
      }
    }
    if (!ok) s_abort = 1;
  } else if (warp >= C::kHelpWarp && warp < C::kTmaWarp) {
    // ---------------- helpers: V in halves, tile by tile, and the rows of the segments after the first, a segment ahead.
    // They meet at named barriers, which have no limit, so a warp whose wait gave up goes on (its waits are over at once)
    // until they leave together.
    const int hw = warp - C::kHelpWarp;
    bool ok = true, all = true, more = sg.first(a, piece);
    if (more) {
      prepare(sg, 0, warp, C::kSoftWarps + 4, 10);
      bar_sync(10, (C::kSoftWarps + 4) * 32);
      if (lane == 0) mbar_arrive1(&qfull[0]);
    }
    for (int i = 0, seg = 0; more; ++seg) {
      const int n = sg.t1 - sg.t0, end = i + n;
      Segments next = sg;
      more = next.step(a);
      if (more) {  // the next segment's rows, once the segment before this has left their buffer
        const int buf = (seg + 1) & 1;
        ok = ok && (seg < 1 || warp_wait(&qempty[buf], ((seg - 1) >> 1) & 1));
        all = !bar_or(11, 128, !ok || s_abort);
        if (!all) break;
        prepare(next, buf, hw, 4, 11);
        if (lane == 0) mbar_arrive1(&qfull[buf]);
      }
      for (int x = 0; x < n; ++x, ++i) {
        const int t = sg.t0 + x, u = i % NB;
        // S first: by then K of this tile has landed, and with it every load that used V's slots before; a wait for V's
        // phase of a slot would not tell the phase two before from it
        ok = ok && warp_wait(&sfull[u], (i / NB) & 1);
        // the product that last read the buffer is done
        if (i >= C::kABufs) ok = ok && warp_wait(&pvdone[(i - C::kABufs) % NB], ((i - C::kABufs) / NB) & 1);
        tc_fence_after();
        // hidden keys take no part whatever their v holds (0 * NaN): they become 0; a tree node's NaN becomes 0 too, and
        // reaches the rows that see it at the segment's end
        bool part = (t + 1) * C::kKeys > min(sg.L, sg.nkeys);
        part = __any_sync(0xffffffffu, part || (lane < KT * kPages && meta[i % kMeta][lane].y < 0.f));
        const int load0 = (min(i + NB, end) + i) * KT;  // V's place in the order of loads
#pragma unroll 1
        for (int h = 0; h < KT; ++h) {
          const int slot = (load0 + h) % NSLOT;
          ok = ok && warp_wait(&full[slot], ((load0 + h) / NSLOT) & 1);
          if (!ok) break;
          const uint8_t *const vt = smem + C::kRing + slot * C::kSlot;
          uint32_t any = 0;
          if constexpr (C::kRowLanes) {  // a lane per key
            const int r = hw * 32 + lane, pos = t * kSub + r;
            const bool gone = part && (meta[i % kMeta][r / kPage].y < 0.f || pos >= sg.nkeys);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {  // 16 codes
              uint4 v = make_uint4(0, 0, 0, 0);
              if (!gone) v = *reinterpret_cast<const uint4 *>(vt + (D == 128 ? sw128(r, c * 16) : sw64(r, c * 16)));
              if (part && pos >= sg.L)
                v = make_uint4(without_nan(v.x, ~0u, any), without_nan(v.y, ~0u, any), without_nan(v.z, ~0u, any),
                               without_nan(v.w, ~0u, any));
              uint32_t x[8];
              halves_of(v.x, x[0], x[1]);
              halves_of(v.y, x[2], x[3]);
              halves_of(v.z, x[4], x[5]);
              halves_of(v.w, x[6], x[7]);
              uint8_t *const to = smem + C::kH + u * C::kHBuf + (c >> 2) * C::kBlock;
              *reinterpret_cast<uint4 *>(to + sw128(r, (c & 3) * 32)) = make_uint4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<uint4 *>(to + sw128(r, (c & 3) * 32 + 16)) = make_uint4(x[4], x[5], x[6], x[7]);
            }
            fence_proxy_async();  // V (generic writes) -> visible to the tensor cores
          } else {  // V^T: 32 keys of this warp's 32 elements (at d = 64 the upper lanes repeat the lower ones) at a time
            const int el = (D == 128 ? hw : hw & 1) * 32 + (lane >> 4) * 16;
            const uint32_t from = smem_u32(vt) + (D == 128 ? sw128(lane & 15, el) : sw64(lane & 15, el));
            const uint32_t to = tmem + C::kACol + (i % C::kABufs) * C::kACols + h * (kSub / 2) +
                                (static_cast<uint32_t>(hw * 32) << 16);
            // a rolled loop: the softmax warps' code has to stay in the instruction cache
#pragma unroll 1
            for (int k0 = 0; k0 < kSub; k0 += 32) {
              uint32_t c[8];
              load_columns(from + k0 * D, c);
              load_columns(from + (k0 + 16) * D, c + 4);
              if (part) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  // this lane's four keys: those that are there, and those that are tree nodes
                  const int key = h * kSub + k0 + b * 16, pos = t * C::kKeys + key + (lane & 3) * 4;
                  auto first = [](int n) { return n <= 0 ? 0u : (n >= 4 ? ~0u : (1u << (8 * n)) - 1u); };
                  const uint32_t there = meta[i % kMeta][key / kPage].y < 0.f ? 0u : first(sg.nkeys - pos);
                  const uint32_t nodes = ~first(sg.L - pos);
#pragma unroll
                  for (int w = 0; w < 4; ++w) c[b * 4 + w] = without_nan(c[b * 4 + w] & there, nodes, any);
                }
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // 16 elements each
                uint32_t v[8];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  halves_of(c[b * 4 + e * 2], v[b * 4], v[b * 4 + 1]);
                  halves_of(c[b * 4 + e * 2 + 1], v[b * 4 + 2], v[b * 4 + 3]);
                }
                tmem_st_16x16(to + k0 / 2 + (static_cast<uint32_t>(e * 16) << 16), v);
              }
            }
            tmem_wait_st();
            tc_fence_before();
          }
          if (any) s_nan[seg & 3] = 1;
          __syncwarp();
          if (lane == 0) mbar_arrive1(&vfull[u][h]);
        }
      }
      sg = next;
    }
    if (!ok || !all) s_abort = 1;
  } else if constexpr (C::kRowLanes) {
    // ---------------- softmax, a lane per row: group g has the keys g * 32 .. + 31 of every tile
    const int g = warp / 4, wg = warp & 3, r = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>(wg * 32) << 16;
    const uint32_t tS = tmem + g * 32 + lane_off, tO = tmem + C::kOCol + g * (D / 4) + lane_off;
    const int bar = 1 + wg;  // the four warps that share 32 rows
    int i0 = 0, seg = 0;     // the segment's first tile in the CTA's count
    uint32_t sphase = 0;     // parities of sfull
    bool dead = false;
    bool more = sg.first(a, piece);
    if (more) {
      prepare(sg, 0, warp, C::kSoftWarps + 4, 10);
      bar_sync(10, (C::kSoftWarps + 4) * 32);
    }
    for (; more; more = sg.step(a), ++seg) {
      const int buf = seg & 1, n = sg.t1 - sg.t0, row = sg.mt * RT + r;
      const bool live = row < a.nrows, some = sg.mt * RT + wg * 32 < a.nrows;  // this row; some row of the warp
      const int qi = min(static_cast<int>((row * a.group_magic) >> 16), kMaxNodes - 1);
      bool ok = warp_wait(&qfull[buf], (seg >> 1) & 1);
      const float qscale = live ? qs[buf][r] : 0.f;
      // the row's m (all four groups keep it), and what is added to its scores; a row behind the last gets p = 0
      float m = NEG_INF, add = live ? 0.f : -1e30f;
      uint64_t l2[2] = {0, 0};
      bool begin = true, unset = live;  // before the segment's first tile; no visible key so far
      for (int x = 0; x < n; ++x) {
        const int i = i0 + x, t = sg.t0 + x, u = i % NB;  // u: S and P buffer
        ok = ok && warp_wait(&sfull[u], sphase >> u & 1);
        sphase ^= 1u << u;  // the scales were there before K was
        tc_fence_after();
        bool part = (t + 1) * kSub > min(sg.L, sg.nkeys);
        part = __any_sync(0xffffffffu, part || (lane < kPages && meta[i % kMeta][lane].y < 0.f));
        if (some) {
          float cq[2], wv[2], lsv[2];
          uint32_t vis = ~0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 sc = meta[i % kMeta][g * 2 + e];
            cq[e] = fminf(sc.x * qscale, 3e38f);
            wv[e] = fmaxf(sc.y, 0.f);
            lsv[e] = sc.z;
            if (sc.y < 0.f) vis &= e ? 0x0000FFFFu : 0xFFFF0000u;
          }
          if (part) {
            const int k0 = t * kSub + g * 32, left = sg.nkeys - k0, node = k0 - sg.L;  // of bit 0
            if (left < 32) vis &= left <= 0 ? 0u : (1u << left) - 1u;
            if (node > -32) {
              const uint32_t *const bits = anc[buf][qi];
              const int word = node >> 5;
              const uint32_t lo = node < 0 ? ~0u : (word < kMaxNodes / 32 ? bits[word] : 0u);
              const uint32_t hi = word + 1 < kMaxNodes / 32 ? bits[word + 1] : 0u;
              vis &= __funnelshift_r(lo, hi, node & 31);
            }
          }
          float y[32];
          // y = x - m + 11 (x for a row without m); hidden keys -inf
          auto scores = [&]() {
            tmem_ld16_async(tS + u * kSub, y);
            tmem_ld16_async(tS + u * kSub + 16, y + 16);
            tmem_wait16(y);
            tmem_wait16(y + 16);
            const uint64_t add2 = pack2(add, add);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t c2 = pack2(cq[e], cq[e]);
#pragma unroll
              for (int j = e * 16; j < e * 16 + 16; j += 2)
                unpack2(fma2(pack2(y[j], y[j + 1]), c2, add2), y[j], y[j + 1]);
            }
            if (part) {
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = ((vis >> j) & 1u) ? y[j] : NEG_INF;
            }
          };
          // y, and whether a row's m has to move; then once more with the new m
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            scores();
            if (pass == 1) break;
            float top = NEG_INF;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t4[4] = {y[e * 16], y[e * 16 + 1], y[e * 16 + 2], y[e * 16 + 3]};
#pragma unroll
              for (int j = 4; j < 16; ++j) t4[j & 3] = fmaxf(t4[j & 3], y[e * 16 + j]);
              top = fmaxf(top, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) + lsv[e]);
            }
            if (!bar_or(bar, 128, top > kGrow || unset || !ok)) break;
            red[g][r] = top;
            // O is rescaled below: every P V before has to be in it
            if (!begin) {
              ok = warp_wait(&pvdone[(i - 1) % NB], ((i - 1) / NB) & 1) && ok;
              tc_fence_after();
            }
            if (bar_or(bar, 128, !ok)) {
              dead = true;
              break;
            }
            const float z = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
            bar_sync(bar, 128);  // read, before the next is written
            float f = 1.f;
            if (live) {
              if (m == NEG_INF) {
                m = z;
                unset = m == NEG_INF;
              } else if (z > kGrow) {
                m += z - kMoved;
                f = ex2(kMoved - z);
              }
              add = unset ? 0.f : kBias - m;
            }
            if (!begin && __any_sync(0xffffffffu, f != 1.f)) {
              const uint64_t f2 = pack2(f, f);
              l2[0] = mul2(l2[0], f2);
              l2[1] = mul2(l2[1], f2);
#pragma unroll 1
              for (int k = 0; k < D / 64; ++k) {  // this group's quarter of O
                const uint32_t at = tO + k * 16;
                float o[16];
                tmem_ld16(at, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_st16(at, o);
              }
            }
          }
          if (dead) break;
          begin = false;
          // the P buffer is free: S of this tile was issued behind P V of tile i - NB
          const uint64_t unit2 = pack2(kSumUnit, kSumUnit);
          uint32_t hp[16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t w2 = pack2(wv[e], wv[e]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint64_t p = pack2(ex2(y[e * 16 + 2 * j]), ex2(y[e * 16 + 2 * j + 1]));
              l2[j & 1] = fma2(p, unit2, l2[j & 1]);
              float a0, a1;
              unpack2(mul2(p, w2), a0, a1);
              hp[e * 8 + j] = half2_of(a0, a1);
            }
          }
          tmem_st16_async(tmem + C::kACol + u * C::kACols + g * 16 + lane_off, hp);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&pfull[u]);
      }
      // ---------------- the segment's end: l, then O from TMEM, a quarter of the row's elements each
      if (dead) ok = false;
      {
        float l0, l1, l3, l4;
        unpack2(l2[0], l0, l1);
        unpack2(l2[1], l3, l4);
        red[g][r] = __fadd_rn(__fadd_rn(l0, l1), __fadd_rn(l3, l4));
      }
      const int il = i0 + n - 1;
      ok = ok && warp_wait(&pvdone[il % NB], (il / NB) & 1);
      tc_fence_after();
      if (bar_or(9, kSoftThreads, !ok)) {
        s_abort = 1;
        break;
      }
      const bool whole = sg.t0 == 0 && sg.t1 == sg.nt, nan = s_nan[seg & 3] != 0;
      if (tid == 0) s_nan[(seg + 2) & 3] = 0;
      if (some) {
        const int slot = blockIdx.x * 2 + (sg.t0 > 0 ? 0 : 1);
        const float L = __fadd_rn(__fadd_rn(red[0][r], red[1][r]), __fadd_rn(red[2][r], red[3][r]));
        const float factor = L == 0.f ? 0.f : (whole ? 1.f / L : 1.f) * kSumUnit;
        const int64_t orow = (static_cast<int64_t>(sg.b) * a.Nq + qi) * a.Hq + sg.hk * a.group + (row - qi * a.group);
        if (live && g == 0) {
          if (!whole)
            a.part_ml[slot * RT + r] = make_float2(m, L);
          else if (a.lse)
            a.lse[orow] = L == 0.f ? NEG_INF : (m - kSumBias + log2f(L)) * 0.69314718055994531f;
        }
#pragma unroll 1
        for (int j0 = 0; j0 < D / 4; j0 += 16) {
          float o[16];
          tmem_ld16(tO + j0, o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] *= factor;
          if (!live) continue;
          const int e0 = g * (D / 4) + j0;
          if (nan) {
            // tree nodes of this segment that this row sees and whose v holds NaN
            const int from = sg.t0 * C::kKeys - sg.L, to = min(sg.nkeys, sg.t1 * C::kKeys) - sg.L;
            for (int node = max(0, from); node < to; ++node) {
              if (!((anc[buf][qi][node >> 5] >> (node & 31)) & 1u)) continue;
              const int pos = sg.L + node, blk = a.table[static_cast<int64_t>(sg.b) * a.maxb + pos / kPage];
              if (blk < 0 || blk >= a.num_blocks) continue;
              const int64_t unit = static_cast<int64_t>(blk) * a.Hkv + sg.hk;
              if (!good_scale(a.ks[unit]) || !good_scale(a.vs[unit])) continue;
              const uint8_t *const code = a.vc + (unit * kPage + pos % kPage) * D + e0;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if ((code[j] & 0x7F) == 0x7F) o[j] = __int_as_float(0x7fc00000);
            }
          }
          if (whole) {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(o[2 * j + 1]), "f"(o[2 * j]));
            uint4 *const to = reinterpret_cast<uint4 *>(a.out + orow * D + e0);
            to[0] = make_uint4(h[0], h[1], h[2], h[3]);
            to[1] = make_uint4(h[4], h[5], h[6], h[7]);
          } else {
            float4 *const to = reinterpret_cast<float4 *>(a.part_o + (static_cast<int64_t>(slot) * RT + r) * D + e0);
#pragma unroll
            for (int j = 0; j < 4; ++j) to[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
      }
      tc_fence_before();
      bar_sync(9, kSoftThreads);  // O and the sums have been read
      if (lane == 0) mbar_arrive1(&qempty[buf]);
      i0 += n;
    }
  } else {
    // ---------------- softmax: group g of the rows, one thread per key
    const int g = warp / 4, wg = warp & 3, tg = tid & 127;
    const int col = g * CG;
    const uint32_t lane_off = static_cast<uint32_t>(wg * 32) << 16;
    const uint32_t tS = tmem + col + lane_off, tO = tmem + C::kOCol + col + lane_off;
    const int bar = 1 + g;
    int i0 = 0, seg = 0;  // the segment's first tile in the CTA's count
    uint32_t sphase = 0;  // parities of sfull
    bool dead = false;
    bool more = sg.first(a, piece);
    if (more) {
      prepare(sg, 0, warp, C::kSoftWarps + 4, 10);
      bar_sync(10, (C::kSoftWarps + 4) * 32);
    }
    for (; more; more = sg.step(a), ++seg) {
      const int buf = seg & 1, n = sg.t1 - sg.t0;
      const int hk = sg.hk, mt = sg.mt;
      const int row0 = mt * RT + col;  // the warp's first row of (b, hk)
      bool ok = warp_wait(&qfull[buf], (seg >> 1) & 1);
      if (tg < CG) {
        s_m[col + tg] = NEG_INF;
        float *const rc = reinterpret_cast<float *>(&rowc[(col + tg) >> 1]) + (tg & 1);
        rc[0] = qs[buf][col + tg];
        rc[2] = 0.f;
      }
      bar_sync(bar, 128);
      uint64_t l2[CG / 2];
#pragma unroll
      for (int j = 0; j < CG / 2; ++j) l2[j] = 0;
      bool begin = true, unset = true;  // before the segment's first tile; a row without a visible key so far
      for (int x = 0; x < n; ++x) {
        const int i = i0 + x, t = sg.t0 + x, u = i % NB;  // u: S and P buffer
        ok = ok && warp_wait(&sfull[u], sphase >> u & 1);
        sphase ^= 1u << u;  // the scales were there before K was
        tc_fence_after();
        // this thread's keys: their scales, and the rows that see them
        float c[KT];
        // what is used once a tile is read where it is used: at 64 rows the warps have 80 registers a thread
        auto scale_of = [&](int h) -> const float4 & { return meta[i % kMeta][h * kPages + tg / kPage]; };
        uint32_t vis[KT];
        bool hidden[KT], part = false;
#pragma unroll
        for (int h = 0; h < KT; ++h) {
          const float2 sc = *reinterpret_cast<const float2 *>(&scale_of(h));
          c[h] = sc.x;
          const int pos = t * C::kKeys + h * kSub + tg;
          hidden[h] = sc.y < 0.f || pos >= sg.nkeys;
          part = part || hidden[h] || pos >= sg.L;
        }
        part = __any_sync(0xffffffffu, part);
        if (part) {
#pragma unroll
          for (int h = 0; h < KT; ++h) {
            const int node = t * C::kKeys + h * kSub + tg - sg.L;
            vis[h] = hidden[h] ? 0u : ~0u;
            if (!hidden[h] && node >= 0) {
              // row j is query (row0 + j) / group: the rows of one query are neighbours
              uint32_t see = 0;
              int qi = static_cast<int>((row0 * a.group_magic) >> 16), j0 = 0;
#pragma unroll 1
              for (int j1 = (qi + 1) * a.group - row0; j0 < CG && qi < a.Nq; ++qi, j0 = j1, j1 += a.group)
                if ((anc[buf][qi][node >> 5] >> (node & 31)) & 1u)
                  see |= (j1 < CG ? (1u << j1) - 1u : ~0u) & (~0u << j0);
              vis[h] = see;
            }
          }
        }
        float y[KT][CG];
        // y = x - m + 11 (x for a row without m); hidden keys -inf
        auto scores = [&]() {
#pragma unroll
          for (int h = 0; h < KT; ++h) tmem_ld16_async(tS + (u * KT + h) * RT, y[h]);
#pragma unroll
          for (int h = 0; h < KT; ++h) tmem_wait16(y[h]);
#pragma unroll
          for (int j = 0; j < CG; j += 2) {
            const float4 rc = rowc[(col + j) / 2];
#pragma unroll
            for (int h = 0; h < KT; ++h)
              unpack2(fma2(mul2(pack2(y[h][j], y[h][j + 1]), pack2(c[h], c[h])), pack2(rc.x, rc.y), pack2(rc.z, rc.w)),
                      y[h][j], y[h][j + 1]);
          }
          if (part) {
#pragma unroll
            for (int h = 0; h < KT; ++h)
#pragma unroll
              for (int j = 0; j < CG; ++j) y[h][j] = ((vis[h] >> j) & 1u) ? y[h][j] : NEG_INF;
          }
        };
        // y, and whether a row's m has to move; then once more with the new m
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          scores();
          if (pass == 1) break;
          float top = NEG_INF;
#pragma unroll
          for (int h = 0; h < KT; ++h) {
            float t4[4] = {y[h][0], y[h][1], y[h][2], y[h][3]};
#pragma unroll
            for (int j = 4; j < CG; ++j) t4[j & 3] = fmaxf(t4[j & 3], y[h][j]);
            top = fmaxf(top, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) + scale_of(h).z);
          }
          if (!bar_or(bar, 128, top > kGrow || unset || !ok)) break;
          // the rows' largest log2 of P v_scale (of a row without a key so far: x + log2 v_scale) in this tile
          float big = NEG_INF;
#pragma unroll
          for (int j = 0; j < CG; ++j) {
            const float z = warp_top(fmaxf(y[0][j] + scale_of(0).z, y[1][j] + scale_of(1).z));
            if (lane == j) big = z;
          }
          if (lane < CG) red[wg][col + lane] = big;
          // O is rescaled below: every P V before has to be in it
          if (!begin) {
            ok = warp_wait(&pvdone[(i - 1) % NB], ((i - 1) / NB) & 1) && ok;
            tc_fence_after();
          }
          if (bar_or(bar, 128, !ok)) {
            dead = true;
            break;
          }
          bool none = false;
          if (tg < CG) {
            const int r = col + tg;
            const float mo = s_m[r];
            const float z = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
            float mn = mo, f = 1.f;
            if (mo == NEG_INF) {
              mn = z;
              none = mn == NEG_INF;
            } else if (z > kGrow) {
              mn = mo + (z - kMoved);
              f = ex2(kMoved - z);
            }
            s_m[r] = mn;
            s_f[r] = f;
            reinterpret_cast<float *>(&rowc[r >> 1])[2 + (tg & 1)] = none ? 0.f : kBias - mn;
          }
          unset = bar_or(bar, 128, none);
          if (!begin) {
            bool moved = false;
#pragma unroll
            for (int j = 0; j < CG; ++j) moved = moved || s_f[col + j] != 1.f;
            if (moved) {
#pragma unroll
              for (int j = 0; j < CG / 2; ++j) l2[j] = mul2(l2[j], pack2(s_f[col + 2 * j], s_f[col + 2 * j + 1]));
              float o[CG];
              tmem_ld16(tO, o);
#pragma unroll
              for (int j = 0; j < CG; ++j) o[j] *= s_f[col + j];
              tmem_st16(tO, o);
            }
          }
        }
        if (dead) break;
        begin = false;
        // the P buffer is free: S of this tile was issued behind P V of tile i - NB
        const uint64_t unit2 = pack2(kSumUnit, kSumUnit);
#pragma unroll
        for (int h = 0; h < KT; ++h) {
          const float wv = fmaxf(scale_of(h).y, 0.f);
          const uint64_t w2 = pack2(wv, wv);
          uint32_t hp[CG / 2];
#pragma unroll
          for (int j = 0; j < CG / 2; ++j) {
            const uint64_t p = pack2(ex2(y[h][2 * j]), ex2(y[h][2 * j + 1]));
            l2[j] = fma2(p, unit2, l2[j]);
            float a0, a1;
            unpack2(mul2(p, w2), a0, a1);
            hp[j] = half2_of(a0, a1);
          }
          uint8_t *const pb = smem + C::kH + u * C::kHBuf + h * C::kBlock;
          *reinterpret_cast<uint4 *>(pb + sw128(tg, col * 2)) = make_uint4(hp[0], hp[1], hp[2], hp[3]);
          *reinterpret_cast<uint4 *>(pb + sw128(tg, col * 2 + 16)) = make_uint4(hp[4], hp[5], hp[6], hp[7]);
        }
        fence_proxy_async();  // P (generic writes) -> visible to the tensor cores
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&pfull[u]);
      }
      // ---------------- the segment's end: l, then O from TMEM
      if (dead) ok = false;
      {
        float z[CG];
#pragma unroll
        for (int j = 0; j < CG; j += 2) unpack2(l2[j / 2], z[j], z[j + 1]);
        const float sum = warp_columns(z, lane);
        if (!(lane & 1)) red[wg][col + (lane >> 1)] = sum;
      }
      const int il = i0 + n - 1;
      ok = ok && warp_wait(&pvdone[il % NB], (il / NB) & 1);
      tc_fence_after();
      if (bar_or(9, kSoftThreads, !ok)) {
        s_abort = 1;
        break;
      }
      const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
      const int slot = blockIdx.x * 2 + (sg.t0 > 0 ? 0 : 1);
      if (tid == 0) s_nan[(seg + 2) & 3] = 0;
      for (int r = tid; r < RT; r += kSoftThreads) {
        const float M = s_m[r], L = __fadd_rn(__fadd_rn(red[0][r], red[1][r]), __fadd_rn(red[2][r], red[3][r]));
        s_f[r] = L == 0.f ? 0.f : (whole ? 1.f / L : 1.f) * kSumUnit;
        const int row = mt * RT + r;
        if (row < a.nrows) {
          if (!whole) a.part_ml[slot * RT + r] = make_float2(M, L);
          else if (a.lse) {
            const int qi = static_cast<int>((row * a.group_magic) >> 16), head = hk * a.group + (row - qi * a.group);
            a.lse[(static_cast<int64_t>(sg.b) * a.Nq + qi) * a.Hq + head] =
                L == 0.f ? NEG_INF : (M - kSumBias + log2f(L)) * 0.69314718055994531f;
          }
        }
      }
      bar_sync(9, kSoftThreads);
      const bool nan = s_nan[seg & 3] != 0;
      // four rows at a time; at d = 64 the upper 64 lanes of O repeat the lower ones and take half of the rows
      constexpr int kShares = C::kGroups * (128 / D);
      const int share = D == 128 ? g : g * 2 + (wg >> 1), el = tg & (D - 1);
      uint16_t *const to = a.out + (static_cast<int64_t>(sg.b) * a.Nq * a.Hq + hk * a.group) * D + el;
#pragma unroll 1
      for (int j0 = share * 4; j0 < RT; j0 += kShares * 4) {
        const int r0 = mt * RT + j0;
        if (r0 >= a.nrows) break;
        float o[4];
        tmem_ld4(tmem + C::kOCol + j0 + lane_off, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] *= s_f[j0 + j];
        if (nan) {
          // tree nodes of this segment whose v holds NaN at this thread's element
          const int from = sg.t0 * C::kKeys - sg.L, to = min(sg.nkeys, sg.t1 * C::kKeys) - sg.L;
          for (int node = max(0, from); node < to; ++node) {
            const int pos = sg.L + node, blk = a.table[static_cast<int64_t>(sg.b) * a.maxb + pos / kPage];
            if (blk < 0 || blk >= a.num_blocks) continue;
            const int64_t unit = static_cast<int64_t>(blk) * a.Hkv + hk;
            if (!good_scale(a.ks[unit]) || !good_scale(a.vs[unit])) continue;
            if ((a.vc[(unit * kPage + pos % kPage) * D + el] & 0x7F) != 0x7F) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int qi = min(static_cast<int>(((r0 + j) * a.group_magic) >> 16), kMaxNodes - 1);
              if ((anc[buf][qi][node >> 5] >> (node & 31)) & 1u) o[j] = __int_as_float(0x7fc00000);
            }
          }
        }
        if (whole) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = r0 + j;
            if (r >= a.nrows) break;
            const int qi = static_cast<int>((r * a.group_magic) >> 16), at = qi * a.Hq + (r - qi * a.group);
            uint32_t b2;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b2) : "f"(0.f), "f"(o[j]));
            to[static_cast<int64_t>(at) * D] = static_cast<uint16_t>(b2 & 0xFFFFu);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) a.part_o[(static_cast<int64_t>(slot) * RT + j0 + j) * D + el] = o[j];
        }
      }
      tc_fence_before();
      bar_sync(9, kSoftThreads);  // O, the factors and the sums have been read
      if (lane == 0) mbar_arrive1(&qempty[buf]);
      i0 += n;
    }
  }
  if (tid == 0 && a.split) {  // what the piece's last item still needs
    int4 need = make_int4(0, 0, 0, 0);
    Segments x;
    for (bool more = x.first(a, piece); more; more = x.step(a))
      if (x.t0 == 0 && x.t1 < x.nt)
        need = make_int4(1 + (x.nt - x.t1 + piece.chunk - 1) / piece.chunk, x.b, x.hk, x.mt);
    a.info[blockIdx.x] = need;
  }
  tc_fence_before();
  __syncthreads();
  if (s_abort && tid == 0) atomicOr(a.status, kFlagWaitTimeout);
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that were cut: block (x, y) the item that CTA x
// began and did not end, eight of its rows, a warp per row.
template <int D, int RT>
__global__ void __launch_bounds__(256) k_attn_q8_merge(const __grid_constant__ Args a) {
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

}  // namespace q8
}  // namespace ssd

using namespace ssd;

namespace {

using q8::Args;

// [num_blocks][Hkv * 16 rows][d codes], boxes of one block's rows of a head
bool make_code_map(CUtensorMap *m, const void *base, int64_t num_blocks, int Hkv, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hkv) * q8::kPage,
                        static_cast<cuuint64_t>(num_blocks)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(d) * Hkv * q8::kPage};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(d), q8::kPage, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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

template <int D, int RT>
cudaError_t launch(const CUtensorMap &kmap, const CUtensorMap &vmap, const Args &a, unsigned grid, cudaStream_t cs) {
  using C = q8::Cfg<D, RT>;
  if (a.keys != C::kKeys) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(q8::k_branch_attn_q8<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  q8::k_branch_attn_q8<D, RT><<<grid, C::kThreads, C::kSmem, cs>>>(kmap, vmap, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.split) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (min(RT, a.nrows) + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = cs;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8::k_attn_q8_merge<D, RT>, a);
}

template <int D>
cudaError_t launch_shape(const Shape &s, const CUtensorMap &kmap, const CUtensorMap &vmap, const Args &a,
                         unsigned grid, cudaStream_t cs) {
  switch (s.RT) {
    case 16: return launch<D, 16>(kmap, vmap, a, grid, cs);
    case 32: return launch<D, 32>(kmap, vmap, a, grid, cs);
    case 48: return launch<D, 48>(kmap, vmap, a, grid, cs);
    case 64: return launch<D, 64>(kmap, vmap, a, grid, cs);
    default: return launch<D, 128>(kmap, vmap, a, grid, cs);
  }
}

}  // namespace

extern "C" {

size_t ssd_attention_q8_workspace_size(int B, int Nq, int Hq, int Hkv, int d) {
  if (B <= 0 || Nq <= 0 || Nq > q8::kMaxNodes || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 16 ||
      (d != 64 && d != 128))
    return 0;
  return workspace_of(shape_of(Nq, Hq, Hkv), d, attn_num_sms()).total;
}

ssd_status_t ssd_branch_attention_q8(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                                     const float *v_scale, const int32_t *block_table, int maxb, int64_t num_blocks,
                                     const int32_t *prefix_len, const int32_t *parent, int B, int N, int Nq, int Hq,
                                     int Hkv, int d, float scale, void *out, float *lse, uint32_t *status, void *ws,
                                     size_t ws_bytes, ssd_stream_t s) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return SSD_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return SSD_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSD_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16 || N < 1 || N > q8::kMaxNodes || Nq < 1 || Nq > N) return SSD_ERR_UNSUPPORTED;
  if (B == 0) return SSD_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len || !parent || !out ||
      !status || maxb < 1 || num_blocks < 1)
    return SSD_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(out)) & 15u)
    return SSD_ERR_UNSUPPORTED;
  if (num_blocks > 0x7fffffffLL || static_cast<int64_t>(B) * Hkv > 0x7fffffffLL / 32) return SSD_ERR_UNSUPPORTED;
  const Shape sh = shape_of(Nq, Hq, Hkv);
  Args a{};
  a.q = static_cast<const uint16_t *>(q);
  a.vc = static_cast<const uint8_t *>(v_cache);
  a.ks = k_scale;
  a.vs = v_scale;
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
  a.keys = sh.RT <= 64 ? 2 * q8::kSub : q8::kSub;
  const int64_t max_keys = static_cast<int64_t>(maxb) * q8::kPage;
  const int64_t max_tiles = (max_keys + a.keys - 1) / a.keys;
  const int64_t units = max_tiles * B * a.per_b;
  const unsigned grid = static_cast<unsigned>(units < sms ? units : sms);
  if ((max_tiles + q8::kEnd) * B * a.per_b / grid > 0x3fffffff) return SSD_ERR_UNSUPPORTED;  // a piece counts in 32 bits
  // short items are not worth cutting; without room for the parts none is cut
  const Workspace w = workspace_of(sh, d, sms);
  a.split = max_keys > q8::kWholeKeys && ws && ws_bytes >= w.total && !(reinterpret_cast<uintptr_t>(ws) & 255u);
  if (a.split) {
    char *const p = static_cast<char *>(ws);
    a.part_o = reinterpret_cast<float *>(p + w.o);
    a.part_ml = reinterpret_cast<float2 *>(p + w.ml);
    a.info = reinterpret_cast<int4 *>(p + w.info);
  }
  CUtensorMap kmap, vmap;
  if (!make_code_map(&kmap, k_cache, num_blocks, Hkv, d) || !make_code_map(&vmap, v_cache, num_blocks, Hkv, d))
    return SSD_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = d == 64 ? launch_shape<64>(sh, kmap, vmap, a, grid, cs)
                                : launch_shape<128>(sh, kmap, vmap, a, grid, cs);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
