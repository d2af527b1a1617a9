// cache_q4.cu -- the append into, and the reading back of, a paged K/V cache
// held in 4 bits: e2m1 codes with a power-of-two scale per 32 elements of a token
// and head.
//
// A group's scale is the smallest power of two that brings it under 6, so x /
// scale is exact and one rounding is made, to the nearest code; values come back
// exactly (a code has two significant bits).  Tokens share no scale: an append
// touches nothing but its own rows.  What neighbours do share is v's byte of two
// positions.
//
//   k_append_q4   a thread has 8 elements of two neighbouring positions (a byte of
//                 v holds both), K and V: four 16-byte loads in flight; four lanes
//                 are a group and find its maximum as 16-bit integers.  Half a
//                 pair (an odd first or even last position) reads the byte first.
//   k_read_q4     the same split the other way.
// Bound by HBM and the issue slots for prompts, by the chain prefix -> block table -> block for a decode step.  8 prompts
// of 4096 to 8191 tokens, 8 heads of 128: append (255 MB) 55 us, 4.6 TB/s, read back 51 us, 5.0 TB/s; 4 prefixes of 16384
// tokens (340 MB) 64 us, 5.3 TB/s; a decode step of 256 tokens 2.5 and 2.9 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/ssd.h"
#include "common.cuh"
#include "e2m1.cuh"
#include "e4m3.cuh"

namespace {

using namespace ssd;

constexpr int kThreads = 256;
constexpr int kPage = 16;
// Reading takes two pairs a thread where there are many, for the loads in flight (prefix of 4 x 16384 tokens, 340 MB: 64 us,
// 69 with one, 70 with four); appending, which has twice the bytes of a pair in flight, one (two took 2 us more).
constexpr int64_t kFewItems = 1 << 15;

struct Place {  // which rows, and where their blocks are
  const int32_t *table;
  int maxb;
  int64_t num_blocks;
  const int32_t *prefix_len, *count;
  int node0, S, Hkv;
  uint32_t items, blocks;  // of a sequence: pairs of positions that its rows may touch, times heads; CTAs
  uint32_t magic;          // item / Hkv = (item * magic >> 32) >> shift, item < 2^31, Hkv > 1
  int shift;
  int64_t grid;
  uint32_t *status;
};
struct AppendArgs {
  Place at;
  const uint16_t *rows[2];
  int64_t ss[2], ts[2];  // strides between sequences and tokens, elements
  uint8_t *cache[2], *scale[2];
};
struct ReadArgs {
  Place at;
  const uint8_t *cache[2], *scale[2];
  void *out[2];
  int64_t ss[2], ts[2];
};

// A thread's two positions: rows i and i + 1 (wanted: which are asked for), their block and slots.
struct Pair {
  int b, h, e0;       // sequence, head, first of the 8 elements
  int64_t i;          // row of the even position (may be -1)
  int64_t pos;        // the even position
  uint32_t wanted;    // bit 0 the even position, bit 1 the odd one
  uint32_t flags;
};
template <int D, int U>
SSD_DEV Pair pair_of(const Place &a, int u) {  // a thread's u-th pair of U
  constexpr int kPieces = D / 8;
  Pair p;
  p.wanted = 0;
  p.flags = 0;
  p.i = p.pos = 0;
  // neighbouring lanes take neighbouring pieces, then heads (adjacent in a token's row)
  const uint32_t b = blockIdx.x / a.blocks;
  const uint32_t item = ((blockIdx.x - b * a.blocks) * U + u) * (kThreads / kPieces) + threadIdx.x / kPieces;
  const uint32_t w = a.Hkv == 1 ? item : __umulhi(item, a.magic) >> a.shift;
  p.b = static_cast<int>(b);
  p.e0 = (threadIdx.x % kPieces) * 8;
  p.h = static_cast<int>(item - w * a.Hkv);
  if (item >= a.items) return p;
  const int L = a.prefix_len[b];
  if (L == -1) return p;  // a slot without a request
  int count = a.S;
  if (a.count) {
    const int c = a.count[b];
    count = min(max(c, 0), a.S);
    if (c != count) p.flags |= kFlagBadPrefix;
  }
  if (L < 0) {
    p.flags |= kFlagBadPrefix;
    return p;
  }
  const int64_t first = static_cast<int64_t>(L) + a.node0;
  p.pos = (first & ~int64_t(1)) + 2 * static_cast<int64_t>(w);
  p.i = p.pos - first;
  if (p.i >= 0 && p.i < count) p.wanted |= 1;
  if (p.i + 1 < count) p.wanted |= 2;  // i + 1 >= 0
  return p;
}
// The block * Hkv + head of a pair that has wanted rows; of a missing or bad block none is wanted any more.
SSD_DEV int64_t unit_of(const Place &a, Pair &p) {
  const int64_t page = p.pos / kPage;
  int blk = -1;
  if (page >= a.maxb) {
    p.flags |= kFlagBadPrefix;
  } else {
    blk = a.table[static_cast<int64_t>(p.b) * a.maxb + page];
    if (blk < 0 || blk >= a.num_blocks) {
      p.flags |= kFlagBadBlock;
      blk = -1;
    }
  }
  if (blk < 0) p.wanted = 0;
  return static_cast<int64_t>(blk) * a.Hkv + p.h;
}

SSD_DEV uint32_t larger_magnitude2(uint32_t a, uint32_t b) {  // of bf16 pairs, NaN if either is; the sign means nothing
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
SSD_DEV uint32_t largest16(const uint4 &x) {  // the largest magnitude of eight, as bits: they order like integers
  const uint32_t m = larger_magnitude2(larger_magnitude2(x.x, x.y), larger_magnitude2(x.z, x.w)) & 0x7FFF7FFFu;
  return max(m & 0xFFFFu, m >> 16);
}
SSD_DEV uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_append_q4(const __grid_constant__ AppendArgs a) {
  Pair p = pair_of<D, 1>(a.at, 0);
  uint4 x[2][2];  // [K or V][even or odd position]
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      x[o][r] = make_uint4(0, 0, 0, 0);
      if ((p.wanted >> r) & 1)
        x[o][r] = __ldg(reinterpret_cast<const uint4 *>(a.rows[o] + p.b * a.ss[o] + (p.i + r) * a.ts[o] +
                                                           static_cast<int64_t>(p.h) * D + p.e0));
    }
  // behind the rows: they are asked for while the table is read
  const int64_t unit = p.wanted ? unit_of(a.at, p) : 0;
  uint32_t flags = p.flags;
  const uint32_t wanted = p.wanted;
  const int e0 = p.e0;
  uint32_t byte[2][2];
  bool bad = false;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    // the group's largest, both positions at once
    uint32_t m = largest16(x[o][0]) | largest16(x[o][1]) << 16;
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t mr = r ? m >> 16 : m & 0xFFFFu;
      byte[o][r] = e8m0_of(mr);
      // exact, but for what is far below the smallest code
      const uint32_t inv = (254u - byte[o][r]) * 0x00800080u;
      if (mr >= 0x7F80u) {  // infinities or NaN: the whole group
        bad = true;
        byte[o][r] = kNanScaleByte;
        x[o][r] = make_uint4(0, 0, 0, 0);
      }
      uint4 &v = x[o][r];
      v = make_uint4(bmul2(v.x, inv), bmul2(v.y, inv), bmul2(v.z, inv), bmul2(v.w, inv));
    }
  }
  if (!wanted) {
    if (flags) atomicOr(a.at.status, flags);
    return;
  }
  if (bad) flags |= kFlagBadValue;
  constexpr int groups = D / kQ4Group;
  const int slot = static_cast<int>(p.pos % kPage);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (!((wanted >> r) & 1)) continue;
    const int64_t row = unit * kPage + slot + r;
    float f[8];
    EBF16::unpack(x[0][r], f);
    *reinterpret_cast<uint32_t *>(a.cache[0] + row * (D / 2) + e0 / 2) = e2m1_pack8(f);
    if ((e0 & (kQ4Group - 1)) == 0) {
      a.scale[0][row * groups + e0 / kQ4Group] = static_cast<uint8_t>(byte[0][r]);
      a.scale[1][row * groups + e0 / kQ4Group] = static_cast<uint8_t>(byte[1][r]);
    }
  }
  uint2 *const to = reinterpret_cast<uint2 *>(a.cache[1] + (unit * (kPage / 2) + slot / 2) * D + e0);
  uint2 v;
  {
    float f[2][8], y[8];
    EBF16::unpack(x[1][0], f[0]);
    EBF16::unpack(x[1][1], f[1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[2 * j] = f[0][j], y[2 * j + 1] = f[1][j];
    v.x = e2m1_pack8(y);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[2 * j] = f[0][4 + j], y[2 * j + 1] = f[1][4 + j];
    v.y = e2m1_pack8(y);
  }
  if (wanted != 3) {  // the other position's codes stay
    const uint32_t mine = wanted == 1 ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
    const uint2 old = *to;
    v.x = (v.x & mine) | (old.x & ~mine);
    v.y = (v.y & mine) | (old.y & ~mine);
  }
  *to = v;
  if (flags) atomicOr(a.at.status, flags);
}

template <bool BF16>
SSD_DEV void store8(void *out, int64_t at, const float *f) {
  if (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(f[2 * j + 1]), "f"(f[2 * j]));
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4 *const to = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
    to[0] = make_float4(f[0], f[1], f[2], f[3]);
    to[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

template <int D, bool BF16, int U>
__global__ void __launch_bounds__(kThreads) k_read_q4(const __grid_constant__ ReadArgs a) {
  constexpr int groups = D / kQ4Group;
  Pair p[U];
  int64_t row[U];
  uint32_t flags = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) p[u] = pair_of<D, U>(a.at, u);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    row[u] = p[u].wanted ? unit_of(a.at, p[u]) * kPage + p[u].pos % kPage : 0;
    flags |= p[u].flags;
  }
  if (flags) atomicOr(a.at.status, flags);
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    if (!a.out[o]) continue;
    uint2 w[U];          // K: eight codes of either position; V: eight bytes of both
    uint32_t scale[U];   // the bytes of the group, in the low and the next half
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = make_uint2(0, 0);
      scale[u] = 0;
      if (!p[u].wanted) continue;
      if (o == 0) {
        const uint8_t *const from = a.cache[0] + row[u] * (D / 2) + p[u].e0 / 2;
        w[u].x = __ldg(reinterpret_cast<const uint32_t *>(from));
        w[u].y = __ldg(reinterpret_cast<const uint32_t *>(from + D / 2));
      } else {
        w[u] = __ldg(reinterpret_cast<const uint2 *>(a.cache[1] + (row[u] / 2) * D + p[u].e0));
      }
      // both positions' scales are neighbours
      const int g = p[u].e0 / kQ4Group;
      if (groups == 4) {
        const uint2 b = __ldg(reinterpret_cast<const uint2 *>(a.scale[o] + row[u] * groups));
        scale[u] = ((b.x >> (8 * g)) & 255u) | ((b.y >> (8 * g)) & 255u) << 16;
      } else {
        const uint32_t b = __ldg(reinterpret_cast<const uint32_t *>(a.scale[o] + row[u] * groups));
        scale[u] = (b >> (8 * g)) & 0x00FF00FFu;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[2][8];
      uint32_t h[8];
      e2m1_halves8(w[u].x, h);
      e2m1_halves8(w[u].y, h + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (o == 0) half2_to_float(h[j], f[j >> 2][2 * (j & 3)], f[j >> 2][2 * (j & 3) + 1]);
        else half2_to_float(h[j], f[0][j], f[1][j]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (!((p[u].wanted >> r) & 1)) continue;
        const float s = e8m0_value((scale[u] >> (16 * r)) & 255u);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[r][j] = __fmul_rn(f[r][j], s);
        store8<BF16>(a.out[o], p[u].b * a.ss[o] + (p[u].i + r) * a.ts[o] + static_cast<int64_t>(p[u].h) * D + p[u].e0, f[r]);
      }
    }
  }
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// The arguments that both calls share; SSD_OK with grid = 0: nothing to do.
ssd_status_t place_of(Place &a, const int32_t *table, int maxb, int64_t num_blocks, const int32_t *prefix_len,
                      const int32_t *count, int node0, int B, int S, int Hkv, int d, uint32_t *status,
                      int each) {
  if (B < 0 || S < 0 || Hkv < 1 || d < 1 || node0 < 0 || maxb < 1 || num_blocks < 1) return SSD_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSD_ERR_UNSUPPORTED;
  a = Place{};
  if (B == 0 || S == 0) return SSD_OK;
  if (!table || !prefix_len || !status) return SSD_ERR_INVALID_ARG;
  const int64_t pairs = static_cast<int64_t>(S) / 2 + 1;
  if (pairs > 0x7fffffffLL / Hkv || pairs * Hkv > 0x7fffffffLL / B) return SSD_ERR_UNSUPPORTED;
  a.table = table;
  a.maxb = maxb;
  a.num_blocks = num_blocks;
  a.prefix_len = prefix_len;
  a.count = count;
  a.node0 = node0;
  a.S = S;
  a.Hkv = Hkv;
  a.items = static_cast<uint32_t>(pairs * Hkv);
  int bits = 0;  // 2^bits >= Hkv; magic = ceil(2^(31 + bits) / Hkv) fits 32 bits
  while ((1ll << bits) < Hkv) ++bits;
  a.magic = Hkv == 1 ? 0u : static_cast<uint32_t>(((1ull << (31 + bits)) + Hkv - 1) / Hkv);
  a.shift = bits - 1;
  const uint32_t per = kThreads / (d / 8);
  a.status = status;
  a.blocks = (a.items + per * each - 1) / (per * each);
  a.grid = static_cast<int64_t>(a.blocks) * B;
  return a.grid > 0x7fffffffLL ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

}  // namespace

extern "C" {

ssd_status_t ssd_kv_append_q4(const void *k_new, int64_t k_ss, int64_t k_ts, const void *v_new, int64_t v_ss,
                              int64_t v_ts, void *k_cache, void *v_cache, uint8_t *k_scale, uint8_t *v_scale,
                              const int32_t *block_table, int maxb, int64_t num_blocks, const int32_t *prefix_len,
                              const int32_t *count, int node0, int B, int S, int Hkv, int d, uint32_t *status,
                              ssd_stream_t s) {
  AppendArgs a{};
  const ssd_status_t st = place_of(a.at, block_table, maxb, num_blocks, prefix_len, count, node0, B, S, Hkv, d, status, 1);
  if (st != SSD_OK || a.at.grid == 0) return st;
  if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale) return SSD_ERR_INVALID_ARG;
  if (misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
      misaligned(k_scale, 16) || misaligned(v_scale, 16) || ((k_ss | k_ts | v_ss | v_ts) & 7))
    return SSD_ERR_UNSUPPORTED;
  a.rows[0] = static_cast<const uint16_t *>(k_new);
  a.rows[1] = static_cast<const uint16_t *>(v_new);
  a.ss[0] = k_ss, a.ts[0] = k_ts, a.ss[1] = v_ss, a.ts[1] = v_ts;
  a.cache[0] = static_cast<uint8_t *>(k_cache);
  a.cache[1] = static_cast<uint8_t *>(v_cache);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  void (*const kernel)(AppendArgs) = d == 64 ? k_append_q4<64> : k_append_q4<128>;
  kernel<<<static_cast<unsigned>(a.at.grid), kThreads, 0, reinterpret_cast<cudaStream_t>(s)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_kv_read_q4(const void *k_cache, const void *v_cache, const uint8_t *k_scale, const uint8_t *v_scale,
                            const int32_t *block_table, int maxb, int64_t num_blocks, const int32_t *prefix_len,
                            const int32_t *count, int node0, void *k_out, int64_t ko_ss, int64_t ko_ts, void *v_out,
                            int64_t vo_ss, int64_t vo_ts, ssd_dtype_t dt, int B, int S, int Hkv, int d,
                            uint32_t *status, ssd_stream_t s) {
  if (dt != SSD_F32 && dt != SSD_BF16) return SSD_ERR_INVALID_ARG;
  ReadArgs a{};
  const int each = (static_cast<int64_t>(S) / 2 + 1) * Hkv > kFewItems / (B > 0 ? B : 1) ? 2 : 1;
  const ssd_status_t st = place_of(a.at, block_table, maxb, num_blocks, prefix_len, count, node0, B, S, Hkv, d, status, each);
  if (st != SSD_OK || a.at.grid == 0) return st;
  if (!k_out && !v_out) return SSD_OK;
  if ((k_out && (!k_cache || !k_scale)) || (v_out && (!v_cache || !v_scale))) return SSD_ERR_INVALID_ARG;
  const int64_t step = dt == SSD_BF16 ? 7 : 3;
  if (misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(k_scale, 16) || misaligned(v_scale, 16) ||
      misaligned(k_out, 16) || misaligned(v_out, 16) || (k_out && ((ko_ss | ko_ts) & step)) ||
      (v_out && ((vo_ss | vo_ts) & step)))
    return SSD_ERR_UNSUPPORTED;
  a.cache[0] = static_cast<const uint8_t *>(k_cache);
  a.cache[1] = static_cast<const uint8_t *>(v_cache);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.ss[0] = ko_ss, a.ts[0] = ko_ts, a.ss[1] = vo_ss, a.ts[1] = vo_ts;
  auto kernel = [&](auto bf16) {
    constexpr bool B16 = decltype(bf16)::value;
    return d == 64 ? (each == 1 ? k_read_q4<64, B16, 1> : k_read_q4<64, B16, 2>)
                   : (each == 1 ? k_read_q4<128, B16, 1> : k_read_q4<128, B16, 2>);
  };
  void (*const run)(ReadArgs) = dt == SSD_BF16 ? kernel(std::true_type{}) : kernel(std::false_type{});
  run<<<static_cast<unsigned>(a.at.grid), kThreads, 0, reinterpret_cast<cudaStream_t>(s)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
