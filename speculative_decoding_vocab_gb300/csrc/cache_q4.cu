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
// Bound by HBM for prompts, by the chain prefix -> block table -> block for a decode step.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "common.cuh"
#include "e2m1.cuh"
#include "e4m3.cuh"

namespace {

using namespace ssd;

constexpr int kThreads = 256;
constexpr int kPage = 16;

struct Place {  // which rows, and where their blocks are
  const int32_t *table;
  int maxb;
  int64_t num_blocks;
  const int32_t *prefix_len, *count;
  int node0, S, Hkv, d, pairs;  // pairs: pairs of positions that a sequence's rows may touch
  int64_t threads;
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
  uint32_t wanted;    // bit 0 the even position, bit 1 the odd one
  int64_t unit;       // block * Hkv + head
  int slot;           // of the even position in its block
  uint32_t flags;
};
SSD_DEV Pair pair_of(const Place &a) {
  Pair p;
  p.wanted = 0;
  p.flags = 0;
  p.unit = 0;
  p.slot = 0;
  p.i = 0;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int pieces = a.d / 8;
  // neighbouring lanes take neighbouring pieces, then heads (adjacent in a token's row)
  const int64_t g1 = g / pieces, g2 = g1 / a.Hkv;
  p.e0 = static_cast<int>(g - g1 * pieces) * 8;
  p.h = static_cast<int>(g1 - g2 * a.Hkv);
  const int64_t b = g2 / a.pairs;
  const int64_t w = g2 - b * a.pairs;
  p.b = static_cast<int>(b);
  if (g >= a.threads) return p;
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
  const int64_t pos = (first & ~int64_t(1)) + 2 * w;
  p.i = pos - first;
  uint32_t want = 0;
  if (p.i >= 0 && p.i < count) want |= 1;
  if (p.i + 1 < count) want |= 2;  // i + 1 >= 0
  if (!want) return p;
  const int64_t page = pos / kPage;
  if (page >= a.maxb) {
    p.flags |= kFlagBadPrefix;
    return p;
  }
  const int blk = a.table[b * a.maxb + page];
  if (blk < 0 || blk >= a.num_blocks) {
    p.flags |= kFlagBadBlock;
    return p;
  }
  p.wanted = want;
  p.unit = static_cast<int64_t>(blk) * a.Hkv + p.h;
  p.slot = static_cast<int>(pos % kPage);
  return p;
}

SSD_DEV uint32_t largest16(const uint4 &x) {  // bf16 magnitudes order like integers
  const uint32_t m = max_u16x2(max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                               max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

__global__ void __launch_bounds__(kThreads) k_append_q4(const __grid_constant__ AppendArgs a) {
  const Pair p = pair_of(a.at);
  const int d = a.at.d;
  uint32_t flags = p.flags;
  uint4 x[2][2];  // [K or V][even or odd position]
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      x[o][r] = make_uint4(0, 0, 0, 0);
      if ((p.wanted >> r) & 1)
        x[o][r] = __ldg(reinterpret_cast<const uint4 *>(a.rows[o] + p.b * a.ss[o] + (p.i + r) * a.ts[o] +
                                                        static_cast<int64_t>(p.h) * d + p.e0));
    }
  int byte[2][2];
  float f[2][2][8];
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t m = largest16(x[o][r]);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      int b = e8m0_of(m << 16);
      EBF16::unpack(x[o][r], f[o][r]);
      const float inv = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[o][r][j] = __fmul_rn(f[o][r][j], inv);
      if (m >= 0x7F80u) {  // infinities or NaN: the whole group
        flags |= kFlagBadValue;
        b = kNanScaleByte;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[o][r][j] = 0.f;
      }
      byte[o][r] = b;
    }
  if (p.wanted) {
    const int groups = d / kQ4Group;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!((p.wanted >> r) & 1)) continue;
      const int64_t row = p.unit * kPage + p.slot + r;
      *reinterpret_cast<uint32_t *>(a.cache[0] + row * (d / 2) + p.e0 / 2) = e2m1_pack8(f[0][r]);
      if ((p.e0 & (kQ4Group - 1)) == 0) {
        a.scale[0][row * groups + p.e0 / kQ4Group] = static_cast<uint8_t>(byte[0][r]);
        a.scale[1][row * groups + p.e0 / kQ4Group] = static_cast<uint8_t>(byte[1][r]);
      }
    }
    uint2 *const to = reinterpret_cast<uint2 *>(a.cache[1] + (p.unit * (kPage / 2) + p.slot / 2) * d + p.e0);
    uint2 v;
    {
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[2 * j] = f[1][0][j], y[2 * j + 1] = f[1][1][j];
      v.x = e2m1_pack8(y);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[2 * j] = f[1][0][4 + j], y[2 * j + 1] = f[1][1][4 + j];
      v.y = e2m1_pack8(y);
    }
    if (p.wanted != 3) {  // the other position's codes stay
      const uint32_t mine = p.wanted == 1 ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
      const uint2 old = *to;
      v.x = (v.x & mine) | (old.x & ~mine);
      v.y = (v.y & mine) | (old.y & ~mine);
    }
    *to = v;
  }
  if (flags) atomicOr(a.at.status, p.wanted ? flags : flags & ~kFlagBadValue);
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

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_read_q4(const __grid_constant__ ReadArgs a) {
  const Pair p = pair_of(a.at);
  const int d = a.at.d, groups = d / kQ4Group;
  if (p.flags) atomicOr(a.at.status, p.flags);
  if (!p.wanted) return;
  const int64_t row = p.unit * kPage + p.slot;
  float f[2][8];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    if (!a.out[o]) continue;
    if (o == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(a.cache[0] + (row + r) * (d / 2) + p.e0 / 2));
        uint32_t h[4];
        e2m1_halves8(w, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) half2_to_float(h[j], f[r][2 * j], f[r][2 * j + 1]);
      }
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2 *>(a.cache[1] + (row / 2) * d + p.e0));
      uint32_t h[8];
      e2m1_halves8(w.x, h);
      e2m1_halves8(w.y, h + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) half2_to_float(h[j], f[0][j], f[1][j]);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!((p.wanted >> r) & 1)) continue;
      const float s = e8m0_value(a.scale[o][(row + r) * groups + p.e0 / kQ4Group]);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[r][j] = __fmul_rn(f[r][j], s);
      store8<BF16>(a.out[o], p.b * a.ss[o] + (p.i + r) * a.ts[o] + static_cast<int64_t>(p.h) * d + p.e0, f[r]);
    }
  }
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// The arguments that both calls share; SSD_OK with threads = 0: nothing to do.
ssd_status_t place_of(Place &a, const int32_t *table, int maxb, int64_t num_blocks, const int32_t *prefix_len,
                      const int32_t *count, int node0, int B, int S, int Hkv, int d, uint32_t *status) {
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
  a.d = d;
  a.pairs = static_cast<int>(pairs);
  a.threads = static_cast<int64_t>(B) * pairs * Hkv * (d / 8);
  a.status = status;
  return SSD_OK;
}
unsigned grid_of(const Place &a) { return static_cast<unsigned>((a.threads + kThreads - 1) / kThreads); }

}  // namespace

extern "C" {

ssd_status_t ssd_kv_append_q4(const void *k_new, int64_t k_ss, int64_t k_ts, const void *v_new, int64_t v_ss,
                              int64_t v_ts, void *k_cache, void *v_cache, uint8_t *k_scale, uint8_t *v_scale,
                              const int32_t *block_table, int maxb, int64_t num_blocks, const int32_t *prefix_len,
                              const int32_t *count, int node0, int B, int S, int Hkv, int d, uint32_t *status,
                              ssd_stream_t s) {
  AppendArgs a{};
  const ssd_status_t st = place_of(a.at, block_table, maxb, num_blocks, prefix_len, count, node0, B, S, Hkv, d, status);
  if (st != SSD_OK || a.at.threads == 0) return st;
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
  k_append_q4<<<grid_of(a.at), kThreads, 0, reinterpret_cast<cudaStream_t>(s)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_kv_read_q4(const void *k_cache, const void *v_cache, const uint8_t *k_scale, const uint8_t *v_scale,
                            const int32_t *block_table, int maxb, int64_t num_blocks, const int32_t *prefix_len,
                            const int32_t *count, int node0, void *k_out, int64_t ko_ss, int64_t ko_ts, void *v_out,
                            int64_t vo_ss, int64_t vo_ts, ssd_dtype_t dt, int B, int S, int Hkv, int d,
                            uint32_t *status, ssd_stream_t s) {
  if (dt != SSD_F32 && dt != SSD_BF16) return SSD_ERR_INVALID_ARG;
  ReadArgs a{};
  const ssd_status_t st = place_of(a.at, block_table, maxb, num_blocks, prefix_len, count, node0, B, S, Hkv, d, status);
  if (st != SSD_OK || a.at.threads == 0) return st;
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
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  if (dt == SSD_BF16)
    k_read_q4<true><<<grid_of(a.at), kThreads, 0, cs>>>(a);
  else
    k_read_q4<false><<<grid_of(a.at), kThreads, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
