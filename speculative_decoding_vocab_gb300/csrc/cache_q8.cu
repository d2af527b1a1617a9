// cache_q8.cu -- the append into a paged K/V cache held in 8 bits, with one
// scale for each block of 16 positions and KV head.
//
// need = the smallest power of two that brings the block's new rows under
// 448; scale' = max(scale, need) where the block already holds rows.  Powers
// of two cost e4m3 nothing (its relative step is the same in every binade;
// only one of its 17 binades of range can be lost), make x / scale' exact, and
// let rows that move to a larger scale keep their bits unless they underflow.
//
//   k_kv_append_q8   one warp per (block, head, K or V): it holds the block's
//                    new rows in registers (16 x d values, 16-byte loads all
//                    in flight), takes their maximum as 16-bit integers, and
//                    writes codes; rows that the block held before are
//                    rewritten only when the scale grew.
// Bound by HBM for prompts (2 bytes read and 1 written per value), by the
// chain prefix -> block table -> block for a decode step.  8 prompts of 4096 to
// 8191 tokens, 8 heads of 128 (302 MB): 55 us, 5.5 TB/s; a decode step of 256
// tokens: 2.7 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "common.cuh"
#include "e4m3.cuh"

namespace {

using namespace ssd;

constexpr int kThreads = 128;
constexpr int kPage = 16;

struct Operand {
  const uint16_t *rows;
  int64_t ss, ts;  // strides between sequences and tokens, elements
  uint8_t *cache;
  float *scale;
};
struct AppendArgs {
  Operand kv[2];
  const int32_t *table;
  int maxb;
  int64_t num_blocks;
  const int32_t *prefix_len, *count;
  int node0, S, Hkv, windows;  // windows: blocks a sequence's rows may touch
  int64_t warps;
  uint32_t *status;
};

// the smallest power of two s >= 2^-100 with amax <= 448 s (448 = 1.75 * 2^8)
SSD_DEV float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // biased exponent of s
  e = max(e, 27);                                                                // 2^-100
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_append_q8(const __grid_constant__ AppendArgs a) {
  constexpr int kLanes = D / 8;         // lanes per row: 8 values each
  constexpr int kRows = 32 / kLanes;    // rows per pass
  constexpr int kPasses = kPage / kRows;
  const int lane = threadIdx.x & 31;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (g >= a.warps) return;
  // neighbouring warps take neighbouring heads (adjacent rows in memory), then K and V
  const int h = static_cast<int>(g % a.Hkv);
  const int64_t g1 = g / a.Hkv;
  const int which = static_cast<int>(g1 & 1);
  const int64_t g2 = g1 >> 1;
  const int win = static_cast<int>(g2 % a.windows), b = static_cast<int>(g2 / a.windows);
  const Operand o = which ? a.kv[1] : a.kv[0];
  uint32_t flags = 0;
  const int L = a.prefix_len[b];
  int count = a.S;
  if (a.count) {
    const int c = a.count[b];
    count = min(max(c, 0), a.S);
    if (c != count) flags |= kFlagBadPrefix;
  }
  if (L < 0) {
    if (L != -1 && lane == 0 && win == 0) atomicOr(a.status, flags | kFlagBadPrefix);  // -1: a slot without a request
    return;
  }
  const int64_t first = static_cast<int64_t>(L) + a.node0;  // position of row 0
  const int64_t page = first / kPage + win;
  const int64_t rel0 = page * kPage - first;  // row at the block's first position (negative: older positions)
  if (count == 0 || rel0 >= count) {  // no new row here
    if (lane == 0 && flags && win == 0) atomicOr(a.status, flags);
    return;
  }
  const int lr = lane / kLanes, e0 = (lane % kLanes) * 8;
  uint4 x[kPasses];
  uint32_t is_new = 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t rel = rel0 + p * kRows + lr;
    x[p] = make_uint4(0, 0, 0, 0);
    if (rel >= 0 && rel < count) {
      is_new |= 1u << p;
      x[p] = __ldg(reinterpret_cast<const uint4 *>(o.rows + b * o.ss + rel * o.ts + static_cast<int64_t>(h) * D + e0));
    }
  }
  int64_t blk = -1;
  if (page >= a.maxb) {
    flags |= kFlagBadPrefix;
  } else {
    blk = a.table[static_cast<int64_t>(b) * a.maxb + page];
    if (blk < 0 || blk >= a.num_blocks) {
      flags |= kFlagBadBlock;
      blk = -1;
    }
  }
  if (blk < 0) {
    if (lane == 0) atomicOr(a.status, flags);
    return;
  }
  const int64_t unit = blk * a.Hkv + h;
  const int held = rel0 < 0 ? static_cast<int>(min(static_cast<int64_t>(kPage), -rel0)) : 0;  // older rows
  float old = 0.f;
  if (held > 0) {
    old = o.scale[unit];
    if (!good_scale(old)) {
      flags |= kFlagBadValue;
      old = 0.f;
    }
  }
  // largest magnitude of the new rows: bf16 magnitudes order like integers
  uint32_t m2 = 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    m2 = max_u16x2(m2, max_u16x2(max_u16x2(x[p].x & 0x7FFF7FFFu, x[p].y & 0x7FFF7FFFu),
                                 max_u16x2(x[p].z & 0x7FFF7FFFu, x[p].w & 0x7FFF7FFFu)));
  }
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  if (__any_sync(0xffffffffu, m >= 0x7F80u)) {  // infinities or NaN: left out of the maximum, stored as NaN
    flags |= kFlagBadValue;
    m = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = w[q] & 0x7FFFu, hi = (w[q] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) m = max(m, lo);
        else w[q] = (w[q] & 0xFFFF0000u) | 0x7FC0u;
        if (hi < 0x7F80u) m = max(m, hi);
        else w[q] = (w[q] & 0xFFFFu) | 0x7FC00000u;
      }
      x[p] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
  const float need = pow2_scale(__uint_as_float(m << 16));
  const float at = fmaxf(old, need);
  uint8_t *const dst = o.cache + unit * (kPage * D);
  const bool grew = held > 0 && at != old;
  // x / at: by the exact reciprocal of a power of two, else (a scale that another program wrote) by division
  const bool pow2 = (__float_as_uint(at) & 0x7FFFFFu) == 0 && at <= 0x1p126f;
  const float inv = 1.f / at;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int r = p * kRows + lr;
    uint2 *const to = reinterpret_cast<uint2 *>(dst + r * D + e0);
    if ((is_new >> p) & 1u) {
      float f[8];
      EBF16::unpack(x[p], f);
      if (pow2) {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = __fmul_rn(f[q], inv);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = __fdiv_rn(f[q], at);
      }
      *to = make_uint2(e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16),
                       e4m3_pair(f[4], f[5]) | (e4m3_pair(f[6], f[7]) << 16));
    } else if (grew && r < held) {
      const uint2 c = *to;
      float f[8];
      e4m3_unpack4(c.x, f);
      e4m3_unpack4(c.y, f + 4);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = __fdiv_rn(__fmul_rn(f[q], old), at);
      *to = make_uint2(e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16),
                       e4m3_pair(f[4], f[5]) | (e4m3_pair(f[6], f[7]) << 16));
    }
  }
  if (lane == 0) {
    if (held == 0 || grew) o.scale[unit] = at;
    if (flags) atomicOr(a.status, flags);
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

extern "C" ssd_status_t ssd_kv_append_q8(const void *k_new, int64_t k_ss, int64_t k_ts, const void *v_new,
                                         int64_t v_ss, int64_t v_ts, void *k_cache, void *v_cache, float *k_scale,
                                         float *v_scale, const int32_t *block_table, int maxb, int64_t num_blocks,
                                         const int32_t *prefix_len, const int32_t *count, int node0, int B, int S,
                                         int Hkv, int d, uint32_t *status, ssd_stream_t s) {
  if (B < 0 || S < 0 || Hkv < 1 || d < 1 || node0 < 0 || maxb < 1 || num_blocks < 1) return SSD_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSD_ERR_UNSUPPORTED;
  if (B == 0 || S == 0) return SSD_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len || !status)
    return SSD_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      ((k_ss | k_ts | v_ss | v_ts) & 7))
    return SSD_ERR_UNSUPPORTED;
  AppendArgs a{};
  a.kv[0] = {static_cast<const uint16_t *>(k_new), k_ss, k_ts, static_cast<uint8_t *>(k_cache), k_scale};
  a.kv[1] = {static_cast<const uint16_t *>(v_new), v_ss, v_ts, static_cast<uint8_t *>(v_cache), v_scale};
  a.table = block_table;
  a.maxb = maxb;
  a.num_blocks = num_blocks;
  a.prefix_len = prefix_len;
  a.count = count;
  a.node0 = node0;
  a.S = S;
  a.Hkv = Hkv;
  a.windows = static_cast<int>((static_cast<int64_t>(S) + kPage - 2) / kPage + 1);
  a.warps = static_cast<int64_t>(B) * a.windows * 2 * Hkv;
  a.status = status;
  const int64_t grid = (a.warps + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  if (d == 64)
    k_kv_append_q8<64><<<static_cast<unsigned>(grid), kThreads, 0, cs>>>(a);
  else
    k_kv_append_q8<128><<<static_cast<unsigned>(grid), kThreads, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
