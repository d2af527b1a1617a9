// attention_q4.cu -- tree-masked decode attention over a paged K/V cache held
// in 4 bits (e2m1 codes, a power-of-two scale byte per 32 elements of a token and
// head): out = softmax(scale q k^T + mask) v.
//
// One warp per query row and head, a key at a time, with the running maximum
// and sum of a softmax; a lane holds d / 32 elements of q, k, v and the output.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <cmath>

#include "../../include/ssd.h"
#include "common.cuh"
#include "device_info.h"
#include "e2m1.cuh"
#include "e4m3.cuh"

namespace {

using namespace ssd;

constexpr int kPage = 16;
constexpr int kMaxNodes = 128;
constexpr int kWarps = 4;

struct Args {
  const uint16_t *q;
  const uint8_t *kc, *vc, *ks, *vs;
  const int32_t *table;
  int maxb;
  int64_t num_blocks;
  const int32_t *prefix_len, *parent;
  int B, N, Nq, Hq, Hkv;
  float scale;
  uint16_t *out;
  float *lse;
  uint32_t *status;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_attn_q4_rows(const __grid_constant__ Args a) {
  constexpr int E = D / 32;  // elements of a lane
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (r >= static_cast<int64_t>(a.B) * a.Nq * a.Hq) return;
  const int head = static_cast<int>(r % a.Hq);
  const int64_t bq = r / a.Hq;
  const int qi = static_cast<int>(bq % a.Nq), b = static_cast<int>(bq / a.Nq);
  const int hk = head / (a.Hq / a.Hkv);
  const float NEG_INF = -__int_as_float(0x7f800000);
  uint32_t flags = 0;
  const int prefix = a.prefix_len[b], L = max(prefix, 0);
  int64_t keys = static_cast<int64_t>(L) + a.N;
  if (prefix == -1) {
    keys = 0;
  } else {
    if (prefix < 0 || keys > static_cast<int64_t>(a.maxb) * kPage) flags |= kFlagBadPrefix;
    keys = min(keys, static_cast<int64_t>(a.maxb) * kPage);
  }
  uint32_t path[kMaxNodes / 32] = {};
  if (keys > 0)
    for (int m = a.N - a.Nq + qi; m >= 0;) {
      path[m >> 5] |= 1u << (m & 31);
      const int up = a.parent[static_cast<int64_t>(b) * a.N + m];
      if (up < -1 || up >= m) {
        flags |= kFlagBadTree;
        break;
      }
      m = up;
    }
  float q[E], o[E], m = NEG_INF, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float(static_cast<uint32_t>(a.q[r * D + lane * E + e]) << 16) * a.scale;
    o[e] = 0.f;
  }
  const int group = lane * E / kQ4Group;
  for (int64_t k = 0; k < keys; ++k) {
    const int node = k < L ? -1 : static_cast<int>(k - L);
    const int blk = a.table[static_cast<int64_t>(b) * a.maxb + k / kPage];
    if (blk < 0 || blk >= a.num_blocks) {
      flags |= kFlagBadBlock;
      continue;
    }
    if (node >= 0 && !((path[node >> 5] >> (node & 31)) & 1u)) continue;
    const int64_t row = (static_cast<int64_t>(blk) * a.Hkv + hk) * kPage + k % kPage;
    const float ks = e8m0_value(a.ks[row * (D / kQ4Group) + group]);
    const uint32_t vb = a.vs[row * (D / kQ4Group) + group];
    const float vs = vb < kMinScaleByte ? 0.f : e8m0_value(vb);
    float kf[E], vf[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = lane * E + e;
      const uint32_t kb = a.kc[row * (D / 2) + at / 2] >> (at & 1) * 4;
      const uint32_t vb4 = a.vc[(row / 2) * D + at] >> (row & 1) * 4;
      uint32_t h[4];
      e2m1_halves8((kb & 15u) | (vb4 & 15u) << 4, h);
      half2_to_float(h[0], kf[e], vf[e]);
    }
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], kf[e] * ks, x);
    x = warp_sum(x);
    const float mn = x > m ? x : m;
    const float f = m == NEG_INF ? 0.f : expf(m - mn), p = expf(x - mn);
    m = mn;
    const float kept = l * f;
    l = kept + p;
    // the weighted mean so far: a sum of values near fp32's largest would pass it
    const float wo = kept / l, wv = p / l;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * wo + wv * (vf[e] * vs);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(0.f), "f"(o[e]));
    a.out[r * D + lane * E + e] = static_cast<uint16_t>(w & 0xFFFFu);
  }
  if (lane == 0) {
    if (a.lse) a.lse[r] = l == 0.f ? NEG_INF : m + logf(l);
    if (flags) atomicOr(a.status, flags);
  }
}

}  // namespace

extern "C" {

size_t ssd_attention_q4_workspace_size(int B, int Nq, int Hq, int Hkv, int d) {
  if (B <= 0 || Nq <= 0 || Nq > kMaxNodes || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 16 ||
      (d != 64 && d != 128))
    return 0;
  return 256;
}

ssd_status_t ssd_branch_attention_q4(const void *q, const void *k_cache, const void *v_cache, const uint8_t *k_scale,
                                     const uint8_t *v_scale, const int32_t *block_table, int maxb, int64_t num_blocks,
                                     const int32_t *prefix_len, const int32_t *parent, int B, int N, int Nq, int Hq,
                                     int Hkv, int d, float scale, void *out, float *lse, uint32_t *status, void *ws,
                                     size_t ws_bytes, ssd_stream_t s) {
  (void)ws;
  (void)ws_bytes;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return SSD_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return SSD_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSD_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16 || N < 1 || N > kMaxNodes || Nq < 1 || Nq > N) return SSD_ERR_UNSUPPORTED;
  if (B == 0) return SSD_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len || !parent || !out ||
      !status || maxb < 1 || num_blocks < 1)
    return SSD_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(k_scale) |
       reinterpret_cast<uintptr_t>(v_scale)) & 15u ||
      (reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 31u)
    return SSD_ERR_UNSUPPORTED;
  if (num_blocks > 0x7fffffffLL || static_cast<int64_t>(B) * Hkv > 0x7fffffffLL / 32) return SSD_ERR_UNSUPPORTED;
  const int64_t row_tiles = (static_cast<int64_t>(Hq / Hkv) * Nq + 127) / 128;
  if (static_cast<int64_t>(maxb) * B * Hkv * row_tiles / 16 / attn_num_sms() > 0x3fffffff) return SSD_ERR_UNSUPPORTED;
  Args a{static_cast<const uint16_t *>(q), static_cast<const uint8_t *>(k_cache), static_cast<const uint8_t *>(v_cache),
         k_scale, v_scale, block_table, maxb, num_blocks, prefix_len, parent, B, N, Nq, Hq, Hkv, scale,
         static_cast<uint16_t *>(out), lse, status};
  const int64_t rows = static_cast<int64_t>(B) * Nq * Hq, grid = (rows + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  if (d == 64)
    k_attn_q4_rows<64><<<static_cast<unsigned>(grid), kWarps * 32, 0, cs>>>(a);
  else
    k_attn_q4_rows<128><<<static_cast<unsigned>(grid), kWarps * 32, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
