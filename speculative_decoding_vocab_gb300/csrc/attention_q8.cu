// attention_q8.cu -- tree-masked decode attention over a paged K/V cache held
// in 8 bits (e4m3 codes, one scale per block of 16 positions and KV head).
//
//   k_branch_attn_q8   one CTA per (sequence, query node, head): a thread per
//                      key for the scores, a thread per element for the
//                      output, an online softmax over tiles of 128 keys.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <cmath>

#include "../../include/ssd.h"
#include "common.cuh"
#include "e4m3.cuh"

namespace {

using namespace ssd;

constexpr int kPage = 16;
constexpr int kMaxNodes = 128;
constexpr int kKeys = 128;

struct AttnArgs {
  const uint16_t *q;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int32_t *table;
  int maxb;
  int64_t num_blocks;
  const int32_t *prefix_len, *parent;
  int N, Nq, Hq, Hkv, group;
  float scale_log2;
  uint16_t *out;
  float *lse;
  uint32_t *status;
};

SSD_DEV float code_value(uint8_t c) {
  float lo, hi;
  half2_to_float(e4m3_to_half2(c), lo, hi);
  return lo;
}

template <int D>
__global__ void __launch_bounds__(kKeys) k_branch_attn_q8(AttnArgs a) {
  __shared__ float sq[D], sp[kKeys], sw[kKeys], red[kKeys / 32 + 1];
  __shared__ int sblk[kKeys / kPage];
  __shared__ uint32_t anc[kMaxNodes / 32];
  const int tid = threadIdx.x;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int64_t row = blockIdx.x;  // (b, qi, h)
  const int h = static_cast<int>(row % a.Hq);
  const int64_t bq = row / a.Hq;
  const int qi = static_cast<int>(bq % a.Nq), b = static_cast<int>(bq / a.Nq);
  const int hk = h / a.group;
  const int L_in = a.prefix_len[b], L = max(L_in, 0);
  const int64_t nkeys64 = static_cast<int64_t>(L) + a.N;
  const int64_t cap = static_cast<int64_t>(a.maxb) * kPage;
  if (tid == 0) {
    if (L_in < 0 || nkeys64 > cap) atomicOr(a.status, kFlagBadPrefix);
    for (int w = 0; w < kMaxNodes / 32; ++w) anc[w] = 0;
    for (int m = a.N - a.Nq + qi; m >= 0;) {
      anc[m >> 5] |= 1u << (m & 31);
      const int up = a.parent[static_cast<int64_t>(b) * a.N + m];
      if (up < -1 || up >= m) {
        atomicOr(a.status, kFlagBadTree);
        break;
      }
      m = up;
    }
  }
  bool bad_q = false;
  for (int e = tid; e < D; e += kKeys) {
    sq[e] = __uint_as_float(static_cast<uint32_t>(a.q[row * D + e]) << 16);
    bad_q |= !(fabsf(sq[e]) <= 3.402823466e38f);
  }
  bad_q = __syncthreads_or(bad_q) != 0;
  const int64_t nkeys = nkeys64 < cap ? nkeys64 : cap;
  float m = NEG_INF, l = 0.f, o = 0.f;
  for (int64_t t = 0; t < nkeys; t += kKeys) {
    __syncthreads();
    if (tid < kKeys / kPage) {
      const int64_t p = t / kPage + tid;
      int blk = -1;
      if (p < a.maxb && p * kPage < nkeys) {
        blk = a.table[static_cast<int64_t>(b) * a.maxb + p];
        if (blk < 0 || blk >= a.num_blocks) {
          atomicOr(a.status, kFlagBadBlock);
          blk = -1;
        } else if (!good_scale(a.ks[static_cast<int64_t>(blk) * a.Hkv + hk]) ||
                   !good_scale(a.vs[static_cast<int64_t>(blk) * a.Hkv + hk])) {
          atomicOr(a.status, kFlagBadValue);
          blk = -1;
        }
      }
      sblk[tid] = blk;
    }
    __syncthreads();
    const int64_t key = t + tid;
    const int blk = sblk[tid / kPage];
    bool vis = blk >= 0 && key < nkeys;
    if (vis && key >= L) {
      const int n = static_cast<int>(key - L);
      vis = (anc[n >> 5] >> (n & 31)) & 1u;
    }
    float x = NEG_INF;
    sw[tid] = 0.f;
    if (vis) {
      const int64_t unit = static_cast<int64_t>(blk) * a.Hkv + hk;
      const uint8_t *k = a.kc + (unit * kPage + key % kPage) * D;
      float s = 0.f;
      for (int e = 0; e < D; e += 4) {
        float f[4];
        e4m3_unpack4(*reinterpret_cast<const uint32_t *>(k + e), f);
        for (int i = 0; i < 4; ++i) s = fmaf(sq[e + i], f[i], s);
      }
      x = s * (a.ks[unit] * a.scale_log2);
      const float vsc = a.vs[unit];
      sw[tid] = vsc < kMinBlockScale ? 0.f : vsc;
    }
    const float wmax = warp_max(x);  // fmaxf leaves NaN out
    if ((tid & 31) == 0) red[tid >> 5] = wmax;
    __syncthreads();
    float top = red[0];
    for (int w = 1; w < kKeys / 32; ++w) top = fmaxf(top, red[w]);
    const float m_new = fmaxf(m, top);
    const float f = m == NEG_INF ? 0.f : ex2(m - m_new);
    const float p = vis ? ex2(x - (m_new == NEG_INF ? 0.f : m_new)) : 0.f;
    sp[tid] = p;
    __syncthreads();
    const float wsum = warp_sum(p);
    if ((tid & 31) == 0) red[tid >> 5] = wsum;
    __syncthreads();
    l = l * f + (red[0] + red[1] + red[2] + red[3]);
    m = m_new;
    if (tid < D) {
      o *= f;
      for (int j = 0; j < kKeys; ++j) {
        if (sp[j] == 0.f) continue;  // hidden
        const int64_t unit = static_cast<int64_t>(sblk[j / kPage]) * a.Hkv + hk;
        o = fmaf(sp[j] * sw[j], code_value(a.vc[(unit * kPage + (t + j) % kPage) * D + tid]), o);
      }
    }
  }
  if (tid < D) {
    const float y = bad_q ? __int_as_float(0x7fc00000) : (l > 0.f || l != l ? o / l : 0.f);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(y));
    a.out[row * D + tid] = static_cast<uint16_t>(r & 0xFFFFu);
  }
  if (tid == 0 && a.lse)
    a.lse[row] = bad_q || l != l ? __int_as_float(0x7fc00000) : (l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : NEG_INF);
}

}  // namespace

extern "C" {

size_t ssd_attention_q8_workspace_size(int B, int Nq, int Hq, int Hkv, int d) {
  if (B <= 0 || Nq <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (d != 64 && d != 128)) return 0;
  return 0;
}

ssd_status_t ssd_branch_attention_q8(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                                     const float *v_scale, const int32_t *block_table, int maxb, int64_t num_blocks,
                                     const int32_t *prefix_len, const int32_t *parent, int B, int N, int Nq, int Hq,
                                     int Hkv, int d, float scale, void *out, float *lse, uint32_t *status, void *ws,
                                     size_t ws_bytes, ssd_stream_t s) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return SSD_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return SSD_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSD_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16 || N < 1 || N > kMaxNodes || Nq < 1 || Nq > N) return SSD_ERR_UNSUPPORTED;
  if (B == 0) return SSD_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len || !parent || !out ||
      !status || maxb < 1 || num_blocks < 1)
    return SSD_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(out)) & 15u)
    return SSD_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(B) * Nq * Hq;
  if (rows > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
  AttnArgs a{};
  a.q = static_cast<const uint16_t *>(q);
  a.kc = static_cast<const uint8_t *>(k_cache);
  a.vc = static_cast<const uint8_t *>(v_cache);
  a.ks = k_scale;
  a.vs = v_scale;
  a.table = block_table;
  a.maxb = maxb;
  a.num_blocks = num_blocks;
  a.prefix_len = prefix_len;
  a.parent = parent;
  a.N = N;
  a.Nq = Nq;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.status = status;
  (void)ws;
  (void)ws_bytes;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  if (d == 64)
    k_branch_attn_q8<64><<<static_cast<unsigned>(rows), kKeys, 0, cs>>>(a);
  else
    k_branch_attn_q8<128><<<static_cast<unsigned>(rows), kKeys, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
