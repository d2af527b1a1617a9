// logprobs.cu -- log probabilities of given tokens, with their rank, the row's
// entropy and its likeliest tokens.
//
// One CTA per row: its maximum, then the sums around it, then the n first
// tokens one after the other.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "common.cuh"

namespace {

using namespace ssd;

constexpr int kThreads = 512;
constexpr int kMaxTop = 64;

struct Args {
  const void *z;
  int64_t ss, rs;
  int R, V, n;
  float T;
  const int32_t *tokens;
  float *logprob, *entropy, *top_logprob;
  int32_t *rank, *top_ids;
  uint32_t *status;
};

template <class E>
__global__ void __launch_bounds__(kThreads) k_token_logprobs(const __grid_constant__ Args a) {
  __shared__ float red[kThreads / 32];
  __shared__ uint64_t best[kThreads / 32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int t = a.tokens ? a.tokens[row] : 0;
  if (t == -1) return;
  const bool good = t >= 0 && t < a.V;
  const char *const z = static_cast<const char *>(a.z) + ((row / a.R) * a.ss + (row % a.R) * a.rs) * E::kSize;
  const float INF = __int_as_float(0x7f800000), NAN_ = __int_as_float(0x7fc00000);
  float m = -INF;
  bool bad = false;
  for (int i = tid; i < a.V; i += kThreads) {
    const float x = E::ld(z, i);
    bad |= !(x < INF);
    m = fmaxf(m, x);
  }
  m = block_max<kThreads>(m, red);
  bad = group_sync_or<kThreads>(bad) || m == -INF;
  if (bad) {
    if (tid == 0) {
      if (a.logprob) a.logprob[row] = NAN_;
      if (a.rank) a.rank[row] = -1;
      if (a.entropy) a.entropy[row] = NAN_;
      for (int j = 0; j < a.n; ++j) {
        if (a.top_ids) a.top_ids[row * a.n + j] = -1;
        if (a.top_logprob) a.top_logprob[row * a.n + j] = NAN_;
      }
      atomicOr(a.status, kFlagBadValue | (good ? 0u : kFlagBadToken));
    }
    return;
  }
  const float zt = good ? E::ld(z, t) : INF;
  const float c = a.T == 0.f ? 0.f : 1.f / a.T;
  float s = 0.f, w = 0.f, before = 0.f;
  for (int i = tid; i < a.V; i += kThreads) {
    const float x = E::ld(z, i), y = (x - m) * c, e = x == -INF ? 0.f : expf(y);
    s += e;
    w += e > 0.f ? e * y : 0.f;
    before += (x > zt || (x == zt && i < t)) ? 1.f : 0.f;  // counts to 2^21: exact
  }
  s = block_sum<kThreads>(s, red);
  w = block_sum<kThreads>(w, red);
  before = block_sum<kThreads>(before, red);
  const float ls = logf(s);
  if (tid == 0) {
    if (!good) atomicOr(a.status, kFlagBadToken);
    if (a.rank) a.rank[row] = good ? static_cast<int>(before) : -1;
    if (a.logprob)
      a.logprob[row] = !good ? NAN_ : (a.T == 0.f ? (before == 0.f ? 0.f : -INF) : (zt - m) * c - ls);
    if (a.entropy) a.entropy[row] = a.T == 0.f ? 0.f : ls - w / s;
  }
  uint64_t last = ~0ull;
  for (int j = 0; j < a.n; ++j) {
    uint64_t k = 0;
    for (int i = tid; i < a.V; i += kThreads) {
      const uint64_t key = cand_key(E::ld(z, i) + 0.f, i);
      if (key < last && key > k) k = key;
    }
    last = block_max_u64<kThreads>(k, best);
    if (tid == 0) {
      if (a.top_ids) a.top_ids[row * a.n + j] = cand_idx(last);
      if (a.top_logprob)
        a.top_logprob[row * a.n + j] =
            a.T == 0.f ? (j == 0 ? 0.f : -INF) : (cand_val(last) - m) * c - ls;
    }
  }
}

}  // namespace

extern "C" ssd_status_t ssd_token_logprobs(const void *logits, ssd_dtype_t dt, int64_t seq_stride, int64_t row_stride,
                                           int B, int R, int V, float T, const int32_t *tokens, float *logprob,
                                           int32_t *rank, float *entropy, int n, int32_t *top_ids, float *top_logprob,
                                           uint32_t *status, ssd_stream_t s) {
  if (dt != SSD_F32 && dt != SSD_BF16) return SSD_ERR_INVALID_ARG;
  const int64_t size = dt == SSD_F32 ? 4 : 2;
  if (B < 0 || R < 0 || V < 1 || n < 0 || !(T >= 0.f) || isinf(T)) return SSD_ERR_INVALID_ARG;
  if ((logprob || rank) && !tokens) return SSD_ERR_INVALID_ARG;
  if (n > kMaxTop || n > V || (T > 0.f && T < 0x1p-60f) || V * size > (4 << 20)) return SSD_ERR_UNSUPPORTED;
  if (B == 0 || R == 0) return SSD_OK;
  if (!logits || !status) return SSD_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * R >= (1 << 28)) return SSD_ERR_UNSUPPORTED;
  if (((reinterpret_cast<uintptr_t>(logits) | static_cast<uintptr_t>(seq_stride * size) |
        static_cast<uintptr_t>(row_stride * size)) & 15u))
    return SSD_ERR_UNSUPPORTED;
  Args a{logits, seq_stride, row_stride, R, V, n, T, tokens, logprob, entropy, top_logprob, rank, top_ids, status};
  const unsigned grid = static_cast<unsigned>(B * R);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  if (dt == SSD_BF16)
    k_token_logprobs<EBF16><<<grid, kThreads, 0, cs>>>(a);
  else
    k_token_logprobs<EF32><<<grid, kThreads, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
