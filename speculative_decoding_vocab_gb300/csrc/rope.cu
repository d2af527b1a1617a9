// rope.cu -- rotary positions of the queries and keys at tree nodes.
//
// A token at position n turns the pair i of every head by the angle n theta_i.
// theta_i is held as a 64-bit fraction of a turn, so n theta_i mod one turn is
// one wrapping integer product: no position, however far, loses angle bits
// (an fp32 product is off by 0.06 rad at a million positions).  The angle
// then enters sincospi as half-turns in [-1, 1), rounded to 24 bits: at most
// 2^-25 pi rad, as much as the two products and the sum of an fp32 rotation round.
//
//   k_tree_rope   one CTA per token.  Its threads first ask for their pieces of
//                 the heads; meanwhile they walk the token's ancestors in
//                 shared memory (position = prefix + depth) and compute the
//                 rot/2 rotations once for all Hq + Hkv heads.
// Bound by HBM: every element is read and written once.  64 + 8 heads of 128
// with 64 rotated, 16396 tokens (604 MB): 104 us, 5.8 TB/s (128 us
// when the pieces were asked for after the rotations; with 2 or 4 pieces per thread
// at a time 3 and 6 us more).  A decode step of 256 tokens: 2.9 us, two dependent
// reads and a launch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <cmath>

#include "../../include/ssd.h"
#include "common.cuh"

namespace {

using namespace ssd;

// At most.  96, 128, 160, 192, 256 threads: the prompts above 102.9, 102.1, 103.6, 103.7, 104.7 us; in fp32, 3075 tokens
// of 40 heads, 18.7, 19.4, 18.3, 18.3, 18.8 us; the decode step 3.2, 3.2, 2.9, 2.9, 2.9 us.
constexpr int kThreads = 192;
constexpr int kMaxNodes = 128;
constexpr int kMaxD = 512;

struct RopeArgs {
  const void *q, *k;
  void *qo, *ko;
  int64_t q_ss, q_ts, qo_ss, qo_ts, k_ss, k_ts, ko_ss, ko_ts;  // elements
  const uint64_t *turns;
  int rot;
  float mscale;
  const int32_t *prefix_len, *parent;
  int N, node0, S, Hq, H, d;  // H = Hq + Hkv
  int pair_units, units;      // per head: rotated pieces, then copied ones
  uint32_t *status;
};

SSD_DEV uint32_t bf16_pair(float lo, float hi) {  // round to nearest even: the output's only rounding
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <class E, int VEC>
struct Piece;  // VEC elements moved in one access
template <>
struct Piece<EF32, 4> {
  using Elem = float;
  using Raw = uint4;
  SSD_DEV static void unpack(const Raw &w, float *f) { EF32::unpack(w, f); }
  SSD_DEV static Raw pack(const float *f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Piece<EF32, 1> {
  using Elem = float;
  using Raw = uint32_t;
  SSD_DEV static void unpack(const Raw &w, float *f) { f[0] = __uint_as_float(w); }
  SSD_DEV static Raw pack(const float *f) { return __float_as_uint(f[0]); }
};
template <>
struct Piece<EBF16, 8> {
  using Elem = uint16_t;
  using Raw = uint4;
  SSD_DEV static void unpack(const Raw &w, float *f) { EBF16::unpack(w, f); }
  SSD_DEV static Raw pack(const float *f) {
    return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
  }
};
template <>
struct Piece<EBF16, 4> {
  using Elem = uint16_t;
  using Raw = uint2;
  SSD_DEV static void unpack(const Raw &w, float *f) {
    f[0] = __uint_as_float(w.x << 16);
    f[1] = __uint_as_float(w.x & 0xFFFF0000u);
    f[2] = __uint_as_float(w.y << 16);
    f[3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
  SSD_DEV static Raw pack(const float *f) { return make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])); }
};
template <>
struct Piece<EBF16, 1> {
  using Elem = uint16_t;
  using Raw = uint16_t;
  SSD_DEV static void unpack(const Raw &w, float *f) { f[0] = __uint_as_float(static_cast<uint32_t>(w) << 16); }
  SSD_DEV static Raw pack(const float *f) { return static_cast<uint16_t>(bf16_pair(f[0], 0.f) & 0xFFFFu); }
};

SSD_DEV void rotate(float2 w, float &a, float &b) {
  const float x = a, y = b;
  a = x * w.x - y * w.y;
  b = x * w.y + y * w.x;
}

// VEC = 1 takes any alignment; there a rotated piece is one pair.
template <class E, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads) k_tree_rope(RopeArgs a) {
  using P = Piece<E, VEC>;
  using Raw = typename P::Raw;
  constexpr bool kOne = INTER && VEC > 1;  // a unit is one piece with whole pairs, else the two halves of VEC pairs
  __shared__ float2 turn[kMaxD / 2];       // mscale (cos, sin) of each pair
  __shared__ int par[kMaxNodes];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int b = blockIdx.x / a.S, i = blockIdx.x % a.S;
  const int half = a.rot / 2, total = a.H * a.units;
  struct Unit {
    Raw x, y;
    Raw *dst;
    int pair, second;  // first pair (-1: a copied piece), elements from x to y
  };
  auto load = [&](int w, Unit &t) {
    const int h = w / a.units, u = w - h * a.units;
    const bool isq = h < a.Hq;
    const int64_t hoff = static_cast<int64_t>(isq ? h : h - a.Hq) * a.d;
    const int64_t si = b * (isq ? a.q_ss : a.k_ss) + i * (isq ? a.q_ts : a.k_ts) + hoff;
    const int64_t di = b * (isq ? a.qo_ss : a.ko_ss) + i * (isq ? a.qo_ts : a.ko_ts) + hoff;
    const bool copy = u >= a.pair_units;
    const int e = copy ? a.rot + (u - a.pair_units) * VEC : (INTER && VEC == 1 ? 2 * u : u * VEC);
    t.pair = copy ? -1 : (kOne ? e / 2 : u * VEC);
    t.second = INTER ? 1 : half;
    const typename P::Elem *const src = static_cast<const typename P::Elem *>(isq ? a.q : a.k) + si + e;
    t.dst = reinterpret_cast<Raw *>(static_cast<typename P::Elem *>(isq ? a.qo : a.ko) + di + e);
    t.x = *reinterpret_cast<const Raw *>(src);
    if (!kOne && !copy) t.y = *reinterpret_cast<const Raw *>(src + t.second);
  };
  auto turned = [&](const Unit &t) {
    if (t.pair < 0) {
      *t.dst = t.x;
      return;
    }
    float x[VEC], y[VEC];
    P::unpack(t.x, x);
    if (kOne) {
#pragma unroll
      for (int v = 0; v < VEC; v += 2) rotate(turn[t.pair + v / 2], x[v], x[v + 1 < VEC ? v + 1 : v]);
      *t.dst = P::pack(x);
    } else {
      P::unpack(t.y, y);
#pragma unroll
      for (int v = 0; v < VEC; ++v) rotate(turn[t.pair + v], x[v], y[v]);
      *t.dst = P::pack(x);
      *reinterpret_cast<Raw *>(reinterpret_cast<typename P::Elem *>(t.dst) + t.second) = P::pack(y);
    }
  };
  // the first unit is on its way while the position and the angles are found
  Unit unit;
  if (tid < total) load(tid, unit);
  const int L = a.prefix_len[b];
  if (L == -1) return;  // a slot without a request
  int64_t pos = static_cast<int64_t>(max(L, 0));
  if (L < 0 && tid == 0) atomicOr(a.status, kFlagBadPrefix);
  if (a.parent) {
    for (int m = tid; m < a.N; m += nt) par[m] = a.parent[static_cast<int64_t>(b) * a.N + m];
    __syncthreads();
    for (int m = a.node0 + i;; ++pos) {
      const int up = par[m];
      if (up < -1 || up >= m) {
        if (tid == 0) atomicOr(a.status, kFlagBadTree);
        break;
      }
      if (up < 0) break;
      m = up;
    }
  } else {
    pos += static_cast<int64_t>(a.node0) + i;
  }
  for (int j = tid; j < half; j += nt) {
    const uint64_t t = static_cast<uint64_t>(pos) * a.turns[j];
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &s, &c);
    turn[j] = make_float2(c * a.mscale, s * a.mscale);
  }
  __syncthreads();
  for (int w = tid; w < total; w += nt) {
    if (w != tid) load(w, unit);
    turned(unit);
  }
}

template <class E, int VEC>
void launch(const RopeArgs &a, bool inter, unsigned grid, cudaStream_t cs) {
  // every thread has the same number of units, but for the last warps'
  const int units = a.H * a.units, rounds = (units + kThreads - 1) / kThreads;
  const int threads = ((units + rounds - 1) / rounds + 31) / 32 * 32;
  if (inter)
    k_tree_rope<E, VEC, true><<<grid, threads, 0, cs>>>(a);
  else
    k_tree_rope<E, VEC, false><<<grid, threads, 0, cs>>>(a);
}

}  // namespace

extern "C" ssd_status_t ssd_rope_frequencies(int rot, double base, double factor, double original_len, double fast,
                                             double slow, uint64_t *turns, float *mscale) {
  if (rot < 2 || rot % 2 || !(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) ||
      !(original_len >= 0.0) || !std::isfinite(original_len) || !turns || !mscale)
    return SSD_ERR_INVALID_ARG;
  if (rot > 1024) return SSD_ERR_UNSUPPORTED;
  const bool parts = factor > 1.0 && original_len > 0.0;
  if (parts && !(slow > 0.0 && fast > slow && std::isfinite(fast))) return SSD_ERR_INVALID_ARG;
  const double tau = 6.283185307179586476925286766559;
  // the (fractional) pair that turns r times in original_len positions
  auto pair_of = [&](double r) { return rot * std::log(original_len / (r * tau)) / (2.0 * std::log(base)); };
  double lo = 0.0, hi = 0.0;
  const bool ramped = parts && pair_of(slow) > 0.0;
  if (ramped) {
    lo = std::fmax(std::floor(pair_of(fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(slow)), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double theta = std::pow(base, -2.0 * i / rot);
    if (ramped) {
      const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
      theta = theta / factor * ramp + theta * (1.0 - ramp);
    } else {  // without parts, or no pair turns `slow` times
      theta /= factor;
    }
    turns[i] = static_cast<uint64_t>(std::nearbyint(theta / tau * 18446744073709551616.0));
  }
  *mscale = parts ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return SSD_OK;
}

extern "C" ssd_status_t ssd_tree_rope(const void *q, int64_t q_ss, int64_t q_ts, void *q_out, int64_t qo_ss,
                                      int64_t qo_ts, const void *k, int64_t k_ss, int64_t k_ts, void *k_out,
                                      int64_t ko_ss, int64_t ko_ts, ssd_dtype_t dt, const uint64_t *turns, int rot,
                                      int interleaved, float mscale, const int32_t *prefix_len, const int32_t *parent,
                                      int N, int node0, int B, int S, int Hq, int Hkv, int d, uint32_t *status,
                                      ssd_stream_t s) {
  if (B < 0 || S < 0 || Hq < 0 || Hkv < 0 || d < 1 || rot < 2 || rot % 2 || rot > d || node0 < 0 || N < 0 ||
      !std::isfinite(mscale) || (dt != SSD_F32 && dt != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  if (d > kMaxD || N > kMaxNodes) return SSD_ERR_UNSUPPORTED;
  if (parent && static_cast<int64_t>(node0) + S > N) return SSD_ERR_INVALID_ARG;
  if (B == 0 || S == 0 || Hq + Hkv == 0) return SSD_OK;
  if ((Hq && (!q || !q_out)) || (Hkv && (!k || !k_out)) || !turns || !prefix_len || !status)
    return SSD_ERR_INVALID_ARG;
  const int64_t grid = static_cast<int64_t>(B) * S;
  if (grid > 0x7fffffffLL || static_cast<int64_t>(Hq + Hkv) * d > (1 << 24)) return SSD_ERR_UNSUPPORTED;
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.qo = q_out;
  a.ko = k_out;
  a.q_ss = q_ss;
  a.q_ts = q_ts;
  a.qo_ss = qo_ss;
  a.qo_ts = qo_ts;
  a.k_ss = k_ss;
  a.k_ts = k_ts;
  a.ko_ss = ko_ss;
  a.ko_ts = ko_ts;
  a.turns = turns;
  a.rot = rot;
  a.mscale = mscale;
  a.prefix_len = prefix_len;
  a.parent = parent;
  a.N = N;
  a.node0 = node0;
  a.S = S;
  a.Hq = Hq;
  a.H = Hq + Hkv;
  a.d = d;
  a.status = status;
  // the widest piece that every address, stride and boundary of the head is a multiple of
  const int elem = dt == SSD_F32 ? 4 : 2;
  uint64_t addr = 0, off = static_cast<uint64_t>(d) | static_cast<uint64_t>(d - rot) |
                           static_cast<uint64_t>(interleaved ? rot : rot / 2);
  if (Hq) {
    addr |= reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out);
    off |= static_cast<uint64_t>(q_ss | q_ts | qo_ss | qo_ts);
  }
  if (Hkv) {
    addr |= reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(k_out);
    off |= static_cast<uint64_t>(k_ss | k_ts | ko_ss | ko_ts);
  }
  const auto whole = [&](int vec) { return addr % (vec * elem) == 0 && off % vec == 0; };
  const int vec = (dt == SSD_BF16 && whole(8)) ? 8 : (whole(4) ? 4 : 1);
  if (vec == 1 && addr % elem) return SSD_ERR_UNSUPPORTED;
  a.pair_units = interleaved ? (vec > 1 ? rot / vec : rot / 2) : rot / 2 / vec;
  const bool in_place = (!Hq || (q == q_out && q_ss == qo_ss && q_ts == qo_ts)) &&
                        (!Hkv || (k == k_out && k_ss == ko_ss && k_ts == ko_ts));
  a.units = a.pair_units + (in_place ? 0 : (d - rot) / vec);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  const unsigned g = static_cast<unsigned>(grid);
  const bool inter = interleaved != 0;
  if (dt == SSD_F32) {
    if (vec == 4) launch<EF32, 4>(a, inter, g, cs);
    else launch<EF32, 1>(a, inter, g, cs);
  } else {
    if (vec == 8) launch<EBF16, 8>(a, inter, g, cs);
    else if (vec == 4) launch<EBF16, 4>(a, inter, g, cs);
    else launch<EBF16, 1>(a, inter, g, cs);
  }
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
