// logprobs.cu -- log probabilities of given tokens, with their rank, the row's
// entropy and its likeliest tokens, in one pass over the logits.
//
// With c = log2(e) / T, a number k near the largest z c, y = z c - k, s = sum 2^y, w = sum y 2^y:
//   ln p(t) = ln2 (y_t - log2 s),   entropy = ln2 (log2 s - w / s),
//   rank(t) = #{z > z_t} + #{i < t: z_i = z_t}.
// A thread keeps k, s and w of what it has read (k = m c rounded, m its largest
// logit so far; s and w move with it); parts meet in a fixed order.  k is a
// number like any other, so y = fma(z, c, -k) rounds once.  Logits are cut at
// -1e30, where the exponential is 0 (0 * -inf would be NaN): tokens of -inf or of
// the type's lowest value cost no test and are nobody's m.  A NaN reaches s.  The
// largest logit's own y is what the rounding of k left over, half a step of k: at most 1
// below 2^25, past the exponential's range from 2^31 on.  A row whose largest logit is
// that far from 0 for its c, or is itself near -1e29, or whose products would pass
// fp32's range, is summed again by a loop that takes differences first, and so is every row
// where c is so small that the cut logits would count (T above 1.4e26).  Of other rows
// nothing below -2^26 / c is anyone's m (a finite mask, which may fill a thread's whole
// part): it lies 2^25 below the row's largest, so its exponential is 0 around any k.
// The first n tokens: each CTA collects candidates in shared memory, those that its
// threshold lets through.  The threshold starts from the first stage: each of
// its (up to 8) whole warps gives the k-th largest of its lanes' maxima, k = ceil(n
// / warps); at least n elements reach the least of these.  From then on the n-th candidate so
// far is the threshold, and only larger values pass (indices rise along the
// part, and equal values rank by index).  Keys (value, ~index) are distinct, so their
// ranks are counted, whatever order they came in.  Where a stage lets more through
// than there is room for, the n-th key is searched bit by bit, 64 passes over the stage: a
// first stage in which a warp has fewer allowed tokens than it gives (a grammar's mask,
// ties: 384 rows of 128256 with 10 allowed tokens 442 us, 40 unmasked), every stage of rising rows (1.6 ms).
//
//   k_token_logprobs  a cluster of cw CTAs (256 threads) per row, a range of the row
//       each, in stages of 32 KB that bulk copies bring into a ring of two (8 or 16 KB,
//       rings of three or four, and 64 to 512 threads were slower); rank 0 joins the
//       parts through distributed shared memory.
// Bound by the issue slots where the first tokens are asked for: 2048 rows of 151936 with 20 of them and the rank
// (622 MB) 142 us, 4.4 TB/s; without the first tokens 103, without the rank too 98 (6.4 TB/s).  384 rows of 128256,
// 56 MB of them wanted, with 5 tokens 19 us.  Five fp32 rows: 10 us, the chain of one part's stages and the two joins.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "common.cuh"

namespace {

using namespace ssd;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = 64;
constexpr int kStageBytes = 32768, kStageVecs = kStageBytes / 16, kStages = 2;
constexpr int kVecs = kStageVecs / kThreads;  // of a thread and stage
constexpr int kRoom = 512;  // of candidates; at least kMaxCluster * kMaxTop
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster <= kWarps && kMaxCluster * kMaxTop <= kRoom, "a warp per CTA, room for their candidates");
static_assert(2 * kMaxTop + 16 + 7 <= kRoom, "room for what is kept and the last elements");
constexpr float kCut = -1e30f, kLow = -1e29f, kFar = 0x1p25f, kFlat = 1e-26f, kSteep = 1e7f;

struct Args {
  const void *z;
  int64_t ss, rs;
  int R, V, n, cw;
  float c, inv_t;  // log2(e) / T, 1 / T
  float low;       // what is not above it is nobody's m
  int greedy;
  const int32_t *tokens;
  float *logprob, *entropy, *top_logprob;
  int32_t *rank, *top_ids;
  uint32_t *status;
};

struct Part {
  float most, m, s, w;  // the largest logit; the largest above low, around which s and w are
  int before, count, buffer;  // buffer: which one holds its candidates
};
struct Shared {
  uint64_t cand[2][kRoom];  // the current ones, and where the best of them go
  uint64_t full[kStages];
  float4 red[kWarps];
  uint32_t low[kWarps];
  int before[kWarps];
  int count[3];  // candidates of a stage, by stage mod 3
  int found;
  Part part;
  Part all[kMaxCluster];
};

SSD_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
SSD_DEV uint32_t peer_address(const void *p, unsigned rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
SSD_DEV uint32_t peer_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
SSD_DEV uint64_t peer_u64(uint32_t at) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}
SSD_DEV float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
SSD_DEV uint32_t max_nan2(uint32_t a, uint32_t b) {  // of bf16 pairs
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// a vector's elements, none below kCut
template <class E>
SSD_DEV uint4 cut(const uint4 &v) {
  if (E::kSize == 2) {
    const uint32_t low = 0xF149F149u;  // -1e30 in bf16
    return make_uint4(max_nan2(v.x, low), max_nan2(v.y, low), max_nan2(v.z, low), max_nan2(v.w, low));
  }
  auto one = [](uint32_t x) { return __float_as_uint(max_nan(__uint_as_float(x), kCut)); };
  return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
}
SSD_DEV uint32_t ord(float x) { return f2ord(x + 0.f); }  // -0 and 0 rank alike
// the next larger value of the type, as fp32
template <class E>
SSD_DEV float above(float x) {
  const uint32_t step = 1u << (E::kSize == 2 ? 16 : 0);
  const uint32_t b = __float_as_uint(x);
  if (x == 0.f) return __uint_as_float(step);
  return __uint_as_float(x > 0.f ? b + step : b - step);
}

// How many of a vector's elements are >= z2's, added to `acc` (bf16: a pair of small counts; fp32: a count)
struct Counter {
  __nv_bfloat162 pair;
  int n;
};
template <class E>
SSD_DEV void count_from(const uint4 &v, float z, Counter &k) {
  if (E::kSize == 2) {
    const __nv_bfloat162 z2 = __float2bfloat162_rn(z);  // z is a bf16 value
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __nv_bfloat162 x;
      *reinterpret_cast<uint32_t *>(&x) = w[j];
      k.pair = __hadd2(k.pair, __hge2(x, z2));
    }
  } else {
    k.n += (__uint_as_float(v.x) >= z) + (__uint_as_float(v.y) >= z) + (__uint_as_float(v.z) >= z) +
           (__uint_as_float(v.w) >= z);
  }
}
template <class E>
SSD_DEV float vec_max(const uint4 &v) {
  if (E::kSize == 2) {
    const uint32_t m = bmax2(bmax2(v.x, v.y), bmax2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}

// The n largest of cand[cur][0 .. c) -> the other buffer, in order (all threads; the candidates are written, c <= kRoom)
SSD_DEV int keep_best(Shared &sh, int &cur, int c, int n) {
  const uint64_t *const cand = sh.cand[cur];
  for (int j = threadIdx.x; j < c; j += kThreads) {
    const uint64_t key = cand[j];
    int r = 0, i = 0;
    for (; i + 8 <= c; i += 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) r += cand[i + k] > key;
    }
    for (; i < c; ++i) r += cand[i] > key;
    if (r < n) sh.cand[cur ^ 1][r] = key;
  }
  __syncthreads();
  cur ^= 1;
  return min(c, n);
}

template <class E>
__global__ void __launch_bounds__(kThreads) k_token_logprobs(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / a.cw;
  const int part = static_cast<int>(blockIdx.x - row * a.cw);
  const int t = a.tokens ? a.tokens[row] : 0;
  if (t == -1) return;  // the whole cluster
  const bool given = a.tokens != nullptr, good = t >= 0 && t < a.V;
  const float INF = __int_as_float(0x7f800000), NAN_ = __int_as_float(0x7fc00000);
  const char *const z = static_cast<const char *>(a.z) + ((row / a.R) * a.ss + (row % a.R) * a.rs) * E::kSize;
  const int nv = a.V / E::kVec, per = (nv + a.cw - 1) / a.cw;
  const int v0 = min(nv, part * per), v1 = min(nv, v0 + per), nst = (v1 - v0 + kStageVecs - 1) / kStageVecs;
  auto load = [&](int st) {  // by thread 0
    const int from = v0 + st * kStageVecs, bytes = min(kStageVecs, v1 - from) * 16;
    mbar_arrive_expect_tx(&sh.full[st % kStages], bytes);
    bulk_g2s(ring + (st % kStages) * kStageBytes, z + static_cast<int64_t>(from) * 16, bytes, &sh.full[st % kStages]);
  };
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1);
    fence_mbar_init();
    fence_proxy_async();
    for (int i = 0; i < min(kStages, nst); ++i) load(i);
    sh.count[0] = sh.count[1] = sh.count[2] = 0;
  }
  const bool ranked = given && good && (a.rank || (a.logprob && a.greedy));
  const float zt = given && good ? E::ld(z, t) : 0.f, zt_above = above<E>(zt);
  const float c = a.c;
  const uint64_t c2 = pack2(c, c);
  float most = -INF, m = -INF, k = 0.f;  // the largest logit; the largest above a.low, and m c
  uint64_t s2 = 0, w2 = 0, neg_k2 = 0;
  int before = 0;
  auto rise = [&](float to) {  // a larger m
    const float kn = __fmul_rn(to, c);
    if (m != -INF) {
      const float d = k - kn, f = ex2(d);
      s2 = mul2(s2, pack2(f, f));
      w2 = f == 0.f ? s2 : fma2(pack2(d, d), s2, mul2(w2, pack2(f, f)));  // d may be anything
    }
    m = to;
    k = kn;
    neg_k2 = pack2(-kn, -kn);
  };
  auto add_pair = [&](uint64_t x) {
    const uint64_t y = fma2(x, c2, neg_k2);
    float y0, y1;
    unpack2(y, y0, y1);
    const uint64_t e = pack2(ex2(y0), ex2(y1));
    s2 = add2(s2, e);
    w2 = fma2(e, y, w2);
  };
  float least = -INF;  // the smallest value that passes
  int kept = 0, turn = 0, cur = 0;  // candidates of the stages before; which counter this one has; which buffer
  // a vector's elements that pass: element e at bit e (of fp32), or e / 2 + 4 (e % 2)
  auto passing = [&](const uint4 &v) {
    uint32_t mask = 0;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (E::kSize == 2) {
      const __nv_bfloat162 least2 = __float2bfloat162_rn(least);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        __nv_bfloat162 x;
        *reinterpret_cast<uint32_t *>(&x) = w[h];
        mask |= __hge2_mask(x, least2) & (0x00010001u << h);
      }
      mask = (mask | mask >> 12) & 0xFFu;
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) mask |= (__uint_as_float(w[h]) >= least ? 1u : 0u) << h;
    }
    return mask;
  };
  __syncthreads();
  auto element = [](const uint4 *buf, int j) {  // of a stage
    return E::kSize == 2 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(buf)[j]) << 16)
                         : reinterpret_cast<const float *>(buf)[j];
  };
  bool ok = true;
  for (int st = 0; st < nst; ++st) {
    const int first = v0 + st * kStageVecs, count = min(kStageVecs, v1 - first);
    const uint4 *const buf = reinterpret_cast<const uint4 *>(ring + (st % kStages) * kStageBytes);
    ok = mbar_wait(&sh.full[st % kStages], (st / kStages) & 1) && ok;
    uint4 v[kVecs];
    float top = -INF;  // of this thread's elements of the stage
    const bool whole = count == kStageVecs;
    // `whole` is tested here alone, in a branch that the whole CTA takes: tested per vector it was a branch each time
    if (whole) {
#pragma unroll
      for (int q = 0; q < kVecs; ++q) v[q] = buf[q * kThreads + tid];
    } else {
#pragma unroll
      for (int q = 0; q < kVecs; ++q) v[q] = q * kThreads + tid < count ? buf[q * kThreads + tid] : E::nothing();
    }
#pragma unroll
    for (int q = 0; q < kVecs; ++q) top = fmaxf(top, vec_max<E>(v[q]));
    most = fmaxf(most, top);
    if (top > m && top > a.low) rise(top);
    if (ranked && top >= zt) {
      Counter n{__float2bfloat162_rn(0.f), 0};
#pragma unroll
      for (int q = 0; q < kVecs; ++q) {
        const int j = q * kThreads + tid, i0 = (first + j) * E::kVec;
        count_from<E>(v[q], i0 + E::kVec <= t && j < count ? zt : zt_above, n);  // what is not there is above nothing
      }
      before += n.n + static_cast<int>(__low2float(n.pair)) + static_cast<int>(__high2float(n.pair));
    }
    if (a.n > 0) {
      if (st == 0) {  // the first threshold
        const int warps = min(kThreads, count) / 32;  // those of which every lane has an element
        const int rounds = warps > 0 ? (a.n + warps - 1) / warps : 33;
        if (rounds <= 32) {  // else at most 64 vectors: all pass
          uint32_t mine = ord(top), kth = 0xffffffffu;
          if (warp < warps)
            for (int i = 0; i < rounds; ++i) {
              kth = __reduce_max_sync(0xffffffffu, mine);
              const uint32_t who = __ballot_sync(0xffffffffu, mine == kth);
              if (lane == __ffs(who) - 1) mine = 0;
            }
          if (lane == 0) sh.low[warp] = kth;
          __syncthreads();
          uint32_t low = sh.low[0];
          for (int i = 1; i < kWarps; ++i) low = min(low, sh.low[i]);
          least = ord2f(low);
        }
      }
      if (__any_sync(0xffffffffu, top >= least)) {
        uint32_t mask[2] = {0, 0};  // kVec bits of each vector
#pragma unroll
        for (int q = 0; q < kVecs; ++q) mask[q / 4] |= passing(v[q]) << (q % 4 * E::kVec);
        if (!whole) {
#pragma unroll
          for (int q = 0; q < kVecs; ++q)
            if (q * kThreads + tid >= count) mask[q / 4] &= ~(((1u << E::kVec) - 1u) << (q % 4 * E::kVec));
        }
        const int mine = __popc(mask[0]) + __popc(mask[1]);
        if (mine) {  // few lanes: an atomic each is less than a scan of the warp
          int at = kept + atomicAdd(&sh.count[turn], mine);
          for (uint64_t left = static_cast<uint64_t>(mask[1]) << 32 | mask[0]; left; left &= left - 1, ++at) {
            const int b = __ffsll(left) - 1, q = (b >> 5) * 4 + (b & 31) / E::kVec, p = (b & 31) % E::kVec;
            const int j = q * kThreads + tid, e = E::kSize == 2 ? 2 * (p & 3) + (p >> 2) : p;
            if (at < kRoom) sh.cand[cur][at] = cand_key(element(buf, j * E::kVec + e) + 0.f, (first + j) * E::kVec + e);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      const uint4 x = cut<E>(v[q]);
#pragma unroll
      for (int h = 0; h < E::kPairs; ++h) add_pair(E::pair(x, h));
    }
    if (a.n > 0) {
      __syncthreads();  // the only one of most stages: who is behind may still read this counter when the next stage's rises
      int now = kept + sh.count[turn];
      turn = turn == 2 ? 0 : turn + 1;
      if (tid == 0) sh.count[turn == 2 ? 0 : turn + 1] = 0;  // the stage after next's
      if (now > kRoom) {
        // Too many: the n-th largest key of what was kept and this stage, from the highest bit down.  (The candidates of
        // this stage are dropped and found again.)
        uint64_t key = 0;
        auto reach = [&](uint64_t from) {  // how many keys are >= from
          int r = 0;
          for (int j = tid; j < count * E::kVec; j += kThreads) {
            const int i = first * E::kVec + j;
            const float x = element(buf, j);
            r += cand_key(x + 0.f, i) >= from;
          }
          for (int j = tid; j < kept; j += kThreads) r += sh.cand[cur][j] >= from;
          if (tid == 0) sh.found = 0;
          __syncthreads();
          r = __reduce_add_sync(0xffffffffu, r);
          if (lane == 0) atomicAdd(&sh.found, r);
          __syncthreads();
          const int all = sh.found;
          __syncthreads();
          return all;
        };
        for (int b = 63; b >= 0; --b) {
          const uint64_t with = key | 1ull << b;
          if (reach(with) >= a.n) key = with;
        }
        if (tid == 0) sh.found = 0;
        __syncthreads();
        for (int j = tid; j < count * E::kVec; j += kThreads) {
          const int i = first * E::kVec + j;
          const float x = element(buf, j);
          if (cand_key(x + 0.f, i) >= key) sh.cand[cur][kept + atomicAdd(&sh.found, 1)] = cand_key(x + 0.f, i);
        }
        __syncthreads();
        now = kept + sh.found;  // at most kept + n <= kRoom
      }
      if (st == 0 || now > 2 * a.n + 16) {
        now = keep_best(sh, cur, now, a.n);
        // only larger values pass from here on; until there are n, all do
        least = now == a.n ? above<E>(cand_val(sh.cand[cur][a.n - 1])) : -INF;
      }
      kept = now;
    } else {
      __syncthreads();
    }
    if (tid == 0 && st + kStages < nst) load(st + kStages);
  }
  // The elements behind the last whole vector, which are candidates in any case.  They come last, as their indices do.
  if (part == a.cw - 1) {
    const int i = nv * E::kVec + tid;
    if (i < a.V) {
      const float x = E::ld(z, i);
      most = fmaxf(most, x);
      if (x > m && x > a.low) rise(x);
      add_pair(pack2(max_nan(x, kCut), kCut));  // the pair's other half adds nothing
      if (ranked) before += i < t ? x >= zt : x > zt;
      if (a.n > 0) sh.cand[cur][kept + tid] = cand_key(x + 0.f, i);
    }
    kept += a.V - nv * E::kVec;
  }
  // equal logits before the token in its own vector, which was counted as if they ranked behind it
  if (ranked && tid == 0) {
    const int v = t / E::kVec;
    if (v >= v0 && v < v1)
      for (int i = v * E::kVec; i < t; ++i) before += E::ld(z, i) == zt;
  }
  // ---------------- the CTA's part
  {
    const float M = warp_max(most), W = warp_max(m);  // W: the warp's largest m
    float s0, s1, w0, w1;
    unpack2(s2, s0, s1);
    unpack2(w2, w0, w1);
    auto move = [&](float from, float to, float &s, float &w) {  // sums around `from` c to `to` c
      if (from == -INF || from == to) return;
      const float d = __fmul_rn(from, c) - __fmul_rn(to, c), f = ex2(d);
      s = s * f;
      w = f == 0.f ? s : fmaf(d, s, w * f);
    };
    float s = s0 + s1, w = w0 + w1;
    move(m, W, s, w);
    s = warp_sum(s);
    w = warp_sum(w);
    const int b = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) {
      sh.red[warp] = make_float4(M, W, s, w);
      sh.before[warp] = b;
    }
    __syncthreads();
    // a lane per part; their sums in the order of the exchanges
    auto join = [&](Part p) {
      Part all = p;
      all.most = warp_max(p.most);
      all.m = warp_max(p.m);
      move(p.m, all.m, p.s, p.w);
      all.s = warp_sum(p.s);
      all.w = warp_sum(p.w);
      all.before = __reduce_add_sync(0xffffffffu, p.before);
      return all;
    };
    const Part nothing{-INF, -INF, 0.f, 0.f, 0, 0, 0};
    if (warp == 0) {
      Part p = nothing;
      if (lane < kWarps) p = Part{sh.red[lane].x, sh.red[lane].y, sh.red[lane].z, sh.red[lane].w, sh.before[lane], 0, 0};
      p = join(p);
      if (lane == 0) sh.part = p;
    }
    if (a.n > 0) {
      const int left = keep_best(sh, cur, kept, a.n);
      if (tid == 0) {
        sh.part.count = left;
        sh.part.buffer = cur;
      }
    }
    __syncthreads();
    // ---------------- the row, by rank 0
    if (a.cw > 1) {
      cluster_sync();
      if (part == 0) {
        if (tid < a.cw) {
          const uint32_t from = peer_address(&sh.part, tid);
          sh.all[tid] = Part{__uint_as_float(peer_u32(from)),      __uint_as_float(peer_u32(from + 4)),
                             __uint_as_float(peer_u32(from + 8)),  __uint_as_float(peer_u32(from + 12)),
                             static_cast<int>(peer_u32(from + 16)), static_cast<int>(peer_u32(from + 20)),
                             static_cast<int>(peer_u32(from + 24))};
        }
        __syncthreads();
        int at = 0;  // a warp per CTA: one trip for all of them
        for (int r = 0; r < a.cw; ++r) {
          const int n = sh.all[r].count;
          if (warp == r && r > 0)
            for (int j = lane; j < n; j += 32) sh.cand[cur][at + j] = peer_u64(peer_address(sh.cand[sh.all[r].buffer], r) + 8 * j);
          at += n;
        }
        if (warp == 0) {
          const Part p = join(lane < a.cw ? sh.all[lane] : nothing);
          if (lane == 0) sh.part = p;
        }
        __syncthreads();
        if (a.n > 0) keep_best(sh, cur, at, a.n);
        __syncthreads();
      }
    }
  }
  if (part == 0) {
    const Part p = sh.part;
    // the row's sums around its largest logit, or, where these are out of the loop's range, again.  (With c >= kFlat the
    // gap between kLow / 2 and kLow is 500 in y: what is not above kLow has the exponential 0, as it was counted.)
    float total = p.s, moment = p.w, k_row = __fmul_rn(p.most, c);
    const float half_most = 0.5f * p.most;  // differences are taken of halves: those of logits may pass fp32's range
    const bool again = !(p.most > 0.5f * kLow) || !(fabsf(k_row) < kFar) || !(c >= kFlat && c < kSteep);
    if (again) {
      // A thread adds up to 8192 terms here, often equal ones, whose additions round the same way each time: what each
      // leaves goes to the next.
      float s = 0.f, w = 0.f, s_left = 0.f, w_left = 0.f;
      auto add = [](float &sum, float &left, float term) {
        const float t = __fadd_rn(term, left), to = __fadd_rn(sum, t);
        left = __fsub_rn(t, __fsub_rn(to, sum));
        sum = to;
      };
      for (int i = tid; i < a.V; i += kThreads) {
        const float x = E::ld(z, i), y = max_nan((0.5f * x - half_most) * (2.f * c), -160.f), e = ex2(y);
        add(s, s_left, e);
        add(w, w_left, __fmul_rn(e, y));
      }
      s = warp_sum(s);
      w = warp_sum(w);
      __syncthreads();
      if (lane == 0) sh.red[warp] = make_float4(s, w, 0.f, 0.f);
      __syncthreads();
      total = moment = 0.f;
      for (int i = 0; i < kWarps; ++i) total += sh.red[i].x, moment += sh.red[i].y;
    }
    const bool none = !(total == total) || p.most == INF || p.most == -INF;  // no distribution
    const float ls = log2f(total), ln2 = 0.69314718055994531f;
    // ln p; of the logits that were cut, times c may pass fp32's range where ln p does not.  Where one token has all of
    // the row, the roundings of ex2 and log2 leave it up to 1e-7 on either side of 0.
    auto ln_of = [&](float x) {
      const float ln = again || x < kCut ? fmaf(-ls, ln2, (0.5f * x - half_most) * (2.f * a.inv_t))
                                         : (fmaf(x, c, -k_row) - ls) * ln2;
      return fminf(ln, 0.f);
    };
    if (tid == 0) {
      const uint32_t flags = (none ? kFlagBadValue : 0u) | (good ? 0u : kFlagBadToken);
      if (flags) atomicOr(a.status, flags);
      if (a.logprob)
        a.logprob[row] = none || !good ? NAN_ : (a.greedy ? (p.before == 0 ? 0.f : -INF) : ln_of(zt));
      if (a.rank) a.rank[row] = none || !good ? -1 : p.before;
      if (a.entropy) a.entropy[row] = none ? NAN_ : (a.greedy ? 0.f : fmaxf((ls - moment / total) * ln2, 0.f));
    }
    if (tid < a.n) {
      const uint64_t key = sh.cand[cur][tid];
      const int64_t at = row * a.n + tid;
      if (a.top_ids) a.top_ids[at] = none ? -1 : cand_idx(key);
      if (a.top_logprob)
        a.top_logprob[at] =
            none ? NAN_ : (a.greedy ? (tid == 0 ? 0.f : -INF) : ln_of(cand_val(key)));
    }
  }
  if (!ok && tid == 0) atomicOr(a.status, kFlagWaitTimeout);
  if (a.cw > 1) cluster_sync();  // no CTA leaves while rank 0 may still read its shared memory
}

// CTAs of a row, doubled while there are less than 608 of them: few, so that a CTA's part is long.  (Three of 73 KB fit an
// SM, 456 on 152.)  The call that it is chosen for, a round's emitted tokens (384 rows of 128256, about half of them
// wanted): up to 304 32 us, 608 22, 1216 28.  Where all rows are wanted 304 is as fast or faster (384 bf16 rows of 128256 33
// us instead of 40, of 32000 16 instead of 23; the same up to 64 rows and from 700 on), 1216 never.
int cluster_of(int64_t rows, int V, int64_t size) {
  const int64_t stages = (V * size + kStageBytes - 1) / kStageBytes;
  int cw = 1;
  while (cw < kMaxCluster && rows * cw < 608 && cw < stages) cw *= 2;
  return cw;
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
  Args a{};
  a.z = logits;
  a.ss = seq_stride;
  a.rs = row_stride;
  a.R = R;
  a.V = V;
  a.n = top_ids || top_logprob ? n : 0;
  a.cw = cluster_of(static_cast<int64_t>(B) * R, V, size);
  a.greedy = T == 0.f;
  a.c = a.greedy ? 1.f : static_cast<float>(1.4426950408889634 / T);
  a.inv_t = a.greedy ? 1.f : 1.f / T;
  a.low = fmaxf(kLow, -2.f * kFar / a.c);
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_logprob = top_logprob;
  a.rank = rank;
  a.top_ids = top_ids;
  a.status = status;
  // the ring, or a whole part where that is less
  const int64_t part = ((V * size / 16 + a.cw - 1) / a.cw) * 16;
  const int ring = static_cast<int>(part < kStages * kStageBytes ? (part + 127) / 128 * 128 : kStages * kStageBytes);
  void (*const kernel)(Args) = dt == SSD_BF16 ? k_token_logprobs<EBF16> : k_token_logprobs<EF32>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * kStageBytes) != cudaSuccess)
    return SSD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * R * a.cw));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(ring);
  cfg.stream = reinterpret_cast<cudaStream_t>(s);
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(a.cw);
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
