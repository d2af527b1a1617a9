// tables.cu -- the block tables of a paged K/V cache, grown and shrunk on the
// GPU from the sequences' lengths, with the free blocks in a ring.
//
// Per sequence b: want_b = ceil((len_b + reserve) / 16), grow_b = max(0, want_b
// - have_b), rel_b = max(0, have_b - want_b).  The i-th new block of b is
// ring[head + sum_{a<b} grow_a + i]; its i-th released one goes to ring[head +
// free + sum_{a<b} rel_a + i] (indices modulo the ring).  The ring holds every
// block at most once, so what is read (head .. head + free) and what is
// written (behind it) never meet, and the CTAs need no order among them.
//
//   k_block_tables  64 sequences per CTA, 1024 threads.  Every CTA scans the
//                   lengths up to its own sequences (one coalesced pass, two
//                   64-bit prefix sums); a warp then moves one sequence's ids,
//                   and the slots are flattened over the CTA.  The page counts
//                   and the pool are what every CTA reads, so they change
//                   last: by the CTA that takes the last ticket.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "common.cuh"

namespace {

using namespace ssd;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSeqs = 64;  // sequences per CTA
constexpr int kPage = 16;

struct TableArgs {
  const int32_t *len;
  int reserve, B;
  int32_t *table;
  int maxb;
  int32_t *pages, *ring;
  uint32_t n;  // blocks
  int32_t *pool, *slots;
  int S;
  uint32_t *status;
};

// One sequence's blocks before and after (`bad`: flags it raises).
struct Seq {
  int have, want;
  uint32_t bad;
};
SSD_DEV Seq sequence(const TableArgs &a, int b) {
  Seq q;
  q.bad = 0;
  const int held = a.pages[b], len = a.len[b];
  q.have = min(max(held, 0), a.maxb);
  if (q.have != held) q.bad = kFlagBadPrefix;
  const int64_t want = len < 0 ? 0 : (static_cast<int64_t>(len) + a.reserve + kPage - 1) / kPage;
  q.want = static_cast<int>(want);
  if (want > a.maxb) {
    q.bad = kFlagBadPrefix;
    q.want = q.have;
  }
  return q;
}

// Inclusive sums of (grow, released) over the block's threads; every thread
// also gets the block's totals.
SSD_DEV void block_scan(uint64_t &g, uint64_t &r, uint64_t &gt, uint64_t &rt, uint64_t (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, g, o), y = __shfl_up_sync(0xffffffffu, r, o);
    if (lane >= o) {
      g += x;
      r += y;
    }
  }
  __syncthreads();  // the parts of the previous scan have been read
  if (lane == 31) {
    part[warp][0] = g;
    part[warp][1] = r;
  }
  __syncthreads();
  uint64_t x = part[lane][0], y = part[lane][1];  // kWarps == 32: one part per lane
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  gt = __shfl_sync(0xffffffffu, x, 31);
  rt = __shfl_sync(0xffffffffu, y, 31);
  const uint64_t bx = __shfl_sync(0xffffffffu, x, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, y, max(warp - 1, 0));
  if (warp > 0) {
    g += bx;
    r += by;
  }
}

// head + i modulo the ring (head < n)
SSD_DEV uint32_t ring_at(uint32_t head, uint64_t i, uint32_t n) { return static_cast<uint32_t>((head + i) % n); }

__global__ void __launch_bounds__(kThreads) k_block_tables(TableArgs a) {
  static_assert(kWarps == 32, "block_scan holds one part per lane");
  __shared__ uint64_t part[kWarps][2];
  __shared__ uint64_t s_grow[kSeqs], s_rel[kSeqs];
  __shared__ int s_have[kSeqs], s_want[kSeqs];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = blockIdx.x * kSeqs, hi = min(a.B, lo + kSeqs);
  const bool alone = gridDim.x == 1;

  uint32_t head = static_cast<uint32_t>(a.pool[0]), free = static_cast<uint32_t>(a.pool[1]);
  if (head >= a.n || free > a.n) {
    if (tid == 0) atomicOr(a.status, kFlagBadPrefix);
    head = free = 0;
  }

  // The sequences' blocks and where their moves start, up to sequence `end`;
  // `update`: the counts are written too, and the pool's new state is returned.
  auto pass = [&](int end, bool update, uint64_t &taken, uint64_t &given) {
    uint64_t g0 = 0, r0 = 0;
    taken = 0;
    for (int c = 0; c < end; c += kThreads) {
      const int b = c + tid;
      Seq q{0, 0, 0};
      if (b < end) q = sequence(a, b);
      const uint64_t grow = max(0, q.want - q.have), rel = max(0, q.have - q.want);
      uint64_t g = grow, r = rel, gt, rt;
      block_scan(g, r, gt, rt, part);
      g += g0;
      r += r0;
      const bool fits = g <= free;
      if (!fits && grow) q.want = q.have;
      if (b >= lo && b < hi && !(update && !alone)) {
        s_have[b - lo] = q.have;
        s_want[b - lo] = q.want;
        s_grow[b - lo] = g - grow;
        s_rel[b - lo] = r - rel;
        if (!fits && grow) q.bad |= kFlagNoBlocks;
        if (q.bad) atomicOr(a.status, q.bad);
      }
      if (update && b < end) a.pages[b] = q.want;
      // growth is served in order: the largest running total that fits
      const uint64_t mine = (b < end && fits) ? g : 0;
      taken = max(taken, mine);
      g0 += gt;
      r0 += rt;
    }
    given = r0;
    if (update) {
#pragma unroll
      for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
      __syncthreads();
      if (lane == 0) part[warp][0] = taken;
      __syncthreads();
      taken = part[lane][0];
#pragma unroll
      for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    }
  };
  auto set_pool = [&](uint64_t taken, uint64_t given) {
    if (tid == 0) {
      a.pool[0] = static_cast<int32_t>(ring_at(head, taken, a.n));
      a.pool[1] = static_cast<int32_t>(min(static_cast<uint64_t>(a.n), free - taken + given));
      a.pool[2] = 0;
    }
  };
  uint64_t taken, given;
  pass(hi, alone, taken, given);
  __syncthreads();
  if (alone) set_pool(taken, given);

  // ids: a warp per sequence
  for (int s = warp; s < hi - lo; s += kWarps) {
    int32_t *row = a.table + static_cast<int64_t>(lo + s) * a.maxb;
    const int have = s_have[s], want = s_want[s];
    for (int p = have + lane; p < want; p += 32) row[p] = a.ring[ring_at(head, s_grow[s] + (p - have), a.n)];
    for (int p = want + lane; p < have; p += 32) {
      a.ring[ring_at(head, free + s_rel[s] + (p - want), a.n)] = row[p];
      row[p] = -1;
    }
  }
  // slots of the S positions from len on
  for (int64_t e = tid; e < static_cast<int64_t>(hi - lo) * a.S; e += kThreads) {
    const int s = static_cast<int>(e / a.S), i = static_cast<int>(e % a.S);
    const int b = lo + s, len = a.len[b], have = s_have[s];
    int slot = -1;
    if (len >= 0) {
      const int64_t pos = static_cast<int64_t>(len) + i, p = pos / kPage;
      if (p < s_want[s]) {
        const int blk = p < have ? a.table[static_cast<int64_t>(b) * a.maxb + p]
                                 : a.ring[ring_at(head, s_grow[s] + (p - have), a.n)];
        if (blk >= 0 && static_cast<uint32_t>(blk) < a.n) slot = blk * kPage + static_cast<int>(pos % kPage);
        else atomicOr(a.status, kFlagBadBlock);
      }
    }
    a.slots[static_cast<int64_t>(b) * a.S + i] = slot;
  }
  if (alone) return;

  // the last CTA to come here changes what the others have read
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(a.pool + 2, 1) == static_cast<int>(gridDim.x) - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  pass(a.B, true, taken, given);
  set_pool(taken, given);
}

}  // namespace

extern "C" ssd_status_t ssd_block_table_update(const int32_t *len, int reserve, int B, int32_t *block_table, int maxb,
                                               int32_t *pages, int32_t *ring, int64_t num_blocks, int32_t *pool,
                                               int32_t *slots, int S, uint32_t *status, ssd_stream_t s) {
  if (B < 0 || reserve < 0 || S < 0 || maxb < 1 || num_blocks < 1) return SSD_ERR_INVALID_ARG;
  if (num_blocks > (1 << 27) || maxb > (1 << 27) || B > 65536) return SSD_ERR_UNSUPPORTED;
  if (B == 0) return SSD_OK;
  if (!len || !block_table || !pages || !ring || !pool || !status || (S > 0 && !slots)) return SSD_ERR_INVALID_ARG;
  TableArgs a{};
  a.len = len;
  a.reserve = reserve;
  a.B = B;
  a.table = block_table;
  a.maxb = maxb;
  a.pages = pages;
  a.ring = ring;
  a.n = static_cast<uint32_t>(num_blocks);
  a.pool = pool;
  a.slots = slots;
  a.S = slots ? S : 0;
  a.status = status;
  k_block_tables<<<(B + kSeqs - 1) / kSeqs, kThreads, 0, reinterpret_cast<cudaStream_t>(s)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
