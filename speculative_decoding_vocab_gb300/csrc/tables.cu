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
//   k_block_tables  1024 threads and 8 to 64 sequences per CTA.  Every CTA scans
//                   the lengths up to its own sequences (one coalesced pass,
//                   two prefix sums); a warp then moves one sequence's ids,
//                   and the slots are flattened over the CTA.  The page counts
//                   and the pool are what every CTA's scan reads, so they
//                   change behind the scans: by the CTA that takes the last
//                   ticket.
// Bound by latency: the scan's dependent reads and barriers, then the ids'.  64
// sequences: 3.6 us; 1024 sequences of up to 32768 positions of which 20 end:
// 6.3 us (22 us with a warp per sequence and one read in flight; 16 or 32
// sequences per CTA instead of 8: 7.5 and 10 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "common.cuh"

namespace {

using namespace ssd;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSeqs = 64;  // sequences per CTA, at most
constexpr uint32_t kCap = 1u << 28;  // prefix sums stop here, above every ring (2^27)
constexpr int kPage = 16;

struct TableArgs {
  const int32_t *len;
  int reserve, B, per;  // per: sequences per CTA
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
  int have, want, len;
  uint32_t bad;
};
SSD_DEV Seq sequence(const TableArgs &a, int b) {
  Seq q;
  q.bad = 0;
  const int held = a.pages[b], len = a.len[b];
  q.len = len;
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

SSD_DEV uint32_t add_cap(uint32_t x, uint32_t y) { return min(x + y, kCap); }

// Inclusive sums of (grow, released) over the block's threads; every thread
// also gets the block's totals.
SSD_DEV void block_scan(uint32_t &g, uint32_t &r, uint32_t &gt, uint32_t &rt, uint2 *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](uint32_t &x, uint32_t &y) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x = add_cap(x, u);
        y = add_cap(y, v);
      }
    }
  };
  scan(g, r);
  __syncthreads();  // the parts of the previous scan have been read
  if (lane == 31) part[warp] = make_uint2(g, r);
  __syncthreads();
  uint32_t x = part[lane].x, y = part[lane].y;  // kWarps == 32: one part per lane
  scan(x, y);
  gt = __shfl_sync(0xffffffffu, x, 31);
  rt = __shfl_sync(0xffffffffu, y, 31);
  const uint32_t bx = __shfl_sync(0xffffffffu, x, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, y, max(warp - 1, 0));
  if (warp > 0) {
    g = add_cap(g, bx);
    r = add_cap(r, by);
  }
}

// head + i modulo the ring (head < n, i < 2^30)
SSD_DEV uint32_t ring_at(uint32_t head, uint32_t i, uint32_t n) { return (head + i) % n; }

__global__ void __launch_bounds__(kThreads) k_block_tables(TableArgs a) {
  static_assert(kWarps == 32, "block_scan holds one part per lane");
  __shared__ uint2 part[kWarps];
  __shared__ uint32_t s_grow[kSeqs], s_rel[kSeqs];
  __shared__ int s_have[kSeqs], s_want[kSeqs], s_len[kSeqs];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = blockIdx.x * a.per, hi = min(a.B, lo + a.per);
  const bool alone = gridDim.x == 1;

  uint32_t head = static_cast<uint32_t>(a.pool[0]), free = static_cast<uint32_t>(a.pool[1]);
  if (head >= a.n || free > a.n) {
    if (tid == 0) atomicOr(a.status, kFlagBadPrefix);
    head = free = 0;
  }

  // The sequences' blocks and where their moves start, up to sequence `end`;
  // `update`: the counts are written too, and the pool's new state is returned.
  auto pass = [&](int end, bool update, uint32_t &taken, uint32_t &given) {
    uint32_t g0 = 0, r0 = 0;
    taken = 0;
    for (int c = 0; c < end; c += kThreads) {
      const int b = c + tid;
      Seq q{0, 0, 0, 0};
      if (b < end) q = sequence(a, b);
      const uint32_t grow = max(0, q.want - q.have), rel = max(0, q.have - q.want);
      uint32_t g = grow, r = rel, gt, rt;
      block_scan(g, r, gt, rt, part);
      g = add_cap(g, g0);
      r = add_cap(r, r0);
      const bool fits = g <= free;
      if (!fits && grow) q.want = q.have;
      if (b >= lo && b < hi && !(update && !alone)) {
        s_have[b - lo] = q.have;
        s_want[b - lo] = q.want;
        s_len[b - lo] = q.len;
        s_grow[b - lo] = g - grow;  // (not used where the sum stopped: nothing fits there)
        s_rel[b - lo] = r - rel;
        if (!fits && grow) q.bad |= kFlagNoBlocks;
        if (q.bad) atomicOr(a.status, q.bad);
      }
      if (update && b < end) a.pages[b] = q.want;
      // growth is served in order: the largest running total that fits
      const uint32_t mine = (b < end && fits) ? g : 0;
      taken = max(taken, mine);
      g0 = add_cap(g0, gt);
      r0 = add_cap(r0, rt);
    }
    given = r0;
    if (update) {
#pragma unroll
      for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
      __syncthreads();
      if (lane == 0) part[warp].x = taken;
      __syncthreads();
      taken = part[lane].x;
#pragma unroll
      for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    }
  };
  auto set_pool = [&](uint32_t taken, uint32_t given) {
    if (tid == 0) {
      a.pool[0] = static_cast<int32_t>(ring_at(head, taken, a.n));
      a.pool[1] = static_cast<int32_t>(min(a.n, free - taken + given));
      a.pool[2] = 0;
    }
  };
  uint32_t taken, given;
  pass(hi, alone, taken, given);
  __syncthreads();
  if (alone) {
    set_pool(taken, given);
  } else if (tid == 0) {  // the CTA's scan is done
    __threadfence();
    s_last = atomicAdd(a.pool + 2, 1) == static_cast<int>(gridDim.x) - 1;
  }

  // ids: the warps shared out among the sequences, kBatch reads of a lane in flight (a request that ends gives back
  // thousands of blocks)
  const int nseq = hi - lo, share = max(1, kWarps / nseq);
  for (int w = warp; w < nseq * share; w += kWarps) {
    const int s = w % nseq, first = w / nseq * 32 + lane, step = share * 32;
    int32_t *const row = a.table + static_cast<int64_t>(lo + s) * a.maxb;
    const int have = s_have[s], want = s_want[s], n = max(want - have, have - want);
    const bool grow = want > have;
    const int p0 = min(want, have);
    const uint32_t r0 = grow ? s_grow[s] : free + s_rel[s];
    constexpr int kBatch = 4;
    for (int i = first; i < n; i += kBatch * step) {
      int32_t id[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int x = i + k * step;
        if (x < n) id[k] = grow ? a.ring[ring_at(head, r0 + x, a.n)] : row[p0 + x];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int x = i + k * step;
        if (x >= n) break;
        row[p0 + x] = grow ? id[k] : -1;
        if (!grow) a.ring[ring_at(head, r0 + x, a.n)] = id[k];
      }
    }
  }
  // slots of the S positions from len on
  for (uint32_t e = tid; e < static_cast<uint32_t>(hi - lo) * a.S; e += kThreads) {
    const int s = e / a.S, i = e - s * a.S;
    const int b = lo + s, len = s_len[s], have = s_have[s];
    int slot = -1;
    if (len >= 0) {
      const int64_t pos = static_cast<int64_t>(len) + i, p = pos / kPage;
      if (p < s_want[s]) {
        const int blk = p < have ? a.table[static_cast<int64_t>(b) * a.maxb + p]
                                 : a.ring[ring_at(head, s_grow[s] + static_cast<uint32_t>(p - have), a.n)];
        if (blk >= 0 && static_cast<uint32_t>(blk) < a.n) slot = blk * kPage + static_cast<int>(pos % kPage);
        else atomicOr(a.status, kFlagBadBlock);
      }
    }
    a.slots[static_cast<int64_t>(b) * a.S + i] = slot;
  }
  if (alone) return;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  pass(a.B, true, taken, given);  // all scans are done: what they read may change
  set_pool(taken, given);
}

}  // namespace

extern "C" ssd_status_t ssd_block_table_update(const int32_t *len, int reserve, int B, int32_t *block_table, int maxb,
                                               int32_t *pages, int32_t *ring, int64_t num_blocks, int32_t *pool,
                                               int32_t *slots, int S, uint32_t *status, ssd_stream_t s) {
  if (B < 0 || reserve < 0 || S < 0 || maxb < 1 || num_blocks < 1) return SSD_ERR_INVALID_ARG;
  if (num_blocks > (1 << 27) || maxb > (1 << 27) || B > 65536 || S > (1 << 24)) return SSD_ERR_UNSUPPORTED;
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
  // one CTA up to 64 sequences (no second scan); else enough CTAs that their sequences' ids and slots take few
  // rounds, but not so many that the scans of long batches outweigh them
  a.per = B <= kSeqs ? kSeqs : (B / 128 < 8 ? 8 : (B / 128 < kSeqs ? B / 128 : kSeqs));
  k_block_tables<<<(B + a.per - 1) / a.per, kThreads, 0, reinterpret_cast<cudaStream_t>(s)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
