// attention_q4.cu -- tree-masked decode attention over a paged K/V cache held
// in 4 bits (e2m1 codes, a power-of-two scale byte per 32 elements of a token and
// head), on the sm_103a tensor cores.
//
// The products are those of the 8-bit kernel: up to 64 rows per KV head the keys
// take the MMA's 128-wide side and the rows its N,
//     S^T [128 keys x rows] = K4 Q^T,      O^T [d x rows] += V^T P^T;
// above, the rows fill that side themselves,
//     S [128 rows x 128 keys] = Q K4^T,    O [128 rows x d] += P V.
// S: key codes go to the tensor cores as they are (kind::mxf8f6f4: TMA spreads them
// to a byte each, the MMA multiplies each 32 elements by their scale byte), the
// queries as two e4m3 terms (prepare_rows).  The scale bytes lie in TMEM, a lane per
// row of 128 elements; queries have the constant 2^-8 (their largest element
// lies in [2^7, 2^8), so S passes fp32's range only where sums of |k| do).
// At d = 64 a row of 128 elements is two positions: the MMAs of the even ones
// take its first half, those of the odd ones its second.
// P V: in halves (kind::f16).  With t the largest scale of a key, v = t 2^-13 h: h =
// code * 2^(13 + scale's exponent - t's) is exact down to 2^-36 of t (a half reaches
// 2^-24, and 6 * 2^13 is below its largest).  P t is rounded to a half, off by
// at most 2^-11 of itself, or by 2^-25 where it is subnormal, 2^-36 of the row's largest
// or less.  A byte of v holds one element of two neighbouring keys, which is what a TMEM
// column of halves takes: four bytes of ldmatrix' transpose become four columns by
// one conversion and one product each.
// Scores are x = s * scale * 2^e, P = 2^(x - m + 11); m is the running maximum of x +
// log2(t) as in the 8-bit kernel (kBias, kMoved, kGrow).
//
// CTA: an MMA warp, two producer warps for K and the scales, one for V, helper warps
// (scale bytes to TMEM, t and the factors of a key's groups, V into halves, the
// next segment's rows; two sets of four, with more than 64 rows one), softmax warps
// (groups of four: 16 rows of the tile each, or with a lane per row a quarter of its
// keys).  A unit is what one K slot holds: 128 rows of 128 elements; where a
// tile has two, each set of helpers has one of them, a tile apart if it so happens.
// Bound by the roles' chains in a CTA (issue slots 61 %, the tensor pipe 21 %, HBM a third), not by bytes; their
// loops together miss the instruction cache (10 % of its requests).  Microseconds (bytes' floor): 64 sequences of 8192 keys, 6 rows of 8 per head, d 128: 186 (86); 16 of 2048, 68 rows of 4, d 64: 67
// (4.0); one of 100003 keys, a token: 38 (16); 48 of up to 16384, 8 rows of 8: 96 (33); 64 of 8192, a token each: 144 (84).
// The 8-bit kernel takes 190 / 62 / 45 / 97.  Measured and slower (first / last shape): S and P V issued by two
// warps 232 / 174 instead of 198 / 168, scale warps of their own 201 / 155 instead of 190 / 147, waits with a suspend hint
// 204 / 176 instead of 201 / 166, the loop over V's words unrolled by two 198 / 152 instead of 190 / 144; one set of
// helpers at 64 rows 111 instead of 96 (the fourth).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <cmath>

#include "../../include/ssd.h"
#include "attention_line.cuh"
#include "e2m1.cuh"

namespace ssd {
namespace q4 {

using namespace line;

constexpr int kSmemBudget = 214 * 1024;
constexpr int kTiles = 4;     // tiles whose scales of v are held
constexpr int kIds = 32;      // units whose block ids are held
constexpr int kVShift = 13;
// O / L's unit.  It goes to O before 1 / L does: with v's smallest scales L passes 2^104 a key, and kOutUnit / L is
// subnormal from 5 keys on; with its largest O / L passes fp32's range.
constexpr float kOutUnit = kSumUnit * 0x1p-13f;
constexpr int kQueryByte = 127 - 8;
constexpr float kQueryUnit = 256.f;

// D[tmem] (+)= A B of one 32-element step of K with scale bytes at sfa, sfb (TMEM columns; the byte by idesc)
SSD_DEV void umma_mx(uint32_t d_tmem, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                     uint32_t sfa, uint32_t sfb, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %8, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %5, [%6], [%7], p;\n\t}\n" ::"r"(
          d_tmem),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum)
      : "memory");
}
// M = 128, e2m1 by e4m3 (or, with a lane per row, e4m3 by e2m1); k: which byte of the codes' scales
__host__ __device__ constexpr uint32_t idesc_mx(bool row_lanes, int N, int k) {
  return (5u << (row_lanes ? 10 : 7)) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (8u << 24) |
         (static_cast<uint32_t>(k) << (row_lanes ? 4 : 29));
}
SSD_DEV void tmem_st4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
SSD_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// arrives when this thread's cp.async copies so far have landed
SSD_DEV void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 2^(e - 15) as a half; 0 below the smallest
SSD_DEV uint32_t half_pow2(int e) { return e > 0 ? static_cast<uint32_t>(e) << 10 : (e > -10 ? 1u << (9 + e) : 0u); }
SSD_DEV uint32_t every_other_bit(uint32_t x) {  // bits 0, 2, 4, .. -> bits 0 .. 15
  x &= 0x55555555u;
  x = (x | x >> 1) & 0x33333333u;
  x = (x | x >> 2) & 0x0F0F0F0Fu;
  x = (x | x >> 4) & 0x00FF00FFu;
  return (x | x >> 8) & 0xFFFFu;
}

struct Args : Line {
  const uint8_t *ks, *vs;
};

template <int D, int RT>
struct Cfg {
  static constexpr bool kRowLanes = RT > 64;               // rows, not keys, on the MMA's 128-wide side
  static constexpr int KT = RT <= 64 ? 2 : 1;              // sub-tiles of 128 keys of a tile
  static constexpr int kKeys = KT * kSub;                  // keys of a tile
  static constexpr int CG = kRowLanes ? 32 : 16;           // rows of a softmax warp (keys, with a lane per row)
  static constexpr int kGroups = RT / CG;                  // groups of four warps
  static constexpr int NB = 2;                             // S buffers; S runs NB tiles ahead
  static constexpr int kSoftWarps = 4 * kGroups;
  // The MMA warp and the producers come first: the schedulers prefer older warps, and these few are what all others wait
  // for.  Then the helpers (warp w of a set's four writes TMEM lanes 32 w .. + 31, those that a warp of its number modulo 4
  // reaches), with the keys on the wide side in two sets, a sub-tile each, and the softmax warps.
  static constexpr int kMmaWarp = 0, kTmaWarp = 1, kKWarps = 2, kVWarps = 1;
  static constexpr int kSets = RT <= 64 ? 2 : 1, kHelpers = 4 * kSets, kHelpWarp = 4, kSoftWarp = kHelpWarp + kHelpers;
  static constexpr int kWarps = kSoftWarp + kSoftWarps, kThreads = kWarps * 32;
  static_assert(kTmaWarp + kKWarps + kVWarps == kHelpWarp, "roles");
  // units of a tile; a unit's keys, its rows of 128 elements, its blocks
  static constexpr int kUnits = D == 128 ? KT : 1;
  static constexpr bool kApart = kSets == 2 && kUnits == 2;  // a set has a unit of each tile for itself
  static constexpr int kVHelp = kApart ? 4 : kHelpers;       // helper warps that turn a unit of V into halves
  static constexpr int kUKeys = kKeys / kUnits, kURows = kUKeys * D / 128, kUPages = kUKeys / kPage;
  static constexpr int kG = D / kQ4Group;                  // scales of a key
  static constexpr int kPageBytes = kPage * D / 2;         // codes of a block and head, K or V
  static constexpr int kScalePage = kPage * kG;
  static constexpr int kBatch = 32 / kUPages;              // units that a producer warp's lanes hold the blocks of, every
                                                           // other one
  static constexpr int kQTile = RT * 128;                  // q1 (or q2) at D = 128; [q1 | q2] at D = 64
  static constexpr int kQBuf = D == 128 ? 2 * kQTile : kQTile;
  // P V's operand in shared memory, halves: P^T of a sub-tile in rows of 128 bytes, a key each; with a lane per row V
  // in blocks of 64 elements, rows of 128 bytes, a key each
  static constexpr int kBlock = kSub * 128;
  static constexpr int kHBuf = kRowLanes ? (D / 64) * kBlock : KT * kBlock;  // of a tile
  static constexpr int kKSlot = kURows * 128, kVSlot = kUKeys * D / 2, kSSlot = 1024;
  static constexpr int kFactors = kURows * 8;              // of a unit: a half per key and group
  static constexpr int kFixed = 2 * kQBuf + NB * kHBuf + kTiles * kKeys * 8 + kTiles * kUnits * kFactors;
  static constexpr int kFit = (kSmemBudget - kFixed) / (kKSlot + kVSlot + kSSlot);
  // Sets that work apart may be two tiles from each other, and a barrier's parity tells a wait only the phase before
  // from the one after: each set has slots of its own, every other one.
  static constexpr int kSlots = (kFit > 8 ? 8 : kFit) & (kApart ? ~1 : ~0);
  static constexpr int kQ = 0, kH = 2 * kQBuf, kKRing = kH + NB * kHBuf, kVRing = kKRing + kSlots * kKSlot,
                       kSRing = kVRing + kSlots * kVSlot, kTop = kSRing + kSlots * kSSlot,
                       kFactor = kTop + kTiles * kKeys * 8;
  static constexpr int kSmem = kFactor + kTiles * kUnits * kFactors + 1024;
  // TMEM: NB x KT x S, O, scale bytes (the queries', then a ring of units'), and at its end P V's other operand in
  // halves: V^T (as many buffers as fit), or P (one)
  static constexpr int kOCol = NB * KT * RT, kOCols = kRowLanes ? D : RT;
  static constexpr int kACols = KT * (kSub / 2);           // of a tile
  static constexpr int kABufs = !kRowLanes && kOCol + kOCols + 16 + NB * kACols <= 512 ? NB : 1;
  static constexpr int kACol = 512 - kABufs * kACols;
  static constexpr int kVBufs = kRowLanes ? NB : kABufs;   // of V in halves, in shared memory or TMEM
  static constexpr int kSfCol = kOCol + kOCols;
  static constexpr int kSfFit = (kACol - kSfCol) / 4 - 1;
  static constexpr int kSf = (kSfFit > kSlots ? kSlots : kSfFit) & (kApart ? ~1 : ~0);
  static_assert(kSmem + 13 * 1024 <= 227 * 1024, "shared memory with the static part");
  // The helpers write the scales of a tile NB tiles ahead of V, and the softmax warps are NB tiles behind S at most.
  static_assert(kTiles >= NB + 2, "scales of v");
  static_assert(kSlots >= (NB + 1) * kUnits || kSlots >= 4, "S runs ahead");
  static_assert(kSf >= kUnits && kSf <= kSlots && kIds >= kSlots + 4 * kBatch, "scale bytes in TMEM, block ids");
  static_assert(!kApart || (kSlots % 2 == 0 && kSf % 2 == 0), "a set's slots are its own");
  static_assert(kVWarps == 1 || kApart || kUnits == 1, "V's producers wait for units that one set gives back in order");
  static_assert(!kRowLanes || (RT == 128 && kGroups == 4), "a lane per row, a quarter of the keys per group");
  static_assert(kRowLanes || (KT == 2 && CG == 16 && RT <= 64), "tiles of two sub-tiles, P in rows of 128 bytes");
  static_assert(kKRing % 1024 == 0 && kVRing % 1024 == 0, "swizzled tiles");
};

template <int D, int RT>
__global__ void __launch_bounds__(Cfg<D, RT>::kThreads, 1)
    k_branch_attn_q4(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ Args a) {
  using C = Cfg<D, RT>;
  constexpr int CG = C::CG, NB = C::NB, NSLOT = C::kSlots, KT = C::KT, U = C::kUnits, UP = C::kUPages, G = C::kG;
  constexpr int kSoftThreads = C::kSoftWarps * 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // by an offset: known to be shared memory
  // Of a tile, by the place of a key's scores (element h * 128 + lane of the S^T pair, or the column of S): t, then log2 t
  // (0 and -inf: hidden)
  float *const top = reinterpret_cast<float *>(smem + C::kTop);
  __shared__ __align__(8) uint64_t kfull[NSLOT], kempty[NSLOT], vfull[NSLOT], vempty[NSLOT], kready[C::kSf];
  __shared__ __align__(8) uint64_t sfull[NB], pfull[NB], vready[NB], pvdone[NB], qfull[2], qempty[2];
  __shared__ uint32_t tmem_base;
  __shared__ __align__(16) int s_ids[2][kIds][UP];          // block ids of a unit (K's and V's producers), -1 for none
  __shared__ int s_row[2][kIds];                            // and its head's first row in a block
  __shared__ uint32_t s_gone[kTiles][U * 4];                // missing blocks of a tile, by helper warp
  __shared__ int par[2][kMaxNodes];
  __shared__ uint32_t anc[2][kMaxNodes][kMaxNodes / 32];    // per query: the nodes that it sees
  __shared__ float qs[2][RT];                               // row scales 2^e
  __shared__ __align__(16) float4 rowc[RT / 2];             // two rows: scale 2^e twice, 11 - m twice
  __shared__ float s_m[RT], s_f[RT], red[4][RT];
  __shared__ int s_nan[4];                                  // a tree node's v has a NaN scale, by segment mod 4 (the
                                                            // helper warps are in the segment behind the softmax warps' at most)
  __shared__ long long scan[32];
  __shared__ Piece s_piece;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes
  const float NEG_INF = -__int_as_float(0x7f800000);

  if (tid == 0) {
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&kfull[s], 33);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], C::kVHelp);
    }
    for (int s = 0; s < C::kSf; ++s) mbar_init(&kready[s], 4);
    for (int u = 0; u < NB; ++u) {
      mbar_init(&sfull[u], 1);
      mbar_init(&pfull[u], 4 * C::kGroups);
      mbar_init(&vready[u], C::kHelpers);
      mbar_init(&pvdone[u], 1);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&qfull[u], C::kHelpers);
      mbar_init(&qempty[u], 1 + C::kSoftWarps);
    }
    fence_mbar_init();
    s_abort = 0;
    s_nan[0] = s_nan[1] = s_nan[2] = s_nan[3] = 0;
    s_piece.left = 0;
    s_piece.tiles = 0;
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  find_piece<C::kThreads, C::kKeys>(a, scan, &s_piece);  // its barriers order the set-up above too
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
  const Piece piece = s_piece;
  const int ntiles = piece.tiles;

  // the rows of segment `sg` into buffer `buf`, by warp w of the n that share it (barrier `bar`)
  auto prepare = [&](const Segments &sg, int buf, int w, int n, int bar) {
    prepare_rows<C, D, RT>(a, sg, smem + C::kQ + buf * C::kQBuf, par[buf], anc[buf], qs[buf], w, n, bar);
  };

  Segments sg;
  if (warp >= C::kTmaWarp && warp < C::kHelpWarp) {
    // ---------------- producers: warps for K's codes and both scales, and for V's codes, a unit each in turn (a copy
    // costs its warp 60 to 70 clocks).  Block ids are fetched for kBatch of a warp's units at a time, one batch ahead: lane l
    // holds block l % UP of the batch's unit l / UP.
    const bool is_k = warp < C::kTmaWarp + C::kKWarps;
    const int pw = is_k ? 0 : 1, mine = warp - C::kTmaWarp - (is_k ? 0 : C::kKWarps), page = lane % UP;
    const int step = is_k ? C::kKWarps : C::kVWarps;
    uint64_t *const full = is_k ? kfull : vfull, *const empty = is_k ? kempty : vempty;
    const CUtensorMap *const map = is_k ? &kmap : &vmap;
    constexpr int kKRows = kPage * D / 128;                // rows of a block and head: K, then V
    const int rows = is_k ? kKRows : kPage / 2;
    const int pitch = is_k ? kKRows * 128 : C::kPageBytes, slot_bytes = is_k ? C::kKSlot : C::kVSlot;
    uint8_t *const ring = smem + (is_k ? C::kKRing : C::kVRing);
    bool more = sg.first(a, piece);
    int t = more ? sg.t0 * U : 0;
    auto advance = [&](int n) {  // this lane's place in the line of units
      t += n;
      while (more && t >= sg.t1 * U) {
        t -= sg.t1 * U;
        more = sg.step(a);
      }
    };
    int row, blk;
    auto ids = [&] {
      row = more ? sg.hk * rows : 0;
      blk = -1;
      const int64_t lp = static_cast<int64_t>(t) * UP + page;
      if (more && lp < a.maxb && lp * kPage < sg.nkeys) {
        blk = a.table[static_cast<int64_t>(sg.b) * a.maxb + lp];
        if (blk < 0 || blk >= a.num_blocks) {
          if (is_k) atomicOr(a.status, kFlagBadBlock);
          blk = -1;
        }
      }
      advance(step * C::kBatch);
    };
    advance(mine + step * (lane / UP));
    ids();
    const int nunits = ntiles * U;
    int slot = mine, i = mine;
    uint32_t phase = 1;  // of empty[slot]; the first round's slots are free
    bool ok = true;
    for (int n = 0; i < nunits; i += step, ++n) {
      if (n % C::kBatch == 0) {
        const int at = (i + step * (lane / UP)) % kIds;
        s_ids[pw][at][page] = blk;
        if (page == 0) s_row[pw][at] = row;
        __syncwarp();
        ids();
      }
      const int x = i % kIds, r = s_row[pw][x];
      int e[UP], all = 0;
#pragma unroll
      for (int k = 0; k < UP; k += 4) {
        const int4 v = *reinterpret_cast<const int4 *>(&s_ids[pw][x][k]);
        e[k] = v.x, e[k + 1] = v.y, e[k + 2] = v.z, e[k + 3] = v.w;
        all |= v.x | v.y | v.z | v.w;
      }
      ok = i < NSLOT || warp_wait(&empty[slot], phase);
      if (!ok) break;
      uint8_t *const dst = ring + slot * slot_bytes;
      if (elect_one()) {
        if (all >= 0) {
          mbar_arrive_expect_tx(&full[slot], UP * C::kPageBytes);
#pragma unroll
          for (int k = 0; k < UP; ++k) tma_load_3d(dst + k * pitch, map, 0, r, e[k], &full[slot]);
        } else {  // some blocks are missing or bad
          int there = 0;
          for (int k = 0; k < UP; ++k) there += s_ids[pw][x][k] >= 0;
          mbar_arrive_expect_tx(&full[slot], there * C::kPageBytes);
#pragma unroll 1
          for (int k = 0; k < UP; ++k)
            if (s_ids[pw][x][k] >= 0) tma_load_3d(dst + k * pitch, map, 0, r, s_ids[pw][x][k], &full[slot]);
        }
      }
      __syncwarp();
      if (is_k) {  // the scales, 16 bytes a lane: K's, then V's (a unit's fill 512 bytes, or 256)
        constexpr int kChunks = C::kScalePage / 16;
        const int p = lane / kChunks, b = p < UP ? s_ids[0][x][p] : -1;
        if (b >= 0) {
          const int64_t from = static_cast<int64_t>(b) * (a.Hkv * C::kScalePage) + r * (C::kScalePage / kKRows) + (lane % kChunks) * 16;
          uint8_t *const to = smem + C::kSRing + slot * C::kSSlot + lane * 16;
          cp_async16(to, a.ks + from);
          cp_async16(to + 512, a.vs + from);
        }
        cp_async_arrive(&kfull[slot]);
      }
      slot += step;
      if (slot >= NSLOT) {
        slot -= NSLOT;
        phase ^= 1;
      }
    }
    if (!ok) {
      s_abort = 1;
      // this warp's copies in flight land before the shared memory is given back
      for (int k = 0; k < (NSLOT + step - 1) / step && (i -= step) >= 0; ++k) (void)warp_wait(&full[i % NSLOT], (i / NSLOT) & 1);
    }
    cp_async_wait_all();
  } else if (warp == C::kMmaWarp) {
    // ---------------- MMA issue (one elected lane): S of up to NB tiles ahead, then P V and S in turn.
    constexpr uint32_t idesc_o = idesc_f16(C::kRowLanes ? D : RT), hi128 = desc_hi(1024, kSw128);
    const uint32_t base = smem_u32(smem);
    const uint32_t ring_k = desc_lo(base + C::kKRing, 16), h_lo = desc_lo(base + C::kH, C::kBlock);
    const uint32_t sf_q = tmem + C::kSfCol;
    bool ok = true;
    int slot = 0, sf = 0, seg = 0;
    uint32_t sf_phase = 0;  // of kready[sf]
    bool more = sg.first(a, piece);
    int t = more ? sg.t0 : 0;
    // S of a unit: D = 128 one sub-tile, D = 64 the even positions of the unit, then the odd ones
    auto umma_s = [&](uint32_t d, uint32_t k, uint32_t q, uint32_t sf_k) {
      constexpr int kHalves = D == 128 ? 1 : 2, kSteps = D / 32;
      constexpr int N = C::kRowLanes ? C::kURows : RT;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) {
            const int b = h * kSteps + kk;
            const uint32_t qk = q + (term * (D == 128 ? C::kQTile : 64) >> 4) + kk * 2, kb = k + b * 2;
            const uint32_t more = (term > 0 || kk > 0) ? 1u : 0u;
            if (C::kRowLanes)
              umma_mx(d + h * N, qk, hi128, kb, hi128, idesc_mx(true, N, b), sf_q, sf_k, more);
            else
              umma_mx(d + h * N, kb, hi128, qk, hi128, idesc_mx(false, N, b), sf_k, sf_q, more);
          }
    };
    auto issue_s = [&](int i) {
      const int buf = seg & 1, u = i % NB;
      if (t == sg.t0) ok = warp_wait(&qfull[buf], (seg >> 1) & 1);
      const uint32_t q = desc_lo(base + C::kQ, 16) + buf * (C::kQBuf >> 4);
      const bool last = ++t == sg.t1;
#pragma unroll
      for (int h = 0; h < U; ++h) {
        // the S buffer is free: P of tile i - NB, made from it, has been waited for
        ok = ok && warp_wait(&kready[sf], sf_phase);  // K has landed, its scale bytes are in TMEM
        tc_fence_after();
        if (!ok) return;
        const uint32_t dd = tmem + (u * KT + h) * (C::kRowLanes ? kSub : RT), kd = ring_k + slot * (C::kKSlot >> 4), qd = q, sd = sf_q + 4 + sf * 4;
        if (elect_one()) {
          umma_s(dd, kd, qd, sd);
          umma_commit(&kempty[slot]);
          if (h == U - 1) {
            umma_commit(&sfull[u]);
            if (last) umma_commit(&qempty[buf]);
          }
        }
        __syncwarp();
        if (++slot == NSLOT) slot = 0;
        if (++sf == C::kSf) {
          sf = 0;
          sf_phase ^= 1;
        }
      }
      if (last) {
        more = sg.step(a);
        t = sg.t0;
        ++seg;
      }
    };
    Order order;
    order.start(a, piece);
    for (int i = 0, j = 0; j < ntiles && ok;) {
      if (i - j < NB && i < order.end) {
        issue_s(i++);
      } else {  // P V of tile j
        const int u = j % NB;
        const uint32_t o = tmem + C::kOCol;
        const uint32_t later = j > order.begin;  // not the segment's first tile
        ok = warp_wait(&vready[u], (j / NB) & 1);
        ok = ok && warp_wait(&pfull[u], (j / NB) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + C::kACol + (j % C::kABufs) * C::kACols, b = h_lo + u * (C::kHBuf >> 4);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < KT; ++h)
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk)  // 16 keys: two groups of 8 rows
              umma_f16(o, at + h * (kSub / 2) + kk * 8, b + h * (C::kBlock >> 4) + kk * (2048 >> 4), hi128, idesc_o,
                       kk > 0 || h > 0 ? 1u : later);
          umma_commit(&pvdone[u]);
        }
        __syncwarp();
        order.done(a, ++j);
      }
    }
    if (!ok) s_abort = 1;
  } else if (warp >= C::kHelpWarp && warp < C::kSoftWarp) {
    // ---------------- helpers, in the order of the MMAs.  They meet at named barriers, which have no limit, so a warp
    // whose wait gave up goes on (its waits are over at once) until they leave together.
    const int hw = warp & 3, set = (warp - C::kHelpWarp) >> 2, r = hw * 32 + lane;
    constexpr int kStep = C::kApart ? 2 : 1;  // units from one of this warp's to the next
    const int h0 = C::kApart ? set : 0, h1 = C::kApart ? set + 1 : U;
    const uint32_t quad = static_cast<uint32_t>(hw * 32) << 16;
    bool ok = true, all = true, more = sg.first(a, piece);
    if (more) {
      constexpr uint32_t q = kQueryByte * 0x01010101u;
      if (set == 0) tmem_st4(tmem + C::kSfCol + quad, q, q, q, q);
      tmem_wait_st();
      tc_fence_before();
      prepare(sg, 0, warp - C::kHelpWarp, C::kSoftWarps + C::kHelpers, 10);
      bar_sync(10, (C::kSoftWarps + C::kHelpers) * 32);
      tc_fence_after();
      tc_fence_before();
      if (lane == 0) mbar_arrive1(&qfull[0]);
    }
    int slot = h0, sf = h0 % C::kSf, vslot = h0;
    uint32_t phase = 0, vphase = 0;  // of kfull[slot], vfull[vslot]
    int nk = h0;                     // number of the unit of K
    // the scales of tile i (number t of the segment)
    auto scales = [&](int i, int t, int seg) {
#pragma unroll 1
      for (int h = h0; h < h1; ++h, nk += kStep) {
        ok = ok && warp_wait(&kfull[slot], phase);
        // the unit whose scale bytes were there has been multiplied
        const int old = nk - C::kSf;  // (with as many places for scale bytes as slots K's landing says so)
        if (C::kSf < NSLOT && old >= 0) ok = ok && warp_wait(&kempty[old % NSLOT], (old / NSLOT) & 1);
        tc_fence_after();
        const uint32_t *const sk = reinterpret_cast<const uint32_t *>(smem + C::kSRing + slot * C::kSSlot), *const sv = sk + 128;
        tmem_st4(tmem + C::kSfCol + 4 + sf * 4 + quad, sk[lane], sk[32 + lane], sk[64 + lane], sk[96 + lane]);
        constexpr int kOf = 128 / D;  // keys of a row of 128 elements
        const int first = t * C::kKeys + h * C::kUKeys + r * kOf;
        const bool live = C::kURows == 128 || r < C::kURows;
        const bool gone = live && s_ids[0][nk % kIds][(r * kOf / kPage) % UP] < 0;
        const uint32_t word = live ? sv[r] : 0x7F7F7F7Fu;
        // the usual case: factors 2^13 .. 2^-14, as halves of pairs of bytes
        const uint32_t lo = __byte_perm(word, 0, 0x4140), hi = __byte_perm(word, 0, 0x4342);
        uint32_t f[2], tb[kOf];
        if (D == 128) {
          const uint32_t m = max_u16x2(lo, hi);
          tb[0] = max(m & 0xFFFFu, m >> 16);
          f[0] = ((lo + 28u * 0x10001u) - tb[0] * 0x10001u) << 10;
          f[1] = ((hi + 28u * 0x10001u) - tb[0] * 0x10001u) << 10;
        } else {
          tb[0] = max(lo & 0xFFFFu, lo >> 16);
          tb[kOf - 1] = max(hi & 0xFFFFu, hi >> 16);
          f[0] = ((lo + 28u * 0x10001u) - tb[0] * 0x10001u) << 10;
          f[1] = ((hi + 28u * 0x10001u) - tb[kOf - 1] * 0x10001u) << 10;
        }
        float top_of[kOf], log_of[kOf];
#pragma unroll
        for (int w = 0; w < kOf; ++w) {
          top_of[w] = __uint_as_float(tb[w] << 23);
          log_of[w] = static_cast<float>(static_cast<int>(tb[w]) - 127);
        }
        const uint32_t least = min_u16x2(lo, hi), most = max(tb[0], tb[kOf - 1]);
        bool nan = false;
        if (__any_sync(0xffffffffu, gone || first + kOf > sg.nkeys || most == kNanScaleByte ||
                                        min(least & 0xFFFFu, least >> 16) < max(kMinScaleByte + 0u, most - 27u))) {
#pragma unroll 1
          for (int w = 0; w < kOf; ++w) {
            const int pos = first + w;
            const bool hidden = gone || pos >= sg.nkeys;
            int big = kMinScaleByte;
            for (int g = 0; g < G; ++g) {
              const int b = (word >> ((w * G + g) * 8)) & 255;
              if (b != kNanScaleByte) big = max(big, b);
            }
            uint32_t x[2] = {0, 0};
            for (int g = 0; g < G; ++g) {
              const int b = (word >> ((w * G + g) * 8)) & 255;
              uint32_t y = b < kMinScaleByte ? 0u : half_pow2(b - big + kVShift + 15);
              if (b == kNanScaleByte) {  // of a tree node: 0 here, and reaches the rows that see it at the segment's end
                y = pos >= sg.L ? 0u : 0x7E00u;
                nan = nan || (pos >= sg.L && !hidden);
              }
              if (!hidden) x[g >> 1] |= y << ((g & 1) * 16);
            }
            const float big_of = hidden ? 0.f : __uint_as_float(static_cast<uint32_t>(big) << 23);
            const float log = hidden ? NEG_INF : static_cast<float>(big - 127);
            if (w == 0) top_of[0] = big_of, log_of[0] = log, f[0] = x[0];
            else top_of[kOf - 1] = big_of, log_of[kOf - 1] = log, f[1] = x[0];
            if (D == 128) f[1] = x[1];
          }
        }
        if (live) {
          uint16_t *const factor = reinterpret_cast<uint16_t *>(smem + C::kFactor + ((i % kTiles) * U + h) * C::kFactors);
          float *const tops = top + (i % kTiles) * (2 * C::kKeys) + (D == 128 ? h * kSub : 0) + r;
#pragma unroll
          for (int w = 0; w < kOf; ++w) {
            tops[w * (C::kKeys / 2)] = top_of[w];
            tops[w * (C::kKeys / 2) + C::kKeys] = log_of[w];
          }
          if (D == 128) {
#pragma unroll
            for (int g = 0; g < 4; ++g) factor[g * C::kUKeys + r] = static_cast<uint16_t>(f[g >> 1] >> ((g & 1) * 16));
          } else {  // two keys' halves of a group
            reinterpret_cast<uint32_t *>(factor)[r] = __byte_perm(f[0], f[1], 0x5410);
            reinterpret_cast<uint32_t *>(factor)[C::kUKeys / 2 + r] = __byte_perm(f[0], f[1], 0x7632);
          }
        }
        const uint32_t any = __ballot_sync(0xffffffffu, gone);
        if (lane == 0) s_gone[i % kTiles][h * 4 + hw] = any;
        if (nan) s_nan[seg & 3] = 1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive1(&kready[sf]);
        slot += kStep;
        if (slot >= NSLOT) {
          slot -= NSLOT;
          phase ^= 1;
        }
        sf += kStep;
        if (sf >= C::kSf) sf -= C::kSf;
      }
    };
    // V of tile i in halves
    auto values = [&](int i) {
      const int u = i % NB;
      bar_sync(12 + (C::kApart ? set : 0), 32 * C::kVHelp);  // the factors of all four warps
      // the product that last read the buffer is done
      if (i >= C::kVBufs) ok = ok && warp_wait(&pvdone[(i - C::kVBufs) % NB], ((i - C::kVBufs) / NB) & 1);
      tc_fence_after();
#pragma unroll 1
      for (int h = h0; h < h1; ++h) {
        ok = ok && warp_wait(&vfull[vslot], vphase);
        if (!ok) break;
        const uint8_t *const vt = smem + C::kVRing + vslot * C::kVSlot;
        const uint8_t *const factor = smem + C::kFactor + ((i % kTiles) * U + h) * C::kFactors;
        if constexpr (C::kRowLanes) {
          // two keys and half of their elements a thread.  S has even positions before odd ones at D = 64.
          const int p = r & 63, e0 = (r >> 6) * (D / 2);
          const int r0 = D == 128 ? 2 * p : p, r1 = D == 128 ? 2 * p + 1 : 64 + p;
          uint8_t *const to = smem + C::kH + u * C::kHBuf;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {  // 16 elements
            const int el = e0 + c * 16;
            const uint4 v = *reinterpret_cast<const uint4 *>(vt + (D == 128 ? sw128(p, el) : sw64(p, el)));
            const uint32_t f = *reinterpret_cast<const uint32_t *>(factor + ((el / kQ4Group) * C::kUKeys + 2 * p) * 2);
            const uint32_t f0 = __byte_perm(f, 0, 0x1010), f1 = __byte_perm(f, 0, 0x3232);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t x[8], y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t hh[4];
              e2m1_halves8(w[k], hh);
              x[2 * k] = hmul2(__byte_perm(hh[0], hh[1], 0x5410), f0);
              x[2 * k + 1] = hmul2(__byte_perm(hh[2], hh[3], 0x5410), f0);
              y[2 * k] = hmul2(__byte_perm(hh[0], hh[1], 0x7632), f1);
              y[2 * k + 1] = hmul2(__byte_perm(hh[2], hh[3], 0x7632), f1);
            }
            uint8_t *const bl = to + (el >> 6) * C::kBlock;
            const int cb = (el & 63) * 2;
            *reinterpret_cast<uint4 *>(bl + sw128(r0, cb)) = make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4 *>(bl + sw128(r0, cb + 16)) = make_uint4(x[4], x[5], x[6], x[7]);
            *reinterpret_cast<uint4 *>(bl + sw128(r1, cb)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4 *>(bl + sw128(r1, cb + 16)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
          fence_proxy_async();  // V (generic writes) -> visible to the tensor cores
        } else {
          // V^T: 32 keys of this warp's 32 elements (at d = 64 the upper lanes repeat the lower ones) at a time.  Row i of
          // ldmatrix' 16 is the pair of keys with bits 1 and 2 of i exchanged, so that a lane's four bytes are two
          // columns of either 16x256b store, keys 4 (l % 4) .. + 3 (bits 3 and 4 of the key exchanged), and eight rows never meet in a bank.
          const int g = D == 128 ? hw : hw & 1, i16 = lane & 15;
          const int pair = (i16 & 9) | (i16 & 2) << 1 | (i16 & 4) >> 1, el = g * 32 + (lane >> 4) * 16;
          // (two sets at D = 64: half of the unit's keys each)
          constexpr int kMine = C::kUKeys * 4 / C::kVHelp;
          const int key0 = C::kApart ? 0 : set * kMine;
          uint32_t from = smem_u32(vt) + key0 / 2 * D + (D == 128 ? sw128(pair, el) : sw64(pair, el));
          const uint8_t *f = factor + (g * C::kUKeys + key0 + (lane & 2) * 8 + (lane & 1) * 4) * 2;
          uint32_t to = tmem + C::kACol + (i % C::kABufs) * C::kACols + h * (kSub / 2) + key0 / 2 + quad;
          // a rolled loop: the softmax warps' code has to stay in the instruction cache; the next keys are read ahead
          uint32_t c[4], next[4];
          load_columns(from, c);
          uint2 m0 = *reinterpret_cast<const uint2 *>(f), m1 = *reinterpret_cast<const uint2 *>(f + 16);
#pragma unroll (C::kSets == 2 ? 1 : 2)
          for (int k0 = 0; k0 < kMine; k0 += 32, to += 16) {
            uint2 n0 = m0, n1 = m1;
            if (k0 + 32 < kMine) {
              from += 16 * D;
              f += 64;
              load_columns(from, next);
              n0 = *reinterpret_cast<const uint2 *>(f);
              n1 = *reinterpret_cast<const uint2 *>(f + 16);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // 16 elements each
              uint32_t x[4], y[4];
              e2m1_halves8(c[e * 2], x);
              e2m1_halves8(c[e * 2 + 1], y);
              const uint32_t v[8] = {hmul2(x[0], m0.x), hmul2(x[1], m0.y), hmul2(y[0], m0.x), hmul2(y[1], m0.y),
                                     hmul2(x[2], m1.x), hmul2(x[3], m1.y), hmul2(y[2], m1.x), hmul2(y[3], m1.y)};
              tmem_st_16x16(to + (static_cast<uint32_t>(e * 16) << 16), v);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) c[q] = next[q];
            m0 = n0;
            m1 = n1;
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive1(&vempty[vslot]);
          if (h == h1 - 1) mbar_arrive1(&vready[u]);
        }
        vslot += kStep;
        if (vslot >= NSLOT) {
          vslot -= NSLOT;
          vphase ^= 1;
        }
      }
    };
    for (int i0 = 0, seg = 0; more; ++seg) {
      const int n = sg.t1 - sg.t0;
      int x = 0;
      const bool scaling = C::kApart || set == 0;
      for (; x < n && x < NB; ++x)
        if (scaling) scales(i0 + x, sg.t0 + x, seg);
      Segments next = sg;
      more = next.step(a);
      // the next segment's rows, once the segment before this has left their buffer
      auto next_rows = [&] {
        const int buf = (seg + 1) & 1;
        ok = ok && (seg < 1 || warp_wait(&qempty[buf], ((seg - 1) >> 1) & 1));
        all = !bar_or(11, C::kHelpers * 32, !ok || s_abort);
        if (!all) return;
        prepare(next, buf, warp - C::kHelpWarp, C::kHelpers, 11);
        if (lane == 0) mbar_arrive1(&qfull[buf]);
      };
      // With 128 rows behind this segment's first tile, which need not wait for that (256 rows of 4096 keys, d 128: 121 us
      // instead of 129); below, where rows are few, in front of it (one token of 64 sequences 144 us instead of 152).
      if (!C::kRowLanes && more) next_rows();
      for (int y = 0; y < n && all; ++y) {
        values(i0 + y);
        if (x < n) {
          if (scaling) scales(i0 + x, sg.t0 + x, seg);
          ++x;
        }
        if (C::kRowLanes && y == 0 && more) next_rows();
      }
      if (!all) break;
      i0 += n;
      sg = next;
    }
    if (!ok || !all) s_abort = 1;
  } else if constexpr (C::kRowLanes) {
    // ---------------- softmax, a lane per row: group g has the keys g * 32 .. + 31 of every tile
    const int g = (warp - C::kSoftWarp) / 4, wg = warp & 3, r = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>(wg * 32) << 16;
    const uint32_t tS = tmem + g * 32 + lane_off, tO = tmem + C::kOCol + g * (D / 4) + lane_off;
    const int bar = 1 + wg;  // the four warps that share 32 rows
    int i0 = 0, seg = 0;     // the segment's first tile in the CTA's count
    uint32_t sphase = 0;     // parities of sfull
    bool dead = false;
    bool more = sg.first(a, piece);
    if (more) {
      prepare(sg, 0, warp - C::kHelpWarp, C::kSoftWarps + C::kHelpers, 10);
      bar_sync(10, (C::kSoftWarps + C::kHelpers) * 32);
    }
    for (; more; more = sg.step(a), ++seg) {
      const int buf = seg & 1, n = sg.t1 - sg.t0, row = sg.mt * RT + r;
      const bool live = row < a.nrows, some = sg.mt * RT + wg * 32 < a.nrows;  // this row; some row of the warp
      const int qi = min(static_cast<int>((row * a.group_magic) >> 16), kMaxNodes - 1);
      bool ok = warp_wait(&qfull[buf], (seg >> 1) & 1);
      const float cq = live ? fminf(qs[buf][r] * (a.scale_log2 * kQueryUnit), 3e38f) : 0.f;
      // the row's m (all four groups keep it), and what is added to its scores; a row behind the last gets p = 0
      float m = NEG_INF, add = live ? 0.f : -1e30f;
      uint64_t l2[2] = {0, 0};
      bool begin = true, unset = live;  // before the segment's first tile; no visible key so far
      for (int x = 0; x < n; ++x) {
        const int i = i0 + x, t = sg.t0 + x, u = i % NB;  // u: S and P buffer
        ok = ok && warp_wait(&sfull[u], sphase >> u & 1);
        sphase ^= 1u << u;  // the scales were there before K was
        tc_fence_after();
        bool part = (t + 1) * kSub > min(sg.L, sg.nkeys);
        part = __any_sync(0xffffffffu, part || (lane < U * 4 && s_gone[i % kTiles][lane] != 0));
        if (some) {
          const float4 *const tops = reinterpret_cast<const float4 *>(top + (i % kTiles) * (2 * C::kKeys) + g * 32);
          const float4 *const logs = tops + C::kKeys / 4;
          uint32_t vis = ~0u;
          if (part) {
            const uint32_t *const bits = anc[buf][qi];
            auto window = [&](int node) {  // nodes node .. + 31; the prefix before them is seen by all
              if (node <= -32) return ~0u;
              const int word = node >> 5;
              const uint32_t lo = node < 0 ? ~0u : (word < kMaxNodes / 32 ? bits[word] : 0u);
              const uint32_t hi = word + 1 < kMaxNodes / 32 ? bits[word + 1] : 0u;
              return __funnelshift_r(lo, hi, node & 31);
            };
            if (D == 128) {
              vis = window(t * kSub + g * 32 - sg.L);
            } else {  // even positions, then odd ones
              const int node = t * kSub + (g & 1) * 64 + (g >> 1) - sg.L;
              vis = every_other_bit(window(node)) | every_other_bit(window(node + 32)) << 16;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 s4 = tops[j];
              vis &= ~((s4.x == 0.f ? 1u : 0u) << (4 * j) | (s4.y == 0.f ? 2u : 0u) << (4 * j) |
                       (s4.z == 0.f ? 4u : 0u) << (4 * j) | (s4.w == 0.f ? 8u : 0u) << (4 * j));
            }
          }
          float y[32];
          // y = x - m + 11 (x for a row without m); hidden keys -inf
          auto scores = [&]() {
            tmem_ld16_async(tS + u * kSub, y);
            tmem_ld16_async(tS + u * kSub + 16, y + 16);
            tmem_wait16(y);
            tmem_wait16(y + 16);
            const uint64_t off2 = pack2(add, add), c2 = pack2(cq, cq);
#pragma unroll
            for (int j = 0; j < 32; j += 2) unpack2(fma2(pack2(y[j], y[j + 1]), c2, off2), y[j], y[j + 1]);
            if (part) {
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = ((vis >> j) & 1u) ? y[j] : NEG_INF;
            }
          };
          // y, and whether a row's m has to move; then once more with the new m
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            scores();
            if (pass == 1) break;
            float t4[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 l4 = logs[j];
              float z[4];
              unpack2(add2(pack2(y[4 * j], y[4 * j + 1]), pack2(l4.x, l4.y)), z[0], z[1]);
              unpack2(add2(pack2(y[4 * j + 2], y[4 * j + 3]), pack2(l4.z, l4.w)), z[2], z[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) t4[k] = fmaxf(t4[k], z[k]);
            }
            const float big = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
            if (!bar_or(bar, 128, big > kGrow || unset || !ok)) break;
            red[g][r] = big;
            // O is rescaled below: every P V before has to be in it
            if (!begin) {
              ok = warp_wait(&pvdone[(i - 1) % NB], ((i - 1) / NB) & 1) && ok;
              tc_fence_after();
            }
            if (bar_or(bar, 128, !ok)) {
              dead = true;
              break;
            }
            const float z = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
            bar_sync(bar, 128);  // read, before the next is written
            float f = 1.f;
            if (live) {
              if (m == NEG_INF) {
                m = z;
                unset = m == NEG_INF;
              } else if (z > kGrow) {
                m += z - kMoved;
                f = ex2(kMoved - z);
              }
              add = unset ? 0.f : kBias - m;
            }
            if (!begin && __any_sync(0xffffffffu, f != 1.f)) {
              const uint64_t f2 = pack2(f, f);
              l2[0] = mul2(l2[0], f2);
              l2[1] = mul2(l2[1], f2);
#pragma unroll 1
              for (int k = 0; k < D / 64; ++k) {  // this group's quarter of O
                const uint32_t at = tO + k * 16;
                float o[16];
                tmem_ld16(at, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_st16(at, o);
              }
            }
          }
          if (dead) break;
          begin = false;
          const uint64_t unit2 = pack2(kSumUnit, kSumUnit);
          uint32_t hp[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 s4 = tops[j];
            const uint64_t w2[2] = {pack2(s4.x, s4.y), pack2(s4.z, s4.w)};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint64_t p = pack2(ex2(y[4 * j + 2 * k]), ex2(y[4 * j + 2 * k + 1]));
              l2[k] = fma2(p, unit2, l2[k]);
              float a0, a1;
              unpack2(mul2(p, w2[k]), a0, a1);
              hp[2 * j + k] = half2_of(a0, a1);
            }
          }
          // the product before has read its P
          if (i > 0) ok = ok && warp_wait(&pvdone[(i - 1) % NB], ((i - 1) / NB) & 1);
          tc_fence_after();
          tmem_st16_async(tmem + C::kACol + g * 16 + lane_off, hp);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&pfull[u]);
      }
      // ---------------- the segment's end: l, then O from TMEM, a quarter of the row's elements each
      if (dead) ok = false;
      {
        float l0, l1, l3, l4;
        unpack2(l2[0], l0, l1);
        unpack2(l2[1], l3, l4);
        red[g][r] = __fadd_rn(__fadd_rn(l0, l1), __fadd_rn(l3, l4));
      }
      const int il = i0 + n - 1;
      ok = ok && warp_wait(&pvdone[il % NB], (il / NB) & 1);
      tc_fence_after();
      if (bar_or(9, kSoftThreads, !ok)) {
        s_abort = 1;
        break;
      }
      const bool whole = sg.t0 == 0 && sg.t1 == sg.nt, nan = s_nan[seg & 3] != 0;
      if (tid == C::kSoftWarp * 32) s_nan[(seg + 2) & 3] = 0;
      if (some) {
        const int slot = blockIdx.x * 2 + (sg.t0 > 0 ? 0 : 1);
        const float L = __fadd_rn(__fadd_rn(red[0][r], red[1][r]), __fadd_rn(red[2][r], red[3][r]));
        const float factor = L == 0.f ? 0.f : (whole ? 1.f / L : 1.f);
        const int64_t orow = (static_cast<int64_t>(sg.b) * a.Nq + qi) * a.Hq + sg.hk * a.group + (row - qi * a.group);
        if (live && g == 0) {
          if (!whole)
            a.part_ml[slot * RT + r] = make_float2(m, L);
          else if (a.lse)
            a.lse[orow] = L == 0.f ? NEG_INF : (m - kSumBias + log2f(L)) * 0.69314718055994531f;
        }
#pragma unroll 1
        for (int j0 = 0; j0 < D / 4; j0 += 16) {
          float o[16];
          tmem_ld16(tO + j0, o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = o[j] * kOutUnit * factor;
          if (!live) continue;
          const int e0 = g * (D / 4) + j0;
          if (nan) {
            // tree nodes of this segment that this row sees and whose v has a NaN scale here
            const int from = sg.t0 * C::kKeys - sg.L, to = min(sg.nkeys, sg.t1 * C::kKeys) - sg.L;
            for (int node = max(0, from); node < to; ++node) {
              if (!((anc[buf][qi][node >> 5] >> (node & 31)) & 1u)) continue;
              const int pos = sg.L + node, blk = a.table[static_cast<int64_t>(sg.b) * a.maxb + pos / kPage];
              if (blk < 0 || blk >= a.num_blocks) continue;
              const int64_t at = (static_cast<int64_t>(blk) * a.Hkv + sg.hk) * kPage + pos % kPage;
              if (a.vs[at * G + e0 / kQ4Group] != kNanScaleByte) continue;
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __int_as_float(0x7fc00000);
            }
          }
          if (whole) {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(o[2 * j + 1]), "f"(o[2 * j]));
            uint4 *const to = reinterpret_cast<uint4 *>(a.out + orow * D + e0);
            to[0] = make_uint4(h[0], h[1], h[2], h[3]);
            to[1] = make_uint4(h[4], h[5], h[6], h[7]);
          } else {
            float4 *const to = reinterpret_cast<float4 *>(a.part_o + (static_cast<int64_t>(slot) * RT + r) * D + e0);
#pragma unroll
            for (int j = 0; j < 4; ++j) to[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
      }
      tc_fence_before();
      bar_sync(9, kSoftThreads);  // O and the sums have been read
      if (lane == 0) mbar_arrive1(&qempty[buf]);
      i0 += n;
    }
  } else {
    // ---------------- softmax: group g of the rows, one thread per key
    const int g = (warp - C::kSoftWarp) / 4, wg = warp & 3, tg = tid & 127;
    const int col = g * CG;
    const uint32_t lane_off = static_cast<uint32_t>(wg * 32) << 16;
    const uint32_t tS = tmem + col + lane_off, tO = tmem + C::kOCol + col + lane_off;
    const int bar = 1 + g;
    int i0 = 0, seg = 0;  // the segment's first tile in the CTA's count
    uint32_t sphase = 0;  // parities of sfull
    bool dead = false;
    bool more = sg.first(a, piece);
    if (more) {
      prepare(sg, 0, warp - C::kHelpWarp, C::kSoftWarps + C::kHelpers, 10);
      bar_sync(10, (C::kSoftWarps + C::kHelpers) * 32);
    }
    for (; more; more = sg.step(a), ++seg) {
      const int buf = seg & 1, n = sg.t1 - sg.t0;
      const int hk = sg.hk, mt = sg.mt;
      const int row0 = mt * RT + col;  // the warp's first row of (b, hk)
      bool ok = warp_wait(&qfull[buf], (seg >> 1) & 1);
      if (tg < CG) {
        s_m[col + tg] = NEG_INF;
        float *const rc = reinterpret_cast<float *>(&rowc[(col + tg) >> 1]) + (tg & 1);
        rc[0] = fminf(qs[buf][col + tg] * (a.scale_log2 * kQueryUnit), 3e38f);
        rc[2] = 0.f;
      }
      bar_sync(bar, 128);
      uint64_t l2[CG / 2];
#pragma unroll
      for (int j = 0; j < CG / 2; ++j) l2[j] = 0;
      bool begin = true, unset = true;  // before the segment's first tile; a row without a visible key so far
      for (int x = 0; x < n; ++x) {
        const int i = i0 + x, t = sg.t0 + x, u = i % NB;  // u: S and P buffer
        ok = ok && warp_wait(&sfull[u], sphase >> u & 1);
        sphase ^= 1u << u;  // the scales were there before K was
        tc_fence_after();
        // this thread's keys: their scales (read where they are used: at 64 rows the warps have 80 registers a thread),
        // and the rows that see them
        const float *const tops = top + (i % kTiles) * (2 * C::kKeys) + tg, *const logs = tops + C::kKeys;
        auto key_of = [&](int h) { return D == 128 ? h * kSub + tg : 2 * tg + h; };
        uint32_t vis[KT];
        bool hidden[KT], part = false;
#pragma unroll
        for (int h = 0; h < KT; ++h) {
          hidden[h] = tops[h * kSub] == 0.f;
          part = part || hidden[h] || t * C::kKeys + key_of(h) >= sg.L;
        }
        part = __any_sync(0xffffffffu, part);
        if (part) {
#pragma unroll
          for (int h = 0; h < KT; ++h) {
            const int node = t * C::kKeys + key_of(h) - sg.L;
            vis[h] = hidden[h] ? 0u : ~0u;
            if (!hidden[h] && node >= 0) {
              // row j is query (row0 + j) / group: the rows of one query are neighbours
              uint32_t see = 0;
              int qi = static_cast<int>((row0 * a.group_magic) >> 16), j0 = 0;
#pragma unroll 1
              for (int j1 = (qi + 1) * a.group - row0; j0 < CG && qi < a.Nq; ++qi, j0 = j1, j1 += a.group)
                if ((anc[buf][qi][node >> 5] >> (node & 31)) & 1u)
                  see |= (j1 < CG ? (1u << j1) - 1u : ~0u) & (~0u << j0);
              vis[h] = see;
            }
          }
        }
        float y[KT][CG];
        // y = x - m + 11 (x for a row without m); hidden keys -inf
        auto scores = [&]() {
#pragma unroll
          for (int h = 0; h < KT; ++h) tmem_ld16_async(tS + (u * KT + h) * RT, y[h]);
#pragma unroll
          for (int h = 0; h < KT; ++h) tmem_wait16(y[h]);
#pragma unroll
          for (int j = 0; j < CG; j += 2) {
            const float4 rc = rowc[(col + j) / 2];
#pragma unroll
            for (int h = 0; h < KT; ++h)
              unpack2(fma2(pack2(y[h][j], y[h][j + 1]), pack2(rc.x, rc.y), pack2(rc.z, rc.w)), y[h][j], y[h][j + 1]);
          }
          if (part) {
#pragma unroll
            for (int h = 0; h < KT; ++h)
#pragma unroll
              for (int j = 0; j < CG; ++j) y[h][j] = ((vis[h] >> j) & 1u) ? y[h][j] : NEG_INF;
          }
        };
        // y, and whether a row's m has to move; then once more with the new m
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          scores();
          if (pass == 1) break;
          float most = NEG_INF;
#pragma unroll
          for (int h = 0; h < KT; ++h) {
            float t4[4] = {y[h][0], y[h][1], y[h][2], y[h][3]};
#pragma unroll
            for (int j = 4; j < CG; ++j) t4[j & 3] = fmaxf(t4[j & 3], y[h][j]);
            most = fmaxf(most, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) + logs[h * kSub]);
          }
          if (!bar_or(bar, 128, most > kGrow || unset || !ok)) break;
          // the rows' largest log2 of P v_scale (of a row without a key so far: x + log2 v_scale) in this tile
          float big = NEG_INF;
#pragma unroll
          for (int j = 0; j < CG; ++j) {
            const float z = warp_top(fmaxf(y[0][j] + logs[0], y[1][j] + logs[kSub]));
            if (lane == j) big = z;
          }
          if (lane < CG) red[wg][col + lane] = big;
          // O is rescaled below: every P V before has to be in it
          if (!begin) {
            ok = warp_wait(&pvdone[(i - 1) % NB], ((i - 1) / NB) & 1) && ok;
            tc_fence_after();
          }
          if (bar_or(bar, 128, !ok)) {
            dead = true;
            break;
          }
          bool none = false;
          if (tg < CG) {
            const int r = col + tg;
            const float mo = s_m[r];
            const float z = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
            float mn = mo, f = 1.f;
            if (mo == NEG_INF) {
              mn = z;
              none = mn == NEG_INF;
            } else if (z > kGrow) {
              mn = mo + (z - kMoved);
              f = ex2(kMoved - z);
            }
            s_m[r] = mn;
            s_f[r] = f;
            reinterpret_cast<float *>(&rowc[r >> 1])[2 + (tg & 1)] = none ? 0.f : kBias - mn;
          }
          unset = bar_or(bar, 128, none);
          if (!begin) {
            bool moved = false;
#pragma unroll
            for (int j = 0; j < CG; ++j) moved = moved || s_f[col + j] != 1.f;
            if (moved) {
#pragma unroll
              for (int j = 0; j < CG / 2; ++j) l2[j] = mul2(l2[j], pack2(s_f[col + 2 * j], s_f[col + 2 * j + 1]));
              float o[CG];
              tmem_ld16(tO, o);
#pragma unroll
              for (int j = 0; j < CG; ++j) o[j] *= s_f[col + j];
              tmem_st16(tO, o);
            }
          }
        }
        if (dead) break;
        begin = false;
        // the P buffer is free: S of this tile was issued behind P V of tile i - NB
        const uint64_t unit2 = pack2(kSumUnit, kSumUnit);
#pragma unroll
        for (int h = 0; h < KT; ++h) {
          const float wv = tops[h * kSub];
          const uint64_t w2 = pack2(wv, wv);
          uint32_t hp[CG / 2];
#pragma unroll
          for (int j = 0; j < CG / 2; ++j) {
            const uint64_t p = pack2(ex2(y[h][2 * j]), ex2(y[h][2 * j + 1]));
            l2[j] = fma2(p, unit2, l2[j]);
            float a0, a1;
            unpack2(mul2(p, w2), a0, a1);
            hp[j] = half2_of(a0, a1);
          }
          const int key = key_of(h), row = (key & 0x67) | (key & 8) << 1 | (key & 16) >> 1;  // where V^T has the key
          uint8_t *const pb = smem + C::kH + u * C::kHBuf + (key >> 7) * C::kBlock;
          *reinterpret_cast<uint4 *>(pb + sw128(row, col * 2)) = make_uint4(hp[0], hp[1], hp[2], hp[3]);
          *reinterpret_cast<uint4 *>(pb + sw128(row, col * 2 + 16)) = make_uint4(hp[4], hp[5], hp[6], hp[7]);
        }
        fence_proxy_async();  // P (generic writes) -> visible to the tensor cores
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&pfull[u]);
      }
      // ---------------- the segment's end: l, then O from TMEM
      if (dead) ok = false;
      {
        float z[CG];
#pragma unroll
        for (int j = 0; j < CG; j += 2) unpack2(l2[j / 2], z[j], z[j + 1]);
        const float sum = warp_columns(z, lane);
        if (!(lane & 1)) red[wg][col + (lane >> 1)] = sum;
      }
      const int il = i0 + n - 1;
      ok = ok && warp_wait(&pvdone[il % NB], (il / NB) & 1);
      tc_fence_after();
      if (bar_or(9, kSoftThreads, !ok)) {
        s_abort = 1;
        break;
      }
      const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
      const int slot = blockIdx.x * 2 + (sg.t0 > 0 ? 0 : 1);
      if (tid == C::kSoftWarp * 32) s_nan[(seg + 2) & 3] = 0;
      for (int r = tid - C::kSoftWarp * 32; r < RT; r += kSoftThreads) {
        const float M = s_m[r], L = __fadd_rn(__fadd_rn(red[0][r], red[1][r]), __fadd_rn(red[2][r], red[3][r]));
        s_f[r] = L == 0.f ? 0.f : (whole ? 1.f / L : 1.f);
        const int row = mt * RT + r;
        if (row < a.nrows) {
          if (!whole) a.part_ml[slot * RT + r] = make_float2(M, L);
          else if (a.lse) {
            const int qi = static_cast<int>((row * a.group_magic) >> 16), head = hk * a.group + (row - qi * a.group);
            a.lse[(static_cast<int64_t>(sg.b) * a.Nq + qi) * a.Hq + head] =
                L == 0.f ? NEG_INF : (M - kSumBias + log2f(L)) * 0.69314718055994531f;
          }
        }
      }
      bar_sync(9, kSoftThreads);
      const bool nan = s_nan[seg & 3] != 0;
      // four rows at a time; at d = 64 the upper 64 lanes of O repeat the lower ones and take half of the rows
      constexpr int kShares = C::kGroups * (128 / D);
      const int share = D == 128 ? g : g * 2 + (wg >> 1), el = tg & (D - 1);
      uint16_t *const to = a.out + (static_cast<int64_t>(sg.b) * a.Nq * a.Hq + hk * a.group) * D + el;
#pragma unroll 1
      for (int j0 = share * 4; j0 < RT; j0 += kShares * 4) {
        const int r0 = mt * RT + j0;
        if (r0 >= a.nrows) break;
        float o[4];
        tmem_ld4(tmem + C::kOCol + j0 + lane_off, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = o[j] * kOutUnit * s_f[j0 + j];
        if (nan) {
          // tree nodes of this segment whose v has a NaN scale at this thread's element
          const int from = sg.t0 * C::kKeys - sg.L, to = min(sg.nkeys, sg.t1 * C::kKeys) - sg.L;
          for (int node = max(0, from); node < to; ++node) {
            const int pos = sg.L + node, blk = a.table[static_cast<int64_t>(sg.b) * a.maxb + pos / kPage];
            if (blk < 0 || blk >= a.num_blocks) continue;
            const int64_t at = (static_cast<int64_t>(blk) * a.Hkv + hk) * kPage + pos % kPage;
            if (a.vs[at * G + el / kQ4Group] != kNanScaleByte) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int qi = min(static_cast<int>(((r0 + j) * a.group_magic) >> 16), kMaxNodes - 1);
              if ((anc[buf][qi][node >> 5] >> (node & 31)) & 1u) o[j] = __int_as_float(0x7fc00000);
            }
          }
        }
        if (whole) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = r0 + j;
            if (r >= a.nrows) break;
            const int qi = static_cast<int>((r * a.group_magic) >> 16), at = qi * a.Hq + (r - qi * a.group);
            uint32_t b2;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b2) : "f"(0.f), "f"(o[j]));
            to[static_cast<int64_t>(at) * D] = static_cast<uint16_t>(b2 & 0xFFFFu);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) a.part_o[(static_cast<int64_t>(slot) * RT + j0 + j) * D + el] = o[j];
        }
      }
      tc_fence_before();
      bar_sync(9, kSoftThreads);  // O, the factors and the sums have been read
      if (lane == 0) mbar_arrive1(&qempty[buf]);
      i0 += n;
    }
  }
  if (tid == 0 && a.split) {  // what the piece's last item still needs
    int4 need = make_int4(0, 0, 0, 0);
    Segments x;
    for (bool more = x.first(a, piece); more; more = x.step(a))
      if (x.t0 == 0 && x.t1 < x.nt)
        need = make_int4(1 + (x.nt - x.t1 + piece.chunk - 1) / piece.chunk, x.b, x.hk, x.mt);
    a.info[blockIdx.x] = need;
  }
  tc_fence_before();
  __syncthreads();
  if (s_abort && tid == 0) atomicOr(a.status, kFlagWaitTimeout);
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}


}  // namespace q4
}  // namespace ssd

using namespace ssd;

namespace {

using q4::Args;

// K: [num_blocks][Hkv * rows of 128 elements][128 elements], boxes of one block's rows of a head, a byte per element in
// shared memory; V: [num_blocks][Hkv * 8 pairs of positions][d bytes]
bool make_key_map(CUtensorMap *m, const void *base, int64_t num_blocks, int Hkv, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint32_t rows = static_cast<cuuint32_t>(line::kPage * d / 128);
  cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(Hkv) * rows, static_cast<cuuint64_t>(num_blocks)};
  cuuint64_t strides[2] = {64, 64 * static_cast<cuuint64_t>(Hkv) * rows};
  cuuint32_t box[3] = {128, rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool make_value_map(CUtensorMap *m, const void *base, int64_t num_blocks, int Hkv, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  constexpr cuuint32_t kRows = line::kPage / 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hkv) * kRows,
                        static_cast<cuuint64_t>(num_blocks)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(d) * Hkv * kRows};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(d), kRows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RT>
cudaError_t launch(const CUtensorMap &kmap, const CUtensorMap &vmap, const Args &a, unsigned grid, cudaStream_t cs) {
  using C = q4::Cfg<D, RT>;
  if (a.keys != C::kKeys) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(q4::k_branch_attn_q4<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  q4::k_branch_attn_q4<D, RT><<<grid, C::kThreads, C::kSmem, cs>>>(kmap, vmap, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.split) return e;
  return launch_merge<D, RT>(a, grid, cs);
}

template <int D>
cudaError_t launch_shape(const Shape &s, const CUtensorMap &kmap, const CUtensorMap &vmap, const Args &a,
                         unsigned grid, cudaStream_t cs) {
  switch (s.RT) {
    case 16: return launch<D, 16>(kmap, vmap, a, grid, cs);
    case 32: return launch<D, 32>(kmap, vmap, a, grid, cs);
    case 48: return launch<D, 48>(kmap, vmap, a, grid, cs);
    case 64: return launch<D, 64>(kmap, vmap, a, grid, cs);
    default: return launch<D, 128>(kmap, vmap, a, grid, cs);
  }
}

}  // namespace

extern "C" {

size_t ssd_attention_q4_workspace_size(int B, int Nq, int Hq, int Hkv, int d) {
  if (B <= 0 || Nq <= 0 || Nq > line::kMaxNodes || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 16 ||
      (d != 64 && d != 128))
    return 0;
  return workspace_of(shape_of(Nq, Hq, Hkv), d, attn_num_sms()).total;
}

ssd_status_t ssd_branch_attention_q4(const void *q, const void *k_cache, const void *v_cache, const uint8_t *k_scale,
                                     const uint8_t *v_scale, const int32_t *block_table, int maxb, int64_t num_blocks,
                                     const int32_t *prefix_len, const int32_t *parent, int B, int N, int Nq, int Hq,
                                     int Hkv, int d, float scale, void *out, float *lse, uint32_t *status, void *ws,
                                     size_t ws_bytes, ssd_stream_t s) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return SSD_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return SSD_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SSD_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16 || N < 1 || N > line::kMaxNodes || Nq < 1 || Nq > N) return SSD_ERR_UNSUPPORTED;
  if (B == 0) return SSD_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len || !parent || !out ||
      !status || maxb < 1 || num_blocks < 1)
    return SSD_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(k_scale) |
       reinterpret_cast<uintptr_t>(v_scale)) & 15u ||
      (reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 31u)
    return SSD_ERR_UNSUPPORTED;
  if (num_blocks > 0x7fffffffLL || static_cast<int64_t>(B) * Hkv > 0x7fffffffLL / 32) return SSD_ERR_UNSUPPORTED;
  const Shape sh = shape_of(Nq, Hq, Hkv);
  Args a{};
  a.ks = k_scale;
  a.vs = v_scale;
  unsigned grid;
  if (!make_line(a, sh, q, block_table, maxb, num_blocks, prefix_len, parent, B, N, Nq, Hq, Hkv, d, scale, out, lse,
                 status, ws, ws_bytes, grid))
    return SSD_ERR_UNSUPPORTED;
  CUtensorMap kmap, vmap;
  if (!make_key_map(&kmap, k_cache, num_blocks, Hkv, d) || !make_value_map(&vmap, v_cache, num_blocks, Hkv, d))
    return SSD_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = d == 64 ? launch_shape<64>(sh, kmap, vmap, a, grid, cs)
                                : launch_shape<128>(sh, kmap, vmap, a, grid, cs);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
