// kv8_dense_body.cuh -- dense prefix backend over the 8-bit cache on the 5th-generation tensor cores
// (tcgen05/TMEM), head_dim 128, bf16 q.
//
// One CTA takes one (prefix group, KV head j, 128-row block, L_p piece), as the 16-bit dense kernel:
// rows are the group's (request, head-in-group) pairs of KV head j, and for each 128-token tile i
//     S(i) = Q K(i)^T       (8 tcgen05.mma 128x128x16, fp16 codes of K from shared memory)
//     P(i) = 2^(z - m)      (softmax warps; fp16, written back over S(i) in TMEM)
//     O   += P(i) V(i)      (8 tcgen05.mma with A = P(i) read from TMEM, fp16 codes of V)
// Number format.  Codes become fp16 exactly; q is brought into fp16's range by a power of two per
// row (exact but for elements 2^-31 below the row's largest).  The scales of a slab are those of
// 64-token blocks counted from its start, so each half of a tile has one K scale ks and one V scale
// vs: z = s ks + log2 vs (base 2) costs the FMA that the softmax needs anyway, P = 2^(z - m) is p times
// vs, which is what meets the V codes, and the row sum adds each half's sum of P once, over vs.  The
// running maximum m is taken over z.  P carries a factor of 2^7: it is at most 2^15 (m may lag the row's
// maximum by 2^8, see below), and fp16 keeps its 11 bits down to 2^-21 of the largest weight.
// Roles (13 warps):
//  * warps 0-7, softmax and epilogue: warp w serves TMEM lanes 32*(w%4).. (row r = lane r), all 128
//    columns of the tiles i with i % 2 == w / 4; the two warps of a row quarter take turns, half a
//    tile apart.  The running max is a chain over the tiles: the warp of tile i reads the max used
//    for tile i-1 from shared memory, keeps it unless the tile's row max exceeds it by more than
//    2^8 (then O is rescaled in TMEM), and publishes its own.
//  * warps 8-9 (K) and 10-11 (V), conversion: the tile's codes arrive by TMA (a box of 128 tokens x
//    128 bytes, two in flight for each of K and V); each thread turns 16 codes at a time into fp16
//    and stores them in the 128-byte-swizzled layout that the MMA operands have.  Rows of V past
//    the piece's end are stored as zeros.  The pair's first lane then refills the box.
//  * warp 12, the MMAs, issued as their inputs become ready: S(j) up to three tiles ahead of the PV
//    products (three S/P buffers in TMEM).
// Every mbarrier wait is bounded in time; on expiry the CTA raises an abort flag, latches an error,
// drains what it issued and frees its TMEM.
#pragma once

#include <cuda.h>

#include "internal.h"
#include "kv8_suffix_body.cuh"
#include "kv8_util.cuh"
#include "launch_util.cuh"
#include "mma_util.cuh"
#include "tc_util.cuh"

namespace granikv {
namespace k8d {
namespace {

using k8s::lg2_approx;
using k8s::pack_f16;

constexpr int kD = 128;
constexpr int kM = kDenseRows;                // 128 query rows per CTA
constexpr int kN = kDenseTile;                // 128 tokens per tile
static_assert(kN == 2 * kKv8Block, "each half of a tile is one block of the slab");
constexpr int kSlots = 2;                     // slots of each ring: fp16 K, fp16 V, codes of K, codes of V
constexpr int kSBufs = 3;                     // S/P buffers in TMEM
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kWarpConv = 8, kConvThreads = 64;  // warps 8, 9: K; 10, 11: V
constexpr int kWarpMma = 12;
constexpr int kThreads = 416;
constexpr int kHalf = kN * 128;               // one 64-dim half of an fp16 tile: 16 KB
constexpr int kTile = 2 * kHalf;              // 32 KB
constexpr int kCodes = kN * kD;               // a tile's codes: 16 KB
constexpr int kQBytes = kM * kD * 2;          // 32 KB (two 64-dim K-blocks)
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kQBytes;
constexpr int kOffV = kOffK + kSlots * kTile;
constexpr int kOffCodes = kOffV + kSlots * kTile;  // codes of K: slots 0, 1; of V: slots 2, 3
constexpr int kOffUnit = kOffCodes + 2 * kSlots * kCodes;  // [kM] power of two that undoes a row's scaling
constexpr int kOffBar = kOffUnit + kM * 4;
constexpr int kBarArea = 320;
// [4 quarters][2 tile parities][32 rows] published maxima: in the unit array's place they would
// have to wait for it to be read, so they have their own
constexpr int kOffMPub = kOffBar + kBarArea;
constexpr int kSmemBytes = kOffMPub + 4 * 2 * 32 * 4 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
static_assert(kSlots * kTile >= kM * kD * 4, "the epilogue stages the fp32 record rows in the K ring");
static_assert(kSlots * kTile >= kM * 8, "the epilogue keeps the rows' record offsets in the V ring");
constexpr uint32_t kTmemCols = 512;           // S/P buffers at 0, 128, 256; O at 384
constexpr uint32_t kColO = 384;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 of the largest growth tolerated in P
constexpr float kShift = 7.0f;                // log2 of the factor that P carries
constexpr uint64_t kWaitLimitNs = 2000000000ull;

enum : int {
  kBarCFull = 0,                            // [2 * kSlots] TMA -> conversion (codes of K, then of V)
  kBarCEmpty = kBarCFull + 2 * kSlots,      // [2 * kSlots] conversion has read the codes -> its first lane
  kBarKFull = kBarCEmpty + 2 * kSlots,      // [kSlots] conversion -> MMA (kConvThreads arrivals)
  kBarKEmpty = kBarKFull + kSlots,          // [kSlots] MMA (S done) -> conversion
  kBarVFull = kBarKEmpty + kSlots,          // [kSlots]
  kBarVEmpty = kBarVFull + kSlots,          // [kSlots] MMA (PV done) -> conversion
  kBarSFull = kBarVEmpty + kSlots,          // [kSBufs] S(i) in TMEM -> softmax
  kBarPFull = kBarSFull + kSBufs,           // [kSBufs] P(i) in TMEM -> MMA (128 arrivals)
  kBarPvDone = kBarPFull + kSBufs,          // [kSBufs] PV(i) done -> softmax
  kBarDrain = kBarPvDone + kSBufs,          // all MMAs done -> teardown
  kBarPair = kBarDrain + 1,                 // [4] the two softmax warps of a row quarter, epilogue (64)
  kBarMPub = kBarPair + 4,                  // [4 quarters][2 parities] max of a tile published (32)
  kNumBars = kBarMPub + 8
};
static_assert(8 * kNumBars + 16 <= kBarArea, "barrier area");

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 A and B, fp32 accumulator, A K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int32_t x, int32_t y, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2_2d(const void* tmap, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Prefix work item `item` (one CTA) on `smem_raw` (at least kSmemBytes), run by kThreads threads.
// tmk/tmv: the layer's K and V pools as byte matrices [n_slots, row bytes], boxes of 128 x 128.
__device__ __forceinline__ void kv8_dense_body(const AttnParams& p, int32_t item, const CUtensorMap* tmk,
                                               const CUtensorMap* tmv, unsigned char* smem_raw) {
  // 1024-byte alignment for the 128-byte-swizzle atoms
  const uint32_t raw_u = smem_u32(smem_raw);
  const uint32_t base = (raw_u + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw_u);
  const uint32_t sQ = base + kOffQ, sK = base + kOffK, sV = base + kOffV, sC = base + kOffCodes;
  // row sums and maxima for the epilogue, [kind][parity][row], in the codes' place (idle by then)
  float* red = reinterpret_cast<float*>(smem + kOffCodes);
  float* units = reinterpret_cast<float*>(smem + kOffUnit);
  const uint32_t sBar = base + kOffBar;
  auto bar = [&](int i) { return sBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 8 * kNumBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kNumBars + 8);

  const DevPrefixItem it = p.pitems[item];
  const DevGroup gr = p.groups[it.group];
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int g = p.g;
  const int j = it.kv_head;
  const int32_t rows = gr.n_req * g;
  int32_t t0, t1;
  piece_range(gr, it.split, t0, t1);
  const int n_tiles = t1 > t0 ? (t1 - t0 + kN - 1) / kN : 0;
  const bool slab_ok = gr.slab_off >= 0 && gr.slab_off + gr.L_p <= p.n_hot && n_tiles > 0;
  const int32_t rbase = it.row_block * kM;
  const int64_t first_slot = gr.slab_off + t0;

  // codes of tile i of K (which = 0) or V into slot i % kSlots
  auto issue_codes = [&](int which, int i) {
    const int c = which * kSlots + i % kSlots;
    mbar_arrive_expect_tx(bar(kBarCFull + c), kCodes);
    tma_load_2d(sC + c * kCodes, which ? tmv : tmk, j * kD, (int32_t)(first_slot + i * kN), bar(kBarCFull + c));
  };
  const int l2_ahead = p.l2_ahead;
  if (warp == kWarpConv && lane == 0) {
    tma_prefetch_desc(tmk);
    tma_prefetch_desc(tmv);
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1u;
      if (i >= kBarCEmpty && i < kBarCEmpty + 2 * kSlots) count = kConvThreads;
      if ((i >= kBarKFull && i < kBarKFull + kSlots) || (i >= kBarVFull && i < kBarVFull + kSlots)) count = kConvThreads;
      if (i >= kBarPFull && i < kBarPFull + kSBufs) count = kSoftmaxThreads / 2;
      if (i >= kBarPair && i < kBarPair + 4) count = 64u;
      if (i >= kBarMPub && i < kBarMPub + 8) count = 32u;
      mbar_init(bar(i), count);
    }
    *abort_flag = slab_ok ? 0 : 1;
    if (!slab_ok) atomicCAS(p.err, 0, (int32_t)kDevBadSlab);
    mbar_fence_init();
    fence_proxy_async_smem();
    grid_dep_wait();  // the slab may have been written by the work before this kernel
    if (slab_ok)
      for (int i = 0; i < min(n_tiles, kSlots); ++i) {
        issue_codes(0, i);
        issue_codes(1, i);
      }
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // q and the records are touched only after the previous kernel in the stream has completed
  grid_dep_wait();
  grid_dep_launch_dependents();
  // Q rows of this block -> shared memory in fp16, K-major with 128-byte swizzle: row r, 16-byte
  // chunk c lives in 64-dim block c/8 at r*128 + ((c%8) ^ (r%8))*16; rows past the group are 0.  The 16
  // lanes that hold a row agree on its power of two.
  {
    constexpr int kQIters = (kM * 16 + kThreads - 1) / kThreads;
    int32_t qoff[kQIters];
#pragma unroll
    for (int k = 0; k < kQIters; ++k) {
      const int idx = tid + k * kThreads;
      const int32_t row = rbase + (idx >> 4);
      qoff[k] = -1;
      if (idx < kM * 16 && row < rows) qoff[k] = p.group_req[gr.req_begin + row / g];
    }
    uint4 qv[kQIters];
#pragma unroll
    for (int k = 0; k < kQIters; ++k) {
      const int idx = tid + k * kThreads;
      const int32_t row = rbase + (idx >> 4);
      qv[k] = make_uint4(0u, 0u, 0u, 0u);
      if (qoff[k] >= 0)
        qv[k] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                               ((int64_t)qoff[k] * p.n_q + j * g + row % g) * kD)[idx & 15];
    }
#pragma unroll
    for (int k = 0; k < kQIters; ++k) {
      const int idx = tid + k * kThreads;  // 16 lanes of a warp hold one row
      uint32_t w[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = fmaxf(amax, bf16x2_finite_max(w[i]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float unit;
      const float f = q_factor(amax, unit);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = bf16x2_to_f16x2(w[i], f);
      if (idx < kM * 16) {
        const int r = idx >> 4, c = idx & 15;
        sts128(sQ + (c >> 3) * (kM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
        if (c == 0) units[r] = unit;
      }
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kWarpConv && warp < kWarpMma) {
    // ---------------- conversion: codes -> fp16 operand tiles ----------------
    const int which = (warp - kWarpConv) >> 1;  // 0: K, 1: V
    const int ct = tid - (kWarpConv + 2 * which) * 32;
    const uint32_t dst0 = which ? sV : sK;
    const int full = which ? kBarVFull : kBarKFull, empty = which ? kBarVEmpty : kBarKEmpty;
    int issued = slab_ok ? min(n_tiles, kSlots) : 0, seen = 0;
    for (int i = 0; slab_ok && i < n_tiles; ++i) {
      const int st = i % kSlots, c = which * kSlots + st;
      bool ok = mbar_wait_bounded(bar(kBarCFull + c), (i / kSlots) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
      if (ok && i >= kSlots)
        ok = mbar_wait_bounded(bar(empty + st), ((i / kSlots) - 1) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
      if (!ok) break;  // the abort flag is up: every other role leaves as well
      const int valid = t1 - t0 - i * kN;  // tokens of the tile in range (may exceed kN)
      const uint32_t src = sC + c * kCodes, dst = dst0 + st * kTile;
      // 16 codes at a time: chunk idx is token idx / 8, dims 16 * (idx % 8) ..; they become two 16-byte
      // chunks of the token's row in 64-dim half idx % 8 / 4.  Lanes of the upper half store theirs
      // in the other order, so a store instruction covers all banks.
      const int k16 = ct & 7, half = k16 >> 2, ch = (k16 & 3) * 2;
#pragma unroll 4
      for (int n = 0; n < kN * 8 / kConvThreads; ++n) {
        const int tok = (ct >> 3) + n * (kConvThreads / 8);
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(src + tok * kD + k16 * 16));
        if (which && tok >= valid) x = make_uint4(0u, 0u, 0u, 0u);  // 0 * whatever lies there must not reach O
        uint32_t lo[4], hi[4];
        e4m3x4_to_f16x4(x.x, lo[0], lo[1]);
        e4m3x4_to_f16x4(x.y, lo[2], lo[3]);
        e4m3x4_to_f16x4(x.z, hi[0], hi[1]);
        e4m3x4_to_f16x4(x.w, hi[2], hi[3]);
        const uint32_t row = dst + half * kHalf + tok * 128;
        const uint32_t a = row + ((ch ^ (tok & 7)) << 4), b = row + (((ch + 1) ^ (tok & 7)) << 4);
        if (half) {
          sts128(b, hi[0], hi[1], hi[2], hi[3]);
          sts128(a, lo[0], lo[1], lo[2], lo[3]);
        } else {
          sts128(a, lo[0], lo[1], lo[2], lo[3]);
          sts128(b, hi[0], hi[1], hi[2], hi[3]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(full + st));
      seen = i + 1;
      if (i + kSlots < n_tiles) {
        mbar_arrive(bar(kBarCEmpty + c));
        if (ct == 0) {
          // the pair has read the codes
          if (!mbar_wait_bounded(bar(kBarCEmpty + c), (i / kSlots) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs))
            break;
          issue_codes(which, i + kSlots);
          if (l2_ahead > 0 && i + kSlots + l2_ahead < n_tiles)
            tma_prefetch_l2_2d(which ? tmv : tmk, j * kD, (int32_t)(first_slot + (int64_t)(i + kSlots + l2_ahead) * kN));
          issued = i + kSlots + 1;
        }
      }
    }
    if (ct == 0) {
      // never leave with a copy in flight
      for (int i = seen; i < issued; ++i) {
        const uint64_t t_start = globaltimer_ns();
        while (!mbar_try_wait(bar(kBarCFull + which * kSlots + i % kSlots), (i / kSlots) & 1)) {
          if (globaltimer_ns() - t_start > kWaitLimitNs) {
            atomicCAS(p.err, 0, kDevTimeout);
            break;
          }
        }
      }
    }
  } else if (warp == kWarpMma) {
    // ---------------- MMA issuer ----------------
    if (lane == 0 && !*abort_flag) {
      constexpr uint32_t idS = idesc_f16_f32(kM, kN, false);
      constexpr uint32_t idO = idesc_f16_f32(kM, kD, true);
      const uint64_t dq0 = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sK, 16, 1024);
      // V tile as an MN-major B operand: 16 tokens per step (2048 bytes), the two 64-dim halves
      // kHalf apart (leading offset), 8-token groups 1024 bytes apart (stride)
      const uint64_t dv0 = smem_desc_sw128(sV, kHalf, 1024);
      int committed = 0;
      // PV(i) as soon as P(i) and V(i) are ready, S(j) as soon as K(j) is and its TMEM buffer is
      // free: S(j) overwrites S(j-3)/P(j-3), so it may go in once PV(j-3) has been issued (MMAs of one
      // thread execute in order; the softmax was done with S(j-3) before it produced P(j-3)).
      int next_s = 0, next_pv = 0;
      uint64_t t_last = globaltimer_ns();
      while (next_pv < n_tiles) {
        bool progressed = false;
        if (next_pv < next_s) {
          const int i = next_pv;
          const int st = i % kSlots;
          const int sb = i % kSBufs;
          if (mbar_test_wait(bar(kBarPFull + sb), (i / kSBufs) & 1) &&
              mbar_test_wait(bar(kBarVFull + st), (i / kSlots) & 1)) {
            tc_fence_after();
            const uint32_t pa = tmem + (uint32_t)(sb * kN);  // P(i): 64 columns, two tokens per column
            const uint64_t dv = dv0 + (uint64_t)((st * kTile) >> 4);
#pragma unroll
            for (int ks = 0; ks < kN / 16; ++ks)
              umma_f16_ts(tmem + kColO, pa + (uint32_t)(ks * 8), dv + (uint64_t)((ks * 2048) >> 4), idO,
                          (i > 0 || ks > 0) ? 1u : 0u);
            umma_commit(bar(kBarVEmpty + st));
            umma_commit(bar(kBarPvDone + sb));
            committed += 2;
            ++next_pv;
            progressed = true;
          }
        }
        if (next_s < n_tiles && next_s < next_pv + kSBufs) {
          const int i = next_s;
          const int st = i % kSlots;
          if (mbar_test_wait(bar(kBarKFull + st), (i / kSlots) & 1)) {
            tc_fence_after();
            const uint32_t dS = tmem + (uint32_t)((i % kSBufs) * kN);
            const uint64_t dk = dk0 + (uint64_t)((st * kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint64_t a = dq0 + (uint64_t)(((kk >> 2) * (kM * 128) + (kk & 3) * 32) >> 4);
              const uint64_t b = dk + (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
              umma_f16(dS, a, b, idS, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar(kBarSFull + i % kSBufs));
            umma_commit(bar(kBarKEmpty + st));
            committed += 2;
            ++next_s;
            progressed = true;
          }
        }
        if (progressed) {
          t_last = globaltimer_ns();
        } else if (*abort_flag) {
          break;
        } else if (globaltimer_ns() - t_last > kWaitLimitNs) {
          *abort_flag = 1;
          atomicCAS(p.err, 0, (int32_t)kDevTimeout);
          break;
        }
      }
      // drain: every tcgen05 op this thread issued completes before the CTA frees TMEM
      if (committed > 0) {
        umma_commit(bar(kBarDrain));
        const uint64_t t_start = globaltimer_ns();
        while (!mbar_try_wait(bar(kBarDrain), 0)) {
          if (globaltimer_ns() - t_start > kWaitLimitNs) {
            atomicCAS(p.err, 0, kDevTimeout);
            break;
          }
        }
      }
    }
  } else {
    // ---------------- softmax warps 0-7: rows of quarter `quad`, tiles of parity `par` ----------------
    const int quad = warp & 3;
    const int par = warp >> 2;
    const int half = par;                           // the epilogue's column half of O
    const int r = quad * 32 + lane;                 // row = TMEM lane
    const uint32_t lane_off = (uint32_t)((quad * 32) << 16);
    const int pair_bar = kBarPair + quad;           // mbarrier of the two warps sharing rows
    float* mpub = reinterpret_cast<float*>(smem + kOffMPub) + quad * 64;  // [tile parity][lane]
    const float scale = p.scale_log2 * units[r];
    // this row's request, head and record, looked up now so the loads finish during the tiles
    const int32_t row = rbase + r;
    int32_t h = 0, rec = -1;
    if (row < rows) {
      const int32_t b = p.group_req[gr.req_begin + row / g];
      h = j * g + row % g;
      rec = p.reqs[b].rec_base + it.split;
    }
    // the scales of tile i's two blocks (the second block's of a tile that ends in its first are
    // not used: the first's again)
    const int64_t scale_at = (int64_t)p.n_kv * kD + 4 * j;
    float ks[2], vs[2];
    auto load_scales = [&](int i) {
      const int64_t a = (first_slot + (int64_t)i * kN) * p.kv8_row + scale_at;
      const int64_t b = a + (t1 - t0 - i * kN > kKv8Block ? kKv8Block * p.kv8_row : 0);
      ks[0] = *reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.kpool) + a);
      ks[1] = *reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.kpool) + b);
      vs[0] = *reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.vpool) + a);
      vs[1] = *reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.vpool) + b);
    };
    float m_own = -INFINITY;   // max (of z, base 2) used for this warp's latest tile
    float l = 0.f;             // this warp's share of the row sum, relative to m_own
    int pair_phase = 0;
    bool ok = !*abort_flag;
    if (ok && par < n_tiles) load_scales(par);
    for (int i = par; ok && i < n_tiles; i += 2) {
      const int sb = i % kSBufs;
      const float ca[2] = {scale * ks[0], scale * ks[1]};
      const float cb[2] = {lg2_approx(vs[0]), lg2_approx(vs[1])};
      if (i + 2 < n_tiles) load_scales(i + 2);
      ok = mbar_wait_bounded(bar(kBarSFull + sb), (i / kSBufs) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
      ok = __all_sync(0xffffffffu, ok);  // the TMEM loads below are warp-collective
      if (!ok) break;
      tc_fence_after();
      const int valid = min(kN, t1 - t0 - i * kN);               // tokens of the tile in range
      const uint32_t ts = tmem + lane_off + (uint32_t)(sb * kN);
      // row max of z over the 128 columns, half by half (the factors are positive); S(i) is read
      // again below for the exponentials, which keeps the thread's registers within the launch's
      float mx = -INFINITY;
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        uint32_t u[2][32];
        GRANIKV_TMEM_LD32(ts + hb * 64, u[0]);
        GRANIKV_TMEM_LD32(ts + hb * 64 + 32, u[1]);
        tmem_wait_ld();
        if (valid < kN) {
#pragma unroll
          for (int k = 0; k < 64; ++k) u[k >> 5][k & 31] = 64 * hb + k < valid ? u[k >> 5][k & 31] : 0xff800000u;
        }
        float t[22], w[7];
        auto sv = [&](int k) { return __uint_as_float(u[k >> 5][k & 31]); };
#pragma unroll
        for (int k = 0; k < 21; ++k) t[k] = max3f(sv(3 * k), sv(3 * k + 1), sv(3 * k + 2));
        t[21] = sv(63);
#pragma unroll
        for (int k = 0; k < 7; ++k) w[k] = max3f(t[3 * k], t[3 * k + 1], t[3 * k + 2]);
        const float hm = max3f(max3f(w[0], w[1], w[2]), max3f(w[3], w[4], w[5]), fmaxf(w[6], t[21]));
        mx = fmaxf(mx, hm * ca[hb] + cb[hb]);
      }
      // the max used for tile i: that of tile i-1 (decided by the other warp of the quarter),
      // moved only when this tile's row max exceeds it by more than 2^kRescaleThreshold
      float m_i = mx;
      bool warp_need = false;
      float m_prev = -INFINITY;
      if (i > 0) {
        const int pp = (i - 1) & 1;
        ok = mbar_wait_bounded(bar(kBarMPub + quad * 2 + pp), ((i - 1) >> 1) & 1, abort_flag, p.err, kDevTimeout,
                               kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        m_prev = mpub[pp * 32 + lane];
        warp_need = __any_sync(0xffffffffu, mx > m_prev + kRescaleThreshold);
        m_i = warp_need ? fmaxf(m_prev, mx) : m_prev;
      }
      // publish at once, so the warp of tile i+1 is not held up by the rescale below (the slot's
      // previous value, tile i-2's, was read by that warp before it published tile i-1's)
      mpub[par * 32 + lane] = m_i;
      mbar_arrive(bar(kBarMPub + quad * 2 + par));
      if (warp_need) {
        // O must hold PV(i-1) before it is rescaled, and PV(i) waits for P(i), written below
        ok = mbar_wait_bounded(bar(kBarPvDone + (i - 1) % kSBufs), ((i - 1) / kSBufs) & 1, abort_flag, p.err,
                               kDevTimeout, kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float alpha = m_prev == m_i ? 1.f : ex2_approx(m_prev - m_i);
        uint32_t u[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t ta = tmem + lane_off + kColO + c * 32;
          GRANIKV_TMEM_LD32(ta, u);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * alpha);
          GRANIKV_TMEM_ST32(ta, u);
        }
        tmem_wait_st();
      }
      if (m_own != m_i && m_own != -INFINITY) l *= ex2_approx(m_own - m_i);
      m_own = m_i;
      // P = 2^(z - m + kShift), packed two per 32-bit column and written over columns [0, 64) of the
      // S(i) buffer: S columns [64*hb, 64*hb + 64) are in registers before their P goes to
      // columns [32*hb, 32*hb + 32)
      const float m_use = m_i == -INFINITY ? 0.f : m_i;
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const float off = cb[hb] - m_use + kShift;
        const uint64_t scale2 = f2_pack(ca[hb], ca[hb]), nm2 = f2_pack(off, off);
        uint64_t acc[2] = {0ull, 0ull};  // packed partial sums of the half (0.0f bit patterns)
        uint32_t u[2][32];
        GRANIKV_TMEM_LD32(ts + hb * 64, u[0]);
        GRANIKV_TMEM_LD32(ts + hb * 64 + 32, u[1]);
        tmem_wait_ld();
        if (valid < kN) {  // masked keys: -inf, so their weight is 0
#pragma unroll
          for (int k = 0; k < 64; ++k) u[k >> 5][k & 31] = 64 * hb + k < valid ? u[k >> 5][k & 31] : 0xff800000u;
        }
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float sa = __uint_as_float(u[k >> 4][(2 * k) & 31]);
          const float sb2 = __uint_as_float(u[k >> 4][(2 * k + 1) & 31]);
          const uint64_t x = f2_fma(f2_pack(sa, sb2), scale2, nm2);
          float xa, xb;
          f2_unpack(x, xa, xb);
          const float ea = ex2_approx(xa), eb = ex2_approx(xb);
          acc[k & 1] = f2_add(acc[k & 1], f2_pack(ea, eb));
          pk[k] = pack_f16(ea, eb);
        }
        GRANIKV_TMEM_ST32(tmem + lane_off + (uint32_t)(sb * kN + hb * 32), pk);
        float la, lb;
        f2_unpack(f2_add(acc[0], acc[1]), la, lb);
        // over vs, by the very logarithm that P has
        l += (la + lb) * ex2_approx(-cb[hb]);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(kBarPFull + sb));
    }
    // epilogue: wait for the last PV, combine the two warps' row sums (each relative to the max
    // of its own latest tile; the last tile's max is the final one), normalise, write the record
    if (ok) {
      const int last = n_tiles - 1;
      ok = mbar_wait_bounded(bar(kBarPvDone + last % kSBufs), (last / kSBufs) & 1, abort_flag, p.err, kDevTimeout,
                             kWaitLimitNs);
    }
    ok = __all_sync(0xffffffffu, ok);
    // swap the row sums and maxima with the other warp at the pair barrier; a warp that left the
    // tile loop early may stop waiting for published maxima, so its partner's bounded waits give
    // up and both skip the record
    // (the codes' slots, where these go, are idle once the last PV is done; a CTA that gave up may
    // still have a copy in flight there, and then writes nothing)
    const bool safe = ok;
    if (safe) {
      red[par * kM + r] = l;
      red[2 * kM + par * kM + r] = m_own;
    }
    mbar_arrive(bar(pair_bar));
    bool pair_ok = mbar_wait_bounded(bar(pair_bar), pair_phase & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
    ++pair_phase;
    ok = __all_sync(0xffffffffu, pair_ok) && ok && !*abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const float l0 = red[r], l1 = red[kM + r];
      const float m_used = red[2 * kM + ((n_tiles - 1) & 1) * kM + r];
      const float m0 = red[2 * kM + r], m1 = red[2 * kM + kM + r];
      // a warp that had no tile left 0; an equal maximum (both may be -inf or NaN) needs no factor
      const float lt = (l0 == 0.f ? 0.f : m0 == m_used ? l0 : l0 * ex2_approx(m0 - m_used)) +
                       (l1 == 0.f ? 0.f : m1 == m_used ? l1 : l1 * ex2_approx(m1 - m_used));
      if (row < rows && (rec < 0 || rec >= p.n_records)) {
        if (half == 0) atomicCAS(p.err, 0, (int32_t)kDevBadRecord);
        rec = -1;
      }
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      uint32_t u[2][32];
      GRANIKV_TMEM_LD32(tmem + lane_off + kColO + half * 64, u[0]);
      GRANIKV_TMEM_LD32(tmem + lane_off + kColO + half * 64 + 32, u[1]);
      tmem_wait_ld();
      // Stage the normalised half row in shared memory (the K and V rings are idle: every MMA
      // has completed), 16-byte chunk c of row r at chunk c ^ (r % 32), so that a warp's 32
      // rows hit all banks; the pair then stores whole 512-byte rows, one per warp instruction.
      fence_proxy_async_smem();
      unsigned char* stage = smem + kOffK;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const int chunk = half * 16 + c * 8 + k / 4;
          *reinterpret_cast<float4*>(stage + r * 512 + ((chunk ^ (r & 31)) << 4)) =
              make_float4(__uint_as_float(u[c][k]) * inv, __uint_as_float(u[c][k + 1]) * inv,
                          __uint_as_float(u[c][k + 2]) * inv, __uint_as_float(u[c][k + 3]) * inv);
        }
      if (half == 0) {
        const float m_fin = m_used == -INFINITY ? 0.f : m_used;
        const float lse_row = lt == 0.f ? -INFINITY : (m_fin - kShift + log2f(lt)) * kLn2;
        reinterpret_cast<int64_t*>(smem + kOffV)[r] = rec >= 0 ? ((int64_t)rec * p.n_q + h) * kD : -1;
        if (rec >= 0) st_record(p.rec_lse + (int64_t)rec * p.n_q + h, lse_row, l2_policy_keep());
      }
    }
    // both halves of the quarter's 32 rows are staged (both warps of a pair agree on `ok`, or the
    // abort flag is up and this wait gives up)
    mbar_arrive(bar(pair_bar));
    bool staged = mbar_wait_bounded(bar(pair_bar), pair_phase & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
    ++pair_phase;
    staged = __all_sync(0xffffffffu, staged) && ok;
    if (staged) {
      const unsigned char* stage = smem + kOffK;
      const int64_t* sdst = reinterpret_cast<const int64_t*>(smem + kOffV);
      const uint64_t keep = l2_policy_keep();
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int rr = quad * 32 + half * 16 + i;
        const int64_t d = sdst[rr];
        if (d < 0) continue;
        const float4 x = *reinterpret_cast<const float4*>(stage + rr * 512 + ((lane ^ (rr & 31)) << 4));
        st_record4(p.rec_o + d + lane * 4, x, keep);
      }
    }
  }

  // ---------------- teardown ----------------
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace
}  // namespace k8d
}  // namespace granikv
