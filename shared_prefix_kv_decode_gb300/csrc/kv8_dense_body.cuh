// kv8_dense_body.cuh -- dense prefix backend over the 8-bit cache on the 5th-generation tensor cores
// (tcgen05/TMEM), head_dim 128, bf16 q.
//
// One CTA takes one (prefix group, KV head j, 128-row block, L_p piece), as the 16-bit dense kernel:
// rows are the group's (request, head-in-group) pairs of KV head j.  For each 64-token tile i, one
// scale block of the slab,
//     S(i) = Q K(i)^T       (8 tcgen05.mma 128x64x32, kind::f8f6f4: the codes of K as they are, Q from TMEM)
//     P(i) = 2^(z - m)      (softmax warps; fp16, written back over S(i) in TMEM)
//     O   += P(i) V(i)      (4 tcgen05.mma 128x128x16, fp16, with A = P(i) read from TMEM)
// A tile passes through S, softmax and PV with about 2,900 clocks of latency (products, commits and
// barrier waits, exponentials), while its products need 564 at the nominal rates and its exponentials 512
// of the exponential unit: five tiles in flight (five S/P buffers of 64 columns, O and Q in the rest of
// TMEM) cover that.  A CTA takes 0.88 us for 128 tokens (15 row blocks on one slab, so that HBM is idle).
// With parts taken out: the loads alone 0.48, loads and products 0.68 (what cuBLAS takes for products of
// this size), with softmax 0.75; the conversion of V adds the rest, by its traffic through shared memory
// next to the operands'.  Other splits of TMEM (four S and two P buffers: 0.92; three and four: 1.02),
// waits that spin instead of suspending (0.87) and one arrival a warp (0.89) are no better.  128-token
// tiles in three buffers: a step of the 32/8-head shape (16K prefix, B = 64) took 32.7 us against 30.6.
// Number format.  S takes K's codes straight from TMA and q as the sum of two e4m3 values: each row is
// scaled by a power of two so that its largest element lies in [2^7, 2^8), hi = e4m3(q) and lo =
// e4m3(q - hi).  bf16 has 8 significant bits and each part 4, so q = hi + lo exactly down to 2^-2, 2^-9
// of the row's largest element at the least; smaller elements are off by at most 2^-10 there, 2^-17 of
// the largest (bf16 itself rounds an element by 2^-9 of its own size).  Two passes at fp8's rate
// take the time of one in fp16, and no conversion stands before S.  V's codes become fp16 exactly:
// P in 8 bits would lose the weights.
// The scales of a slab are those of 64-token blocks counted from its start, so a tile has one K scale
// ks and one V scale vs: z = s ks + log2 vs (base 2) costs the FMA that the softmax needs anyway, P =
// 2^(z - m) is p times vs, which is what meets the V codes, and the row sum adds the tile's sum of P
// once, over vs / v, v the piece's smallest V scale.  The running maximum m is taken over z.  P carries a
// factor of 2^7: it is at most 2^15 (m may lag the row's maximum by 2^8, see below), and fp16 keeps its 11
// bits down to 2^-21 of the largest weight.
// V scales lie between 2^-104.9 (of zeros) and 2^119.2.  Where those of a piece span more than 2^32, a tile's P
// may underflow while its weights count: the row sum then has a running maximum and exponentials of its own, over
// s ks alone.  Below that span P reaches weights of 2^-94 of the largest.
// Roles (15 warps; the 16th only takes part in the block's barriers here):
//  * warps 0-7, softmax and epilogue: warp w serves TMEM lanes 32*(w%4).. (row r = lane r), all 64
//    columns of the tiles i with i % 2 == w / 4; the two warps of a row quarter take turns, half a
//    tile apart.  The running max is a chain over the tiles: the warp of tile i reads the max used
//    for tile i-1 from shared memory, keeps it unless the tile's row max exceeds it by more than
//    2^8 (then O is rescaled in TMEM), and publishes its own.  First they bring Q into TMEM.
//  * warps 8-11, V conversion: each takes 32 tokens of every 128 of V.  It loads their codes by TMA into
//    its own ring of four, turns 16 codes at a time into fp16 and stores them in the
//    128-byte-swizzled layout that the MMA operand has (rows past the piece's end as zeros).
//  * warps 12 and 13, the MMAs: one issues S(i), up to five tiles ahead, the
//    other PV(i), so that neither's waits hold up the other's products.
//  * warp 14, the TMA loads of K.
// Every mbarrier wait is bounded in time; on expiry the CTA raises an abort flag, latches an error,
// drains what it issued and frees its TMEM.
#pragma once

#include <cuda.h>

#include <cfloat>

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
constexpr int kN = kKv8Block;                 // 64 tokens per tile
constexpr int kPair = kDenseTile;             // 128 tokens: what the K and V rings hold in a slot
static_assert(kPair == 2 * kN && kPair / 4 == kKv8VBox, "a conversion warp's part of a V slot is one box");
constexpr int kKSlots = 4;                    // slots of the K ring (codes)
constexpr int kVSlots = 3;                    // slots of the V ring (fp16)
constexpr int kCSlots = 4;                    // slots of each conversion warp's ring of V codes
constexpr int kSBufs = 5;                     // S/P buffers in TMEM
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kWarpConv = 8, kConvWarps = 4;
constexpr int kPart = kPair / kConvWarps;     // tokens of a V slot that one warp converts
constexpr int kWarpS = 12, kWarpPv = 13, kWarpTmaK = 14;
constexpr int kThreads = 512;  // one more warp, for the suffix body's producers
constexpr int kHalf = kPair * 128;            // one 64-dim half of an fp16 slot: 16 KB
constexpr int kTile = 2 * kHalf;              // 32 KB
constexpr int kCodes = kPair * kD;            // a slot's codes: 16 KB
constexpr int kPartCodes = kPart * kD;        // 4 KB
constexpr int kOffK = 0;
constexpr int kOffV = kOffK + kKSlots * kCodes;
constexpr int kOffCodes = kOffV + kVSlots * kTile;
constexpr int kOffUnit = kOffCodes + kConvWarps * kCSlots * kPartCodes;  // [kM] power of two that undoes a row's scaling
constexpr int kOffMPub = kOffUnit + kM * 4;   // [4 quarters][2 tile parities][32 rows] published maxima
constexpr int kOffBar = kOffMPub + 4 * 2 * 32 * 4;
constexpr int kBarArea = 512;
constexpr int kSmemBytes = kOffBar + kBarArea + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
static_assert(kConvWarps * kCSlots * kPartCodes >= 6 * kM * 4, "the epilogue's sums and maxima");
constexpr uint32_t kTmemCols = 512;           // S/P buffers at 0, 64, 128, 192, 256; Q (hi, lo) at 320; O at 384
constexpr uint32_t kColQ = kSBufs * kN, kColO = 384;
static_assert(kColQ + 2 * kD / 4 <= kColO && kColO + kD <= kTmemCols, "TMEM columns");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 of the largest growth tolerated in P
constexpr float kShift = 7.0f;                // log2 of the factor that P carries
constexpr uint32_t kWideSpan = 32;            // log2 of a wide span of V scales
constexpr uint64_t kWaitLimitNs = 2000000000ull;

enum : int {
  kBarKFull = 0,                            // [kKSlots] TMA -> MMA
  kBarKEmpty = kBarKFull + kKSlots,         // [kKSlots] MMA (S of the slot's tiles done) -> TMA
  kBarCFull = kBarKEmpty + kKSlots,         // [kConvWarps][kCSlots] TMA -> conversion (codes of V)
  kBarVFull = kBarCFull + kConvWarps * kCSlots,  // [kVSlots] conversion -> MMA (kConvWarps arrivals)
  kBarVEmpty = kBarVFull + kVSlots,         // [kVSlots] MMA (PV of the slot's tiles done) -> conversion
  kBarSFull = kBarVEmpty + kVSlots,         // [kSBufs] S(i) in TMEM -> softmax
  kBarPFull = kBarSFull + kSBufs,           // [kSBufs] P(i) in TMEM -> MMA (128 arrivals)
  kBarPvDone = kBarPFull + kSBufs,          // [kSBufs] PV(i) done -> softmax, and S(i + kSBufs)
  kBarDrain = kBarPvDone + kSBufs,          // [2] all S (all PV) products done -> teardown
  kBarPair = kBarDrain + 2,                 // [4] the two softmax warps of a row quarter, epilogue (64)
  kBarMPub = kBarPair + 4,                  // [4 quarters][2 parities] max of a tile published (32)
  kNumBars = kBarMPub + 8
};
static_assert(8 * kNumBars + 16 <= kBarArea, "barrier area");

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f8f6f4 (A: M rows = TMEM lanes, four 8-bit elements per
// 32-bit column along K), issued by one thread
__device__ __forceinline__ void umma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor with A and B of the kind's format 0 (fp16 of kind::f16, e4m3 of
// kind::f8f6f4), fp32 accumulator, A K-major.
__host__ __device__ constexpr uint32_t idesc_fmt0_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// 32 bytes of a record (32-byte aligned), kept in L2 for the merge
__device__ __forceinline__ void st_record8(float* a, const float (&x)[8], uint64_t pol) {
  asm volatile("st.global.L2::cache_hint.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(a), "f"(x[0]),
               "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "l"(pol)
               : "memory");
}
// Two bf16 times f -> fp16; four fp16 -> four e4m3 codes (nearest even, NaN kept).
__device__ __forceinline__ __half2 f16x2_of(uint32_t w, float f) {
  return __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}
__device__ __forceinline__ uint32_t f16x4_to_e4m3x4(__half2 a, __half2 b) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t*>(&a)));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t*>(&b)));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// 16 columns of this warp's TMEM lanes
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
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
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
  return x;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Prefix work item `item` (one CTA) on `smem_raw` (at least kSmemBytes), run by kThreads threads.
// tmk/tmv: the layer's K and V pools as byte matrices [n_slots, row bytes]: K in boxes of 128 slots x
// 128 bytes with the 128-byte swizzle, V in boxes of 32 slots x 128 bytes, row after row.
__device__ __forceinline__ void kv8_dense_body(const AttnParams& p, int32_t item, const CUtensorMap* tmk,
                                               const CUtensorMap* tmv, unsigned char* smem_raw) {
  // 1024-byte alignment for the 128-byte-swizzle atoms
  const uint32_t raw_u = smem_u32(smem_raw);
  const uint32_t base = (raw_u + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw_u);
  const uint32_t sK = base + kOffK, sV = base + kOffV, sC = base + kOffCodes;
  // row sums, exponents and maxima for the epilogue, [kind][parity][row], in the codes' place (idle by then)
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
  const int n_pairs = (n_tiles + 1) / 2;  // ring slots used
  const bool slab_ok = gr.slab_off >= 0 && gr.slab_off + gr.L_p <= p.n_hot && n_tiles > 0;
  const int32_t rbase = it.row_block * kM;
  const int64_t first_slot = gr.slab_off + t0;

  // slot contents: tokens kPair * i .. of the piece
  auto issue_k = [&](int i) {
    const int st = i % kKSlots;
    mbar_arrive_expect_tx(bar(kBarKFull + st), kCodes);
    tma_load_2d(sK + st * kCodes, tmk, j * kD, (int32_t)(first_slot + (int64_t)i * kPair), bar(kBarKFull + st));
  };
  // conversion warp w's part of V's slot contents i
  auto issue_v = [&](int w, int i) {
    const int c = w * kCSlots + i % kCSlots;
    mbar_arrive_expect_tx(bar(kBarCFull + c), kPartCodes);
    tma_load_2d(sC + c * kPartCodes, tmv, j * kD, (int32_t)(first_slot + (int64_t)i * kPair + w * kPart), bar(kBarCFull + c));
  };
  const int l2_ahead = p.l2_ahead;
  // softmax warps: this lane's row (the same for the two warps of a row quarter), its request, head and
  // record.  The plan is not written by the work before this kernel, so these loads need not wait for it.
  const int qrow = (warp & 3) * 32 + lane, qhalf = warp >> 2;
  const int32_t row = rbase + qrow;
  const bool have = warp < kSoftmaxWarps && row < rows;
  int32_t req = 0, h = 0, rec = -1;
  if (have) {
    req = p.group_req[gr.req_begin + row / g];
    h = j * g + row % g;
    rec = p.reqs[req].rec_base + it.split;
  }
  if (warp == kWarpTmaK && lane == 0) {
    tma_prefetch_desc(tmk);
    tma_prefetch_desc(tmv);
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1u;
      if (i >= kBarVFull && i < kBarVFull + kVSlots) count = kConvWarps;
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
    if (slab_ok) {
      for (int i = 0; i < min(n_pairs, kKSlots); ++i) issue_k(i);
      for (int i = 0; i < min(n_pairs, kCSlots); ++i)
        for (int w = 0; w < kConvWarps; ++w) issue_v(w, i);
    }
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // q and the records are touched only after the previous kernel in the stream has completed
  grid_dep_wait();
  grid_dep_launch_dependents();
  // Q: the two softmax warps of a row quarter take half of their rows' dims each, agree on each row's
  // power of two through shared memory, and split the elements into hi and lo, four to a word; rows
  // past the group are 0
  uint32_t qw[32];
  float* part = reinterpret_cast<float*>(smem + kOffMPub);  // [2][kM], used for the maxima of tiles later
  // the scales of tile i; a softmax warp's first ones are on their way with its rows
  const int64_t scale_at = (int64_t)p.n_kv * kD + 4 * j;
  float ks = 0.f, vs = 0.f;
  auto load_scales = [&](int i) {
    const int64_t a = (first_slot + (int64_t)i * kN) * p.kv8_row + scale_at;
    ks = *reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.kpool) + a);
    vs = *reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.vpool) + a);
  };
  // V scales of the piece's tiles lane, lane + 32, .. as the bits of positive floats, for their span; requested
  // here and used when the set-up is done
  constexpr int kSpan = 4;
  uint32_t v_bits[kSpan] = {};
  auto v_scale_bits = [&](int i) {
    return *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.vpool) + (first_slot + (int64_t)i * kN) * p.kv8_row + scale_at);
  };
  if (warp < kSoftmaxWarps) {
    if (slab_ok && qhalf < n_tiles) load_scales(qhalf);
    if (slab_ok) {
#pragma unroll
      for (int k = 0; k < kSpan; ++k)
        if (lane + 32 * k < n_tiles) v_bits[k] = v_scale_bits(lane + 32 * k);
    }
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                      ((int64_t)req * p.n_q + h) * kD + qhalf * (kD / 2));
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 x = have ? src[k] : make_uint4(0u, 0u, 0u, 0u);
      qw[4 * k] = x.x;
      qw[4 * k + 1] = x.y;
      qw[4 * k + 2] = x.z;
      qw[4 * k + 3] = x.w;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) amax = fmaxf(amax, bf16x2_finite_max(qw[k]));
    part[qhalf * kM + qrow] = amax;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp < kSoftmaxWarps) {
    float unit;
    const float f = q_factor<7>(fmaxf(part[qrow], part[kM + qrow]), unit);
    if (qhalf == 0) units[qrow] = unit;
    // in fp16 pairs: below 2^8 with 8 significant bits they are exact there down to 2^-17
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const __half2 x = q_no_inf(f16x2_of(qw[2 * k], f)), y = q_no_inf(f16x2_of(qw[2 * k + 1], f));
      hi[k] = f16x4_to_e4m3x4(x, y);
      uint32_t u, v;
      e4m3x4_to_f16x4(hi[k], u, v);
      lo[k] = f16x4_to_e4m3x4(__hsub2(x, *reinterpret_cast<__half2*>(&u)), __hsub2(y, *reinterpret_cast<__half2*>(&v)));
    }
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColQ + qhalf * 16;
    tmem_st16(at, hi);
    tmem_st16(at + 32, lo);
    tmem_wait_st();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp >= kWarpConv && warp < kWarpConv + kConvWarps) {
    // ---------------- conversion: codes of V -> fp16 operand tiles ----------------
    // lane: dims 16 * (lane % 8) .. of tokens lane / 8 + 4 n of the part, which become two 16-byte chunks
    // of the token's row in 64-dim half lane % 8 / 4.  Lanes of the upper half store theirs in the other
    // order, so a store instruction covers all banks.
    constexpr int kPer = kPart / 4;
    const int w = warp - kWarpConv;
    const bool upper = (lane & 7) >= 4;
    const int lt = lane >> 3;
    const uint32_t src_off = (uint32_t)lt * kD + (lane & 7) * 16;
    const uint32_t row_off = (uint32_t)w * kPart * 128 + (upper ? kHalf : 0) + (uint32_t)lt * 128;
    const uint32_t ch = (lane & 3) * 2;
    // tokens lt and lt + 4 modulo 8 have two swizzles
    const uint32_t lo0 = row_off + ((ch ^ lt) << 4), hi0 = row_off + (((ch + 1) ^ lt) << 4);
    const uint32_t lo1 = row_off + ((ch ^ (lt + 4)) << 4), hi1 = row_off + (((ch + 1) ^ (lt + 4)) << 4);
    int issued = slab_ok ? min(n_pairs, kCSlots) : 0, seen = 0;
    for (int i = 0; slab_ok && i < n_pairs; ++i) {
      const int c = w * kCSlots + i % kCSlots, st = i % kVSlots;
      bool ok = mbar_wait_bounded(bar(kBarCFull + c), (i / kCSlots) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;  // the abort flag is up: every other role leaves as well
      seen = i + 1;
      const uint32_t src = sC + c * kPartCodes + src_off, dst = sV + st * kTile;
      uint4 x[kPer];
#pragma unroll
      for (int n = 0; n < kPer; ++n) x[n] = lds128(src + n * 4 * kD);
      const int valid = t1 - t0 - i * kPair - w * kPart;  // tokens of the part in range, or more
      if (valid < kPart) {  // 0 * whatever lies past the piece must not reach O
#pragma unroll
        for (int n = 0; n < kPer; ++n)
          if (lt + 4 * n >= valid) x[n] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (i >= kVSlots) {
        ok = mbar_wait_bounded(bar(kBarVEmpty + st), ((i / kVSlots) - 1) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
#pragma unroll
      for (int n = 0; n < kPer; ++n) {
        uint32_t y[8];
        e4m3x4_to_f16x4(x[n].x, y[0], y[1]);
        e4m3x4_to_f16x4(x[n].y, y[2], y[3]);
        e4m3x4_to_f16x4(x[n].z, y[4], y[5]);
        e4m3x4_to_f16x4(x[n].w, y[6], y[7]);
        const uint32_t lo = dst + n * 4 * 128 + (n & 1 ? lo1 : lo0), hi = dst + n * 4 * 128 + (n & 1 ? hi1 : hi0);
        if (upper) {
          sts128(hi, y[4], y[5], y[6], y[7]);
          sts128(lo, y[0], y[1], y[2], y[3]);
        } else {
          sts128(lo, y[0], y[1], y[2], y[3]);
          sts128(hi, y[4], y[5], y[6], y[7]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();  // the warp has stored its part, and read its codes
      if (lane == 0) {
        mbar_arrive(bar(kBarVFull + st));
        if (i + kCSlots < n_pairs) {
          issue_v(w, i + kCSlots);
          if (l2_ahead > 0 && i + kCSlots + l2_ahead < n_pairs)
            tma_prefetch_l2_2d(tmv, j * kD, (int32_t)(first_slot + (int64_t)(i + kCSlots + l2_ahead) * kPair + w * kPart));
          issued = i + kCSlots + 1;
        }
      }
    }
    // never leave with a copy in flight
    if (lane == 0) {
      for (int i = seen; i < issued; ++i) {
        const uint64_t t_start = globaltimer_ns();
        while (!mbar_try_wait(bar(kBarCFull + w * kCSlots + i % kCSlots), (i / kCSlots) & 1)) {
          if (globaltimer_ns() - t_start > kWaitLimitNs) {
            atomicCAS(p.err, 0, kDevTimeout);
            break;
          }
        }
      }
    }
  } else if (warp == kWarpTmaK) {
    // ---------------- TMA loads of K ----------------
    if (lane == 0) {
      int issued = slab_ok ? min(n_pairs, kKSlots) : 0;
      for (int i = issued; slab_ok && i < n_pairs; ++i) {
        if (!mbar_wait_bounded(bar(kBarKEmpty + i % kKSlots), ((i / kKSlots) - 1) & 1, abort_flag, p.err, kDevTimeout,
                               kWaitLimitNs))
          break;
        issue_k(i);
        if (l2_ahead > 0 && i + l2_ahead < n_pairs)
          tma_prefetch_l2_2d(tmk, j * kD, (int32_t)(first_slot + (int64_t)(i + l2_ahead) * kPair));
        issued = i + 1;
      }
      // never leave with a copy in flight
      for (int i = max(0, issued - kKSlots); i < issued; ++i) {
        const uint64_t t_start = globaltimer_ns();
        while (!mbar_try_wait(bar(kBarKFull + i % kKSlots), (i / kKSlots) & 1)) {
          if (globaltimer_ns() - t_start > kWaitLimitNs) {
            atomicCAS(p.err, 0, kDevTimeout);
            break;
          }
        }
      }
    }
  } else if (warp == kWarpS || warp == kWarpPv) {
    // ---------------- MMA issuers ----------------
    // The whole warp runs the loop and one elected lane issues: with the operands' descriptors uniform
    // over the warp, an MMA is issued every 32 clocks; from inside a one-lane branch, every 45, which is
    // more than these 128x64x32 products take.
    if (!*abort_flag) {
      constexpr uint32_t idS = idesc_fmt0_f32(kM, kN, false);
      constexpr uint32_t idO = idesc_fmt0_f32(kM, kD, true);
      const bool el = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      auto wait = [&](int b, int slots, int i) {
        const bool ok = mbar_wait_bounded(bar(b + i % slots), (i / slots) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
        return __all_sync(0xffffffffu, ok) != 0;
      };
      int committed = 0;
      if (warp == kWarpS) {
        const uint64_t dk0 = smem_desc_sw128(sK, 16, 1024);
        for (int i = 0; i < n_tiles; ++i) {
          // S(i) overwrites S(i-5)/P(i-5), whose last reader is PV(i-5)
          if (i >= kSBufs && !wait(kBarPvDone, kSBufs, i - kSBufs)) break;
          if ((i & 1) == 0 && !wait(kBarKFull, kKSlots, i >> 1)) break;
          tc_fence_after();
          const uint32_t dS = tm + (uint32_t)((i % kSBufs) * kN);
          const int st = (i >> 1) % kKSlots;
          const uint64_t dk = dk0 + (uint64_t)((st * kCodes + (i & 1) * kN * kD) >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // lo, the smaller, first
            if (el)
              umma_f8_ts(dS, tm + kColQ + (kk < 4 ? 32 : 0) + (kk & 3) * 8, dk + (uint64_t)(((kk & 3) * 32) >> 4), idS,
                         kk > 0 ? 1u : 0u);
          if (el) {
            umma_commit(bar(kBarSFull + i % kSBufs));
            if (i & 1) umma_commit(bar(kBarKEmpty + st));
          }
          __syncwarp();
          committed += 1;
        }
      } else {
        // V slot as an MN-major B operand: 16 tokens per step (2048 bytes), the two 64-dim halves
        // kHalf apart (leading offset), 8-token groups 1024 bytes apart (stride)
        const uint64_t dv0 = smem_desc_sw128(sV, kHalf, 1024);
        for (int i = 0; i < n_tiles; ++i) {
          if ((i & 1) == 0 && !wait(kBarVFull, kVSlots, i >> 1)) break;
          if (!wait(kBarPFull, kSBufs, i)) break;
          tc_fence_after();
          const uint32_t pa = tm + (uint32_t)((i % kSBufs) * kN);  // P(i): 32 columns, two tokens per column
          const int st = (i >> 1) % kVSlots;
          const uint64_t dv = dv0 + (uint64_t)((st * kTile + (i & 1) * (kN / 16) * 2048) >> 4);
#pragma unroll
          for (int ks = 0; ks < kN / 16; ++ks)
            if (el)
              umma_f16_ts(tm + kColO, pa + (uint32_t)(ks * 8), dv + (uint64_t)((ks * 2048) >> 4), idO,
                          (i > 0 || ks > 0) ? 1u : 0u);
          if (el) {
            umma_commit(bar(kBarPvDone + i % kSBufs));
            if (i & 1) umma_commit(bar(kBarVEmpty + st));
          }
          __syncwarp();
          committed += 1;
        }
      }
      // drain: every tcgen05 op the elected lane issued completes before the CTA frees TMEM
      if (committed > 0 && el) {
        const uint32_t drain = bar(kBarDrain + (warp == kWarpS ? 0 : 1));
        umma_commit(drain);
        const uint64_t t_start = globaltimer_ns();
        while (!mbar_try_wait(drain, 0)) {
          if (globaltimer_ns() - t_start > kWaitLimitNs) {
            atomicCAS(p.err, 0, kDevTimeout);
            break;
          }
        }
      }
    }
  } else if (warp < kSoftmaxWarps) {
    // ---------------- softmax warps 0-7: rows of quarter `quad`, tiles of parity `par` ----------------
    const int quad = warp & 3;
    const int par = warp >> 2;
    const int half = par;                           // the epilogue's column half of O
    const int r = qrow;                             // row = TMEM lane
    const uint32_t lane_off = (uint32_t)((quad * 32) << 16);
    const int pair_bar = kBarPair + quad;           // mbarrier of the two warps sharing rows
    float* mpub = reinterpret_cast<float*>(smem + kOffMPub) + quad * 64;  // [tile parity][lane]
    const float scale = p.scale_log2 * units[r];
    float m_own = -INFINITY;   // max (of z, base 2) used for this warp's latest tile
    float l = 0.f;             // this warp's share of the row sum, over 2^(m_own - kShift - least), or, wide, 2^n
    float n = -INFINITY;
    bool ok = !*abort_flag;
    uint32_t v_min = 0xffffffffu, v_max = 0u;
    auto span_of = [&](uint32_t x) {
      v_min = min(v_min, x - 1u);  // (0: no tile there)
      v_max = max(v_max, x);
    };
#pragma unroll
    for (int k = 0; k < kSpan; ++k) span_of(v_bits[k]);
    for (int i = lane + 32 * kSpan; ok && i < n_tiles; i += 32) span_of(v_scale_bits(i));
    v_min = __reduce_min_sync(0xffffffffu, v_min) + 1u;
    const bool wide = __reduce_max_sync(0xffffffffu, v_max) - v_min > kWideSpan << 23;
    const float least = lg2_approx(__uint_as_float(v_min));  // log2 of the piece's smallest V scale
    // (a loop for each: in one loop the untaken branch cost 2 % of a 16K prefix)
    auto all_tiles = [&](auto wide_span) {
      constexpr bool kWide = decltype(wide_span)::value;
      for (int i = par; ok && i < n_tiles; i += 2) {
        const int sb = i % kSBufs;
        // (at least the smallest normal number: 0 * -inf of a masked key would be NaN)
        const float ca = fmaxf(scale * ks, FLT_MIN), cb = lg2_approx(vs);
        if (i + 2 < n_tiles) load_scales(i + 2);
        // the max used for tile i-1, decided by the other warp of the quarter
        float m_prev = -INFINITY;
        if (i > 0) {
          const int pp = (i - 1) & 1;
          ok = mbar_wait_bounded(bar(kBarMPub + quad * 2 + pp), ((i - 1) >> 1) & 1, abort_flag, p.err, kDevTimeout,
                                 kWaitLimitNs);
          m_prev = mpub[pp * 32 + lane];
        }
        ok = ok && mbar_wait_bounded(bar(kBarSFull + sb), (i / kSBufs) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);  // the TMEM loads below are warp-collective
        if (!ok) break;
        tc_fence_after();
        const int valid = min(kN, t1 - t0 - i * kN);               // tokens of the tile in range
        const uint32_t ts = tmem + lane_off + (uint32_t)(sb * kN);
        uint32_t u[2][32];
        GRANIKV_TMEM_LD32(ts, u[0]);
        GRANIKV_TMEM_LD32(ts + 32, u[1]);
        tmem_wait_ld();
        if (valid < kN) {  // masked keys: -inf, so their weight is 0
#pragma unroll
          for (int k = 0; k < kN; ++k) u[k >> 5][k & 31] = k < valid ? u[k >> 5][k & 31] : 0xff800000u;
        }
        // row max of z (the factor is positive)
        float mx;
        {
          float t[22], w[7];
          auto sv = [&](int k) { return __uint_as_float(u[k >> 5][k & 31]); };
#pragma unroll
          for (int k = 0; k < 21; ++k) t[k] = max3f(sv(3 * k), sv(3 * k + 1), sv(3 * k + 2));
          t[21] = sv(63);
#pragma unroll
          for (int k = 0; k < 7; ++k) w[k] = max3f(t[3 * k], t[3 * k + 1], t[3 * k + 2]);
          mx = max3f(max3f(w[0], w[1], w[2]), max3f(w[3], w[4], w[5]), fmaxf(w[6], t[21])) * ca + cb;
        }
        // the max used for tile i: moved only when this tile's row max exceeds the last one by more
        // than 2^kRescaleThreshold
        float m_i = mx;
        bool warp_need = false;
        if (i > 0) {
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
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t x[16];
            const uint32_t ta = tmem + lane_off + kColO + c * 16;
            tmem_ld16(ta, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * alpha);
            tmem_st16(ta, x);
          }
          tmem_wait_st();
        }
        if constexpr (kWide) {  // S(i) once more, for the row sum over its own maximum
          const float top = fmaxf(n, mx - cb);
          l *= ex2_approx(n - top);
          n = top;
#pragma unroll 1
          for (int c = 0; c < kN / 16; ++c) {
            uint32_t x[16];
            tmem_ld16(ts + c * 16, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) l += c * 16 + k < valid ? ex2_approx(fmaf(__uint_as_float(x[k]), ca, -n)) : 0.f;
          }
        } else if (m_own != m_i && m_own != -INFINITY) {
          l *= ex2_approx(m_own - m_i);
        }
        m_own = m_i;
        // P = 2^(z - m + kShift), packed two per 32-bit column and written over columns [0, 32) of the
        // S(i) buffer, whose 64 columns are in registers
        const float m_use = m_i == -INFINITY ? 0.f : m_i;
        {
          const float off = cb - m_use + kShift;
          const uint64_t scale2 = f2_pack(ca, ca), nm2 = f2_pack(off, off);
          uint64_t acc[2] = {0ull, 0ull};  // packed partial sums (0.0f bit patterns)
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
          GRANIKV_TMEM_ST32(ts, pk);
          float la, lb;
          f2_unpack(f2_add(acc[0], acc[1]), la, lb);
          // over vs, by the very logarithm that P has
          if constexpr (!kWide) l += (la + lb) * ex2_approx(least - cb);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarPFull + sb));
      }
    };
    if (wide) all_tiles(std::true_type{});
    else all_tiles(std::false_type{});
    // epilogue: wait for the last PV, combine the two warps' row sums (each with its exponent), normalise
    // (O is relative to the last tile's max), write the record
    if (ok) {
      const int last = n_tiles - 1;
      ok = mbar_wait_bounded(bar(kBarPvDone + last % kSBufs), (last / kSBufs) & 1, abort_flag, p.err, kDevTimeout,
                             kWaitLimitNs);
    }
    ok = __all_sync(0xffffffffu, ok);
    // swap the row sums, exponents and maxima with the other warp at the pair barrier; a warp that left the
    // tile loop early may stop waiting for published maxima, so its partner's bounded waits give
    // up and both skip the record
    // (the codes' slots, where these go, are idle once the last PV is done; a CTA that gave up may
    // still have a copy in flight there, and then writes nothing)
    const bool safe = ok;
    if (safe) {
      red[par * kM + r] = l;
      red[2 * kM + par * kM + r] = wide ? n : m_own - kShift - least;
      red[4 * kM + par * kM + r] = m_own;
    }
    mbar_arrive(bar(pair_bar));
    const bool pair_ok = mbar_wait_bounded(bar(pair_bar), 0, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
    ok = __all_sync(0xffffffffu, pair_ok) && ok && !*abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const float l0 = red[r], l1 = red[kM + r], e0 = red[2 * kM + r], e1 = red[3 * kM + r];
      const float m_used = red[4 * kM + ((n_tiles - 1) & 1) * kM + r];
      const float top = fmaxf(e0, e1);
      // a warp that had no tile left 0 and -inf
      const float lt = l0 * ex2_approx(e0 - top) + l1 * ex2_approx(e1 - top);
      if (row < rows && (rec < 0 || rec >= p.n_records)) {
        if (half == 0) atomicCAS(p.err, 0, (int32_t)kDevBadRecord);
        rec = -1;
      }
      const float inv = 1.f / lt, unit = ex2_approx(m_used - kShift - top);  // (a tile has a valid token)
      uint32_t u[2][32];
      GRANIKV_TMEM_LD32(tmem + lane_off + kColO + half * 64, u[0]);
      GRANIKV_TMEM_LD32(tmem + lane_off + kColO + half * 64 + 32, u[1]);
      tmem_wait_ld();
      // every lane stores its half row, a whole 32-byte sector at a time
      if (rec >= 0) {
        const uint64_t keep = l2_policy_keep();
        float* dst = p.rec_o + ((int64_t)rec * p.n_q + h) * kD + half * 64;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(u[c >> 2][(c & 3) * 8 + k]) * inv * unit;
          st_record8(dst + c * 8, x, keep);
        }
        if (half == 0) {
          st_record(p.rec_lse + (int64_t)rec * p.n_q + h, kv8_record_lse(lt, (top + log2f(lt)) * kLn2), keep);
        }
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
