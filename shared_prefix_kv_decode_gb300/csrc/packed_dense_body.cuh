// packed_dense_body.cuh -- dense prefix backend over the 8- or 4-bit cache on the 5th-generation tensor cores
// (tcgen05/TMEM), head_dim 128 (4 bits: or 64), bf16 q.  (8 bits first; what 4 bits change stands at the end.)
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
// V scales lie between 2^-104.9 (of zeros) and 2^119.2.  A tile's P is that much smaller than another's of equal weights
// as its V scale is, and a block's scale may come from a token without weight, so in fp16 the weights that make up the
// output may vanish beside others.  Where the scales of a piece span more than 2^8, their powers of two therefore go into
// V's operands, which are bf16 then (a code, or a code times its 4-bit scale, has 4 or 6 significant bits; the piece's largest
// scale becomes 2^90, what lies 2^216 below it 0), and P has the significand of vs alone: P = 2^(z - m - 8) as the sum of two
// bf16 values (16 bits, at most 1, down to 2^-118 of the largest weight), over all of S, in twice the products, with small
// loops, so that the others' instructions stay close: unrolled as those are they cost every piece 3 to 4 %.  With every
// eighth block of V zero the step of a 16K prefix with 64 requests takes 56 us (8 bits 51) instead of 34 (31).
// Elsewhere P is one fp16 value, 11 bits: a weight below 2^-13 of the piece's largest may be off by 2^-24 of that.  The rounding,
// 2^-12.8 of a weight on average, moves about 2 % of the bf16 results to a neighbour (8e-4 of them in the root mean square, where
// their own rounding is 1.7e-3): chosen, since a second part would double the products with P and put a subtraction, a
// conversion and a store more into the rounds that set the pace.
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
//
// 4 bits.  An element is code * b * u, b the e4m3 scale of its 16 dims and u the power of two of its block of 64 slab
// tokens and head, that is, of a tile.  code * b is exact in fp16, so the conversion warps make fp16 operand tiles of
// K as of V (an fp16x2 conversion and a product for each pair), S is an fp16 product with q in fp16 (scaled by a power of two
// to [2^14, 2^15): exact down to 2^-31 of the row's largest element), and u takes the place of ks and vs.  Eight
// warps convert, four of K and four of V (four for both: 104.9 us where eight take 86.7, see below for the shape).  A
// warp's ring holds its 32 tokens' codes, by a TMA box, and scales, 8 bytes a token by cp.async from the warp
// itself.  The K and V rings have five slots of one tile in fp16 (two and three of two tiles: a step of a 16K prefix with
// 64 requests 37.4 us, so 36.7).
// The conversion warps go ahead from the first barrier on, beside q's way to TMEM (one request on 8K 11.2 us, so 10.8).
// What bounds it: the softmax warps' rounds, next to the conversion on the same issue slots and the same shared memory.
// 480 requests on a slab of 8K (32/8 heads of 128, two waves of CTAs) take 73.8 us, in 8 bits 64.  With parts taken out (of 75 us,
// before wide pieces had loops of their own): the products 73.6, three quarters of the conversion's products and stores 69.7, both 67.7; the exponentials, the maxima or the row
// sums 1 to 2 % each, the scales' loads nothing.  Codes and scales of all conversion warps fetched by two warps of their own, in
// boxes of 128 rows: 77.
#pragma once

#include <cuda.h>

#include <cfloat>

#include "internal.h"
#include "kv4_util.cuh"
#include "kv8_util.cuh"
#include "launch_util.cuh"
#include "mma_util.cuh"
#include "packed_suffix_body.cuh"
#include "tc_util.cuh"

#include <type_traits>

namespace granikv {
namespace pkd {
namespace {

using pks::lg2_approx;
using pks::pack_f16;
using pks::block_barrier;
using pks::part_barrier;
using pks::regs_down;
using pks::regs_up;

constexpr int kM = kDenseRows;                // 128 query rows per CTA
constexpr int kN = kPackedBlock;              // 64 tokens per tile
constexpr int kPair = kDenseTile;             // 128 tokens: what is loaded at a time
static_assert(kPair == 2 * kN && kPair / 4 == kPackedBox, "a conversion warp's part is one box");
constexpr int kSBufs = 5;                     // S/P buffers in TMEM
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kWarpConv = 8, kParts = 4;
constexpr int kPart = kPair / kParts;         // tokens that one warp converts at a time
template <int BITS, int D>
struct Layout {
  static_assert(D == 128 || (BITS == 4 && D == 64), "head_dim");
  // 8 bits: kParts warps convert V.  4 bits: as many convert K, before them.  (One more warp, for the suffix body's producers.)
  static constexpr int kConvWarps = BITS == 8 ? kParts : 2 * kParts;
  static constexpr int kWarpS = kWarpConv + kConvWarps, kWarpPv = kWarpS + 1, kWarpTmaK = kWarpS + 2;
  static constexpr int kThreads = (kWarpS + 4) * 32;
  // 4 bits: 20 warps start with 96 registers; the softmax warps go on with 128, the others with 72
  static constexpr bool kSplitRegs = BITS == 4;
  // A slot of the fp16 rings holds 128 tokens, which four warps fill, or (4 bits) a tile of 64, filled by the two warps whose
  // parts it is: what S and PV have read is free a tile earlier
  static constexpr int kSlotTiles = BITS == 8 ? 2 : 1;
  static constexpr int kFill = kParts * kSlotTiles / 2;   // warps that fill a slot
  static constexpr int kHalf = kSlotTiles * kN * 128;     // one 64-dim half of a slot
  static constexpr int kSlot = D / 64 * kHalf;            // 32 KB or (4 bits) 16, heads of 64: 8
  static constexpr int kVSlots = BITS == 8 ? 3 : 5;       // slots of the V ring (fp16)
  static constexpr int kKSlots = BITS == 8 ? 4 : 5;       // slots of the K ring (codes of 128 tokens, 4 bits: fp16)
  static constexpr int kKSlotBytes = BITS == 8 ? kPair * D : kSlot;
  static constexpr int kCSlots = BITS == 8 ? 4 : 3;       // slots of each conversion warp's ring (codes, 4 bits: and scales)
  static constexpr int kHead = D * BITS / 8;              // bytes of a head's codes
  static constexpr int kScale = D / kKv4Group;            // 4 bits: of its scales
  static constexpr int kCSlotBytes = kPart * (kHead + (BITS == 8 ? 0 : kScale));
  static constexpr int kRedBytes = 6 * kM * 4;            // the epilogue's sums, exponents and maxima
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kKSlots * kKSlotBytes;
  static constexpr int kOffCodes = kOffV + kVSlots * kSlot;
  static constexpr int kOffUnit = kOffCodes + kConvWarps * kCSlots * kCSlotBytes;  // [kM] power of two that undoes a row's scaling
  static constexpr int kOffMPub = kOffUnit + kM * 4;      // [4 quarters][2 tile parities][32 rows] published maxima
  static constexpr int kOffBar = kOffMPub + 4 * 2 * 32 * 4;
  static constexpr int kBarArea = BITS == 8 ? 512 : 640;
  static constexpr int kSmemBytes = kOffBar + kBarArea + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(kFill * kCSlots * kCSlotBytes >= kRedBytes,
                "the epilogue's sums and maxima lie in rings whose parts fill every content's first tile");
  // barriers
  static constexpr int kBarKFull = 0;                            // [kKSlots] TMA (4 bits: conversion, kFill arrivals) -> MMA
  static constexpr int kBarKEmpty = kBarKFull + kKSlots;         // [kKSlots] MMA (S of the slot's tiles done) -> TMA (conversion)
  static constexpr int kBarCFull = kBarKEmpty + kKSlots;         // [kConvWarps][kCSlots] TMA -> conversion
  static constexpr int kBarVFull = kBarCFull + kConvWarps * kCSlots;  // [kVSlots] conversion -> MMA (kFill arrivals)
  static constexpr int kBarVEmpty = kBarVFull + kVSlots;         // [kVSlots] MMA (PV of the slot's tiles done) -> conversion
  static constexpr int kBarSFull = kBarVEmpty + kVSlots;         // [kSBufs] S(i) in TMEM -> softmax
  static constexpr int kBarPFull = kBarSFull + kSBufs;           // [kSBufs] P(i) in TMEM -> MMA (128 arrivals)
  static constexpr int kBarPvDone = kBarPFull + kSBufs;          // [kSBufs] PV(i) done -> softmax, and S(i + kSBufs)
  static constexpr int kBarDrain = kBarPvDone + kSBufs;          // [2] all S (all PV) products done -> teardown
  static constexpr int kBarPair = kBarDrain + 2;                 // [4] the two softmax warps of a row quarter, epilogue (64)
  static constexpr int kBarMPub = kBarPair + 4;                  // [4 quarters][2 parities] max of a tile published (32)
  static constexpr int kNumBars = kBarMPub + 8;
  static_assert(8 * kNumBars + 16 <= kBarArea, "barrier area");
};
constexpr uint32_t kTmemCols = 512;           // S/P buffers at 0, 64, 128, 192, 256; Q (hi, lo) at 320; O at 384
constexpr uint32_t kColQ = kSBufs * kN, kColO = 384;
static_assert(kColQ + 128 / 2 <= kColO && kColO + 128 <= kTmemCols, "TMEM columns");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 of the largest growth tolerated in P
constexpr float kShift = 7.0f;                // log2 of the factor that P carries
constexpr uint32_t kWideSpan = 8;             // log2 of a wide span of V scales
constexpr float kWideShift = -8.0f;           // there: log2 of P's factor (P <= 1)
constexpr int kWideTop = 90;                  // and of what the largest V scale's power of two becomes in V's operands
constexpr uint64_t kWaitLimitNs = 2000000000ull;

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
// Two fp16 times f -> bf16 (exact: see kWideSpan).
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t w, float f) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
  const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * f, x.y * f);
  return *reinterpret_cast<const uint32_t*>(&y);
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
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a));
  return x;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// A conversion lane's place in a slot of fp16 operands (two halves of 64 dims, 128-byte rows, 128-byte swizzle).  The
// lanes take 16 bytes of codes each: 16 dims of four tokens, or (4 bits) 32 dims of eight.  A store instruction's
// eight lanes at a time have to cover eight 16-byte chunks that differ in their place within 128 bytes, which the swizzle
// XORs with the token's last bits; the lanes of the upper 64 dims, whose chunks have the same places as the lower
// ones', take the token whose bits differ by one step: 1, or 2 (where the bit 1 already tells two tokens apart).
// (With the stores of the upper half in another order, by a branch, and scales in TMA boxes: 90.4 us where this takes 76.1.)
template <int BITS, int D>
struct ConvLane {
  using Lay = Layout<BITS, D>;
  static constexpr int kDims = 128 / BITS;             // 16 or 32
  static constexpr int kLanes = D / kDims;             // of a token: 8 or 4, heads of 64: 2
  static constexpr int kStep = 32 / kLanes;            // tokens of a load: 4 or 8
  static constexpr int kPer = kPart / kStep;           // loads of a part
  int dim, token;                                      // first dim; token of load 0
  uint32_t row, ch;                                    // of the operand tile: the row's offset, first chunk
  __device__ __forceinline__ ConvLane(int part, int lane) {
    const int c = lane % kLanes;
    dim = c * kDims;
    token = (lane / kLanes) ^ (dim >= 64 ? kStep / 4 : 0);
    row = (uint32_t)(part % Lay::kFill * kPart + token) * 128 + (dim >= 64 ? Lay::kHalf : 0);
    ch = (uint32_t)(dim % 64 / 8);
  }
  // chunk k (8 dims) of load n
  __device__ __forceinline__ void store(uint32_t tile, int n, int k, uint32_t x, uint32_t y, uint32_t z, uint32_t w) const {
    const uint32_t swizzle = (uint32_t)(token + n * kStep) & 7u;
    sts128(tile + row + n * kStep * 128 + (((ch + k) ^ swizzle) << 4), x, y, z, w);
  }
};

// Prefix work item `item` (one CTA) on `smem_raw` (at least Layout<BITS, D>::kSmemBytes), run by Layout<BITS, D>::kThreads threads.
template <int BITS, int D>
__device__ __forceinline__ void packed_dense_body(const AttnParams& p, int32_t item, const PackedMaps* maps,
                                                  unsigned char* smem_raw) {
  using Lay = Layout<BITS, D>;
  constexpr int kKSlots = Lay::kKSlots, kVSlots = Lay::kVSlots, kCSlots = Lay::kCSlots, kConvWarps = Lay::kConvWarps;
  constexpr int kSlotTiles = Lay::kSlotTiles, kHalf = Lay::kHalf, kFill = Lay::kFill;
  constexpr int kWarpS = Lay::kWarpS, kWarpPv = Lay::kWarpPv, kWarpTmaK = Lay::kWarpTmaK;
  constexpr int kOffK = Lay::kOffK, kOffV = Lay::kOffV, kOffCodes = Lay::kOffCodes, kOffUnit = Lay::kOffUnit, kOffMPub = Lay::kOffMPub,
                kOffBar = Lay::kOffBar;
  constexpr int kBarKFull = Lay::kBarKFull, kBarKEmpty = Lay::kBarKEmpty, kBarCFull = Lay::kBarCFull, kBarVFull = Lay::kBarVFull,
                kBarVEmpty = Lay::kBarVEmpty, kBarSFull = Lay::kBarSFull, kBarPFull = Lay::kBarPFull, kBarPvDone = Lay::kBarPvDone,
                kBarDrain = Lay::kBarDrain, kBarPair = Lay::kBarPair, kBarMPub = Lay::kBarMPub, kNumBars = Lay::kNumBars;
  // 1024-byte alignment for the 128-byte-swizzle atoms
  const uint32_t raw_u = smem_u32(smem_raw);
  const uint32_t base = (raw_u + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw_u);
  const uint32_t sK = base + kOffK, sV = base + kOffV, sC = base + kOffCodes;
  // row sums, exponents and maxima for the epilogue, [kind][parity][row], in the first codes' place (idle by then)
  float* red = reinterpret_cast<float*>(smem + kOffCodes);
  float* units = reinterpret_cast<float*>(smem + kOffUnit);
  const uint32_t sBar = base + kOffBar;
  auto bar = [&](int i) { return sBar + 8u * i; };
  // after the barriers four words: the abort flag, V's smallest scale, the tensor memory's address, V's wide top
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
  const int n_pairs = (n_tiles + 1) / 2;
  const bool slab_ok = gr.slab_off >= 0 && gr.slab_off + gr.L_p <= p.n_hot && n_tiles > 0;
  const int32_t rbase = it.row_block * kM;
  const int64_t first_slot = gr.slab_off + t0;

  // slot contents: tokens kPair * i .. of the piece
  auto issue_k = [&](int i) {
    const int st = i % kKSlots;
    mbar_arrive_expect_tx(bar(kBarKFull + st), Lay::kKSlotBytes);
    tma_load_2d(sK + st * Lay::kKSlotBytes, &maps->k, j * D, (int32_t)(first_slot + (int64_t)i * kPair), bar(kBarKFull + st));
  };
  // conversion warp w's part of V's (4 bits, w < kParts: K's) slot contents i
  auto issue_c = [&](int w, int i) {
    const int c = w * kCSlots + i % kCSlots;
    const uint32_t dst = sC + c * Lay::kCSlotBytes, full = bar(kBarCFull + c);
    const int32_t slot = (int32_t)(first_slot + (int64_t)i * kPair + w % kParts * kPart);
    mbar_arrive_expect_tx(full, kPart * Lay::kHead);
    tma_load_2d(dst, BITS == 4 && w < kParts ? &maps->k : &maps->v, j * Lay::kHead, slot, full);
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
    tma_prefetch_desc(&maps->k);
    tma_prefetch_desc(&maps->v);
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1u;
      if (i >= kBarVFull && i < kBarVFull + kVSlots) count = kFill;
      if (BITS == 4 && i >= kBarKFull && i < kBarKFull + kKSlots) count = kFill;
      if (i >= kBarPFull && i < kBarPFull + kSBufs) count = kSoftmaxThreads / 2;
      if (i >= kBarPair && i < kBarPair + 4) count = 64u;
      if (i >= kBarMPub && i < kBarMPub + 8) count = 32u;
      if (i == kBarVFull && p.inject_stall == 2 && blockIdx.x == 0) count += 1u;  // test hook: an arrival that does not come
      mbar_init(bar(i), count);
    }
    *abort_flag = slab_ok ? 0 : 1;
    if (!slab_ok) atomicCAS(p.err, 0, (int32_t)kDevBadSlab);
    mbar_fence_init();
    fence_proxy_async_smem();
    if constexpr (BITS == 8) {
      grid_dep_wait();  // the slab may have been written by the work before this kernel
      if (slab_ok) {
        for (int i = 0; i < min(n_pairs, kKSlots); ++i) issue_k(i);
        for (int i = 0; i < min(n_pairs, kCSlots); ++i)
          for (int w = 0; w < kConvWarps; ++w) issue_c(w, i);
      }
    }
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if constexpr (BITS == 4) __syncthreads();  // the barriers are ready: the conversion warps go ahead from here
  // q and the records are touched only after the previous kernel in the stream has completed
  grid_dep_wait();
  grid_dep_launch_dependents();
  // Q: the two softmax warps of a row quarter take half of their rows' dims each, agree on each row's
  // power of two through shared memory, and split the elements into hi and lo, four to a word; rows
  // past the group are 0
  constexpr int kQw = D / 4;  // words of half a row
  uint32_t qw[kQw];
  float* part = reinterpret_cast<float*>(smem + kOffMPub);  // [2][kM], used for the maxima of tiles later
  // the scales of tile i; a softmax warp's first ones are on their way with its rows
  const int64_t scale_at = BITS == 8 ? (int64_t)p.n_kv * D + 4 * j : kv4_units_at(p.n_kv, D) + j;
  using Scale = std::conditional_t<BITS == 8, float, uint8_t>;  // as it stands in the row
  Scale ks{}, vs{};
  auto load_scales = [&](int i) {
    const int64_t a = (first_slot + (int64_t)i * kN) * p.packed_row + scale_at;
    ks = *reinterpret_cast<const Scale*>(static_cast<const uint8_t*>(p.kpool) + a);
    vs = *reinterpret_cast<const Scale*>(static_cast<const uint8_t*>(p.vpool) + a);
  };
  // V scales of the piece's tiles as the bits of positive floats: the smallest one's, and, where they span widely, the
  // biased exponent of the largest (else 0).  The PV warp finds them beside q's way for the warps that wait for that;
  // the 4-bit conversion warps, which do not, for themselves.
  auto v_scale_bits = [&](int i) {
    const uint8_t* at = static_cast<const uint8_t*>(p.vpool) + (first_slot + (int64_t)i * kN) * p.packed_row + scale_at;
    if constexpr (BITS == 8) return *reinterpret_cast<const uint32_t*>(at);
    else return (uint32_t)*at << 23;
  };
  auto v_span = [&](uint32_t& lo) {
    uint32_t hi = 0u;
    lo = 0xffffffffu;
    for (int i = lane; slab_ok && i < n_tiles; i += 32) {
      const uint32_t x = v_scale_bits(i);
      lo = min(lo, x);
      hi = max(hi, x);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    return hi > lo && hi - lo > kWideSpan << 23 ? hi >> 23 : 0u;
  };
  volatile uint32_t* v_least = reinterpret_cast<volatile uint32_t*>(smem + kOffBar + 8 * kNumBars + 4);
  volatile uint32_t* v_top = v_least + 2;
  if (warp == kWarpPv) {
    uint32_t lo;
    const uint32_t top = v_span(lo);
    if (lane == 0) {
      *v_least = lo;
      *v_top = top;
    }
  }
  if (warp < kSoftmaxWarps) {
    if (slab_ok && qhalf < n_tiles) load_scales(qhalf);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                      ((int64_t)req * p.n_q + h) * D + qhalf * (D / 2));
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kQw / 4; ++k) {
      const uint4 x = have ? src[k] : make_uint4(0u, 0u, 0u, 0u);
      qw[4 * k] = x.x;
      qw[4 * k + 1] = x.y;
      qw[4 * k + 2] = x.z;
      qw[4 * k + 3] = x.w;
    }
#pragma unroll
    for (int k = 0; k < kQw; ++k) amax = fmaxf(amax, bf16x2_finite_max(qw[k]));
    part[qhalf * kM + qrow] = amax;
  }
  // 4 bits: K has to be converted before the first product, which q's way to TMEM need not hold up
  const bool ahead = BITS == 4 && warp >= kWarpConv && warp < kWarpS;
  auto q_barrier = [&] {
    if constexpr (BITS == 8) __syncthreads();
    else if (!ahead) part_barrier<Lay::kThreads - 32 * kConvWarps>();
  };
  tc_fence_before();
  q_barrier();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp < kSoftmaxWarps) {
    float unit;
    const float f = q_factor<BITS == 8 ? 7 : 14>(fmaxf(part[qrow], part[kM + qrow]), unit);
    if (qhalf == 0) units[qrow] = unit;
    if constexpr (BITS == 4) {
#pragma unroll
      for (int k = 0; k < kQw; ++k) {
        const __half2 x = q_no_inf(f16x2_of(qw[k], f));
        qw[k] = *reinterpret_cast<const uint32_t*>(&x);
      }
      const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColQ + qhalf * kQw;
      if constexpr (D == 128) GRANIKV_TMEM_ST32(at, qw);
      else tmem_st16(at, qw);
      tmem_wait_st();
    } else {
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
  }
  tc_fence_before();
  q_barrier();
  tc_fence_after();

  if (warp >= kSoftmaxWarps) {
    if constexpr (Lay::kSplitRegs) regs_down<72>();
    if (warp < kWarpConv + kConvWarps) {
      // ---------------- conversion: codes of V (4 bits: of K and V) -> fp16 operand tiles ----------------
      const int w = warp - kWarpConv;
      const int part = w % kParts;
      const bool to_k = BITS == 4 && w < kParts;
      using Conv = ConvLane<BITS, D>;
      constexpr int kPer = Conv::kPer;
      const Conv cl(part, lane);
      const uint32_t ring = to_k ? sK : sV;
      const int slots = to_k ? kKSlots : kVSlots, full = to_k ? kBarKFull : kBarVFull, empty = to_k ? kBarKEmpty : kBarVEmpty;
      int issued = slab_ok ? min(n_pairs, kCSlots) : 0, seen = 0;
      // 4 bits: the scales of contents i, a token a lane (zeros past the piece's end); a group for every i
      const uint8_t* scale_src = static_cast<const uint8_t*>(to_k ? p.kpool : p.vpool) + (first_slot + part * kPart + lane) * p.packed_row +
                                 kv4_scales_at(p.n_kv, D) + j * Lay::kScale;
      auto copy_scales = [&](int i) {
        if constexpr (BITS == 4) {
          const uint32_t dst = sC + (w * kCSlots + i % kCSlots) * Lay::kCSlotBytes + kPart * Lay::kHead + lane * Lay::kScale;
          const bool in = t0 + i * kPair + part * kPart + lane < t1;
          if (slab_ok && i < n_pairs) {
            const uint8_t* src = in ? scale_src + (int64_t)i * kPair * p.packed_row : static_cast<const uint8_t*>(p.kpool);
            if constexpr (D == 128) cp_async8(dst, src, in ? 8 : 0);
            else cp_async4(dst, src, in ? 4 : 0);
          }
          cp_async_commit();
        }
      };
      if constexpr (BITS == 4) {
        if (lane == 0)
          for (int i = 0; i < issued; ++i) issue_c(w, i);
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < kCSlots; ++i) copy_scales(i);
      uint32_t lo;
      const int wide_top = to_k ? 0 : BITS == 8 ? (int)*v_top : (int)v_span(lo);
      // wide: what code (times scale) is multiplied by in V's operands, which are bf16 then: the tile's power of two, that of the
      // piece's largest made 2^kWideTop
      auto v_size = [&](int tile) {
        const int e = tile < n_tiles ? (int)(v_scale_bits(tile) >> 23) - wide_top + kWideTop + 127 : 0;
        return e > 0 ? __uint_as_float((uint32_t)e << 23) : 0.f;
      };
      auto all_parts = [&](auto wide_span) {
        constexpr bool kWide = decltype(wide_span)::value;
        for (int i = 0; slab_ok && i < n_pairs; ++i) {
          const int c = w * kCSlots + i % kCSlots;
          const int use = BITS == 8 ? i : 2 * i + part / kFill, st = use % slots;  // the slot's use, of all of the ring's
          bool ok = mbar_wait_bounded(bar(kBarCFull + c), (i / kCSlots) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;  // the abort flag is up: every other role leaves as well
          seen = i + 1;
          if constexpr (BITS == 4) {
            cp_async_wait<kCSlots - 1>();
            __syncwarp();
          }
          const uint32_t src = sC + c * Lay::kCSlotBytes, dst = ring + st * Lay::kSlot;
          const int valid = t1 - t0 - i * kPair - part * kPart;  // tokens of the part in range, or more
          auto codes = [&](int n, uint32_t& b) {  // of load n, and (4 bits) their two scales
            const uint32_t t = (uint32_t)(cl.token + n * Conv::kStep);
            if constexpr (BITS == 4) b = lds16(src + kPart * Lay::kHead + t * Lay::kScale + cl.dim / 16);
            return lds128(src + t * Lay::kHead + cl.dim * BITS / 8);
          };
          // 0 * whatever lies past the piece must not reach O
          auto mask = [&](int n, uint4& x, uint32_t& b) {
            if (cl.token + n * Conv::kStep >= valid) {
              x = make_uint4(0u, 0u, 0u, 0u);
              b = 0u;
            }
          };
          uint4 x[kWide ? 1 : kPer];
          uint32_t b[kWide ? 1 : kPer];
          if constexpr (!kWide) {
#pragma unroll
            for (int n = 0; n < kPer; ++n) x[n] = codes(n, b[n]);
            if (valid < kPart) {
#pragma unroll
              for (int n = 0; n < kPer; ++n) mask(n, x[n], b[n]);
            }
          }
          const bool fills = BITS == 8 || use < n_tiles;  // (4 bits: the last two parts may have no tile)
          if (fills && use >= slots) {
            ok = mbar_wait_bounded(bar(empty + st), ((use / slots) - 1) & 1, abort_flag, p.err, kDevTimeout, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          [[maybe_unused]] float size = 1.f;
          if constexpr (kWide) size = v_size(2 * i + part / 2);
          auto put = [&](int n, const uint4& x, uint32_t b) {
            if constexpr (BITS == 8) {
              uint32_t y[8];
              e4m3x4_to_f16x4(x.x, y[0], y[1]);
              e4m3x4_to_f16x4(x.y, y[2], y[3]);
              e4m3x4_to_f16x4(x.z, y[4], y[5]);
              e4m3x4_to_f16x4(x.w, y[6], y[7]);
              if constexpr (kWide) {
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = f16x2_to_bf16x2(y[k], size);
              }
              cl.store(dst, n, 0, y[0], y[1], y[2], y[3]);
              cl.store(dst, n, 1, y[4], y[5], y[6], y[7]);
            } else {
              const uint32_t f = e4m3x2_to_f16x2((uint16_t)b), f2[2] = {__byte_perm(f, f, 0x1010), __byte_perm(f, f, 0x3232)};
              const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t y[4];
                e2m1x8_to_f16x8(u[k], y);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                  y[h] = f16x2_mul(y[h], f2[k / 2]);
                  if constexpr (kWide) y[h] = f16x2_to_bf16x2(y[h], size);
                }
                cl.store(dst, n, k, y[0], y[1], y[2], y[3]);
              }
            }
          };
          if constexpr (kWide) {
#pragma unroll 1
            for (int n = 0; fills && n < kPer; ++n) {
              x[0] = codes(n, b[0]);
              mask(n, x[0], b[0]);
              put(n, x[0], b[0]);
            }
          } else {
#pragma unroll
            for (int n = 0; n < kPer; ++n) {
              if (!fills) break;
              put(n, x[n], b[n]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();  // the warp has stored its part, and read its codes
          copy_scales(i + kCSlots);
          if (lane == 0) {
            if (fills) mbar_arrive(bar(full + st));
            if (i + kCSlots < n_pairs) {
              issue_c(w, i + kCSlots);
              if (l2_ahead > 0 && i + kCSlots + l2_ahead < n_pairs)
                tma_prefetch_l2_2d(to_k ? &maps->k : &maps->v, j * Lay::kHead,
                                   (int32_t)(first_slot + (int64_t)(i + kCSlots + l2_ahead) * kPair + part * kPart));
              issued = i + kCSlots + 1;
            }
          }
        }
      };
      // (a loop for each)
      if (wide_top) all_parts(std::true_type{});
      else all_parts(std::false_type{});
      // never leave with a copy in flight
      if constexpr (BITS == 4) cp_async_wait<0>();
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
      // ---------------- TMA loads of K (8 bits) ----------------
      if (BITS == 8 && lane == 0) {
        int issued = slab_ok ? min(n_pairs, kKSlots) : 0;
        for (int i = issued; slab_ok && i < n_pairs; ++i) {
          if (!mbar_wait_bounded(bar(kBarKEmpty + i % kKSlots), ((i / kKSlots) - 1) & 1, abort_flag, p.err, kDevTimeout,
                                 kWaitLimitNs))
            break;
          issue_k(i);
          if (l2_ahead > 0 && i + l2_ahead < n_pairs)
            tma_prefetch_l2_2d(&maps->k, j * D, (int32_t)(first_slot + (int64_t)(i + l2_ahead) * kPair));
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
            if (i % kSlotTiles == 0 && !wait(kBarKFull, kKSlots, i / kSlotTiles)) break;
            tc_fence_after();
            const uint32_t dS = tm + (uint32_t)((i % kSBufs) * kN);
            const int st = i / kSlotTiles % kKSlots;
            const uint64_t dk = dk0 + (uint64_t)((st * Lay::kKSlotBytes + i % kSlotTiles * kN * 128) >> 4);  // rows of 128 bytes
#pragma unroll
            // 8 bits: lo, the smaller, first; 4 bits: 16 dims each, four of a 64-dim half
            for (int kk = 0; kk < (BITS == 8 ? 8 : D / 16); ++kk)
              if (el && BITS == 4)
                umma_f16_ts(dS, tm + kColQ + kk * 8, dk + (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), idS, kk > 0 ? 1u : 0u);
              else if (el)
                umma_f8_ts(dS, tm + kColQ + (kk < 4 ? 32 : 0) + (kk & 3) * 8, dk + (uint64_t)(((kk & 3) * 32) >> 4), idS,
                           kk > 0 ? 1u : 0u);
            if (el) {
              umma_commit(bar(kBarSFull + i % kSBufs));
              if (i % kSlotTiles == kSlotTiles - 1) umma_commit(bar(kBarKEmpty + st));
            }
            __syncwarp();
            committed += 1;
          }
        } else {
          // V slot as an MN-major B operand: 16 tokens per step (2048 bytes), the two 64-dim halves
          // kHalf apart (leading offset), 8-token groups 1024 bytes apart (stride)
          const uint64_t dv0 = smem_desc_sw128(sV, kHalf, 1024);
          auto all_products = [&](auto wide_span) {
            constexpr bool kWide = decltype(wide_span)::value;
            constexpr uint32_t idO = kWide ? idesc_bf16_f32(kM, D, true) : idesc_fmt0_f32(kM, D, true);
            constexpr int kTerms = kWide ? 2 : 1;  // of P, 8 columns each for 16 tokens
            for (int i = 0; i < n_tiles; ++i) {
              if (i % kSlotTiles == 0 && !wait(kBarVFull, kVSlots, i / kSlotTiles)) break;
              if (!wait(kBarPFull, kSBufs, i)) break;
              tc_fence_after();
              const uint32_t pa = tm + (uint32_t)((i % kSBufs) * kN);  // P(i): 32 columns, two tokens per column
              const int st = i / kSlotTiles % kVSlots;
              const uint64_t dv = dv0 + (uint64_t)((st * Lay::kSlot + i % kSlotTiles * (kN / 16) * 2048) >> 4);
#pragma unroll
              for (int ks = 0; ks < kN / 16 * kTerms; ++ks)
                if (el)
                  umma_f16_ts(tm + kColO, pa + (uint32_t)(ks * 8), dv + (uint64_t)((ks / kTerms * 2048) >> 4), idO,
                              (i > 0 || ks > 0) ? 1u : 0u);
              if (el) {
                umma_commit(bar(kBarPvDone + i % kSBufs));
                if (i % kSlotTiles == kSlotTiles - 1) umma_commit(bar(kBarVEmpty + st));
              }
              __syncwarp();
              committed += 1;
            }
          };
          if (*v_top) all_products(std::true_type{});
          else all_products(std::false_type{});
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
    }
    if constexpr (Lay::kSplitRegs) {
      // (between the two barriers the softmax warps give back what they took)
      __syncwarp();
      block_barrier<Lay::kThreads>();
      block_barrier<Lay::kThreads>();
      regs_up<96>();
    }
  } else {
    if constexpr (Lay::kSplitRegs) regs_up<128>();
    // ---------------- softmax warps 0-7: rows of quarter `quad`, tiles of parity `par` ----------------
    const int quad = warp & 3;
    const int par = warp >> 2;
    const int half = par;                           // the epilogue's column half of O
    const int r = qrow;                             // row = TMEM lane
    const uint32_t lane_off = (uint32_t)((quad * 32) << 16);
    const int pair_bar = kBarPair + quad;           // mbarrier of the two warps sharing rows
    float* mpub = reinterpret_cast<float*>(smem + kOffMPub) + quad * 64;  // [tile parity][lane]
    const float scale = p.scale_log2 * units[r];
    // (a loop and an epilogue for each: in one loop the untaken branch cost 2 % of a 16K prefix, with the epilogue in common
    // heads of 64 took 36.4 us where they take 33.8)
    auto all_tiles = [&](auto wide_span) {
      constexpr bool kWide = decltype(wide_span)::value;
      float m_own = -INFINITY;   // max (of z, base 2) used for this warp's latest tile
      float l = 0.f;             // this warp's share of the row sum, over 2^(m_own - (shift + least))
      bool ok = !*abort_flag;
      // log2 of the piece's smallest V scale; wide: P has no power of two of V's scales
      const float least = kWide ? 0.f : BITS == 8 ? lg2_approx(__uint_as_float(*v_least)) : (float)((int)(*v_least >> 23) - 127);
      for (int i = par; ok && i < n_tiles; i += 2) {
        const int sb = i % kSBufs;
        // (from the smallest normal number to the largest: 0 * -inf of a masked key and inf * 0 of a score would be NaN)
        float ca, cb;
        if constexpr (BITS == 8) {
          ca = scale * ks;
          cb = lg2_approx(kWide ? __uint_as_float((__float_as_uint(vs) & 0x7fffffu) | 0x3f800000u) : vs);
        } else {
          ca = scale * kv4_unit(ks);
          cb = kWide ? 0.f : (float)((int)vs - 127);
        }
        ca = fminf(fmaxf(ca, FLT_MIN), FLT_MAX);
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
        // row max of z (the factor is positive); masked keys: -inf, so their weight is 0
        [[maybe_unused]] uint32_t u[2][32];
        float mx;
        if constexpr (kWide) {
          mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kN / 16; ++c) {
            uint32_t x[16];
            tmem_ld16(ts + c * 16, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) mx = fmaxf(mx, c * 16 + k < valid ? __uint_as_float(x[k]) : -INFINITY);
          }
          mx = mx * ca + cb;
        } else {
          GRANIKV_TMEM_LD32(ts, u[0]);
          GRANIKV_TMEM_LD32(ts + 32, u[1]);
          tmem_wait_ld();
          if (valid < kN) {
#pragma unroll
            for (int k = 0; k < kN; ++k) u[k >> 5][k & 31] = k < valid ? u[k >> 5][k & 31] : 0xff800000u;
          }
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
          for (int c = 0; c < D / 16; ++c) {
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
        if (m_own != m_i && m_own != -INFINITY) l *= ex2_approx(m_own - m_i);
        m_own = m_i;
        // P = 2^(z - m + shift), packed two per 32-bit column and written over columns [0, 32) of the
        // S(i) buffer, whose 64 columns are in registers; wide: 16 tokens at a time, the nearest bf16 over the first 8 columns
        // of their S and what that leaves out over the others
        const float m_use = m_i == -INFINITY ? 0.f : m_i;
        {
          const float off = cb - m_use + (kWide ? kWideShift : kShift);
          float la, lb;
          if constexpr (kWide) {
            la = lb = 0.f;
#pragma unroll 1
            for (int c = 0; c < kN / 16; ++c) {
              uint32_t x[16];
              tmem_ld16(ts + c * 16, x);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int t = c * 16 + 2 * k;
                const float ea = t < valid ? ex2_approx(fmaf(__uint_as_float(x[2 * k]), ca, off)) : 0.f;
                const float eb = t + 1 < valid ? ex2_approx(fmaf(__uint_as_float(x[2 * k + 1]), ca, off)) : 0.f;
                la += ea, lb += eb;
                const __nv_bfloat162 hi = __floats2bfloat162_rn(ea, eb);
                const float2 h = __bfloat1622float2(hi);
                const __nv_bfloat162 lo = __floats2bfloat162_rn(ea - h.x, eb - h.y);
                x[2 * k] = *reinterpret_cast<const uint32_t*>(&hi);
                x[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&lo);
              }
              const uint32_t parts[16] = {x[0], x[2], x[4], x[6], x[8], x[10], x[12], x[14],
                                          x[1], x[3], x[5], x[7], x[9], x[11], x[13], x[15]};
              tmem_st16(ts + c * 16, parts);
            }
          } else {
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
            f2_unpack(f2_add(acc[0], acc[1]), la, lb);
          }
          // over vs (wide: its significand), by the very logarithm that P has
          l += (la + lb) * ex2_approx(least - cb);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarPFull + sb));
      }
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
      // (they go into the rings of the first kFill conversion warps.  Those have read all their codes once the last PV is done:
      // their parts belong to the first tile of each content, which some product waited for.  The other parts' last
      // content may have no tile, and its copies may still be landing.  A CTA that gave up may have copies in flight
      // in any ring, and writes nothing)
      const bool safe = ok;
      constexpr float shift = kWide ? kWideShift : kShift;
      if (safe) {
        red[par * kM + r] = l;
        red[2 * kM + par * kM + r] = m_own - (shift + least);
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
        // (a tile has a valid token); wide: V's operands back to their size, by half of the power of two each
        const int size = kWide ? (int)*v_top - 127 - kWideTop : 0, half_size = size >> 1;
        const float inv = 1.f / lt * __uint_as_float((uint32_t)(127 + half_size) << 23);
        const float unit = ex2_approx(m_used - shift - top) * __uint_as_float((uint32_t)(127 + size - half_size) << 23);
        // every lane stores its half row, a whole 32-byte sector at a time
        const uint64_t keep = l2_policy_keep();
        const uint32_t cols = tmem + lane_off + kColO + half * (D / 2);
        float* dst = p.rec_o + ((int64_t)rec * p.n_q + h) * D + half * (D / 2);
        auto store8 = [&](const uint32_t* u, int at) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(u[k]) * inv * unit;
          st_record8(dst + at, x, keep);
        };
        if constexpr (kWide) {
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 16) {
            uint32_t u[16];
            tmem_ld16(cols + c, u);
            tmem_wait_ld();
            if (rec >= 0) {
              store8(u, c);
              store8(u + 8, c + 8);
            }
          }
        } else {
          uint32_t u[D / 64][32];
          GRANIKV_TMEM_LD32(cols, u[0]);
          if constexpr (D == 128) GRANIKV_TMEM_LD32(cols + 32, u[1]);
          tmem_wait_ld();
          if (rec >= 0) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) store8(u[c >> 2] + (c & 3) * 8, c * 8);
          }
        }
        if (rec >= 0 && half == 0)
          st_record(p.rec_lse + (int64_t)rec * p.n_q + h, packed_record_lse(lt, (top + log2f(lt)) * kLn2), keep);
      }
    };
    if (__builtin_expect(*v_top == 0u, 1)) all_tiles(std::false_type{});
    else all_tiles(std::true_type{});
    if constexpr (Lay::kSplitRegs) {
      __syncwarp();
      block_barrier<Lay::kThreads>();
      regs_down<96>();
      block_barrier<Lay::kThreads>();
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
}  // namespace pkd
}  // namespace granikv
