// kv8_suffix_body.cuh -- COLD suffix partial attention over the 8-bit cache: bulk-copy gather of
// packed rows, warp-level fp16 tensor cores.
//
// Shape: head_dim 128, bf16 q, g = n_q/n_kv <= 8.  A consumer warp owns one KV head of one request
// segment; tokens are the MMA's M dimension, the g query heads its N dimension (8 columns):
//     S^T[16 tok x 8] = K[16 tok x 128] . Q^T[128 x 8]       (8 mma.m16n8k16, fp16)
//     O^T[128 x 8]   += V^T[128 x 16 tok] . P^T[16 tok x 8]  (8 mma.m16n8k16, fp16)
// Number format.  Codes become fp16 exactly (one conversion per pair, on the way from ldmatrix to
// the MMA); q is brought into fp16's range by a power of two per query head (exact but for elements
// 2^-31 below the row's largest).  With ks, vs the token's scales, y = s ks and z = y + log2 vs (base 2), the
// running maximum m is taken over z and P = 2^(z - m) is what meets the V codes (p times vs), so a token with
// a small V scale cannot push the weights of the others out of fp16's range.  P carries a factor of
// 2^14 (it is at most 2^14), so that fp16 keeps its 11 bits down to weights of 2^-28; m, the sums and
// O are fp32.
// The row sum adds 2^(y - m + 10).  A scale lies between 2^-104.9 (of zeros) and 2^119.2, so y - m is at most 104.9, and
// the 4,096 tokens a CTA may have sum to less than 2^127; the heaviest token has y - m of -119.2 or more, so what it
// adds is a normal number, and a weight down to 2^-40 of it a subnormal one.  (P / vs in place of this exponential
// would lose the tokens whose P underflows, and with P's factor overflow on 600 zero rows.)
// ldmatrix moves 16-bit pairs, here two codes: a lane's 4 codes of a row serve one k-step of S^T in
// a permuted order of head_dim (q is loaded in the same order), and the transposed form gives two
// tokens x two dims, which one byte permutation turns into the two A registers of O^T's dims 2 r
// and 2 r + 1.
//
// Loads: the plan's token-CTA runs, as in the 16-bit kernel.  Producer warps stream 16-token
// tiles through a 6-stage shared-memory ring, one cp.async.bulk for each token's packed K and V row
// (1,056 bytes for eight heads: codes and scales arrive together), so a CTA keeps up to 200 KB in
// flight.  Rows are 1,072 bytes apart, which puts the eight rows an ldmatrix reads into eight
// different 16-byte bank groups.  Rows past a segment's end come from a zero row.  Every mbarrier wait is
// bounded in time; on expiry the CTA raises an abort flag, latches an error, and the producer
// waits (again bounded) for its copies in flight before the CTA exits.
// Bound by HBM on scattered rows: 71K tokens (150 MB, 128 requests) alone take 31.6 us with the merge, about
// 5.8 TB/s once the rings are full; without the conversions the time is the same.  One tile at a time and one
// producer warp took 48.1.
#pragma once

#include "internal.h"
#include "kv8_util.cuh"
#include "launch_util.cuh"
#include "mma_util.cuh"
#include "tc_util.cuh"

#include <type_traits>

namespace granikv {
namespace k8s {
namespace {

constexpr int kD = 128;
constexpr int kTile = 16;                          // tokens per tile (MMA M)
constexpr int kStages = 6;
constexpr int kWarps = 8;                          // consumer warps: KV heads per CTA
constexpr int kProducers = 8;                      // producer warps: two of a tile's rows each
constexpr int kRowsEach = kTile / kProducers;
constexpr int kThreads = (kWarps + kProducers) * 32;
constexpr int kRowMax = kWarps * (kD + 4);         // packed row of eight heads: 1,056 B
constexpr int kRowStride = kRowMax + 16;           // 1,072 B: 48 modulo 128
constexpr int kTileBytes = kTile * kRowStride;
constexpr int kStageBytes = 2 * kTileBytes;        // K + V: 34,304 B
constexpr int kOffSlots = kStages * kStageBytes;
constexpr int kOffSegs = kOffSlots + kSuffixMaxCtaTokens * 4;
constexpr int kSegSmem = 256;                      // segment descriptors staged in shared memory
constexpr int kOffBar = kOffSegs + kSegSmem * (int)sizeof(DevSuffixItem);
constexpr int kSmemBytes = kOffBar + 8 * 2 * kStages + 16;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
static_assert(kRowStride % 128 == 48, "ldmatrix bank groups");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kShift = 14.f;                     // log2 of the factor that P carries
constexpr float kSumShift = 10.f;                  // and that the row sum does
static_assert(kSuffixMaxCtaTokens <= 4096, "the row sum's range");
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Source of the rows of masked tokens (zero-initialised at module load, never written).
__device__ __align__(128) uint4 g_zero_row[kRowMax / 16];

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void st_record2(float* a, float x, float y, uint64_t pol) {
  asm volatile("st.global.L2::cache_hint.v2.f32 [%0], {%1, %2}, %3;" ::"l"(a), "f"(x), "f"(y), "l"(pol) : "memory");
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One token-CTA `cta` of the suffix work list, for KV-head group `group`, on `smem` (at least
// kSmemBytes, 128-byte aligned), run by kThreads or more threads (the extra warps only take
// part in the set-up barriers).
__device__ __forceinline__ void kv8_suffix_body(const AttnParams& p, const int32_t* __restrict__ cta_begin, int cta,
                                                int group, unsigned char* smem) {
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int seg_begin = cta_begin[cta];
  const int seg_end = cta_begin[cta + 1];
  if (seg_begin >= seg_end) return;
  const int j0 = group * kWarps;                      // first KV head of this CTA's group
  const int nh = min(kWarps, p.n_kv - j0);            // heads in the group
  const uint32_t code_bytes = (uint32_t)nh * kD;
  const uint32_t scale_bytes = (uint32_t)(nh + 3) / 4 * 16;  // the row is padded to 16 bytes
  const uint32_t sbase = smem_u32(smem);
  auto full_bar = [&](int st) { return sbase + kOffBar + 8 * st; };
  auto empty_bar = [&](int st) { return sbase + kOffBar + 8 * (kStages + st); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 16 * kStages);

  // The slot ids of all of this CTA's tokens (its segments back to back) and its segment
  // descriptors go to shared memory once.  The plan keeps a CTA's tokens within
  // kSuffixMaxCtaTokens; descriptors beyond kSegSmem are read from global memory.
  int32_t* sslot = reinterpret_cast<int32_t*>(smem + kOffSlots);
  DevSuffixItem* sseg = reinterpret_cast<DevSuffixItem*>(smem + kOffSegs);
  const int n_seg = seg_end - seg_begin;
  // this thread's descriptor (the plan is not written by the work before this kernel)
  static_assert(kSegSmem <= kThreads, "a descriptor a thread");
  DevSuffixItem mine{};
  if (threadIdx.x < min(n_seg, kSegSmem)) mine = p.sitems[seg_begin + threadIdx.x];
  // the token tables, lengths, pools and q are read only after the previous kernel in the
  // stream completed
  grid_dep_wait();
  grid_dep_launch_dependents();
  // a plan made for more tokens than exist yet: each segment ends at its request's live length
  auto live = [&](DevSuffixItem it) {
    if (p.live_len) it.t1 = max(it.t0, min(it.t1, p.live_len[it.b]));
    return it;
  };
  auto item = [&](int k) { return live(p.sitems[seg_begin + k]); };
  if (threadIdx.x < min(n_seg, kSegSmem)) sseg[threadIdx.x] = live(mine);
  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(full_bar(st), kProducers);
      mbar_init(empty_bar(st), (uint32_t)nh);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();
  auto seg_at = [&](int k) { return k < kSegSmem ? sseg[k] : item(k); };
  int n_tok = 0;
  for (int k = 0; k < n_seg; ++k) {
    const DevSuffixItem seg = seg_at(k);
    const int len = seg.t1 - seg.t0;
    const int32_t* row = p.req_to_slot + (int64_t)seg.b * p.cap + seg.t0;
    for (int i = threadIdx.x; i < len && n_tok + i < kSuffixMaxCtaTokens; i += blockDim.x) sslot[n_tok + i] = row[i];
    n_tok += len;
  }
  if (threadIdx.x == 0 && n_tok > kSuffixMaxCtaTokens) latch_err(p.err, kDevBadRecord);
  __syncthreads();
  if (n_tok > kSuffixMaxCtaTokens) return;

  if (warp >= kWarps) {
    // ---------------- producers: one packed row per lane (lanes 0-1 K, 2-3 V) -------------
    const int part = warp - kWarps;
    if (part >= kProducers) return;
    const bool is_v = (lane & (2 * kRowsEach - 1)) >= kRowsEach;
    const uint8_t* pool = static_cast<const uint8_t*>(is_v ? p.vpool : p.kpool);
    const int64_t code_off = (int64_t)j0 * kD, scale_off = (int64_t)p.n_kv * kD + 4 * j0;
    const bool whole = p.n_kv <= kWarps;  // codes and scales are one run of bytes
    const int r = part * kRowsEach + (lane & (kRowsEach - 1));
    int n = 0;    // tiles issued
    int pos = 0;  // position of the current segment's first token in sslot
    bool stop = false;
    // test hook: token-CTA 0 of group 0 withholds its first tile
    const bool skip0 = p.inject_stall != 0 && cta == 0 && group == 0;
    for (int sg = 0; sg < n_seg && !stop; ++sg) {
      const DevSuffixItem seg = seg_at(sg);
      for (int t = seg.t0; t < seg.t1; t += kTile, ++n) {
        const int st = n % kStages;
        // every lane polls; the warp goes on only if all of them saw the phase complete
        const bool free_ok = n < kStages || mbar_wait_bounded(empty_bar(st), ((n / kStages) - 1) & 1, abort_flag,
                                                              p.err, kDevTimeout, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, free_ok)) {
          stop = true;
          break;
        }
        const uint8_t* row = nullptr;
        if (lane < 2 * kRowsEach && t + r < seg.t1) {
          const int32_t slot = sslot[pos + (t - seg.t0) + r];
          if (slot >= p.n_hot && slot < p.n_slots) row = pool + (int64_t)slot * p.kv8_row;
          else latch_err(p.err, kDevBadSlot);
        }
        if (skip0 && n == 0) continue;
        if (lane == 0) mbar_arrive_expect_tx(full_bar(st), 2u * kRowsEach * (code_bytes + scale_bytes));
        __syncwarp();
        if (lane >= 2 * kRowsEach) continue;
        const uint32_t dst = sbase + st * kStageBytes + (is_v ? kTileBytes : 0) + r * kRowStride;
        const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
        if (whole) {
          bulk_load(dst, row ? row : zero, code_bytes + scale_bytes, full_bar(st));
        } else {
          bulk_load(dst, row ? row + code_off : zero, code_bytes, full_bar(st));
          bulk_load(dst + code_bytes, row ? row + scale_off : zero, scale_bytes, full_bar(st));
        }
      }
      pos += seg.t1 - seg.t0;
    }
    // never leave with a copy in flight: wait for the last issued tiles to land (every producer's
    // part of a tile: they issue the same tiles unless one gave up, and then this gives up as well)
    if (lane == 0) {
      for (int i = max(skip0 ? 1 : 0, n - kStages); i < n; ++i) {
        const uint64_t t_start = globaltimer_ns();
        while (!mbar_try_wait(full_bar(i % kStages), (i / kStages) & 1)) {
          if (globaltimer_ns() - t_start > kWaitLimitNs) {
            atomicCAS(p.err, 0, kDevTimeout);
            break;
          }
        }
      }
    }
    return;
  }
  if (warp >= nh) return;  // no CTA-wide barrier is used below

  // ---------------- consumers: warp `warp` owns KV head j ----------------
  const int j = j0 + warp;
  const int g = p.g;
  const int r = lane >> 2, c = lane & 3;
  const int h0 = 2 * c;  // this thread's two head columns: h0, h0 + 1
  // Q^T as B fragments in the order of the K codes: k-step i takes dims 16 i + 4 c + {0, 1} and {2, 3}
  // of column r (query head j*g + r); the next segment's rows are loaded one segment ahead
  uint32_t qn[16];
  auto load_q = [&](int sg) {
    if (sg < n_seg && r < g) {
      const uint2* qrow = reinterpret_cast<const uint2*>(
          static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)seg_at(sg).b * p.n_q + j * g + r) * kD);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint2 x = qrow[4 * i + c];
        qn[2 * i] = x.x;
        qn[2 * i + 1] = x.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) qn[i] = 0u;
    }
  };
  load_q(0);
  const uint32_t head_off = (uint32_t)warp * kD;
  const uint32_t scale_at = code_bytes + 4 * (uint32_t)warp;
  int tile = 0;  // tiles consumed so far
  for (int sg = 0; sg < n_seg; ++sg) {
    const DevSuffixItem seg = seg_at(sg);
    uint32_t qf[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) qf[i] = qn[i];
    load_q(sg + 1);
    float unit;
    q_to_f16<16>(qf, unit);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half2 x = q_no_inf(*reinterpret_cast<const __half2*>(&qf[i]));
      qf[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    const float f0 = __shfl_sync(0xffffffffu, unit, 8 * c) * p.scale_log2;
    const float f1 = __shfl_sync(0xffffffffu, unit, 8 * c + 4) * p.scale_log2;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[8][4];
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    bool ok = true;
    // V tiles from token t on: one running-max update for both, and their products side by side, so
    // that a warp has two chains to issue from (two warps a scheduler leave most of a chain's
    // latency open)
    auto tiles = [&](auto count, int t) {
      constexpr int V = decltype(count)::value;
      const int mi = lane >> 3;
      const uint32_t frag = head_off + ((lane & 7) + (mi & 1) * 8) * kRowStride + (mi >> 1) * 16;
      uint32_t at[V];  // this lane's ldmatrix row of each tile
      float sa[V], sb[V], la[V], lb[V], s[V][4], s2[V][4];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int st = (tile + v) % kStages;
        const bool landed = mbar_wait_bounded(full_bar(st), ((tile + v) / kStages) & 1, abort_flag, p.err, kDevTimeout,
                                              kWaitLimitNs);
        if (!__all_sync(0xffffffffu, landed)) return false;
        at[v] = sbase + st * kStageBytes + frag;
        // the scales of tokens r and r + 8
        const unsigned char* ksp = smem + st * kStageBytes + r * kRowStride + scale_at;
        sa[v] = *reinterpret_cast<const float*>(ksp);
        sb[v] = *reinterpret_cast<const float*>(ksp + 8 * kRowStride);
        la[v] = *reinterpret_cast<const float*>(ksp + kTileBytes);
        lb[v] = *reinterpret_cast<const float*>(ksp + kTileBytes + 8 * kRowStride);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[v][e] = s2[v][e] = 0.f;
      }
      // S^T = K . Q^T, in two accumulation chains a tile
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[V][4];
#pragma unroll
        for (int v = 0; v < V; ++v) ldsm_x4(at[v] + i * 32, w[v][0], w[v][1], w[v][2], w[v][3]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x4(w[v][0], a0, a2);
          e4m3x4_to_f16x4(w[v][1], a1, a3);
          mma_f16_16816(s[v], a0, a1, a2, a3, qf[4 * i], qf[4 * i + 1]);
          e4m3x4_to_f16x4(w[v][2], a0, a2);
          e4m3x4_to_f16x4(w[v][3], a1, a3);
          mma_f16_16816(s2[v], a0, a1, a2, a3, qf[4 * i + 2], qf[4 * i + 3]);
        }
      }
      const int rem = seg.t1 - t;  // valid tokens from the first tile on
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // (the zero row of a token that does not count has scale 0)
        const bool in_a = v * kTile + r < rem && la[v] != 0.f, in_b = v * kTile + r + 8 < rem && lb[v] != 0.f;
        la[v] = lg2_approx(la[v]);
        lb[v] = lg2_approx(lb[v]);
        s[v][0] = in_a ? (s[v][0] + s2[v][0]) * (f0 * sa[v]) : -INFINITY;
        s[v][1] = in_a ? (s[v][1] + s2[v][1]) * (f1 * sa[v]) : -INFINITY;
        s[v][2] = in_b ? (s[v][2] + s2[v][2]) * (f0 * sb[v]) : -INFINITY;
        s[v][3] = in_b ? (s[v][3] + s2[v][3]) * (f1 * sb[v]) : -INFINITY;
        mx0 = max3f(mx0, s[v][0] + la[v], s[v][2] + lb[v]);
        mx1 = max3f(mx1, s[v][1] + la[v], s[v][3] + lb[v]);
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
      }
      const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
      const float mu0 = (mn0 == -INFINITY ? 0.f : mn0), mu1 = (mn1 == -INFINITY ? 0.f : mn1);
      if (__any_sync(0xffffffffu, mn0 != m0 || mn1 != m1)) {
        // (a step of m may pass 2^126, by which O is 0, but not the row sum)
        const float half0 = ex2_approx(0.5f * (m0 - mu0)), half1 = ex2_approx(0.5f * (m1 - mu1));
        const float al0 = half0 * half0, al1 = half1 * half1;
        l0 = l0 * half0 * half0;
        l1 = l1 * half1 * half1;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          o[mt][0] *= al0;
          o[mt][2] *= al0;
          o[mt][1] *= al1;
          o[mt][3] *= al1;
        }
        m0 = mn0;
        m1 = mn1;
      }
      const float hm0 = 0.5f * (kSumShift - mu0), hm1 = 0.5f * (kSumShift - mu1);
      uint32_t b0[V], b1[V];  // P^T in B-operand layout
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float p0 = ex2_approx(s[v][0] + la[v] - mu0 + kShift), p1 = ex2_approx(s[v][1] + la[v] - mu1 + kShift);
        const float p2 = ex2_approx(s[v][2] + lb[v] - mu0 + kShift), p3 = ex2_approx(s[v][3] + lb[v] - mu1 + kShift);
        // the row sum's weights as squares of 2^((y - m + kSumShift) / 2), which stays above ex2's smallest result
        const float e0 = ex2_approx(fmaf(0.5f, s[v][0], hm0)), e1 = ex2_approx(fmaf(0.5f, s[v][1], hm1));
        const float e2 = ex2_approx(fmaf(0.5f, s[v][2], hm0)), e3 = ex2_approx(fmaf(0.5f, s[v][3], hm1));
        l0 = fmaf(e2, e2, fmaf(e0, e0, l0));
        l1 = fmaf(e3, e3, fmaf(e1, e1, l1));
        b0[v] = movmatrix_t(pack_f16(p0, p1));
        b1[v] = movmatrix_t(pack_f16(p2, p3));
      }
      // O^T += V^T . P^T: m-tile mt holds dims 16 mt + 2 r (row r) and 16 mt + 2 r + 1 (row r + 8)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[V][4];
#pragma unroll
        for (int v = 0; v < V; ++v) ldsm_x4_t(at[v] + kTileBytes + i * 32, w[v][0], w[v][1], w[v][2], w[v][3]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x4(__byte_perm(w[v][0], 0, 0x3120), a0, a1);
          e4m3x4_to_f16x4(__byte_perm(w[v][1], 0, 0x3120), a2, a3);
          mma_f16_16816(o[2 * i], a0, a1, a2, a3, b0[v], b1[v]);
          e4m3x4_to_f16x4(__byte_perm(w[v][2], 0, 0x3120), a0, a1);
          e4m3x4_to_f16x4(__byte_perm(w[v][3], 0, 0x3120), a2, a3);
          mma_f16_16816(o[2 * i + 1], a0, a1, a2, a3, b0[v], b1[v]);
        }
      }
      // this warp is done reading the stages
      __syncwarp();
      if (lane == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) mbar_arrive(empty_bar((tile + v) % kStages));
      tile += V;
      return true;
    };
    for (int t = seg.t0; ok && t < seg.t1;) {
      if (seg.t1 - t > kTile) {
        ok = tiles(std::integral_constant<int, 2>{}, t);
        t += 2 * kTile;
      } else {
        ok = tiles(std::integral_constant<int, 1>{}, t);
        t += kTile;
      }
    }
    if (!ok) break;

    // finish the segment: full column sums, normalise, write the record
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    const int32_t rec = seg.rec;
    if (rec < 0 || rec >= p.n_records) {
      if (lane == 0) latch_err(p.err, kDevBadRecord);
      continue;
    }
    constexpr float kUnit = 1.f / (float)(1 << (int)(kShift - kSumShift));
    const float inv0 = l0 == 0.f ? 0.f : kUnit / l0;
    const float inv1 = l1 == 0.f ? 0.f : kUnit / l1;
    const int hq0 = j * g + h0;
    float* dst0 = p.rec_o + ((int64_t)rec * p.n_q + hq0) * kD + 2 * r;
    const bool w0 = h0 < g, w1 = h0 + 1 < g;
    const uint64_t keep = l2_policy_keep();
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      if (w0) st_record2(dst0 + mt * 16, o[mt][0] * inv0, o[mt][2] * inv0, keep);
      if (w1) st_record2(dst0 + kD + mt * 16, o[mt][1] * inv1, o[mt][3] * inv1, keep);
    }
    if (lane < 4) {
      float* ldst = p.rec_lse + (int64_t)rec * p.n_q + hq0;
      if (w0) st_record(ldst, kv8_record_lse(l0, (m0 - kSumShift + log2f(l0)) * kLn2), keep);
      if (w1) st_record(ldst + 1, kv8_record_lse(l1, (m1 - kSumShift + log2f(l1)) * kLn2), keep);
    }
  }
}

}  // namespace
}  // namespace k8s
}  // namespace granikv
