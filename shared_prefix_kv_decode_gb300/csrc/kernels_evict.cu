// kernels_evict.cu -- eviction of COLD tokens by accumulated attention weight: the weight each
// COLD token received in a step, and the selection and removal of the lightest tokens of a row.
//
// The token-level COLD pool (GraniKV, arXiv:2608.15584, "3 GraniKV": page size 1) lets single
// tokens leave a request: their table entries close up and their slots go back to the free ring.
#include "kv4_util.cuh"
#include "kv8_util.cuh"
#include "launch_util.cuh"
#include "mma_util.cuh"
#include "tc_util.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

namespace granikv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void latch(int32_t* err, int32_t code) { atomicCAS(err, 0, code); }

// ---- weighing ---------------------------------------------------------------------------------
// The rows' token counts travel as a kernel parameter, with the number of chunks before each row,
// so the grid has one CTA for each chunk of tokens that a row may hold and none for empty ones.
template <int N>
struct WeighRows {
  int32_t first[N + 1];  // chunks of the rows before
  int32_t len[N];
  int32_t n, b0;         // rows here; row r is request b0 + r
  int32_t tokens;        // of a chunk
};

// Chunk -> (row of the parameter, first token); a chunk that begins past the row's live tokens has n <= 0.
template <int N>
__device__ __forceinline__ void chunk_of(const WeighRows<N>& rows, const int32_t* live_len, int32_t chunk, int tokens,
                                         int32_t& b, int32_t& t0, int32_t& n) {
  int lo = 0, hi = rows.n;  // the last row with first <= chunk
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (rows.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  b = rows.b0 + lo;
  t0 = (chunk - rows.first[lo]) * tokens;
  n = min(min(live_len[b], rows.len[lo]) - t0, tokens);
}

// Any shape:
// A CTA takes 32 tokens of a request: KV head by KV head the tokens' K rows go to shared memory in
// fp32, each warp takes every eighth query head of the group, its lanes the tokens.  A lane sums
// its heads in order, the warps' sums are added in warp order.
constexpr int kTok = 32;

template <typename T, int BITS, int N>
__global__ void __launch_bounds__(256) weigh_generic_kernel(WeighParams p, const __grid_constant__ WeighRows<N> rows) {
  extern __shared__ float sm[];
  float* sK = sm;                       // [kTok][d + 1]
  float* sSum = sK + kTok * (p.d + 1);  // [8][kTok]
  __shared__ int32_t s_slot[kTok];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t d = p.d;
  int32_t b, t0, n;
  chunk_of(rows, p.live_len, blockIdx.x, kTok, b, t0, n);
  if (n > 0) {
    if (threadIdx.x < kTok) {
      int32_t slot = -1;
      if (threadIdx.x < n) {
        slot = p.req_to_slot[(int64_t)b * p.cap + t0 + threadIdx.x];
        if (slot < p.n_hot || slot >= p.n_slots) {
          latch(p.err, kDevBadSlot);
          slot = -1;
        }
      }
      s_slot[threadIdx.x] = slot;
    }
    float sum = 0.f;
    for (int32_t j = 0; j < p.n_kv; ++j) {
      __syncthreads();
      for (int i = threadIdx.x; i < kTok * (d / 4); i += blockDim.x) {
        const int tok = i / (d / 4), c = i % (d / 4) * 4;
        const int32_t slot = s_slot[tok];
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (slot >= 0) {
          if constexpr (BITS == 4) {
            const uint8_t* row = (const uint8_t*)p.kpool + (int64_t)slot * p.packed_row;
            uint32_t y[4];
            e2m1x8_to_f16x8(*reinterpret_cast<const uint16_t*>(row + (int64_t)j * (d / 2) + c / 2), y);
            const uint32_t scale = kv4_scale2(row[kv4_scales_at(p.n_kv, d) + (int64_t)j * (d / kKv4Group) + c / kKv4Group]);
            const float unit = kv4_unit(row[kv4_units_at(p.n_kv, d) + j]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t h = f16x2_mul(y[u], scale);
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
              x[2 * u] = f.x * unit;
              x[2 * u + 1] = f.y * unit;
            }
          } else if constexpr (BITS == 8) {
            const uint8_t* row = (const uint8_t*)p.kpool + (int64_t)slot * p.packed_row;
            e4m3x4_to_f32x4(*reinterpret_cast<const uint32_t*>(row + (int64_t)j * d + c), x);
            const float s = *reinterpret_cast<const float*>(row + (int64_t)p.n_kv * d + 4 * j);
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] *= s;
          } else {
            const T* row = (const T*)p.kpool + ((int64_t)slot * p.n_kv + j) * d + c;
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = (float)row[u];
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) sK[tok * (d + 1) + c + u] = x[u];
      }
      __syncthreads();
      for (int32_t h = j * p.g + warp; h < (j + 1) * p.g; h += 8) {
        const T* q = (const T*)p.q + ((int64_t)b * p.n_q + h) * d;
        float s = 0.f;
        for (int i = 0; i < d; ++i) s += (float)q[i] * sK[lane * (d + 1) + i];
        const float lse = p.lse[(int64_t)b * p.n_q + h];
        if (lse != -INFINITY) sum += exp2f(s * p.scale_log2 - lse * kLog2e);
      }
    }
    sSum[warp * kTok + lane] = sum;
    __syncthreads();
    if (warp == 0 && lane < n) {
      float w = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) w += sSum[i * kTok + lane];
      if (s_slot[lane] < 0) w = 0.f;
      float* dst = p.weight + (int64_t)b * p.cap + t0 + lane;
      *dst = p.keep != 0.f ? p.keep * *dst + w : w;
    }
  }
}

// bf16 q, head_dim 64 or 128: one unit is 16 tokens of one KV head, on warp-level tensor cores,
//     S^T[16 tok x 8 heads] = K[16 tok x d] . Q^T[d x 8]     (d / 16 mma.m16n8k16 for each 8 query heads)
// The sum over d may be taken in any order, so the lanes of a row take 16-byte pieces of it (whole
// sectors) that serve as the A operand as they are, and Q^T is loaded in the same order.  Every lane
// copies its own pieces into shared memory some units ahead (cp.async) and reads them back when their
// turn comes: K is read once, no lane waits for another, and the bytes in flight are not bound by
// registers.
// Of a 16-bit row lane c = lane % 4 holds dims 32 i + 8 c + 0..7 of load i; k-step 2 i + u takes its dims
// 4 u + {0, 1} and 4 u + {2, 3}.  Of a packed 8-bit row it holds dims 64 i + 16 c + 0..15; k-step
// 4 i + u takes dims 4 u + {0, 1} and 4 u + {2, 3}, converted to fp16 (exact); the row's scale
// multiplies the scores, and q is brought into fp16's range by a power of two per query head
// (exact but for elements 2^-31 below the row's largest).  Of a packed 4-bit row it holds dims D / 4 c and on in one
// piece of 16 bytes (d 64: 8), with the four bytes that its 16-dim scales are among and the four that the row's unit is; the
// piece's word w takes k-steps 2 w and 2 w + 1 (dims 8 w + 4 u + {0, 1} and {2, 3}), converted to fp16 times scale (exact).
// The units' sums go to shared memory and are added in KV-head order: the result has one order.
// A CTA takes a chunk of 64 to 512 tokens, sized so that all chunks run at once: with 256 tokens a CTA the
// 877 chunks of 224K tokens made 1.44 waves of 608 CTAs (49.5 us against 47.8), and a CTA's start (length, slots, q, first rows: four
// trips to memory one after the other) costs about 4 us each time.
constexpr int kChunkMin = 64, kChunkMax = 512;
constexpr int kMaxHeads = 64;  // KV heads: the sums of a chunk of kChunkMin tokens take 16 KB

// Two units in shared memory a warp, and as many warps as registers allow: 224K tokens of packed rows
// 47.8 us (5.0 TB/s of its 237 MB), 30K of 16-bit rows 13.9 us.  Fewer CTAs with deeper rings were
// slower (224K tokens, on an earlier form: 50.8 us with four CTAs an SM, 52.9 with three and three units,
// 58.9 with two and four), and so were units ahead in registers (58.8).
template <int BITS, int D>
struct WeighUnit {
  static constexpr bool KV8 = BITS == 8;
  static constexpr int kPieces = BITS == 4 ? 1 : KV8 ? D / 64 : D / 32;  // 16-byte pieces of a row a lane
  // rows lane / 4 and lane / 4 + 8, and their scales (4 bits: scales and units)
  static constexpr int kBytes = 2 * kPieces * 512 + (BITS == 4 ? 512 : KV8 ? 256 : 0);
  static constexpr int kDepth = 2;
  static constexpr int kRing = 8 * kDepth * kBytes;
  static constexpr int kBlocks = BITS ? 4 : 3;
  // shared memory for a chunk's sums that leaves room for kBlocks CTAs an SM
  static constexpr int kSums = BITS ? 16 * 1024 : 8 * 1024;
};

template <int BITS, int D, int N>
__global__ void __launch_bounds__(256, WeighUnit<BITS, D>::kBlocks) weigh_mma_kernel(WeighParams p, const __grid_constant__ WeighRows<N> rows) {
  using Unit = WeighUnit<BITS, D>;
  constexpr bool KV8 = BITS == 8, KV4 = BITS == 4;
  extern __shared__ __align__(16) unsigned char s_ring[];  // [8 warps][kDepth] units, then the sums
  float* s_sum = reinterpret_cast<float*>(s_ring + Unit::kRing);  // [n_kv][rows.tokens]
  __shared__ int32_t s_slot[kChunkMax];
  const int kChunk = rows.tokens;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  int32_t b, t0, n;
  chunk_of(rows, p.live_len, blockIdx.x, kChunk, b, t0, n);
  if (n <= 0) return;
  // every place up to the last unit's end has a slot or -1
  for (int32_t i = tid; i < (n + 15) / 16 * 16; i += 256) {
    int32_t slot = -1;
    if (i < n) {
      slot = p.req_to_slot[(int64_t)b * p.cap + t0 + i];
      if (slot < p.n_hot || slot >= p.n_slots) {
        latch(p.err, kDevBadSlot);
        slot = -1;
      }
    }
    s_slot[i] = slot;
  }
  const uint32_t ring = smem_u32(s_ring) + warp * (Unit::kDepth * Unit::kBytes);
  // a warp takes every eighth unit; unit u is KV head j = u % n_kv of the tokens from tile = u / n_kv * 16 on
  struct Place {
    int32_t j, tile;
  };
  const int32_t step_j = 8 % p.n_kv, step_tile = 8 / p.n_kv * 16;
  auto next = [&](Place& x) {
    x.j += step_j;
    x.tile += step_tile;
    if (x.j >= p.n_kv) {
      x.j -= p.n_kv;
      x.tile += 16;
    }
  };
  const int32_t row_bytes = BITS ? (int32_t)p.packed_row : p.n_kv * D * 2;
  // this lane's pieces of the rows of a unit into stage st (zeros for a slot that does not count)
  auto load_unit = [&](const Place& x, int st) {
    if (x.tile < n) {
      const int32_t j = x.j, tile = x.tile;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t slot = s_slot[tile + r + 8 * h];
        const uint8_t* row = (const uint8_t*)p.kpool + (int64_t)max(slot, 0) * row_bytes;
        const uint32_t dst = ring + st * Unit::kBytes + (h * Unit::kPieces * 32 + lane) * 16;
        if constexpr (KV4) {
          const uint8_t* src = row + j * (D / 2) + c * (D / 8);
          if constexpr (D == 128) cp_async16(dst, src, slot < 0 ? 0 : 16);
          else cp_async8(dst, src, slot < 0 ? 0 : 8);
          const uint32_t meta = ring + st * Unit::kBytes + 1024 + (h * 32 + lane) * 8;
          cp_async4(meta, row + kv4_scales_at(p.n_kv, D) + j * (D / kKv4Group) + (D == 128 ? c / 2 * 4 : 0), slot < 0 ? 0 : 4);
          cp_async4(meta + 4, row + kv4_units_at(p.n_kv, D) + j / 4 * 4, slot < 0 ? 0 : 4);
          continue;
        }
        const uint4* src = reinterpret_cast<const uint4*>(row + j * (KV8 ? D : 2 * D)) + c;
#pragma unroll
        for (int i = 0; i < Unit::kPieces; ++i) cp_async16(dst + i * 512, src + 4 * i, slot < 0 ? 0 : 16);
        if constexpr (KV8)
          cp_async4(ring + st * Unit::kBytes + 2 * Unit::kPieces * 512 + (h * 32 + lane) * 4,
                    row + p.n_kv * D + 4 * j, slot < 0 ? 0 : 4);
      }
    }
    cp_async_commit();
  };
  constexpr int kSteps = D / 16;
  uint32_t qf[kSteps][2];
  float c0 = 0.f, c1 = 0.f, e0 = -INFINITY, e1 = -INFINITY;  // heads 2 c and 2 c + 1: score factor, -lse in base 2
  int32_t have = -1;                                          // the query heads whose q is in qf
  // q of query heads h0 .. (at most 8, below h_end): column lane / 4
  auto load_q = [&](int32_t h0, int32_t h_end) {
    have = h0;
    const bool mine = h0 + r < h_end;
    const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.q + ((int64_t)b * p.n_q + h0 + r) * D);
    float unit = 1.f;  // what one step of the scaled q stands for
    if constexpr (KV4) {
      uint32_t w[D / 32][4];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = mine ? __ldg(src + (D / 32) * c + i) : make_uint4(0u, 0u, 0u, 0u);
        w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
      }
      q_to_f16<D / 8>(&w[0][0], unit);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) qf[2 * i + u][0] = w[i][2 * u], qf[2 * i + u][1] = w[i][2 * u + 1];
    } else if constexpr (!KV8) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = mine ? __ldg(src + 4 * i + c) : make_uint4(0u, 0u, 0u, 0u);
        qf[2 * i][0] = x.x, qf[2 * i][1] = x.y, qf[2 * i + 1][0] = x.z, qf[2 * i + 1][1] = x.w;
      }
    } else {
      uint32_t w[D / 64][8];
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint4 x = mine ? __ldg(src + 8 * i + 2 * c + u) : make_uint4(0u, 0u, 0u, 0u);
          w[i][4 * u] = x.x, w[i][4 * u + 1] = x.y, w[i][4 * u + 2] = x.z, w[i][4 * u + 3] = x.w;
        }
      q_to_f16<D / 8>(&w[0][0], unit);
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) qf[4 * i + u][0] = w[i][2 * u], qf[4 * i + u][1] = w[i][2 * u + 1];
    }
    const float lse = mine ? p.lse[(int64_t)b * p.n_q + h0 + r] : -INFINITY;
    const float factor = unit * p.scale_log2, minus = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    c0 = __shfl_sync(0xffffffffu, factor, 8 * c);
    c1 = __shfl_sync(0xffffffffu, factor, 8 * c + 4);
    e0 = __shfl_sync(0xffffffffu, minus, 8 * c);
    e1 = __shfl_sync(0xffffffffu, minus, 8 * c + 4);
  };
  auto unit = [&](const Place& x, int st) {
    const int32_t j = x.j, tile = x.tile;
    const unsigned char* mine = s_ring + warp * (Unit::kDepth * Unit::kBytes) + st * Unit::kBytes;
    const uint4* ka = reinterpret_cast<const uint4*>(mine) + lane;
    float sa = 1.f, sb = 1.f;
    if constexpr (KV8) {
      const float* sc = reinterpret_cast<const float*>(mine + 2 * Unit::kPieces * 512);
      sa = sc[lane];
      sb = sc[32 + lane];
    }
    uint2 ma, mb;  // 4 bits: the rows' scales and units
    if constexpr (KV4) {
      const uint2* meta = reinterpret_cast<const uint2*>(mine + 1024) + lane;
      ma = meta[0];
      mb = meta[32];
      sa = kv4_unit(ma.y >> (j % 4 * 8) & 255u);
      sb = kv4_unit(mb.y >> (j % 4 * 8) & 255u);
      // this lane's one or two scales in the low bytes
      ma.x >>= D == 128 ? c % 2 * 16 : c * 8;
      mb.x >>= D == 128 ? c % 2 * 16 : c * 8;
    }
    float w0 = 0.f, w1 = 0.f;
    for (int32_t h0 = j * p.g; h0 < (j + 1) * p.g; h0 += 8) {
      if (have != h0) load_q(h0, (j + 1) * p.g);
      float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};  // two accumulation chains
#pragma unroll
      for (int i = 0; i < Unit::kPieces; ++i) {
        const uint4 x = ka[32 * i], y = ka[32 * (Unit::kPieces + i)];
        const uint32_t a[4] = {x.x, x.y, x.z, x.w}, z[4] = {y.x, y.y, y.z, y.w};
        if constexpr (KV4) {
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            const uint32_t fa = kv4_scale2(ma.x >> (w / 2 * 8) & 255u), fb = kv4_scale2(mb.x >> (w / 2 * 8) & 255u);
            uint32_t ka4[4], kb4[4];
            e2m1x8_to_f16x8(a[w], ka4);
            e2m1x8_to_f16x8(z[w], kb4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ka4[k] = f16x2_mul(ka4[k], fa);
              kb4[k] = f16x2_mul(kb4[k], fb);
            }
            mma_f16_16816(s, ka4[0], kb4[0], ka4[1], kb4[1], qf[2 * w][0], qf[2 * w][1]);
            mma_f16_16816(s2, ka4[2], kb4[2], ka4[3], kb4[3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
          }
        } else if constexpr (KV8) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a2, b0, b2;
            e4m3x4_to_f16x4(a[w], a0, a2);
            e4m3x4_to_f16x4(z[w], b0, b2);
            mma_f16_16816(w & 1 ? s2 : s, a0, b0, a2, b2, qf[4 * i + w][0], qf[4 * i + w][1]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 2; ++w)
            mma_bf16_16816(w & 1 ? s2 : s, a[2 * w], z[2 * w], a[2 * w + 1], z[2 * w + 1], qf[2 * i + w][0], qf[2 * i + w][1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += s2[e];
      // a head without weight (lse -inf, or past the group) adds 2^-inf = 0, whatever its score
      const float a0 = score_factor<BITS>(c0, sa), a1 = score_factor<BITS>(c1, sa);
      const float b0 = score_factor<BITS>(c0, sb), b1 = score_factor<BITS>(c1, sb);
      w0 += (e0 == -INFINITY ? 0.f : exp2f(s[0] * a0 + e0)) + (e1 == -INFINITY ? 0.f : exp2f(s[1] * a1 + e1));
      w1 += (e0 == -INFINITY ? 0.f : exp2f(s[2] * b0 + e0)) + (e1 == -INFINITY ? 0.f : exp2f(s[3] * b1 + e1));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      w0 += __shfl_xor_sync(0xffffffffu, w0, o);
      w1 += __shfl_xor_sync(0xffffffffu, w1, o);
    }
    if (c == 0) {
      s_sum[j * kChunk + tile + r] = w0;
      s_sum[j * kChunk + tile + r + 8] = w1;
    }
  };
  Place now{warp % p.n_kv, warp / p.n_kv * 16}, ahead = now;
  // q of the warp's first units' heads is on its way with the slots
  if (now.tile < n) load_q(now.j * p.g, (now.j + 1) * p.g);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < Unit::kDepth - 1; ++i) {
    load_unit(ahead, i);
    next(ahead);
  }
  int st = 0;
  for (; now.tile < n; next(now)) {
    load_unit(ahead, (st + Unit::kDepth - 1) % Unit::kDepth);
    next(ahead);
    cp_async_wait<Unit::kDepth - 1>();
    unit(now, st);
    st = (st + 1) % Unit::kDepth;
  }
  __syncthreads();
  for (int32_t i = tid; i < n; i += 256) {
    float w = 0.f;
    for (int32_t j = 0; j < p.n_kv; ++j) w += s_sum[j * kChunk + i];
    if (s_slot[i] < 0) w = 0.f;
    float* dst = p.weight + (int64_t)b * p.cap + t0 + i;
    *dst = p.keep != 0.f ? p.keep * *dst + w : w;
  }
}

// ---- eviction ---------------------------------------------------------------------------------
// Ordering key of a weight: unsigned order = float order, -0 equal to 0, NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

template <int N>
struct EvictRows {
  EvictRow r[N];
};

constexpr int kEvictThreads = 1024;

// Sum of v over the threads before this one, and over all (block of kEvictThreads); s: 33 words.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* s, uint32_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = upto;
  __syncthreads();
  uint32_t x = s[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  total = __shfl_sync(0xffffffffu, x, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, x, warp ? warp - 1 : 0);
  return (warp ? before : 0u) + upto - v;
}

// Rows of up to 8 * 1024 * PER tokens: a cluster of CTAs per row, each with a slice of it in registers
// (PER tokens a thread: slot and weight).  The whole row is read once and written once; what it costs
// is latency.  A radix selection in three digits (11, 11 and 10 bits: the first one, sign, exponent
// and two mantissa bits, already spreads softmax weights over many bins) finds the key of the
// n_evict-th lightest candidate: each CTA counts its slice in shared memory, and after a cluster
// barrier adds up the others' counts.  Then every CTA knows how many leave before its slice, and
// places each token by ballots.  All of a row's tokens are in registers before the barrier that
// precedes the first write, so the row is closed up in place.  Counts are whole numbers: the result
// does not depend on the order of the atomics.
template <int PER, int N>
__global__ void __launch_bounds__(kEvictThreads, 1)
    evict_cluster_kernel(const __grid_constant__ EvictRows<N> rows, int32_t row0, int32_t keep_last, int32_t cs,
                         int32_t* __restrict__ req_to_slot, int32_t* __restrict__ suffix_len,
                         float* __restrict__ weight, int32_t cap, int32_t* __restrict__ slots_out) {
  namespace cg = cooperative_groups;
  constexpr int kBins = 2048;
  __shared__ uint32_t s_hist[3][kBins];
  __shared__ uint32_t s_scan[33];
  __shared__ uint32_t s_cnt[PER * 32];  // tokens of (k, warp): below | equal << 16
  __shared__ uint32_t s_total, s_prefix;
  __shared__ int32_t s_left;
  const EvictRow r = rows.r[blockIdx.x / cs];
  const int32_t b = row0 + blockIdx.x / cs, rank = blockIdx.x % cs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0 && rank == 0 && suffix_len) suffix_len[b] = r.len - r.n_evict;
  if (r.n_evict <= 0) return;  // the whole cluster
  cg::cluster_group cluster = cg::this_cluster();
  int32_t* tab = req_to_slot + (int64_t)b * cap;
  float* wt = weight + (int64_t)b * cap;
  const int32_t slice = (r.len + cs - 1) / cs;
  const int32_t p0 = rank * slice + tid, p1 = min(r.len, (rank + 1) * slice);  // slice <= PER * 1024
  const int32_t c0 = r.first, c1 = r.len - keep_last;                          // candidates
  float w[PER];
  int32_t slot[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int32_t p = p0 + k * kEvictThreads;
    const bool in = p < p1;
    w[k] = in ? wt[p] : 0.f;
    slot[k] = in ? tab[p] : 0;
  }
  auto candidate = [&](int k) {
    const int32_t p = p0 + k * kEvictThreads;
    return p < p1 && p >= c0 && p < c1;
  };
  for (int i = tid; i < 3 * kBins; i += kEvictThreads) (&s_hist[0][0])[i] = 0u;
  __syncthreads();
  uint32_t prefix = 0;
  int32_t left = r.n_evict;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const uint32_t key = weight_key(w[k]);
      const bool match = pass == 0 || (key >> (sh + bits)) == (prefix >> (sh + bits));
      if (candidate(k) && match) atomicAdd(&s_hist[pass][(key >> sh) & ((1u << bits) - 1u)], 1u);
    }
    cluster.sync();  // (for one CTA, a block barrier)
    uint32_t a = 0, c = 0;  // the row's counts of bins 2 tid and 2 tid + 1
    for (int q = 0; q < cs; ++q) {
      const uint2 x = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&s_hist[pass][2 * tid], q));
      a += x.x;
      c += x.y;
    }
    uint32_t total;
    const int32_t before = (int32_t)block_exclusive(a + c, s_scan, total);
    if (before < left && left <= before + (int32_t)(a + c)) {
      const bool second = left > before + (int32_t)a;
      s_prefix = prefix | ((uint32_t)(2 * tid + (second ? 1 : 0)) << sh);
      s_left = left - before - (second ? (int32_t)a : 0);
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // leavers: keys below `prefix`, and the first `left` with that key
  uint32_t below[PER], equal[PER];  // ballots of this warp's tokens
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const uint32_t key = weight_key(w[k]);
    below[k] = __ballot_sync(0xffffffffu, candidate(k) && key < prefix);
    equal[k] = __ballot_sync(0xffffffffu, candidate(k) && key == prefix);
    if (lane == 0) s_cnt[k * 32 + warp] = (uint32_t)__popc(below[k]) | ((uint32_t)__popc(equal[k]) << 16);
  }
  __syncthreads();
  {
    uint32_t total;
    const uint32_t v = tid < PER * 32 ? s_cnt[tid] : 0u;
    const uint32_t ex = block_exclusive(v, s_scan, total);
    if (tid < PER * 32) s_cnt[tid] = ex;
    if (tid == 0) s_total = total;
  }
  cluster.sync();  // every slice is in registers and counted
  int32_t base_b = 0, base_e = 0;
  for (int q = 0; q < rank; ++q) {
    const uint32_t x = *cluster.map_shared_rank(&s_total, q);
    base_b += (int32_t)(x & 0xffffu);
    base_e += (int32_t)(x >> 16);
  }
  const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int32_t p = p0 + k * kEvictThreads;
    if (p >= p1) continue;
    const uint32_t ex = s_cnt[k * 32 + warp];
    const int32_t nb = base_b + (int32_t)(ex & 0xffffu) + __popc(below[k] & lower);
    const int32_t ne = base_e + (int32_t)(ex >> 16) + __popc(equal[k] & lower);
    const int32_t gone = nb + min(ne, left);  // leavers before this place
    const bool leaves = ((below[k] >> lane) & 1u) || (((equal[k] >> lane) & 1u) && ne < left);
    if (leaves) {
      slots_out[r.out + gone] = slot[k];
    } else if (gone > 0) {
      tab[p - gone] = slot[k];
      wt[p - gone] = w[k];
    }
    if (p >= r.len - r.n_evict) wt[p] = 0.f;
  }
  cluster.sync();  // no CTA leaves while another reads its counts
}

// Longer rows.  One CTA per row: a radix selection (four passes of 8 bits) finds the key of the n_evict-th
// lightest candidate; one pass in place then closes the row up, tile by tile.  A tile's places are
// read before any is written, and tokens only move towards the row's start, so no place is
// overwritten before it is read.
template <int N>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictRows<N> rows, int32_t row0,
                                                              int32_t keep_last, int32_t* __restrict__ req_to_slot,
                                                              int32_t* __restrict__ suffix_len,
                                                              float* __restrict__ weight, int32_t cap,
                                                              int32_t* __restrict__ slots_out) {
  __shared__ int32_t s_hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int32_t s_left;
  __shared__ uint32_t s_scan[32];
  const EvictRow r = rows.r[blockIdx.x];
  const int32_t b = row0 + blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0 && suffix_len) suffix_len[b] = r.len - r.n_evict;
  if (r.n_evict <= 0) return;
  int32_t* tab = req_to_slot + (int64_t)b * cap;
  float* wt = weight + (int64_t)b * cap;
  const int32_t c0 = r.first, c1 = r.len - keep_last;  // candidates
  // the n_evict-th smallest key: after the pass of bits [sh, sh + 8) the key's bits above sh are
  // `prefix`, and `left` of the candidates with those bits are still to leave
  uint32_t prefix = 0;
  int32_t left = r.n_evict;
  for (int sh = 24; sh >= 0; sh -= 8) {
    for (int i = tid; i < 256; i += kEvictThreads) s_hist[i] = 0;
    __syncthreads();
    for (int32_t t = c0 + tid; t < c1; t += kEvictThreads) {
      const uint32_t key = weight_key(wt[t]);
      if (sh == 24 || (key >> (sh + 8)) == (prefix >> (sh + 8))) atomicAdd(&s_hist[(key >> sh) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {  // lane: bins 8 * lane ..
      int32_t c[8], mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += c[i] = s_hist[lane * 8 + i];
      int32_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      int32_t before = upto - mine;
      if (before < left && left <= upto) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < left && left <= before + c[i]) {
            s_prefix = prefix | ((uint32_t)(lane * 8 + i) << sh);
            s_left = left - before;
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // leavers: keys below `prefix`, and the first `left` with that key
  int32_t below = 0, equal = 0;  // of the places before this tile
  for (int32_t t0 = c0; t0 < r.len; t0 += kEvictThreads) {
    const int32_t t = t0 + tid;
    int32_t slot = 0;
    float w = 0.f;
    uint32_t flag = 0;  // 1: below, 1 << 16: equal
    if (t < r.len) {
      slot = tab[t];
      w = wt[t];
      if (t < c1) {
        const uint32_t key = weight_key(w);
        flag = key < prefix ? 1u : key == prefix ? 0x10000u : 0u;
      }
    }
    uint32_t upto = flag;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    uint32_t base = 0, total = 0;
    {
      uint32_t v = s_scan[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      total = __shfl_sync(0xffffffffu, v, 31);
      base = warp ? __shfl_sync(0xffffffffu, v, warp - 1) : 0u;
    }
    const uint32_t ex = base + upto - flag;
    const int32_t nb = below + (int32_t)(ex & 0xffffu), ne = equal + (int32_t)(ex >> 16);
    const int32_t gone = nb + min(ne, left);  // leavers before this place
    if (t < r.len) {
      const bool leaves = (flag & 1u) || ((flag >> 16) && ne < left);
      if (leaves) {
        slots_out[r.out + gone] = slot;
      } else if (gone > 0) {
        tab[t - gone] = slot;
        wt[t - gone] = w;
      }
    }
    below += (int32_t)(total & 0xffffu);
    equal += (int32_t)(total >> 16);
    __syncthreads();  // s_scan is read; the writes are done before the next tile's
  }
  for (int32_t t = r.len - r.n_evict + tid; t < r.len; t += kEvictThreads) wt[t] = 0.f;
}

template <int PER, int N>
cudaError_t evict_cluster(const EvictRows<N>& a, int32_t row0, int32_t n, int32_t cs, int32_t keep_last,
                          int32_t* req_to_slot, int32_t* suffix_len, float* weight, int32_t cap, int32_t* slots_out,
                          cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(n * cs));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_cluster_kernel<PER, N>, a, row0, keep_last, cs, req_to_slot, suffix_len, weight,
                            cap, slots_out);
}

template <int N>
cudaError_t evict_n(const EvictRow* rows, int32_t row0, int32_t n, int32_t num_sms, int32_t keep_last,
                    int32_t* req_to_slot, int32_t* suffix_len, float* weight, int32_t cap, int32_t* slots_out, cudaStream_t s) {
  EvictRows<N> a{};
  int32_t longest = 1;
  for (int32_t i = 0; i < n; ++i) {
    a.r[i] = rows[i];
    if (rows[i].n_evict > 0 && rows[i].len > longest) longest = rows[i].len;
  }
  // the fewest CTAs (a power of two, 8 at most) whose threads hold the longest row at PER tokens each.  Two a
  // thread where that is one CTA a row, or two or four and all run at once (a CTA's 1,024 threads take an SM), else
  // eight or sixteen.  With 2 and 8 a thread (us): rows of 2,048, B = 152 6.9 and 9.0, B = 608 25.5 and 33.8; of 4,000,
  // B = 76 8.0 and 9.4, B = 100 14.9 and 9.5; of 8,000, B = 32 10.1 and 10.0, B = 64 19.3 and 10.2; of 16,000
  // (clusters of eight), B = 8 13.0 and 11.3
  auto ctas = [&](int per) {
    int32_t cs = 1;
    while ((int64_t)cs * per * kEvictThreads < longest) cs *= 2;
    return cs;
  };
  if (ctas(2) == 1 || (ctas(2) <= 4 && n * ctas(2) <= num_sms))
    return evict_cluster<2>(a, row0, n, ctas(2), keep_last, req_to_slot, suffix_len, weight, cap, slots_out, s);
  if (ctas(8) <= 8)
    return evict_cluster<8>(a, row0, n, ctas(8), keep_last, req_to_slot, suffix_len, weight, cap, slots_out, s);
  if (ctas(16) <= 8)
    return evict_cluster<16>(a, row0, n, ctas(16), keep_last, req_to_slot, suffix_len, weight, cap, slots_out, s);
  evict_kernel<N><<<n, kEvictThreads, 0, s>>>(a, row0, keep_last, req_to_slot, suffix_len, weight, cap, slots_out);
  return cudaGetLastError();
}

template <typename T>
bool weigh_on_mma(const WeighParams& p) {
  return std::is_same_v<T, __nv_bfloat16> && (p.d == 128 || p.d == 64) && p.n_kv <= kMaxHeads;
}

template <int BITS, int D, int N>
cudaError_t weigh_mma(const WeighParams& p, const WeighRows<N>& rows, int32_t chunks, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem_once(weigh_mma_kernel<BITS, D, N>, WeighUnit<BITS, D>::kRing + 4 * kMaxHeads * kChunkMin, allowed, 4 * kChunkMax);
  if (e != cudaSuccess) return e;
  const int smem = WeighUnit<BITS, D>::kRing + (int)sizeof(float) * p.n_kv * rows.tokens;
  weigh_mma_kernel<BITS, D, N><<<chunks, 256, smem, s>>>(p, rows);
  return cudaGetLastError();
}

template <typename T, int BITS, int N>
cudaError_t weigh_launch(const WeighParams& p, const WeighRows<N>& rows, int32_t chunks, cudaStream_t s) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    if (weigh_on_mma<T>(p)) {
      return p.d == 128 ? weigh_mma<BITS, 128, N>(p, rows, chunks, s) : weigh_mma<BITS, 64, N>(p, rows, chunks, s);
    }
  }
  const int smem = (int)sizeof(float) * (kTok * (p.d + 1) + 8 * kTok);
  weigh_generic_kernel<T, BITS, N><<<chunks, 256, smem, s>>>(p, rows);
  return cudaGetLastError();
}

template <typename T, int BITS, int N>
cudaError_t weigh_rows(const WeighParams& p, const int32_t* seq_len, int32_t b0, int32_t n, int tokens, cudaStream_t s) {
  WeighRows<N> rows;
  int64_t chunks = 0;
  for (int32_t r = 0; r < n; ++r) {
    rows.first[r] = (int32_t)chunks;
    rows.len[r] = seq_len[b0 + r];
    chunks += (seq_len[b0 + r] + tokens - 1) / tokens;
    if (chunks > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  }
  rows.first[n] = (int32_t)chunks;
  rows.n = n;
  rows.b0 = b0;
  rows.tokens = tokens;
  return chunks ? weigh_launch<T, BITS, N>(p, rows, (int32_t)chunks, s) : cudaSuccess;
}

template <typename T, int BITS>
cudaError_t weigh_all(const WeighParams& p, const int32_t* seq_len, cudaStream_t s) {
  constexpr int kSmall = 64, kLarge = kRowsPerLaunch;
  int tokens = kTok;
  if (weigh_on_mma<T>(p)) {
    using Unit = WeighUnit<BITS, 128>;
    const int most = std::max(kChunkMin, std::min(kChunkMax, Unit::kSums / (4 * p.n_kv) / 16 * 16));
    const int64_t slots = (int64_t)Unit::kBlocks * p.num_sms;
    // the fewest tokens a chunk, in steps of 16, with which the grid is one wave
    tokens = kChunkMin;
    for (int pass = 0; pass < 8 && tokens < most; ++pass) {
      int64_t chunks = 0;
      for (int32_t b = 0; b < p.B; ++b) chunks += (seq_len[b] + tokens - 1) / tokens;
      if (chunks <= slots) break;
      const int64_t want = (chunks * tokens / slots + 15) / 16 * 16;
      tokens = (int)std::min<int64_t>(most, std::max<int64_t>(want, tokens + 16));
    }
  }
  cudaError_t e = cudaSuccess;
  for (int32_t b = 0; b < p.B && e == cudaSuccess;) {
    const int32_t n = p.B - b < kLarge ? p.B - b : kLarge;
    e = n <= kSmall ? weigh_rows<T, BITS, kSmall>(p, seq_len, b, n, tokens, s)
                    : weigh_rows<T, BITS, kLarge>(p, seq_len, b, n, tokens, s);
    b += n;
  }
  return e;
}

}  // namespace

cudaError_t launch_cold_weigh(int32_t dtype, const WeighParams& p, const int32_t* seq_len, cudaStream_t s) {
  auto all = [&](auto t) {
    using T = decltype(t);
    return p.packed_bits == 4 ? weigh_all<T, 4>(p, seq_len, s) : p.packed_bits == 8 ? weigh_all<T, 8>(p, seq_len, s) : weigh_all<T, 0>(p, seq_len, s);
  };
  return dtype == 1 ? all(__nv_bfloat16{}) : all(0.f);
}

cudaError_t launch_cold_evict(const EvictRow* rows, int32_t B, int32_t num_sms, int32_t keep_last,
                              int32_t* req_to_slot, int32_t* suffix_len, float* weight, int32_t cap, int32_t* slots_out, cudaStream_t s) {
  // the rows' counts travel as a kernel parameter: nothing is staged in memory that two calls (or
  // a captured and an eager one) could share
  constexpr int kSmall = 64, kLarge = kRowsPerLaunch;
  cudaError_t e = cudaSuccess;
  for (int32_t b = 0; b < B && e == cudaSuccess;) {
    const int32_t n = B - b < kLarge ? B - b : kLarge;
    e = n <= kSmall ? evict_n<kSmall>(rows + b, b, n, num_sms, keep_last, req_to_slot, suffix_len, weight, cap, slots_out, s)
                    : evict_n<kLarge>(rows + b, b, n, num_sms, keep_last, req_to_slot, suffix_len, weight, cap, slots_out, s);
    b += n;
  }
  return e;
}

}  // namespace granikv
