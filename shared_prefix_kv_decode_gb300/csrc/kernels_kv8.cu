// kernels_kv8.cu -- 8-bit cache: the kernels that quantise K/V rows into packed slots, and the
// CUDA-core decode attention over such slots for any head_dim that is a multiple of 32 (up to
// 256) and either type of q.
#include "kv8_util.cuh"
#include "launch_util.cuh"
#include "tc_util.cuh"

#include <cmath>

namespace granikv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void latch(int32_t* err, int32_t code) { atomicCAS(err, 0, code); }

// 16 bytes of a row, kept as they came: 8 bf16 or 4 fp32 elements.  amax_of: the largest finite magnitude
// of N pieces.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kElems = 8;
  uint4 w;
  __device__ __forceinline__ void store(uint8_t* dst, float inv) const {
    const uint64_t inv2 = f2_pack(inv, inv);
    auto codes = [&](uint32_t x) {
      float a, b;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), inv2), a, b);
      return (uint32_t)f32x2_to_e4m3x2(a, b);
    };
    *reinterpret_cast<uint2*>(dst) = make_uint2(codes(w.x) | codes(w.y) << 16, codes(w.z) | codes(w.w) << 16);
  }
  template <int N>
  __device__ static __forceinline__ float amax_of(const Piece (&x)[N]) {
    // magnitudes order as their bits do, two to a word; only where one is not finite are they told apart
    uint32_t m = 0u;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      m = __vmaxu2(m, __vmaxu2(x[c].w.x & 0x7fff7fffu, x[c].w.y & 0x7fff7fffu));
      m = __vmaxu2(m, __vmaxu2(x[c].w.z & 0x7fff7fffu, x[c].w.w & 0x7fff7fffu));
    }
    const uint32_t top = max(m & 0xffffu, m >> 16);
    float amax = __uint_as_float(top << 16);
    if (top >= 0x7f80u) {
      amax = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c)
        amax = fmaxf(amax, fmaxf(fmaxf(bf16x2_finite_max(x[c].w.x), bf16x2_finite_max(x[c].w.y)),
                                 fmaxf(bf16x2_finite_max(x[c].w.z), bf16x2_finite_max(x[c].w.w))));
    }
    return amax;
  }
};
template <>
struct Piece<float> {
  static constexpr int kElems = 4;
  uint4 w;
  __device__ __forceinline__ void store(uint8_t* dst, float inv) const {
    *reinterpret_cast<uint32_t*>(dst) = f32x4_to_e4m3x4(__uint_as_float(w.x) * inv, __uint_as_float(w.y) * inv,
                                                        __uint_as_float(w.z) * inv, __uint_as_float(w.w) * inv);
  }
  template <int N>
  __device__ static __forceinline__ float amax_of(const Piece (&x)[N]) {
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c)
      amax = fmaxf(amax, fmaxf(fmaxf(finite_abs(__uint_as_float(x[c].w.x)), finite_abs(__uint_as_float(x[c].w.y))),
                               fmaxf(finite_abs(__uint_as_float(x[c].w.z)), finite_abs(__uint_as_float(x[c].w.w)))));
    return amax;
  }
};

// One block of kKv8Block slab tokens of one KV head (the heads of a block are neighbours in the grid, so
// that its rows are read and written whole at about the same time), of K (blockIdx.y = 0) or V.  The block stays in
// registers between its amax and its codes (pieces of 16 bytes, all of a thread's requested at once), so
// the rows are read once: 3 bytes moved for each bf16 element (16K tokens of 8 x 128: 17.5 us at six CTAs an
// SM; its 100 MB take 14.9).  What it costs beyond HBM is issue: with head_dim at run time, the pieces'
// places cost two divisions each, the warps issued in 77 % of the cycles, and it took 23.2 us.
template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) * D <= 256 ? 6 : 1) kv8_fill_kernel(
    const T* __restrict__ k, const T* __restrict__ v, int32_t L_p, uint8_t* __restrict__ kpool,
    uint8_t* __restrict__ vpool, int64_t first_slot, int32_t n_kv) {
  constexpr int kElems = Piece<T>::kElems;
  constexpr int kPerRow = D / kElems;              // pieces of a head's row
  constexpr int kPieces = kKv8Block * kPerRow / 256;  // of a thread
  __shared__ float s_max[8];
  const int32_t j = blockIdx.x % n_kv;
  const int32_t t0 = blockIdx.x / n_kv * kKv8Block;
  const int32_t n = min(kKv8Block, L_p - t0);
  const T* src = (blockIdx.y ? v : k) + ((int64_t)t0 * n_kv + j) * D;
  Piece<T> x[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int32_t idx = threadIdx.x + c * 256, t = idx / kPerRow;
    x[c].w = t < n ? __ldcs(reinterpret_cast<const uint4*>(src + t * (n_kv * D) + idx % kPerRow * kElems))
                   : make_uint4(0u, 0u, 0u, 0u);
  }
  float amax = Piece<T>::amax_of(x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = fmaxf(amax, s_max[w]);
  const float inv = kv8_inverse(amax), scale = kv8_scale(amax);
  const int32_t row = (int32_t)kv8_row_bytes(n_kv, D);
  uint8_t* dst = (blockIdx.y ? vpool : kpool) + (first_slot + t0) * row;
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int32_t idx = threadIdx.x + c * 256, t = idx / kPerRow;
    if (t < n) x[c].store(dst + t * row + j * D + idx % kPerRow * kElems, inv);
  }
  for (int32_t t = threadIdx.x; t < n; t += 256) *reinterpret_cast<float*>(dst + t * row + n_kv * D + 4 * j) = scale;
}

// One warp quantises head j of one K (or V) row into a packed slot: a lane holds VPL consecutive
// elements, and stores VPL codes (VPL bytes, at a VPL-byte offset).
template <typename T, int VPL>
__device__ __forceinline__ void kv8_write_row(const T* __restrict__ src, uint8_t* __restrict__ slot_row, int32_t j,
                                              int32_t n_kv, int32_t d, int lane) {
  float x[VPL];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    x[i] = (float)src[lane * VPL + i];
    amax = fmaxf(amax, finite_abs(x[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float inv = kv8_inverse(amax);
  uint8_t* dst = slot_row + (int64_t)j * d + lane * VPL;
  if constexpr (VPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4)
      *reinterpret_cast<uint32_t*>(dst + i) =
          f32x4_to_e4m3x4(x[i] * inv, x[i + 1] * inv, x[i + 2] * inv, x[i + 3] * inv);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) dst[i] = (uint8_t)f32x2_to_e4m3x2(x[i] * inv, 0.f);
  }
  if (lane == 0) *reinterpret_cast<float*>(slot_row + (int64_t)n_kv * d + 4 * j) = kv8_scale(amax);
}

// Rows at slots[i] (one scale per token and head): one warp per (row, head), K and V.
template <typename T, int VPL>
__global__ void __launch_bounds__(256) kv8_append_kernel(const T* __restrict__ k_new, const T* __restrict__ v_new,
                                                         const int32_t* __restrict__ slots, int32_t N,
                                                         uint8_t* __restrict__ kpool, uint8_t* __restrict__ vpool,
                                                         int32_t n_kv, int32_t d, int64_t row, int64_t n_hot,
                                                         int64_t n_slots, int32_t* err) {
  const int lane = threadIdx.x & 31;
  const int64_t total = (int64_t)N * n_kv;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += (int64_t)gridDim.x * 8) {
    const int32_t t = (int32_t)(w / n_kv), j = (int32_t)(w % n_kv);
    const int32_t slot = slots[t];
    if (slot < n_hot || slot >= n_slots) {
      if (lane == 0) latch(err, kDevBadSlot);
      continue;
    }
    kv8_write_row<T, VPL>(k_new + w * d, kpool + (int64_t)slot * row, j, n_kv, d, lane);
    kv8_write_row<T, VPL>(v_new + w * d, vpool + (int64_t)slot * row, j, n_kv, d, lane);
  }
}

// Row b of k_new/v_new at the slot of request b's newest token (the fused append's write).
template <typename T, int VPL>
__global__ void __launch_bounds__(256) kv8_append_newest_kernel(AttnParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)p.B * p.n_kv) return;
  const int32_t b = (int32_t)(w / p.n_kv), j = (int32_t)(w % p.n_kv);
  int32_t n = p.reqs[b].seq_len;
  if (p.live_len) n = min(n, p.live_len[b]);
  if (n < 1) return;
  const int32_t slot = p.req_to_slot[(int64_t)b * p.cap + n - 1];
  if (slot < p.n_hot || slot >= p.n_slots) {
    if (lane == 0) latch(p.err, kDevBadSlot);
    return;
  }
  kv8_write_row<T, VPL>((const T*)p.k_new + w * p.d, (uint8_t*)p.kpool + (int64_t)slot * p.kv8_row, j, p.n_kv, p.d, lane);
  kv8_write_row<T, VPL>((const T*)p.v_new + w * p.d, (uint8_t*)p.vpool + (int64_t)slot * p.kv8_row, j, p.n_kv, p.d, lane);
}

// ---- decode attention on CUDA cores -----------------------------------------------------------
// A CTA takes up to kGenericRows query rows of one KV head and a run of tokens.  Tiles of 64
// tokens are unpacked into shared memory once for all rows (a thread holds the next tile's codes
// and scales while it computes this one).  Warps w and w + 4 hold the same four rows, each over its half
// of a tile: the lanes are the half's tokens for the scores and head_dim's columns for the weighted
// sum, and the two join at the end.  A token's scales multiply its score and its weight.
// Bound by the latency of small problems and by reads of shared memory: four rows a warp use what it
// reads of K and V four times, and products go two to an instruction where a lane's columns pair up
// (head_dim a multiple of 64).  fp32, 1,500-token prefix, 48 requests of 8/2 heads of 64 with up to 80 COLD
// tokens: 22.4 us with two rows a warp and 32-token tiles, 19.9 so, with the merge, at three CTAs an SM.
constexpr int kRows = kGenericRows;
constexpr int kTok = 64, kHalfTok = 32;
constexpr int kWarpRows = 4;
static_assert(kRows == 4 * kWarpRows && kTok % kGenericTile == 0, "eight warps: four row groups, two halves of a tile");

// floats: V [kTok][d], q [kRows][d], K [kTok][d + 4], weights [8][kTok / 2][kWarpRows], scales [2][kTok]
__host__ __device__ inline int generic_smem(int d) {
  return (int)sizeof(float) * (kTok * (d + 4) + kTok * d + kRows * d + 8 * kHalfTok * kWarpRows + 2 * kTok);
}

// slot_of(t): the token's slot, or -1 for one that does not count.
template <typename T, int VPL, typename SlotOf, typename ReqOf, typename HeadOf, typename RecOf>
__device__ __forceinline__ void kv8_generic_run(const AttnParams& p, int32_t j, int32_t t0, int32_t t1, int n_rows,
                                                SlotOf slot_of, ReqOf req_of, HeadOf head_of, RecOf rec_of) {
  constexpr int d = VPL * 32;
  constexpr int kPer = VPL % 2 ? 1 : 2;  // neighbouring columns a lane takes
  constexpr int kCols = VPL / kPer;      // column of (i, e): (lane + 32 i) * kPer + e
  extern __shared__ __align__(16) float sm[];
  float* sV = sm;                 // codes
  float* sQ = sV + kTok * d;
  float* sK = sQ + kRows * d;     // codes: 16-byte reads of eight tokens cover all banks
  float4* sW = reinterpret_cast<float4*>(sK + kTok * (d + 4));
  float* sScale = reinterpret_cast<float*>(sW + 8 * kHalfTok);  // of K (0: the token does not count), of V
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = (warp & 3) * kWarpRows, half = warp >> 2;
  float4* w_mine = sW + warp * kHalfTok;  // weights times the V scale of this warp's four rows, by token
  for (int i = threadIdx.x; i < kRows * d; i += blockDim.x)
    sQ[i] = i < n_rows * d ? (float)((const T*)p.q)[((int64_t)req_of(i / d) * p.n_q + head_of(i / d)) * d + i % d] * p.scale_log2 : 0.f;
  int32_t rec[kWarpRows];  // looked up now, so that the loads finish during the tiles
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) rec[r] = half == 0 && r0 + r < n_rows ? rec_of(r0 + r) : -1;
  float m[kWarpRows], l[kWarpRows], acc[kWarpRows][VPL];
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[r][i] = 0.f;
  }
  // this thread's share of a tile: VPL pieces of eight codes, piece i of token (thread + 256 i) / (d / 8)
  uint2 kw[VPL], vw[VPL];
  float ks[VPL], vs[VPL];
  auto load = [&](int32_t t) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int w = threadIdx.x + 256 * i, tok = w / (d / 8), c = w % (d / 8) * 8;
      const int32_t slot = t + tok < t1 ? slot_of(t + tok) : -1;
      kw[i] = vw[i] = make_uint2(0u, 0u);
      ks[i] = vs[i] = 0.f;
      if (slot >= 0) {
        const uint8_t* kr = (const uint8_t*)p.kpool + (int64_t)slot * p.kv8_row;
        const uint8_t* vr = (const uint8_t*)p.vpool + (int64_t)slot * p.kv8_row;
        kw[i] = *reinterpret_cast<const uint2*>(kr + (int64_t)j * d + c);
        vw[i] = *reinterpret_cast<const uint2*>(vr + (int64_t)j * d + c);
        if (c == 0) {
          ks[i] = *reinterpret_cast<const float*>(kr + (int64_t)p.n_kv * d + 4 * j);
          vs[i] = *reinterpret_cast<const float*>(vr + (int64_t)p.n_kv * d + 4 * j);
        }
      }
    }
  };
  auto unpack = [](float* dst, uint2 w) {
    float x[4];
    e4m3x4_to_f32x4(w.x, x);
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    e4m3x4_to_f32x4(w.y, x);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(x[0], x[1], x[2], x[3]);
  };
  load(t0);
  for (int32_t t = t0; t < t1; t += kTok) {
    __syncthreads();  // the tile before is read
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int w = threadIdx.x + 256 * i, tok = w / (d / 8), c = w % (d / 8) * 8;
      unpack(sK + tok * (d + 4) + c, kw[i]);
      unpack(sV + tok * d + c, vw[i]);
      if (c == 0) {
        sScale[tok] = ks[i];
        sScale[kTok + tok] = vs[i];
      }
    }
    __syncthreads();
    if (t + kTok < t1) load(t + kTok);
    const int first = half * kHalfTok;  // of the warp's tokens in the tile
    const int n_tok = min(kHalfTok, t1 - t - first);
    if (r0 >= n_rows || n_tok <= 0) continue;
    const float k_scale = sScale[first + lane], v_scale = sScale[kTok + first + lane];
    const ulonglong2* q = reinterpret_cast<const ulonglong2*>(sQ + r0 * d);
    const ulonglong2* kr = reinterpret_cast<const ulonglong2*>(sK + (first + lane) * (d + 4));
    uint64_t s2[kWarpRows][2];  // two partial sums each
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) s2[r][0] = s2[r][1] = 0ull;  // 0.0f bit patterns
#pragma unroll 4
    for (int i = 0; i < d / 4; ++i) {
      const ulonglong2 k = kr[i];
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) {
        const ulonglong2 a = q[r * (d / 4) + i];
        s2[r][0] = f2_fma(a.x, k.x, s2[r][0]);
        s2[r][1] = f2_fma(a.y, k.y, s2[r][1]);
      }
    }
    float s[kWarpRows], mx[kWarpRows], w[kWarpRows], sum[kWarpRows];
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      float x, y;
      f2_unpack(f2_add(s2[r][0], s2[r][1]), x, y);
      mx[r] = s[r] = k_scale != 0.f ? (x + y) * k_scale : -INFINITY;  // (a written row's scale is above 0)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], o));
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      const float mn = fmaxf(m[r], mx[r]);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float a = exp2f(m[r] - base);
      sum[r] = w[r] = exp2f(s[r] - base);
      l[r] *= a;
      m[r] = mn;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[r][i] *= a;
    }
    w_mine[lane] = make_float4(w[0] * v_scale, w[1] * v_scale, w[2] * v_scale, w[3] * v_scale);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) l[r] += sum[r];
    __syncwarp();
    const float* v_mine = sV + first * d;
    if constexpr (kPer == 2) {
      uint64_t o2[kWarpRows][kCols];
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r)
#pragma unroll
        for (int i = 0; i < kCols; ++i) o2[r][i] = f2_pack(acc[r][2 * i], acc[r][2 * i + 1]);
#pragma unroll 4
      for (int tok = 0; tok < n_tok; ++tok) {
        const float4 x = w_mine[tok];
        const uint64_t x2[kWarpRows] = {f2_pack(x.x, x.x), f2_pack(x.y, x.y), f2_pack(x.z, x.z), f2_pack(x.w, x.w)};
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const uint64_t v = *reinterpret_cast<const uint64_t*>(v_mine + tok * d + (lane + 32 * i) * 2);
#pragma unroll
          for (int r = 0; r < kWarpRows; ++r) o2[r][i] = f2_fma(x2[r], v, o2[r][i]);
        }
      }
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r)
#pragma unroll
        for (int i = 0; i < kCols; ++i) f2_unpack(o2[r][i], acc[r][2 * i], acc[r][2 * i + 1]);
    } else {
#pragma unroll 4
      for (int tok = 0; tok < n_tok; ++tok) {
        const float4 x = w_mine[tok];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const float v = v_mine[tok * d + lane + 32 * i];
          acc[0][i] += x.x * v;
          acc[1][i] += x.y * v;
          acc[2][i] += x.z * v;
          acc[3][i] += x.w * v;
        }
      }
    }
    __syncwarp();  // the weights are read
  }
  // the second halves' states go to shared memory (K and V are read), the first join them
  __syncthreads();
  float* other = sV + (warp & 3) * (kWarpRows * (d + 2));  // [kWarpRows][d], then the maxima and sums
  if (half == 1 && r0 < n_rows) {
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) other[r * d + i * 32 + lane] = acc[r][i];
      if (lane == 0) {
        other[kWarpRows * d + r] = m[r];
        other[kWarpRows * (d + 1) + r] = l[r];
      }
    }
  }
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) {
    if (r0 + r >= n_rows) break;
    if (rec[r] < 0 || rec[r] >= p.n_records) {
      if (lane == 0) latch(p.err, kDevBadRecord);
      continue;
    }
    const float m1 = other[kWarpRows * d + r], l1 = other[kWarpRows * (d + 1) + r];
    const float mn = fmaxf(m[r], m1), base = mn == -INFINITY ? 0.f : mn;
    const float a0 = exp2f(m[r] - base), a1 = exp2f(m1 - base);
    const float sum = l[r] * a0 + l1 * a1;
    const int64_t at = (int64_t)rec[r] * p.n_q + head_of(r0 + r);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float* dst = p.rec_o + at * d;
#pragma unroll
    for (int i = 0; i < kCols; ++i)
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        dst[(lane + 32 * i) * kPer + e] = (acc[r][i * kPer + e] * a0 + other[r * d + (i * kPer + e) * 32 + lane] * a1) * inv;
    if (lane == 0) p.rec_lse[at] = kv8_record_lse(sum, (mn + log2f(sum)) * kLn2);
  }
}

// CTAs [0, n_prefix) take prefix items first_item.., the rest (suffix item, KV head, block of kRows of
// its query heads): one launch, so that short prefixes and suffixes share the SMs.
template <typename T, int VPL>
__global__ void __launch_bounds__(256, VPL <= 2 ? 3 : VPL <= 6 ? 2 : 1) kv8_generic_kernel(AttnParams p, int32_t first_item, int32_t n_prefix) {
  // (the plan is not written by the work before this kernel; everything else waits for that work)
  if ((int32_t)blockIdx.x < n_prefix) {
    const DevPrefixItem it = p.pitems[first_item + blockIdx.x];
    const DevGroup gr = p.groups[it.group];
    grid_dep_wait();
    grid_dep_launch_dependents();  // the merge waits for this grid before it reads a record
    if (gr.slab_off < 0 || gr.slab_off + gr.L_p > p.n_hot) {
      if (threadIdx.x == 0) latch(p.err, kDevBadSlab);
      return;
    }
    int32_t t0, t1;
    piece_range(gr, it.split, t0, t1);
    const int32_t r0 = it.row_block * gr.rows_per_cta;
    const int n_rows = min(gr.n_req * p.g - r0, kRows);
    auto req = [&](int r) { return p.group_req[gr.req_begin + (r0 + r) / p.g]; };
    kv8_generic_run<T, VPL>(
        p, it.kv_head, t0, t1, n_rows, [&](int32_t t) { return (int32_t)(gr.slab_off + t); },
        req, [&](int r) { return it.kv_head * p.g + (r0 + r) % p.g; },
        [&](int r) { return p.reqs[req(r)].rec_base + it.split; });
    return;
  }
  const int blocks = (p.g + kRows - 1) / kRows, per = p.n_kv * blocks;
  const int32_t w = blockIdx.x - n_prefix;
  DevSuffixItem it = p.sitems[w / per];
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (p.live_len) it.t1 = max(it.t0, min(it.t1, p.live_len[it.b]));
  const int32_t j = w % per / blocks, h0 = j * p.g + w % blocks * kRows;
  const int n_rows = min(kRows, (j + 1) * p.g - h0);
  kv8_generic_run<T, VPL>(
      p, j, it.t0, it.t1, n_rows,
      [&](int32_t t) {
        const int32_t slot = p.req_to_slot[(int64_t)it.b * p.cap + t];
        if (slot >= p.n_hot && slot < p.n_slots) return slot;
        latch(p.err, kDevBadSlot);
        return (int32_t)-1;
      },
      [&](int) { return it.b; }, [&](int r) { return h0 + r; }, [&](int) { return it.rec; });
}

// Runs f with VPL = d / 32 as a compile-time constant.
template <typename F>
cudaError_t with_vpl(int32_t d, F f) {
  switch (d / 32) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5: return f(std::integral_constant<int, 5>{});
    case 6: return f(std::integral_constant<int, 6>{});
    case 7: return f(std::integral_constant<int, 7>{});
    case 8: return f(std::integral_constant<int, 8>{});
    default: return cudaErrorInvalidValue;
  }
}

template <typename T>
cudaError_t fill_t(const T* k, const T* v, int32_t L_p, uint8_t* kpool, uint8_t* vpool, int64_t first_slot,
                   int32_t n_kv, int32_t d, cudaStream_t s) {
  const int64_t ctas = (int64_t)((L_p + kKv8Block - 1) / kKv8Block) * n_kv;
  if (ctas > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas, 2);
  return with_vpl(d, [&](auto vpl) {
    kv8_fill_kernel<T, 32 * decltype(vpl)::value><<<grid, 256, 0, s>>>(k, v, L_p, kpool, vpool, first_slot, n_kv);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t append_t(const T* k, const T* v, const int32_t* slots, int32_t N, uint8_t* kpool, uint8_t* vpool,
                     int32_t n_kv, int32_t d, int64_t n_hot, int64_t n_slots, int32_t* err, cudaStream_t s) {
  const int64_t ctas = ((int64_t)N * n_kv + 7) / 8;
  const unsigned grid = (unsigned)(ctas < 16384 ? ctas : 16384);
  return with_vpl(d, [&](auto vpl) {
    kv8_append_kernel<T, decltype(vpl)::value><<<grid, 256, 0, s>>>(k, v, slots, N, kpool, vpool, n_kv, d,
                                                                    kv8_row_bytes(n_kv, d), n_hot, n_slots, err);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_kv8_fill(int32_t dtype, const void* k, const void* v, int32_t L_p, uint8_t* kpool, uint8_t* vpool,
                            int64_t first_slot, int32_t n_kv, int32_t d, cudaStream_t s) {
  return dtype == 1 ? fill_t((const __nv_bfloat16*)k, (const __nv_bfloat16*)v, L_p, kpool, vpool, first_slot, n_kv, d, s)
                    : fill_t((const float*)k, (const float*)v, L_p, kpool, vpool, first_slot, n_kv, d, s);
}

cudaError_t launch_kv8_append(int32_t dtype, const void* k_new, const void* v_new, const int32_t* slots, int32_t N,
                              uint8_t* kpool, uint8_t* vpool, int32_t n_kv, int32_t d, int64_t n_hot,
                              int64_t n_slots, int32_t* err, cudaStream_t s) {
  return dtype == 1 ? append_t((const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, slots, N, kpool, vpool, n_kv,
                               d, n_hot, n_slots, err, s)
                    : append_t((const float*)k_new, (const float*)v_new, slots, N, kpool, vpool, n_kv, d, n_hot,
                               n_slots, err, s);
}

cudaError_t launch_kv8_append_newest(int32_t dtype, const AttnParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(((int64_t)p.B * p.n_kv + 7) / 8);
  return with_vpl(p.d, [&](auto vpl) {
    constexpr int n = decltype(vpl)::value;
    if (dtype == 1) kv8_append_newest_kernel<__nv_bfloat16, n><<<grid, 256, 0, s>>>(p);
    else kv8_append_newest_kernel<float, n><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  });
}

cudaError_t launch_kv8_generic(int32_t dtype, const AttnParams& p, int32_t first_item, int32_t n_items, bool suffix,
                               cudaStream_t s, bool pdl) {
  const int64_t ctas = n_items + (suffix ? (int64_t)p.n_sitems * p.n_kv * ((p.g + kRows - 1) / kRows) : 0);
  if (ctas <= 0) return cudaSuccess;
  if (ctas > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  const int smem = generic_smem(p.d);
  return with_vpl(p.d, [&](auto vpl) {
    constexpr int n = decltype(vpl)::value;
    auto kernel = dtype == 1 ? kv8_generic_kernel<__nv_bfloat16, n> : kv8_generic_kernel<float, n>;
    cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)ctas), dim3(256), (size_t)smem, s, pdl, p, first_item, n_items);
  });
}

}  // namespace granikv
