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
  // (kv8_quotient, two elements to an instruction)
  __device__ __forceinline__ void store(uint8_t* dst, const Kv8Divisor& by, bool finite) const {
    const uint64_t f2 = f2_pack(by.minus_f, by.minus_f), inv2 = f2_pack(by.minus_inv, by.minus_inv), a2 = f2_pack(by.a, by.a);
    auto codes = [&](uint32_t w) {
      const float x = __uint_as_float(w << 16), y = __uint_as_float(w & 0xffff0000u);
      float a, b;
      if (finite) {
        const uint64_t n = f2_mul(f2_pack(x, y), f2), q0 = f2_mul(n, inv2), r = f2_fma(q0, a2, n);
        f2_unpack(f2_fma(r, inv2, q0), a, b);
      } else {
        a = kv8_quotient<__nv_bfloat16>(x, by);
        b = kv8_quotient<__nv_bfloat16>(y, by);
      }
      return (uint32_t)f32x2_to_e4m3x2(a, b);
    };
    *reinterpret_cast<uint2*>(dst) = make_uint2(codes(w.x) | codes(w.y) << 16, codes(w.z) | codes(w.w) << 16);
  }
  template <int N>
  __device__ static __forceinline__ float amax_of(const Piece (&x)[N], bool& finite) {
    // magnitudes order as their bits do, two to a word; only where one is not finite are they told apart
    uint32_t m = 0u;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      m = __vmaxu2(m, __vmaxu2(x[c].w.x & 0x7fff7fffu, x[c].w.y & 0x7fff7fffu));
      m = __vmaxu2(m, __vmaxu2(x[c].w.z & 0x7fff7fffu, x[c].w.w & 0x7fff7fffu));
    }
    const uint32_t top = max(m & 0xffffu, m >> 16);
    float amax = __uint_as_float(top << 16);
    finite = top < 0x7f80u;
    if (!finite) {
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
  __device__ __forceinline__ void store(uint8_t* dst, const Kv8Divisor& by, bool) const {
    auto q = [&](uint32_t u) { return kv8_quotient<float>(__uint_as_float(u), by); };
    *reinterpret_cast<uint32_t*>(dst) = f32x4_to_e4m3x4(q(w.x), q(w.y), q(w.z), q(w.w));
  }
  template <int N>
  __device__ static __forceinline__ float amax_of(const Piece (&x)[N], bool&) {
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
// the rows are read once: 3 bytes moved for each bf16 element (16K tokens of 8 x 128: 18.7 us at six CTAs an
// SM; its 100 MB take 14.9).  What it costs beyond HBM is issue: 17.4 us with one product an element in place of
// the quotient (which rounds twice), 23.2 with head_dim at run time (two divisions for each piece's place).
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
  bool finite = true;  // this thread's elements
  float amax = Piece<T>::amax_of(x, finite);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = fmaxf(amax, s_max[w]);
  const Kv8Divisor by = kv8_divisor(amax);
  const float scale = kv8_scale(amax);
  const int32_t row = (int32_t)kv8_row_bytes(n_kv, D);
  uint8_t* dst = (blockIdx.y ? vpool : kpool) + (first_slot + t0) * row;
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int32_t idx = threadIdx.x + c * 256, t = idx / kPerRow;
    if (t < n) x[c].store(dst + t * row + j * D + idx % kPerRow * kElems, by, finite);
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
  const Kv8Divisor by = kv8_divisor(amax);
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] = kv8_quotient<T>(x[i], by);
  uint8_t* dst = slot_row + (int64_t)j * d + lane * VPL;
  if constexpr (VPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4)
      *reinterpret_cast<uint32_t*>(dst + i) = f32x4_to_e4m3x4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) dst[i] = (uint8_t)f32x2_to_e4m3x2(x[i], 0.f);
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
// A CTA takes up to kGenericRows (16) query rows of one KV head and a run of tokens.  Its warps take the
// run's 16-token tiles in turn, each all rows of its tiles, with a softmax state of its own; the states
// join at the end.  A warp unpacks a tile into its own part of shared memory (its lanes hold the next
// one's codes and scales meanwhile), so nothing in the loop waits for another warp.
// A lane (x = lane % 8, y = lane / 8) has the scores of tokens x, x + 8 and rows y, y + 4, y + 8, y + 12, then the
// sums of these rows over columns 4 (x + 8 k) .. + 3: what is read of shared memory serves 8 and 16 products an
// element.  Products go two to an instruction, with no branch among them.  A token's scales multiply its score
// and its weight.  Bound by latency in small problems, by issue in large ones.  fp32, 8/2 heads of 64, with the
// merge: 1,500-token prefix, B = 48 16.5 us; 2,900 tokens, B = 64 26.8; 34 and 1,995 tokens, B = 4 9.7.  (With a warp's
// lanes as tokens and four rows a warp, reads of shared memory took most of the time: 19.7, 39.0 and 12.5.)
constexpr int kRows = kGenericRows, kTok = 16, kRowSets = 4;
static_assert(kRows == 4 * kRowSets, "rows y + 4 i of lanes y");
__host__ __device__ constexpr int generic_warps(int d) { return d <= 128 ? 8 : 4; }

// floats: q [kRows][d + 4]; a warp's K [kTok][d + 4] (then weights [kTok][kRows]) and V [kTok][d] (then, over both, its
// sums [kRows][d]); the warps' maxima and row sums [warps][2][kRows]
__host__ __device__ constexpr int generic_warp_floats(int d) { return kTok * (2 * d + 4); }
__host__ __device__ constexpr int generic_smem(int d) {
  return (int)sizeof(float) * (kRows * (d + 4) + generic_warps(d) * (generic_warp_floats(d) + 2 * kRows));
}

// slot_of(t): the token's slot, or -1 for one that does not count.
template <typename T, int VPL, typename SlotOf, typename ReqOf, typename HeadOf, typename RecOf>
__device__ __forceinline__ void kv8_generic_run(const AttnParams& p, int32_t j, int32_t t0, int32_t t1, int n_rows,
                                                SlotOf slot_of, ReqOf req_of, HeadOf head_of, RecOf rec_of) {
  constexpr int d = VPL * 32, kWarps = generic_warps(d), kPer = kRows / kWarps;
  extern __shared__ __align__(16) float sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = lane & 7, y = lane >> 3;
  float* sQ = sm;
  float* sK = sQ + kRows * (d + 4) + warp * generic_warp_floats(d);
  float* sV = sK + kTok * (d + 4);
  float4* sP = reinterpret_cast<float4*>(sK);  // [kTok][4]: of lane y's rows
  float* sState = sQ + kRows * (d + 4) + kWarps * generic_warp_floats(d);  // [warp][max, sum][row]
  // q, and where the warp's rows go: rows warp, warp + kWarps, ..
  int32_t rec[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = warp + i * kWarps;
    rec[i] = -1;
    const T* q = nullptr;
    if (r < n_rows) {
      rec[i] = rec_of(r);
      q = (const T*)p.q + ((int64_t)req_of(r) * p.n_q + head_of(r)) * d;
    }
#pragma unroll
    for (int c = 0; c < VPL; ++c) sQ[r * (d + 4) + lane + 32 * c] = q ? q_no_inf((float)q[lane + 32 * c]) * p.scale_log2 : 0.f;
  }
  // this lane's share of a tile: VPL pieces of 16 codes, piece i of token (lane + 32 i) / (d / 16), and the K
  // (lanes below 16) or V scale of token lane % 16 (0 for one that does not count)
  uint4 kw[VPL], vw[VPL];
  float scale;
  auto load = [&](int32_t t) {
    const int32_t mine = t + (lane & 15) < t1 ? slot_of(t + (lane & 15)) : -1;
    const uint8_t* pool = (const uint8_t*)(lane < 16 ? p.kpool : p.vpool);
    scale = mine < 0 ? 0.f : *reinterpret_cast<const float*>(pool + (int64_t)mine * p.kv8_row + (int64_t)p.n_kv * d + 4 * j);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int w = lane + 32 * i;
      const int32_t slot = __shfl_sync(0xffffffffu, mine, w / (d / 16));
      kw[i] = vw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (slot >= 0) {
        const int64_t at = (int64_t)slot * p.kv8_row + (int64_t)j * d + w % (d / 16) * 16;
        kw[i] = *reinterpret_cast<const uint4*>((const uint8_t*)p.kpool + at);
        vw[i] = *reinterpret_cast<const uint4*>((const uint8_t*)p.vpool + at);
      }
    }
  };
  // (the lanes of a store phase start at different pieces of theirs, which spreads them over the banks)
  auto unpack = [lane](float* dst, const uint4& w) {
    const bool odd = lane & 1, up = lane & 2;
    const uint32_t a = odd ? w.y : w.x, b = odd ? w.x : w.y, c = odd ? w.w : w.z, e = odd ? w.z : w.w;
    const uint32_t u[4] = {up ? c : a, up ? e : b, up ? a : c, up ? b : e};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[4];
      e4m3x4_to_f32x4(u[i], f);
      *reinterpret_cast<float4*>(dst + 4 * (i ^ (lane & 3))) = make_float4(f[0], f[1], f[2], f[3]);
    }
  };
  // the products, of the row sets that hold rows (y + 4 i for i < 1, 2 or 4), without a branch among them
  auto with_sets = [&](auto f) {
    if (n_rows <= 4) f(std::integral_constant<int, 1>{});
    else if (n_rows <= 8) f(std::integral_constant<int, 2>{});
    else f(std::integral_constant<int, kRowSets>{});
  };
  float m[kRowSets], l[kRowSets];
  uint64_t o2[kRowSets][VPL][2];  // pairs of columns
#pragma unroll
  for (int i = 0; i < kRowSets; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < VPL; ++k) o2[i][k][0] = o2[i][k][1] = 0ull;  // 0.0f bit patterns
  }
  int32_t t = t0 + warp * kTok;
  if (t < t1) load(t);
  __syncthreads();  // q
  for (; t < t1; t += kWarps * kTok) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int w = lane + 32 * i, tok = w / (d / 16), c = w % (d / 16) * 16;
      unpack(sK + tok * (d + 4) + c, kw[i]);
      unpack(sV + tok * d + c, vw[i]);
    }
    const float ks[2] = {__shfl_sync(0xffffffffu, scale, x), __shfl_sync(0xffffffffu, scale, x + 8)};
    const float vs[2] = {__shfl_sync(0xffffffffu, scale, x + 16), __shfl_sync(0xffffffffu, scale, x + 24)};
    __syncwarp();
    if (t + kWarps * kTok < t1) load(t + kWarps * kTok);
    uint64_t s2[2][kRowSets];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < kRowSets; ++i) s2[u][i] = 0ull;
    const ulonglong2* k0 = reinterpret_cast<const ulonglong2*>(sK + x * (d + 4));
    const ulonglong2* k1 = reinterpret_cast<const ulonglong2*>(sK + (x + 8) * (d + 4));
    const ulonglong2* q0 = reinterpret_cast<const ulonglong2*>(sQ + y * (d + 4));
    with_sets([&](auto n) {
#pragma unroll 4
      for (int c = 0; c < d / 4; ++c) {
        const ulonglong2 a = k0[c], b = k1[c];
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const ulonglong2 q = q0[i * (d + 4) + c];  // (4 rows of d + 4 floats are d + 4 pieces)
          s2[0][i] = f2_fma(q.y, a.y, f2_fma(q.x, a.x, s2[0][i]));
          s2[1][i] = f2_fma(q.y, b.y, f2_fma(q.x, b.x, s2[1][i]));
        }
      }
    });
    __syncwarp();  // K is read: the weights take its place
    float w0[kRowSets], w1[kRowSets], alpha[kRowSets];
    bool moved = false;
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      float lo, hi;
      f2_unpack(s2[0][i], lo, hi);
      w0[i] = ks[0] != 0.f ? (lo + hi) * ks[0] : -INFINITY;  // (a written row's scale is above 0)
      f2_unpack(s2[1][i], lo, hi);
      w1[i] = ks[1] != 0.f ? (lo + hi) * ks[1] : -INFINITY;
      float mx = fmaxf(w0[i], w1[i]);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
      alpha[i] = exp2f(m[i] - base);
      moved = moved || mn != m[i];
      m[i] = mn;
      w0[i] = exp2f(w0[i] - base);
      w1[i] = exp2f(w1[i] - base);
      l[i] = l[i] * alpha[i] + (w0[i] + w1[i]);  // this lane's tokens; the lanes' sums are added at the end
    }
    sP[x * 4 + y] = make_float4(w0[0] * vs[0], w0[1] * vs[0], w0[2] * vs[0], w0[3] * vs[0]);
    sP[(x + 8) * 4 + y] = make_float4(w1[0] * vs[1], w1[1] * vs[1], w1[2] * vs[1], w1[3] * vs[1]);
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < kRowSets; ++i) {
        const uint64_t a2 = f2_pack(alpha[i], alpha[i]);
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
          o2[i][k][0] = f2_mul(o2[i][k][0], a2);
          o2[i][k][1] = f2_mul(o2[i][k][1], a2);
        }
      }
    }
    __syncwarp();
    with_sets([&](auto n) {
#pragma unroll 4
      for (int tok = 0; tok < kTok; ++tok) {  // (a token that does not count has weight 0 and V 0)
        const float4 w = sP[tok * 4 + y];
        const uint64_t w2[kRowSets] = {f2_pack(w.x, w.x), f2_pack(w.y, w.y), f2_pack(w.z, w.z), f2_pack(w.w, w.w)};
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sV + tok * d + (x + 8 * k) * 4);
#pragma unroll
          for (int i = 0; i < n; ++i) {
            o2[i][k][0] = f2_fma(w2[i], v.x, o2[i][k][0]);
            o2[i][k][1] = f2_fma(w2[i], v.y, o2[i][k][1]);
          }
        }
      }
    });
    __syncwarp();  // the tile is read
  }
  // the warps' states meet in shared memory, each warp's sums in its own tile's place
#pragma unroll
  for (int i = 0; i < kRowSets; ++i) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
#pragma unroll
    for (int k = 0; k < VPL; ++k)
      *reinterpret_cast<ulonglong2*>(sK + (y + 4 * i) * d + (x + 8 * k) * 4) = make_ulonglong2(o2[i][k][0], o2[i][k][1]);
    if (x == 0) {
      sState[warp * 2 * kRows + y + 4 * i] = m[i];
      sState[warp * 2 * kRows + kRows + y + 4 * i] = l[i];
    }
  }
  __syncthreads();
  const float* sums = sQ + kRows * (d + 4);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = warp + i * kWarps;
    if (r >= n_rows) break;
    if (rec[i] < 0 || rec[i] >= p.n_records) {
      if (lane == 0) latch(p.err, kDevBadRecord);
      continue;
    }
    float top = -INFINITY, total = 0.f, o[VPL];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sState[w * 2 * kRows + r]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int c = 0; c < VPL; ++c) o[c] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = exp2f(sState[w * 2 * kRows + r] - base);
      total += sState[w * 2 * kRows + kRows + r] * a;
#pragma unroll
      for (int c = 0; c < VPL; ++c) o[c] += sums[w * generic_warp_floats(d) + r * d + lane + 32 * c] * a;
    }
    const int64_t at = (int64_t)rec[i] * p.n_q + head_of(r);
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int c = 0; c < VPL; ++c) p.rec_o[at * d + lane + 32 * c] = o[c] * inv;
    if (lane == 0) p.rec_lse[at] = kv8_record_lse(total, (base + log2f(total)) * kLn2);
  }
}

// CTAs [0, n_prefix) take prefix items first_item.., the rest (suffix item, KV head, block of kRows of
// its query heads): one launch, so that short prefixes and suffixes share the SMs.
template <typename T, int VPL>
__global__ void __launch_bounds__(generic_warps(32 * VPL) * 32, VPL <= 1 ? 3 : VPL <= 2 ? 2 : 1) kv8_generic_kernel(AttnParams p, int32_t first_item, int32_t n_prefix) {
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
    return launch_kernel(kernel, dim3((unsigned)ctas), dim3(generic_warps(32 * n) * 32), (size_t)smem, s, pdl, p, first_item, n_items);
  });
}

}  // namespace granikv
