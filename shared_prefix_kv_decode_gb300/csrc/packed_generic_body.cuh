// packed_generic_body.cuh -- CUDA-core decode attention over the packed slots of an 8- or 4-bit cache, for any
// head_dim that is a multiple of 32 (up to 256) and either type of q.
#pragma once

#include "kv4_util.cuh"
#include "kv8_util.cuh"
#include "launch_util.cuh"
#include "tc_util.cuh"

#include <cmath>
#include <type_traits>

namespace granikv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void latch(int32_t* err, int32_t code) { atomicCAS(err, 0, code); }

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

// 16 elements of a packed head: their bytes in a row, and their way into shared memory as floats.
template <int BITS>
struct PackedPiece;
template <>
struct PackedPiece<8> {
  uint4 w;
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const uint8_t* row, int32_t, int32_t d, int32_t j, int piece) {
    w = *reinterpret_cast<const uint4*>(row + (int64_t)j * d + piece * 16);
  }
  // (the lanes of a store phase start at different pieces of theirs, which spreads them over the banks)
  __device__ __forceinline__ void unpack(float* dst, int lane) const {
    const bool odd = lane & 1, up = lane & 2;
    const uint32_t a = odd ? w.y : w.x, b = odd ? w.x : w.y, c = odd ? w.w : w.z, e = odd ? w.z : w.w;
    const uint32_t u[4] = {up ? c : a, up ? e : b, up ? a : c, up ? b : e};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[4];
      e4m3x4_to_f32x4(u[i], f);
      *reinterpret_cast<float4*>(dst + 4 * (i ^ (lane & 3))) = make_float4(f[0], f[1], f[2], f[3]);
    }
  }
  // what the row's codes of head j are multiplied by
  __device__ static __forceinline__ float scale(const uint8_t* row, int32_t n_kv, int32_t d, int32_t j) {
    return *reinterpret_cast<const float*>(row + (int64_t)n_kv * d + 4 * j);
  }
};
template <>
struct PackedPiece<4> {
  uint2 w;
  uint32_t b;
  __device__ __forceinline__ void clear() {
    w = make_uint2(0u, 0u);
    b = 0u;
  }
  __device__ __forceinline__ void load(const uint8_t* row, int32_t n_kv, int32_t d, int32_t j, int piece) {
    w = *reinterpret_cast<const uint2*>(row + (int64_t)j * (d / 2) + piece * 8);
    b = row[kv4_scales_at(n_kv, d) + (int64_t)j * (d / kKv4Group) + piece];
  }
  __device__ __forceinline__ void unpack(float* dst, int lane) const {
    const uint32_t s = kv4_scale2(b);
    uint32_t y[4], z[4];
    e2m1x8_to_f16x8(w.x, y);
    e2m1x8_to_f16x8(w.y, z);
    const bool odd = lane & 1, up = lane & 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // elements 4 (i ^ lane % 4) ..
      uint32_t h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t lo = (i & 2) ? z[u] : y[u], lo2 = (i & 2) ? z[2 + u] : y[2 + u];
        const uint32_t hi = (i & 2) ? y[u] : z[u], hi2 = (i & 2) ? y[2 + u] : z[2 + u];
        const bool second = (i & 1) != 0;
        const uint32_t a = second != odd ? lo2 : lo, c = second != odd ? hi2 : hi;
        h[u] = f16x2_mul(up ? c : a, s);
      }
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[0])), g = __half22float2(*reinterpret_cast<__half2*>(&h[1]));
      *reinterpret_cast<float4*>(dst + 4 * (i ^ (lane & 3))) = make_float4(f.x, f.y, g.x, g.y);
    }
  }
  __device__ static __forceinline__ float scale(const uint8_t* row, int32_t n_kv, int32_t d, int32_t j) {
    return kv4_unit(row[kv4_units_at(n_kv, d) + j]);
  }
};

// slot_of(t): the token's slot, or -1 for one that does not count.
template <int BITS, typename T, int VPL, typename SlotOf, typename ReqOf, typename HeadOf, typename RecOf>
__device__ __forceinline__ void packed_generic_run(const AttnParams& p, int32_t j, int32_t t0, int32_t t1, int n_rows,
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
  // (lanes below 16) or V scale (4 bits: unit) of token lane % 16 (0 for one that does not count)
  PackedPiece<BITS> kw[VPL], vw[VPL];
  float scale;
  auto load = [&](int32_t t) {
    const int32_t mine = t + (lane & 15) < t1 ? slot_of(t + (lane & 15)) : -1;
    const uint8_t* pool = (const uint8_t*)(lane < 16 ? p.kpool : p.vpool);
    scale = mine < 0 ? 0.f : PackedPiece<BITS>::scale(pool + (int64_t)mine * p.packed_row, p.n_kv, d, j);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int w = lane + 32 * i;
      const int32_t slot = __shfl_sync(0xffffffffu, mine, w / (d / 16));
      kw[i].clear();
      vw[i].clear();
      if (slot >= 0) {
        const int64_t at = (int64_t)slot * p.packed_row;
        kw[i].load((const uint8_t*)p.kpool + at, p.n_kv, d, j, w % (d / 16));
        vw[i].load((const uint8_t*)p.vpool + at, p.n_kv, d, j, w % (d / 16));
      }
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
      kw[i].unpack(sK + tok * (d + 4) + c, lane);
      vw[i].unpack(sV + tok * d + c, lane);
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
    if (lane == 0) p.rec_lse[at] = packed_record_lse(total, (base + log2f(total)) * kLn2);
  }
}

// CTAs [0, n_prefix) take prefix items first_item.., the rest (suffix item, KV head, block of kRows of
// its query heads): one launch, so that short prefixes and suffixes share the SMs.
template <int BITS, typename T, int VPL>
__global__ void __launch_bounds__(generic_warps(32 * VPL) * 32, VPL <= 1 ? 3 : VPL <= 2 ? 2 : 1) packed_generic_kernel(AttnParams p, int32_t first_item, int32_t n_prefix) {
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
    packed_generic_run<BITS, T, VPL>(
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
  packed_generic_run<BITS, T, VPL>(
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

template <int BITS>
cudaError_t launch_packed_generic(int32_t dtype, const AttnParams& p, int32_t first_item, int32_t n_items, bool suffix,
                                  cudaStream_t s, bool pdl) {
  const int64_t ctas = n_items + (suffix ? (int64_t)p.n_sitems * p.n_kv * ((p.g + kRows - 1) / kRows) : 0);
  if (ctas <= 0) return cudaSuccess;
  if (ctas > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  const int smem = generic_smem(p.d);
  return with_vpl(p.d, [&](auto vpl) {
    constexpr int n = decltype(vpl)::value;
    auto kernel = dtype == 1 ? packed_generic_kernel<BITS, __nv_bfloat16, n> : packed_generic_kernel<BITS, float, n>;
    cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)ctas), dim3(generic_warps(32 * n) * 32), (size_t)smem, s, pdl, p, first_item, n_items);
  });
}

}  // namespace
}  // namespace granikv
