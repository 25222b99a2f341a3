// Cross attention: what stands before and behind its products.
//
// * fp32 preprocess: D_i = rowsum(dO o O) and L_i, stored negated as the backward's
//   addends, for every query row that takes part (-inf and 0 elsewhere, which makes
//   the row's probabilities 0);
// * join of the forward's splits: with their log-sum-exps l_s,
//   O = sum_s 2^(l_s - l) O_s, l = log2 sum_s 2^l_s;
// * joins of dQ and of dK, dV: sums over the splits in ascending order, so that the
//   same inputs give the same bits on every run.
//
// All are bound by memory; a thread takes 16 bytes of a 16-bit result.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fa_cross.h"
#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kJoinThreads = 256;

// -L * log2(e) of a real row (a row without keys: -inf).
__device__ __forceinline__ float neg_lse2(float l) { return l == -INFINITY ? l : -(l * 1.4426950408889634f); }

// fp32, any d: one warp a query row (b, h, i), i fastest over the padded rows.
__global__ void __launch_bounds__(kJoinThreads) cross_preprocess_f32_kernel(const __grid_constant__ CrossParams p) {
  let_next_begin();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.B * p.Hq * p.nq_pad, apart = (long long)gridDim.x * (kJoinThreads / 32);
  for (long long row = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5); row < rows; row += apart) {
    const long long bh = row / p.nq_pad;
    const int i = (int)(row - bh * p.nq_pad), b = (int)(bh / p.Hq), h = (int)(bh - (long long)b * p.Hq);
    float acc = 0.f, nl = -INFINITY;
    if (i < cross_q_len(p, b)) {
      const float* o = static_cast<const float*>(p.o) + b * p.o_st.b + i * p.o_st.n + h * p.o_st.h;
      const float* g = static_cast<const float*>(p.dout) + b * p.do_st.b + i * p.do_st.n + h * p.do_st.h;
      for (int e = lane; e < p.d; e += 32) acc = fmaf(o[e], g[e], acc);
      acc = row_sum<32>(acc);
      nl = neg_lse2(p.lse[bh * p.Nq + i]);
    }
    if (lane == 0) {
      p.nD[row] = -acc;
      p.nL2[row] = nl;
    }
  }
}

// Four consecutive values as T.
template <typename T>
__device__ __forceinline__ void store4(T* to, const float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) to[e] = static_cast<T>(v[e]);
}
template <>
__device__ __forceinline__ void store4<__half>(__half* to, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(to) = make_uint2(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]));
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* to, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(to) = make_uint2(pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3]));
}

// Four values of a split's row (d is a multiple of 4 for 16-bit types; fp32 rows of any d by single values).
__device__ __forceinline__ void load_part(const float* from, int left, bool vec, float (&v)[4]) {
  if (vec) {
    const float4 a = *reinterpret_cast<const float4*>(from);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < left ? from[e] : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store_row(T* to, int left, const float (&v)[4]) {
  if (left >= 4) {
    store4(to, v);
  } else {
    for (int e = 0; e < left; ++e) to[e] = static_cast<T>(v[e]);
  }
}

// kWide warps take a row (b, t, h) of [B, Nq, Hq, d], each every kWide-th split: a lane has one split's weight and
// four values (lanes past d / 4 none), and eight splits' loads are under way at once. (A thread a
// row piece with the splits one after the other took 45 us for 32 rows of 76 splits, one load's latency each.)
template <typename T, int kWide>
__global__ void __launch_bounds__(kJoinThreads) cross_join_fwd_kernel(const __grid_constant__ CrossParams p) {
  constexpr int kRowsBlock = kJoinThreads / 32 / kWide;
  __shared__ __align__(16) float part_sum[kJoinThreads / 32][128];
  let_next_begin();
  wait_for_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp % kWide;
  const long long rows = (long long)p.B * p.Nq * p.Hq, row = (long long)blockIdx.x * kRowsBlock + warp / kWide;
  const bool vec = (p.d & 3) == 0, in = row < rows;
  const long long bt = row / p.Hq;
  const int h = (int)(row - bt * p.Hq), b = (int)(bt / p.Nq), t = (int)(bt - (long long)b * p.Nq), e = 4 * lane;
  const long long at = ((long long)b * p.Hq + h) * p.Nq + t;
  const int n = p.plan.k_splits;
  float m = -INFINITY, sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
  if (in) {
    for (int s = lane; s < n; s += 32) m = fmaxf(m, p.part_lse[s * rows + at]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  for (int s0 = 0; s0 < n; s0 += 32) {  // 32 splits' weights, one a lane
    const int s = s0 + lane;
    const float w = in && s < n ? exp2f(p.part_lse[s * rows + at] - base) : 0.f;
    sum += row_sum<32>(w);
#pragma unroll 1
    for (int y0 = mine; y0 < 32 && s0 + y0 < n; y0 += 8 * kWide) {
      float a[8][4], f[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const int from = y0 + y * kWide;
        f[y] = __shfl_sync(0xffffffffu, w, from & 31);
        if (from >= 32 || s0 + from >= n) f[y] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[y][i] = 0.f;
        if (f[y] != 0.f && e < p.d)  // (without keys a split has no output there)
          load_part(p.part + ((long long)(s0 + from) * rows + row) * p.d + e, p.d - e, vec, a[y]);
      }
#pragma unroll
      for (int y = 0; y < 8; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(f[y], a[y][i], v[i]);
    }
  }
  if (kWide > 1) {
    *reinterpret_cast<float4*>(&part_sum[warp][e]) = make_float4(v[0], v[1], v[2], v[3]);
    __syncthreads();
    if (mine != 0) return;
#pragma unroll
    for (int w = 1; w < kWide; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += part_sum[warp + w][e + i];
  }
  if (!in) return;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;  // (a NaN sum is there)
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= inv;
  if (e < p.d) store_row(static_cast<T*>(p.out) + b * p.out_st.b + t * p.out_st.n + h * p.out_st.h + e, p.d - e, v);
  if (lane == 0) p.lse_out[at] = sum != 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Sums over the splits of [splits][.., N, H, d] from `part`, `apart` floats between
// splits, times `mul`; rows from their sequence's length on get zeros.
template <typename T, bool kKeys>
__device__ __forceinline__ void join_rows(const CrossParams& p, const float* part, long long apart, int splits, int N,
                                          int H, void* out, const fa_strides& st, float mul) {
  const int quads = (p.d + 3) >> 2;
  const long long n = (long long)p.B * N * H * quads;
  const bool vec = (p.d & 3) == 0;
  const long long apart_x = (long long)gridDim.x * kJoinThreads;
  for (long long x = (long long)blockIdx.x * kJoinThreads + threadIdx.x; x < n; x += apart_x) {
    const long long row = x / quads, bt = row / H;
    const int e = 4 * (int)(x - row * quads), h = (int)(row - bt * H), b = (int)(bt / N);
    const int t = (int)(bt - (long long)b * N);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (t < (kKeys ? cross_k_len(p, b) : cross_q_len(p, b))) {
      // (in order; eight loads under way at once)
      for (int s0 = 0; s0 < splits; s0 += 8) {
        float a[8][4];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
#pragma unroll
          for (int i = 0; i < 4; ++i) a[s][i] = 0.f;
          if (s0 + s < splits) load_part(part + (s0 + s) * apart + row * p.d + e, p.d - e, vec, a[s]);
        }
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += a[s][i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= mul;
    }
    store_row(static_cast<T*>(out) + b * st.b + t * st.n + h * st.h + e, p.d - e, v);
  }
}

// y: 0 dQ, 1 dK, 2 dV, as far as they are in splits.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) cross_join_bwd_kernel(const __grid_constant__ CrossParams p) {
  let_next_begin();
  wait_for_previous();
  if (blockIdx.y == 0) {
    if (p.plan.k_splits > 1)
      join_rows<T, false>(p, p.part, (long long)p.B * p.Nq * p.Hq * p.d, p.plan.k_splits, p.Nq, p.Hq, p.out, p.out_st,
                          p.scale);
    return;
  }
  if (p.plan.q_splits == 1) return;
  const long long size = (long long)p.B * p.Nk * p.Hk * p.d;
  const bool is_v = blockIdx.y == 2;
  join_rows<T, true>(p, p.part_kv + (is_v ? size : 0), 2 * size, p.plan.q_splits, p.Nk, p.Hk, is_v ? p.dv : p.dk,
                     is_v ? p.dv_st : p.dk_st, is_v ? 1.f : p.scale);
}

int join_blocks(const CrossParams& p, int N, int H) {
  const long long n = (long long)p.B * N * H * ((p.d + 3) / 4);
  const long long blocks = (n + kJoinThreads - 1) / kJoinThreads;
  return (int)(blocks < 152 * 16 ? blocks : 152 * 16);
}

}  // namespace

cudaError_t launch_cross_preprocess_f32(const CrossParams& p, cudaStream_t st) {
  const long long blocks = ((long long)p.B * p.Hq * p.nq_pad + 7) / 8;
  return launch_chained(cross_preprocess_f32_kernel, dim3((unsigned)(blocks < 152 * 32 ? blocks : 152 * 32)),
                        kJoinThreads, 0, 1, p, st);
}

template <typename T>
static cudaError_t launch_join_fwd(const CrossParams& p, cudaStream_t st) {
  const long long rows = (long long)p.B * p.Nq * p.Hq;
  const int n = p.plan.k_splits;
  if (n > 16) return launch_chained(cross_join_fwd_kernel<T, 8>, dim3((unsigned)rows), kJoinThreads, 0, 1, p, st);
  if (n > 8)
    return launch_chained(cross_join_fwd_kernel<T, 2>, dim3((unsigned)((rows + 3) / 4)), kJoinThreads, 0, 1, p, st);
  return launch_chained(cross_join_fwd_kernel<T, 1>, dim3((unsigned)((rows + 7) / 8)), kJoinThreads, 0, 1, p, st);
}

cudaError_t launch_cross_join_fwd(const CrossParams& p, int dtype, cudaStream_t st) {
  if (dtype == FA_F32) return launch_join_fwd<float>(p, st);
  return dtype == FA_BF16 ? launch_join_fwd<__nv_bfloat16>(p, st) : launch_join_fwd<__half>(p, st);
}

cudaError_t launch_cross_join_bwd(const CrossParams& p, int dtype, cudaStream_t st) {
  const dim3 grid(std::max(p.plan.k_splits > 1 ? join_blocks(p, p.Nq, p.Hq) : 1,
                           p.plan.q_splits > 1 ? join_blocks(p, p.Nk, p.Hk) : 1),
                  3);
  if (dtype == FA_F32) return launch_chained(cross_join_bwd_kernel<float>, grid, kJoinThreads, 0, 1, p, st);
  return dtype == FA_BF16 ? launch_chained(cross_join_bwd_kernel<__nv_bfloat16>, grid, kJoinThreads, 0, 1, p, st)
                          : launch_chained(cross_join_bwd_kernel<__half>, grid, kJoinThreads, 0, 1, p, st);
}

}  // namespace fa
