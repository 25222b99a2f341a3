// Cross attention: what stands before and behind its products.
//
// * preprocess: D_i = rowsum(dO o O) (or, over few keys, sum_j P_ij dP_ij, which it
//   is) and L_i, stored negated as the backward's addends, for every query row that
//   takes part (-inf and 0 elsewhere, which makes the row's probabilities 0); in fp16
//   with the norms that bound dS (cross_exponent);
// * join of the forward's splits: with their log-sum-exps l_s,
//   O = sum_s 2^(l_s - l) O_s, l = log2 sum_s 2^l_s;
// * joins of dQ and of dK, dV: sums over the splits in ascending order, so that the
//   same inputs give the same bits on every run.
//
// All are bound by memory; a thread takes 16 bytes of a 16-bit result.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

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

// A block's maxima x and y (not negative, no NaN) into those of a (batch, key head), the same in any order.
// Once a block.
__device__ __forceinline__ void put_maxima(unsigned int* to_x, float x, unsigned int* to_y, float y) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ unsigned int tops[2 * kWarps];
  const unsigned int top_x = __reduce_max_sync(0xffffffffu, __float_as_uint(x));
  const unsigned int top_y = __reduce_max_sync(0xffffffffu, __float_as_uint(y));
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    tops[threadIdx.x >> 5] = top_x;
    tops[kWarps + (threadIdx.x >> 5)] = top_y;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const unsigned int all_x = __reduce_max_sync(0xffffffffu, lane < kWarps ? tops[lane] : 0u);
  const unsigned int all_y = __reduce_max_sync(0xffffffffu, lane < kWarps ? tops[kWarps + lane] : 0u);
  if (lane == 0) atomicMax(to_x, all_x);
  if (lane == 0 && to_y != nullptr) atomicMax(to_y, all_y);
}

__global__ void __launch_bounds__(kJoinThreads) cross_clear_maxima_kernel(const __grid_constant__ CrossParams p) {
  let_next_begin();
  wait_for_previous();
  const long long n = (long long)p.B * p.Hk;
  const long long apart = (long long)gridDim.x * kJoinThreads;
  for (long long i = (long long)blockIdx.x * kJoinThreads + threadIdx.x; i < n; i += apart)
    p.maxima[i] = {0u, 0u, 0u, 0u};
}

// fp16: the maximum of |V_j|^2 over kNormRows keys of a (batch, key head). (A sum that is NaN is passed over: where V
// has one, every gradient that this scales is NaN.)
constexpr int kNormRows = 256;

template <int D>
__device__ __forceinline__ void value_norms(const CrossParams& p, int idx) {
  constexpr int kLanes = D / 8, kApart = kJoinThreads / kLanes, kRowsEach = 8;
  const int parts = (p.Nk + kNormRows - 1) / kNormRows, bh = idx / parts, b = bh / p.Hk, h = bh - b * p.Hk;
  const int begin = (idx - bh * parts) * kNormRows, end = min(cross_k_len(p, b), begin + kNormRows);
  if (begin >= end) return;
  const __half* v = static_cast<const __half*>(p.v) + b * p.v_st.b + h * p.v_st.h + 8 * (threadIdx.x % kLanes);
  float top = 0.f;
#pragma unroll 1
  for (int first = begin; first < end; first += kRowsEach * kApart) {
    Raw8<__half> rv[kRowsEach];
#pragma unroll
    for (int r = 0; r < kRowsEach; ++r) {
      const int j = first + r * kApart + threadIdx.x / kLanes;
      zero8(rv[r]);
      if (j < end) load8(rv[r], v + j * p.v_st.n);
    }
#pragma unroll
    for (int r = 0; r < kRowsEach; ++r) {
      uint64_t x[4], s0 = 0ull;
      rv[r].unpack(x);
#pragma unroll
      for (int c = 0; c < 4; ++c) s0 = f2_fma(x[c], x[c], s0);
      top = fmaxf(top, row_sum<kLanes>(f2_sum(s0)));
    }
  }
  put_maxima(&p.maxima[bh].v, top, nullptr, 0.f);
}

// 16-bit types, D = rowsum(dO o O) of the rows [row0, row0 + preprocess_rows) of one (b, h): D / 8 lanes a row, 16
// bytes of O and of dO each, four rows a thread with all their loads under way at once. (A warp a row with 2 bytes a
// lane took 34 us at 4x16x2048x128, where the copy rate allows 10.)
template <int D>
constexpr int preprocess_rows() { return kJoinThreads / (D / 8) * 4; }

template <typename T, int D>
__device__ __forceinline__ void rows_from_output(const CrossParams& p, int bh, int b, int h, int nq, int row0) {
  constexpr int kLanes = D / 8, kApart = kJoinThreads / kLanes, kRowsEach = 4;
  constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;
  const int e = 8 * (threadIdx.x % kLanes), first = row0 + threadIdx.x / kLanes;
  const T* o = static_cast<const T*>(p.o) + b * p.o_st.b + h * p.o_st.h + e;
  const T* g = static_cast<const T*>(p.dout) + b * p.do_st.b + h * p.do_st.h + e;
  Raw8<T> ro[kRowsEach], rg[kRowsEach];
#pragma unroll
  for (int r = 0; r < kRowsEach; ++r) {
    const int i = first + r * kApart;
    zero8(ro[r]);
    zero8(rg[r]);
    if (i < nq) {
      load8(ro[r], o + i * p.o_st.n);
      load8(rg[r], g + i * p.do_st.n);
    }
  }
  float most = 0.f, most_D = 0.f;
#pragma unroll
  for (int r = 0; r < kRowsEach; ++r) {
    const int i = first + r * kApart;
    uint64_t x[4], y[4], s0 = 0ull;
    ro[r].unpack(x);
    rg[r].unpack(y);
#pragma unroll
    for (int c = 0; c < 4; ++c) s0 = f2_fma(x[c], y[c], s0);
    const float acc = row_sum<kLanes>(f2_sum(s0));
    if (e == 0 && i < p.nq_pad) {
      const long long row = (long long)bh * p.nq_pad + i;
      p.nD[row] = -acc;
      p.nL2[row] = i < nq ? neg_lse2(p.lse[(long long)bh * p.Nq + i]) + kCrossPLog2<kBf16> : -INFINITY;
    }
    if constexpr (!kBf16) {
      uint64_t s1 = 0ull;
#pragma unroll
      for (int c = 0; c < 4; ++c) s1 = f2_fma(y[c], y[c], s1);
      const float norm = sqrtf(row_sum<kLanes>(f2_sum(s1)));  // (0 where there is no row, and so is acc)
      if (e == 0 && i < p.nq_pad) p.dout_norm[(long long)bh * p.nq_pad + i] = norm;
      most = fmaxf(most, norm);
      most_D = fmaxf(most_D, fabsf(acc));
    }
  }
  if constexpr (!kBf16) {
    CrossMaxima& m = p.maxima[b * p.Hk + h / p.G];
    put_maxima(&m.dout, most, &m.D, most_D);
  }
}

// 16-bit types, sequences of up to kFewKeysMost keys (real ones: a sequence's gradients do not depend on what its
// batch is padded to): D = sum_j P_ij dP_ij from the scores instead. rowsum(dO o O) has the
// rounding of O to 16 bits in it, and over a handful of keys, where O is as large as V, or a few dozen where q, k
// and v have large channels, that was the larger part of the error of dQ and dK (1.6 to 2.4 times the results' own
// rounding; 1.0 to 1.4 so). A warp takes 16 of the 128 rows [row0, ..), S and dP by m16n8k16, the block's keys and
// values in shared memory, 16-byte pieces swizzled by row. The backward of 2x16/4 4095 over 16 keys, d = 64, takes
// 53.6 us with it and 51.2 without, over 64 keys 59.6 and 51.0, 4x16 2048 over 64 keys, d = 128, 97 and 84, 1x2 128
// over 5 9.8 and 9.6; with more keys the two products cost more, and O is smaller.
constexpr int kFewKeysMost = 64;

template <int D, bool kBf16>
__device__ __forceinline__ void rows_from_scores(const CrossParams& p, int bh, int b, int h, int nq, int nk, int row0) {
  __shared__ __align__(128) uint16_t sk[kFewKeysMost * D], sv[kFewKeysMost * D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, in_quad = lane & 3;
  const int tiles = (nk + 7) / 8;
  row0 += warp * 16;
  const uint16_t* k = static_cast<const uint16_t*>(p.k) + b * p.k_st.b + h / p.G * p.k_st.h;
  const uint16_t* v = static_cast<const uint16_t*>(p.v) + b * p.v_st.b + h / p.G * p.v_st.h;
  for (int x = threadIdx.x; x < 8 * tiles * (D / 8); x += kJoinThreads) {
    const int j = x / (D / 8), piece = x % (D / 8), to = j * D + 8 * (piece ^ (j & 7));
    uint4 kv[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (j < nk) {
      kv[0] = *reinterpret_cast<const uint4*>(k + j * p.k_st.n + 8 * piece);
      kv[1] = *reinterpret_cast<const uint4*>(v + j * p.v_st.n + 8 * piece);
    }
    *reinterpret_cast<uint4*>(sk + to) = kv[0];
    *reinterpret_cast<uint4*>(sv + to) = kv[1];
  }
  // Q and dO as A operands: rows quad and quad + 8, columns 2 in_quad and + 8 of every 16 (zeros where there is none)
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.q_st.b + h * p.q_st.h + 2 * in_quad;
  const uint16_t* g = static_cast<const uint16_t*>(p.dout) + b * p.do_st.b + h * p.do_st.h + 2 * in_quad;
  uint32_t aq[D / 16][4], ag[D / 16][4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int i = row0 + quad + 8 * (x & 1);
    const uint16_t *qi = q + (i < nq ? i * p.q_st.n : 0), *gi = g + (i < nq ? i * p.do_st.n : 0);
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      const int col = 16 * st + 8 * (x >> 1);
      aq[st][x] = i < nq ? *reinterpret_cast<const uint32_t*>(qi + col) : 0u;
      ag[st][x] = i < nq ? *reinterpret_cast<const uint32_t*>(gi + col) : 0u;
    }
  }
  float nl[2], acc[2] = {0.f, 0.f};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = row0 + quad + 8 * half;
    nl[half] = i < nq ? neg_lse2(p.lse[(long long)bh * p.Nq + i]) : -INFINITY;
  }
  __syncthreads();
  const int mat = lane >> 3, mrow = lane & 7;  // ldmatrix: lane i gives the address of row i % 8 of matrix i / 8
  for (int n = 0; n < tiles; ++n) {
    float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int st = 0; st < D / 32; ++st) {
      uint32_t kb[4], vb[4];
      const int at = (8 * n + mrow) * D + 8 * ((4 * st + mat) ^ mrow);
      ldmatrix4(kb, smem_u32(sk + at));
      ldmatrix4(vb, smem_u32(sv + at));
      mma16816<kBf16>(s, aq[2 * st], kb[0], kb[1]);
      mma16816<kBf16>(dp, ag[2 * st], vb[0], vb[1]);
      mma16816<kBf16>(s, aq[2 * st + 1], kb[2], kb[3]);
      mma16816<kBf16>(dp, ag[2 * st + 1], vb[2], vb[3]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (nl[e >> 1] != -INFINITY && 8 * n + 2 * in_quad + (e & 1) < nk)
        acc[e >> 1] = fmaf(exp2f(fmaf(s[e], p.scale_log2, nl[e >> 1])), dp[e], acc[e >> 1]);
  }
  float most = 0.f, most_D = 0.f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    acc[half] += __shfl_xor_sync(0xffffffffu, acc[half], 1);
    acc[half] += __shfl_xor_sync(0xffffffffu, acc[half], 2);
    const long long row = (long long)bh * p.nq_pad + row0 + quad + 8 * half;
    const bool there = in_quad == 0 && row0 + quad + 8 * half < p.nq_pad;
    if (there) {
      p.nD[row] = -acc[half];
      p.nL2[row] = nl[half] + kCrossPLog2<kBf16>;
    }
    if constexpr (!kBf16) {
      float square = 0.f;
#pragma unroll
      for (int st = 0; st < D / 16; ++st)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float lo, hi;
          unpack2<kBf16>(ag[st][half + 2 * x], lo, hi);
          square = fmaf(lo, lo, fmaf(hi, hi, square));
        }
      square += __shfl_xor_sync(0xffffffffu, square, 1);
      square += __shfl_xor_sync(0xffffffffu, square, 2);
      const float norm = sqrtf(square);  // (0 where there is no row, and so is acc)
      if (there) p.dout_norm[row] = norm;
      most = fmaxf(most, norm);
      most_D = fmaxf(most_D, fabsf(acc[half]));
    }
  }
  if constexpr (!kBf16) {
    CrossMaxima& m = p.maxima[b * p.Hk + h / p.G];
    put_maxima(&m.dout, most, &m.D, most_D);
  }
}

// kForm: the form of all of the call's sequences, or of those whose length calls for it (kByLength; the others' blocks
// leave); kEither: each block its sequence's.
enum PreprocessForm { kScores, kOutput, kEither };

template <int D, bool kBf16, PreprocessForm kForm, bool kByLength>
__global__ void __launch_bounds__(kJoinThreads) cross_preprocess_kernel(const __grid_constant__ CrossParams p) {
  using T = std::conditional_t<kBf16, __nv_bfloat16, __half>;
  constexpr int kRows = kForm == kOutput ? preprocess_rows<D>() : 128;
  static_assert(kForm != kEither || preprocess_rows<D>() == 128, "a block has the same rows in both forms");
  let_next_begin();
  wait_for_previous();
  const int blocks = (p.nq_pad + kRows - 1) / kRows, all = p.B * p.Hq * blocks;
  if constexpr (!kBf16) {  // (the blocks behind those of the rows)
    if ((int)blockIdx.x >= all) {
      value_norms<D>(p, blockIdx.x - all);
      return;
    }
  }
  const int bh = blockIdx.x / blocks, b = bh / p.Hq, h = bh - b * p.Hq;
  const int nq = cross_q_len(p, b), nk = cross_k_len(p, b), row0 = (blockIdx.x - bh * blocks) * kRows;
  const bool scores = kByLength ? nk <= kFewKeysMost : kForm == kScores;
  if (scores && kForm != kOutput) rows_from_scores<D, kBf16>(p, bh, b, h, nq, nk, row0);
  if (!scores && kForm != kScores) rows_from_output<T, D>(p, bh, b, h, nq, row0);
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

template <int D, bool kBf16>
cudaError_t launch_preprocess(const CrossParams& p, cudaStream_t st) {
  const long long norms = kBf16 ? 0 : (long long)p.B * p.Hk * ((p.Nk + kNormRows - 1) / kNormRows);
  const auto launch = [&](auto kernel, int rows, long long more) {
    const long long blocks = (long long)p.B * p.Hq * ((p.nq_pad + rows - 1) / rows) + more;
    return launch_chained(kernel, dim3((unsigned)blocks), kJoinThreads, 0, 1, p, st);
  };
  if (!kBf16) {
    const long long blocks = ((long long)p.B * p.Hk + kJoinThreads - 1) / kJoinThreads;
    const cudaError_t e = launch_chained(cross_clear_maxima_kernel, dim3((unsigned)(blocks < 152 ? blocks : 152)),
                                         kJoinThreads, 0, 1, p, st);
    if (e != cudaSuccess) return e;
  }
  if (p.Nk <= kFewKeysMost) return launch(cross_preprocess_kernel<D, kBf16, kScores, false>, 128, norms);
  if (!p.k_lens) return launch(cross_preprocess_kernel<D, kBf16, kOutput, false>, preprocess_rows<D>(), norms);
  // One kernel for both with d = 64, two with d = 128, where the scores' 118 registers leave two blocks an SM
  // (backward, us, one / two kernels: 4x16 2048 over 512, d = 64, 96 / 96, with short sequences among them 78 / 80,
  // 2x16/4 4095 over 77 54 / 56; d = 128 136 / 125, 113 / 113 and 91 / 93).
  if constexpr (D == 64) {
    return launch(cross_preprocess_kernel<D, kBf16, kEither, true>, 128, norms);
  } else {
    const cudaError_t e = launch(cross_preprocess_kernel<D, kBf16, kScores, true>, 128, 0);
    return e == cudaSuccess ? launch(cross_preprocess_kernel<D, kBf16, kOutput, true>, preprocess_rows<D>(), norms) : e;
  }
}

}  // namespace

cudaError_t launch_cross_preprocess(const CrossParams& p, int dtype, cudaStream_t st) {
  const long long heads = (long long)p.B * p.Hq;
  if (dtype == FA_F32) {
    const long long blocks = (heads * p.nq_pad + 7) / 8;
    return launch_chained(cross_preprocess_f32_kernel, dim3((unsigned)(blocks < 152 * 32 ? blocks : 152 * 32)),
                          kJoinThreads, 0, 1, p, st);
  }
  if (p.d == 64) return dtype == FA_BF16 ? launch_preprocess<64, true>(p, st) : launch_preprocess<64, false>(p, st);
  return dtype == FA_BF16 ? launch_preprocess<128, true>(p, st) : launch_preprocess<128, false>(p, st);
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
