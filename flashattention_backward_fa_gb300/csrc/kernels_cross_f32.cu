// Cross attention on the CUDA cores, in fp32 (d <= 128), forward and backward.
//
//   S = scale q k^T over the keys j < k_len, O = softmax(S) V, L = log sum exp S
//   P = exp(S - L), dP = dO V^T, dS = P o (dP - D), D = rowsum(dO o O)
//   dQ = scale dS K;  dV = sum P^T dO, dK = scale sum dS^T Q over a group's heads
//
// fp32 needs about 1e-7 relative accuracy, which the tf32 tensor-core kind cannot
// give, so the products are FFMA. A block holds 32 rows (query rows of a group of heads;
// keys in the dK/dV kernel) and walks 64 columns at a time (keys; query rows).
// 128 threads as 8 x 16: a thread has 4 x 4 of the 32 x 64 products (rows ty + 8 i,
// columns tx + 16 j, both operands read in 16-byte pieces of rows DP + 4 floats
// apart, which no two threads of a quarter warp have in the same bank) and 4 rows x
// DP / 16 columns of the 32 x DP sums. Rows and columns past a sequence's length are
// zeros in shared memory, so nothing of what lies there reaches a product.
//
// Bound by the FFMA pipe and the staging between barriers: 1x32/8 2048x2048x64 933 us forward
// (37 TFLOP/s), 3215 us backward (37); 2x8 1024x1024x128 267 and 1235 us (32 and 24 TFLOP/s). Small
// calls are bound by their launches (2 + 3 us for 1x2 128x77x64 on the GPU).
#include "fa_cross.h"
#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kRows = 32, kCols = 64, kThreads = 128;
constexpr int kPad = kCols + 4;  // floats between the rows of a 32 x 64 tile

template <int DP>
struct Tile {
  static constexpr int kApart = DP + 4;  // floats between rows
  static constexpr int bytes(int rows) { return rows * kApart * 4; }
};

// Where a row of a (batch, head) is in its tensor: the rows of one key head, or those of all query heads of its
// group, the heads of a query side by side (so that few queries fill a tile, the real ones are the first, and
// keys are read once for a group).
struct KeyRows {
  int64_t at, n;
  __device__ __forceinline__ KeyRows(const fa_strides& st, int b, int h, int first)
      : at(b * st.b + h * st.h + first * st.n), n(st.n) {}
  __device__ __forceinline__ int64_t operator()(int r) const { return at + r * n; }
};
struct GroupRows {
  int64_t at, n, h;
  int first, G;
  __device__ __forceinline__ GroupRows(const fa_strides& st, int b, int hk, int G_, int first_)
      : at(b * st.b + (int64_t)(hk * G_) * st.h), n(st.n), h(st.h), first(first_), G(G_) {}
  __device__ __forceinline__ int64_t operator()(int r) const {
    const int t = (first + r) / G;
    return at + t * n + (first + r - t * G) * h;
  }
};

// Rows [0, rows) of a tensor (d values each) to shared memory as [kMost][DP], zeros past `rows` and d; by
// 16 bytes where the tensor's strides allow it (vec), all of a thread's loads under way at once.
template <int DP, int kMost, typename Rows>
__device__ __forceinline__ void stage(float* to, const void* tensor, const Rows& row, int rows, int d, bool vec) {
  const float* from = static_cast<const float*>(tensor);
  if (vec) {
    constexpr int kEach = kMost * DP / 4 / kThreads;
    float4 v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int x = threadIdx.x + i * kThreads, r = x / (DP / 4), e = 4 * (x % (DP / 4));
      v[i] = r < rows && e < d ? *reinterpret_cast<const float4*>(from + row(r) + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int x = threadIdx.x + i * kThreads, r = x / (DP / 4), e = 4 * (x % (DP / 4));
      *reinterpret_cast<float4*>(to + r * Tile<DP>::kApart + e) = v[i];
    }
    return;
  }
#pragma unroll 8
  for (int x = threadIdx.x; x < kMost * DP; x += kThreads) {
    const int r = x / DP, e = x - r * DP;
    to[r * Tile<DP>::kApart + e] = r < rows && e < d ? from[row(r) + e] : 0.f;
  }
}

__device__ __forceinline__ bool vec_rows(const CrossParams& p, const fa_strides& st) {
  return ((p.d | (int)(st.b & 3) | (int)(st.n & 3) | (int)(st.h & 3)) & 3) == 0;
}

// s[i][j] = row ty + 8 i of a . row tx + 16 j of b.
template <int DP>
__device__ __forceinline__ void rows_by_rows(const float* a, const float* b, float (&s)[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  uint64_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
#pragma unroll 4
  for (int e = 0; e < DP; e += 4) {
    uint64_t x[4][2], y[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(a + (ty + 8 * i) * Tile<DP>::kApart + e);
      const float4 w = *reinterpret_cast<const float4*>(b + (tx + 16 * i) * Tile<DP>::kApart + e);
      x[i][0] = f2_pack(u.x, u.y), x[i][1] = f2_pack(u.z, u.w);
      y[i][0] = f2_pack(w.x, w.y), y[i][1] = f2_pack(w.z, w.w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f2_fma(x[i][1], y[j][1], f2_fma(x[i][0], y[j][0], acc[i][j]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      f2_unpack(acc[i][j], lo, hi);
      s[i][j] = lo + hi;
    }
}

// acc[i][c] += sum over the columns x of row ty + 8 i of w (32 x 64) times row x of b; a thread's columns
// of DP are 4 tx + 64 c ..  + 3 (as two pairs).
template <int DP>
__device__ __forceinline__ void weights_by_rows(const float* w, const float* b, uint64_t (&acc)[4][DP / 64][2]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
  for (int x = 0; x < kCols; x += 4) {
    float f[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(w + (ty + 8 * i) * kPad + x);
      f[i][0] = u.x, f[i][1] = u.y, f[i][2] = u.z, f[i][3] = u.w;
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(b + (x + y) * Tile<DP>::kApart + 4 * tx + 64 * c);
        const uint64_t lo = f2_pack(v.x, v.y), hi = f2_pack(v.z, v.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t ff = f2_pack(f[i][y], f[i][y]);
          acc[i][c][0] = f2_fma(ff, lo, acc[i][c][0]);
          acc[i][c][1] = f2_fma(ff, hi, acc[i][c][1]);
        }
      }
  }
}

// A thread's 4 x 4 into a 32 x 64 tile.
__device__ __forceinline__ void put_tile(float* to, const float (&s)[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) to[(ty + 8 * i) * kPad + tx + 16 * j] = s[i][j];
}

// A thread's sums of row ty + 8 i, times mul, to `to` (a row of d values).
template <int DP>
__device__ __forceinline__ void put_row(float* to, const uint64_t (&acc)[DP / 64][2], float mul, int d) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c) {
    float v[4];
    f2_unpack(acc[c][0], v[0], v[1]);
    f2_unpack(acc[c][1], v[2], v[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * (threadIdx.x & 15) + 64 * c + e < d) to[4 * (threadIdx.x & 15) + 64 * c + e] = v[e] * mul;
  }
}

template <int DP>
__device__ __forceinline__ void clear(uint64_t (&acc)[4][DP / 64][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) acc[i][c][0] = acc[i][c][1] = 0ull;
}

// Place of row r of a group in the backward's -L and -D.
__device__ __forceinline__ int64_t stats_row(const CrossParams& p, int b, int hk, int r) {
  const int t = r / p.G;
  return ((int64_t)b * p.Hq + hk * p.G + r - t * p.G) * p.nq_pad + t;
}

// Over the 16 threads that share a row.
__device__ __forceinline__ float row_max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Grid: x the tile of the group's query rows, y key head, z batch * split.
template <int DP>
__global__ void __launch_bounds__(kThreads) cross_fwd_f32_kernel(const __grid_constant__ CrossParams p) {
  extern __shared__ __align__(16) float sm[];
  let_next_begin();
  wait_for_previous();
  float *q = sm, *k = q + kRows * Tile<DP>::kApart, *v = k + kCols * Tile<DP>::kApart;
  float* w = v + kCols * Tile<DP>::kApart;
  const int splits = p.plan.k_splits, b = blockIdx.z / splits, split = blockIdx.z - b * splits, hk = blockIdx.y;
  const int r0 = blockIdx.x * kRows, live = cross_q_len(p, b) * p.G - r0, nk = cross_k_len(p, b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int per = ((nk + kCols - 1) / kCols + splits - 1) / splits * kCols, j_end = min(nk, (split + 1) * per);
  uint64_t acc[4][DP / 64][2];
  clear<DP>(acc);
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
  if (live > 0) stage<DP, kRows>(q, p.q, GroupRows(p.q_st, b, hk, p.G, r0), live, p.d, vec_rows(p, p.q_st));
  for (int j0 = split * per; live > 0 && j0 < j_end; j0 += kCols) {
    __syncthreads();
    stage<DP, kCols>(k, p.k, KeyRows(p.k_st, b, hk, j0), j_end - j0, p.d, vec_rows(p, p.k_st));
    stage<DP, kCols>(v, p.v, KeyRows(p.v_st, b, hk, j0), j_end - j0, p.d, vec_rows(p, p.v_st));
    __syncthreads();
    float s[4][4];
    rows_by_rows<DP>(q, k, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = j0 + tx + 16 * j < j_end ? s[i][j] * p.scale_log2 : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
      const float now = fmaxf(m[i], row_max16(top));
      const float base = now == -INFINITY ? 0.f : now;  // every score so far is -inf
      const float was = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - base);
        sum += s[i][j];
      }
      l[i] = l[i] * was + row_sum<16>(sum);
      m[i] = now;
      const uint64_t f = f2_pack(was, was);
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        acc[i][c][0] = f2_mul(acc[i][c][0], f);
        acc[i][c][1] = f2_mul(acc[i][c][1], f);
      }
    }
    put_tile(w, s);
    __syncthreads();
    weights_by_rows<DP>(w, v, acc);
  }
  const long long rows = (long long)p.B * p.Nq * p.Hq;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 8 * i, t = (r0 + r) / p.G, h = hk * p.G + r0 + r - t * p.G;
    if (t >= p.Nq) continue;
    const bool has = r < live && l[i] != 0.f;  // (a NaN sum counts as there)
    const long long at = ((long long)b * p.Hq + h) * p.Nq + t;
    const float lse2 = has ? m[i] + log2f(l[i]) : -INFINITY;
    if (splits > 1) {
      if (tx == 0) p.part_lse[split * rows + at] = lse2;
      if (has)
        put_row<DP>(p.part + (split * rows + ((long long)b * p.Nq + t) * p.Hq + h) * p.d, acc[i], 1.f / l[i], p.d);
    } else {
      if (!has)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) acc[i][c][0] = acc[i][c][1] = 0ull;
      if (tx == 0) p.lse_out[at] = has ? lse2 * 0.6931471805599453f : -INFINITY;
      put_row<DP>(static_cast<float*>(p.out) + b * p.out_st.b + t * p.out_st.n + h * p.out_st.h, acc[i],
                     has ? 1.f / l[i] : 0.f, p.d);
    }
  }
}

// dQ of a tile x of a group's query rows over the keys of one split (z: batch * split).
template <int DP>
__device__ __forceinline__ void dq_block(const CrossParams& p, float* sm, int x, int hk, int z) {
  float *q = sm, *g = q + kRows * Tile<DP>::kApart, *k = g + kRows * Tile<DP>::kApart,
        *v = k + kCols * Tile<DP>::kApart, *w = v + kCols * Tile<DP>::kApart;
  const int splits = p.plan.k_splits, b = z / splits, split = z - b * splits;
  const int r0 = x * kRows, live = cross_q_len(p, b) * p.G - r0, nk = cross_k_len(p, b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int per = ((nk + kCols - 1) / kCols + splits - 1) / splits * kCols, j_end = min(nk, (split + 1) * per);
  uint64_t acc[4][DP / 64][2];
  clear<DP>(acc);
  float nl[4], nd[4];
  if (live > 0) {
    stage<DP, kRows>(q, p.q, GroupRows(p.q_st, b, hk, p.G, r0), live, p.d, vec_rows(p, p.q_st));
    stage<DP, kRows>(g, p.dout, GroupRows(p.do_st, b, hk, p.G, r0), live, p.d, vec_rows(p, p.do_st));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 8 * i;
      const int64_t at = stats_row(p, b, hk, r0 + r);
      nl[i] = r < live ? p.nL2[at] : -INFINITY;
      nd[i] = r < live ? p.nD[at] : 0.f;
    }
  }
  for (int j0 = split * per; live > 0 && j0 < j_end; j0 += kCols) {
    __syncthreads();
    stage<DP, kCols>(k, p.k, KeyRows(p.k_st, b, hk, j0), j_end - j0, p.d, vec_rows(p, p.k_st));
    stage<DP, kCols>(v, p.v, KeyRows(p.v_st, b, hk, j0), j_end - j0, p.d, vec_rows(p, p.v_st));
    __syncthreads();
    float s[4][4], dp[4][4];
    rows_by_rows<DP>(q, k, s);
    rows_by_rows<DP>(g, v, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = j0 + tx + 16 * j < j_end && nl[i] != -INFINITY
                      ? exp2f(fmaf(s[i][j], p.scale_log2, nl[i])) * (dp[i][j] + nd[i])
                      : 0.f;
    put_tile(w, s);
    __syncthreads();
    weights_by_rows<DP>(w, k, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 8 * i, t = (r0 + r) / p.G, h = hk * p.G + r0 + r - t * p.G;
    if (t >= p.Nq) continue;
    if (splits > 1) {
      if (r < live)
        put_row<DP>(p.part + (((long long)split * p.B + b) * p.Nq + t) * p.Hq * p.d + (long long)h * p.d, acc[i],
                           1.f, p.d);
    } else {
      put_row<DP>(static_cast<float*>(p.out) + b * p.out_st.b + t * p.out_st.n + h * p.out_st.h, acc[i], p.scale, p.d);
    }
  }
}

// dK and dV of a key tile x and key head hk over one split of the query steps (64 rows of the group; z: batch * split).
template <int DP>
__device__ __forceinline__ void dkdv_block(const CrossParams& p, float* sm, int x, int hk, int z) {
  float *k = sm, *v = k + kRows * Tile<DP>::kApart, *q = v + kRows * Tile<DP>::kApart,
        *g = q + kCols * Tile<DP>::kApart, *w = g + kCols * Tile<DP>::kApart, *u = w + kRows * kPad;
  const int splits = p.plan.q_splits, b = z / splits, split = z - b * splits;
  const int j0 = x * kRows, rows = cross_q_len(p, b) * p.G, nk = cross_k_len(p, b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int steps = (rows + kCols - 1) / kCols, per = (steps + splits - 1) / splits;
  const int s_end = min(steps, (split + 1) * per);
  uint64_t dk[4][DP / 64][2], dv[4][DP / 64][2];
  clear<DP>(dk);
  clear<DP>(dv);
  if (j0 < nk) {
    stage<DP, kRows>(k, p.k, KeyRows(p.k_st, b, hk, j0), nk - j0, p.d, vec_rows(p, p.k_st));
    stage<DP, kRows>(v, p.v, KeyRows(p.v_st, b, hk, j0), nk - j0, p.d, vec_rows(p, p.v_st));
  }
  for (int st = split * per; j0 < nk && st < s_end; ++st) {
    const int r0 = st * kCols;
    __syncthreads();
    stage<DP, kCols>(q, p.q, GroupRows(p.q_st, b, hk, p.G, r0), rows - r0, p.d, vec_rows(p, p.q_st));
    stage<DP, kCols>(g, p.dout, GroupRows(p.do_st, b, hk, p.G, r0), rows - r0, p.d, vec_rows(p, p.do_st));
    float nl[4], nd[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + tx + 16 * j;
      const int64_t at = stats_row(p, b, hk, r);
      nl[j] = r < rows ? p.nL2[at] : -INFINITY;
      nd[j] = r < rows ? p.nD[at] : 0.f;
    }
    __syncthreads();
    float s[4][4], dp[4][4];
    rows_by_rows<DP>(k, q, s);
    rows_by_rows<DP>(v, g, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = j0 + ty + 8 * i < nk && nl[j] != -INFINITY;
        s[i][j] = in ? exp2f(fmaf(s[i][j], p.scale_log2, nl[j])) : 0.f;
        dp[i][j] = in ? s[i][j] * (dp[i][j] + nd[j]) : 0.f;
      }
    put_tile(w, s);
    put_tile(u, dp);
    __syncthreads();
    weights_by_rows<DP>(w, g, dv);
    weights_by_rows<DP>(u, q, dk);
  }
  const long long size = (long long)p.B * p.Nk * p.Hk * p.d;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + ty + 8 * i;
    if (j >= p.Nk) continue;
    if (splits > 1) {
      if (j >= nk) continue;
      float* to = p.part_kv + 2 * split * size + (((long long)b * p.Nk + j) * p.Hk + hk) * p.d;
      put_row<DP>(to, dk[i], 1.f, p.d);
      put_row<DP>(to + size, dv[i], 1.f, p.d);
    } else {
      put_row<DP>(static_cast<float*>(p.dk) + b * p.dk_st.b + j * p.dk_st.n + hk * p.dk_st.h, dk[i], p.scale, p.d);
      put_row<DP>(static_cast<float*>(p.dv) + b * p.dv_st.b + j * p.dv_st.n + hk * p.dv_st.h, dv[i], 1.f, p.d);
    }
  }
}

// One launch for both: the blocks of dK/dV, then those of dQ.
template <int DP>
__global__ void __launch_bounds__(kThreads) cross_bwd_f32_kernel(const __grid_constant__ CrossParams p) {
  extern __shared__ __align__(16) float sm[];
  let_next_begin();
  wait_for_previous();
  const int k_tiles = (p.Nk + kRows - 1) / kRows, q_tiles = (p.Nq * p.G + kRows - 1) / kRows;
  const int kv = k_tiles * p.Hk * p.B * p.plan.q_splits;
  const bool is_kv = (int)blockIdx.x < kv;
  const int idx = is_kv ? blockIdx.x : blockIdx.x - kv, tiles = is_kv ? k_tiles : q_tiles;
  const int rest = idx / tiles, x = idx - rest * tiles, z = rest / p.Hk, hk = rest - z * p.Hk;
  if (is_kv)
    dkdv_block<DP>(p, sm, x, hk, z);
  else
    dq_block<DP>(p, sm, x, hk, z);
}

template <int DP>
cudaError_t launch_fwd_t(const CrossParams& p, cudaStream_t st) {
  constexpr int bytes = Tile<DP>::bytes(kRows + 2 * kCols) + kRows * kPad * 4;
  const cudaError_t e = allow_smem<cross_fwd_f32_kernel<DP>>(bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.Nq * p.G + kRows - 1) / kRows, p.Hk, p.B * p.plan.k_splits);
  return launch_chained(cross_fwd_f32_kernel<DP>, grid, kThreads, bytes, 1, p, st);
}

template <int DP>
cudaError_t launch_bwd_t(const CrossParams& p, cudaStream_t st) {
  constexpr int bytes = Tile<DP>::bytes(2 * kRows + 2 * kCols) + 2 * kRows * kPad * 4;
  const cudaError_t e = allow_smem<cross_bwd_f32_kernel<DP>>(bytes);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)((p.Nk + kRows - 1) / kRows) * p.Hk * p.B * p.plan.q_splits +
                           (long long)((p.Nq * p.G + kRows - 1) / kRows) * p.Hk * p.B * p.plan.k_splits;
  return launch_chained(cross_bwd_f32_kernel<DP>, dim3((unsigned)blocks), kThreads, bytes, 1, p, st);
}

}  // namespace

cudaError_t launch_cross_fwd_f32(const CrossParams& p, cudaStream_t st) {
  return p.d <= 64 ? launch_fwd_t<64>(p, st) : launch_fwd_t<128>(p, st);
}
cudaError_t launch_cross_bwd_f32(const CrossParams& p, cudaStream_t st) {
  return p.d <= 64 ? launch_bwd_t<64>(p, st) : launch_bwd_t<128>(p, st);
}

}  // namespace fa
