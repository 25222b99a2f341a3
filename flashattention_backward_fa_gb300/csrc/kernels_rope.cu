// Per-head RMS norm of queries and keys with their position rotation, forward
// and backward (the formulas and the lane layout: rope_common.cuh).
//
// Backward, with dy = R(pos)^T dout, xn = x r, g = w o dy:
//   dx = r (g - xn mean(g o xn));  dw = sum over rows of dy o xn
// r is formed again from x, which the backward reads anyway, so nothing but
// the inputs is kept between the two passes. dw: every lane keeps the sums of
// its eight columns over its rows, a block adds its lanes' sums in a fixed
// order into one row of the workspace, and a second kernel adds the blocks'
// rows in a fixed order, so the gradients are the same bits on every run.
//
// Both are bound by memory: about 30 (forward) and 80 (backward) operations an
// element against 4 and 6 bytes. The row is in registers between its one load
// and its one store, and every lane has several rows' loads in flight.
#include <algorithm>

#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kFwdRows = 4;  // consecutive rows a row group of the forward takes
constexpr int kBwdRows = 2;  // rows a row group of the backward loads at a time
constexpr int kBwdBlocks = 152 * 3;  // most blocks of the backward (and rows of partial weight gradients)

// Row `row` of a [B, N, H] enumeration; next() moves to the row after it. The
// divisions are 32-bit wherever the row number is (a 64-bit division costs as
// much as the rest of a row's index arithmetic together).
struct RowAt {
  long long b;
  int n, head;
  __device__ __forceinline__ RowAt(long long row, int N, int H) {
    long long token;
    if (row >> 32) {
      token = row / H;
      b = token / N;
    } else {
      token = (unsigned)row / (unsigned)H;
      b = (unsigned)token / (unsigned)N;
    }
    head = (int)(row - token * H);
    n = (int)(token - b * N);
  }
  __device__ __forceinline__ void next(int N, int H) {
    if (++head < H) return;
    head = 0;
    if (++n < N) return;
    n = 0;
    ++b;
  }
  __device__ __forceinline__ long long offset(const fa_strides& st) const {
    return b * st.b + (long long)n * st.n + (long long)head * st.h;
  }
};

// The token's row in the tables: its position, clamped into them.
__device__ __forceinline__ long long table_row(const RopeParams& p, const RowAt& a) {
  const int pos = p.positions ? __ldg(p.positions + a.b * p.pos_stride + a.n) : a.n;
  return (long long)min(max(pos, 0), p.max_pos - 1) * (p.rot >> 1);
}

template <typename T, int D, bool kNeighbours>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int G = D / 8;
  const int lane = threadIdx.x & 31, e0 = (lane % G) * 8;
  const bool is_k = blockIdx.x >= (unsigned)p.q_blocks;
  const RopeSide& sd = is_k ? p.k : p.q;
  const long long rows = (long long)p.B * p.N * sd.H;
  const long long first =
      ((long long)(blockIdx.x - (is_k ? p.q_blocks : 0)) * (kRopeThreads / G) + threadIdx.x / G) * kFwdRows;
  const int partner = partner_lane<kNeighbours>(lane, e0, p.rot);
  Raw8<T> raw[kFwdRows];
  RowAt a(first, p.N, sd.H);
  const RowAt a0 = a;
#pragma unroll
  for (int r = 0; r < kFwdRows; ++r) {
    raw[r].zero();
    if (first + r < rows) raw[r].load(static_cast<const T*>(sd.x) + a.offset(sd.x_st) + e0);
    a.next(p.N, sd.H);
  }
  float w[8], w_p[8], c[8], s[8];
  load_weight8<T>(sd.w, p.w_f32, e0, w);
  load_weight8<T>(sd.w, p.w_f32, (partner % G) * 8, w_p);
  a = a0;
#pragma unroll
  for (int r = 0; r < kFwdRows; ++r) {
    const bool live = first + r < rows;
    if (r == 0 || a.head == 0) {  // a new token
      const long long at = live && p.rot ? table_row(p, a) : 0;
      load_rotation<kNeighbours>(p.cos + at, p.sin + at, e0, live ? p.rot : 0, c, s);
    }
    float out[8];
    norm_rope_chunk<T, D, kNeighbours>(raw[r], partner, w, w_p, c, s, p.eps, out);
    if (live) {
      raw[r].pack(out);
      raw[r].store(static_cast<T*>(sd.out) + a.offset(sd.out_st) + e0);
    }
    a.next(p.N, sd.H);
  }
}

template <typename T, int D, bool kNeighbours>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int G = D / 8, kGroups = kRopeThreads / G;
  __shared__ float sums[kGroups][D];
  const int lane = threadIdx.x & 31, e0 = (lane % G) * 8, group = threadIdx.x / G;
  const bool is_k = blockIdx.x >= (unsigned)p.q_blocks;
  const RopeSide& sd = is_k ? p.k : p.q;
  const int blk = blockIdx.x - (is_k ? p.q_blocks : 0), blks = is_k ? gridDim.x - p.q_blocks : p.q_blocks;
  const long long rows = (long long)p.B * p.N * sd.H;
  const int partner = partner_lane<kNeighbours>(lane, e0, p.rot);
  float w[8], dw[8], c[8], s[8];
  load_weight8<T>(sd.w, p.w_f32, e0, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  const long long step = (long long)blks * kGroups * kBwdRows;
  // every lane of a warp runs the same number of turns (the shuffles need all of them)
  for (long long base = (long long)blk * kGroups * kBwdRows; base < rows; base += step) {
    const long long first = base + (long long)group * kBwdRows;
    Raw8<T> raw[kBwdRows], grad[kBwdRows];
    RowAt a(first, p.N, sd.H);
    const RowAt a0 = a;
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r) {
      raw[r].zero();
      grad[r].zero();
      if (first + r < rows) {
        raw[r].load(static_cast<const T*>(sd.x) + a.offset(sd.x_st) + e0);
        grad[r].load(static_cast<const T*>(sd.dout) + a.offset(sd.out_st) + e0);
      }
      a.next(p.N, sd.H);
    }
    a = a0;
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r) {
      const bool live = first + r < rows;
      if (r == 0 || a.head == 0) {  // a new token
        const long long at = live && p.rot ? table_row(p, a) : 0;
        load_rotation<kNeighbours>(p.cos + at, p.sin + at, e0, live ? p.rot : 0, c, s);
      }
      float x[8], g[8], dy[8];
      raw[r].unpack(x);
      grad[r].unpack(g);
      if (kNeighbours) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[i] = fmaf(g[i], c[i], -g[i ^ 1] * s[i]);
      } else {
        float gp[8];
        grad[r].from_lane(partner).unpack(gp);
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[i] = fmaf(g[i], c[i], -gp[i] * s[i]);
      }
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(x[i], x[i], ss);
        gx = fmaf(dy[i] * w[i], x[i], gx);
      }
      ss = row_sum<G>(ss);
      gx = row_sum<G>(gx);
      const float rr = rsqrtf(fmaf(ss, 1.f / D, p.eps));
      const float k1 = gx * (1.f / D) * rr;  // mean(g o xn)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xn = x[i] * rr;
        dw[i] = fmaf(dy[i], xn, dw[i]);
        g[i] = rr * fmaf(-xn, k1, dy[i] * w[i]);
      }
      if (live) {
        raw[r].pack(g);
        raw[r].store(static_cast<T*>(sd.dx) + a.offset(sd.dx_st) + e0);
      }
      a.next(p.N, sd.H);
    }
  }
  if (sd.w == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[group][e0 + i] = dw[i];
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kRopeThreads) {
    float t = 0.f;
#pragma unroll 8
    for (int g = 0; g < kGroups; ++g) t += sums[g][e];
    p.part[(long long)blockIdx.x * D + e] = t;
  }
}

// Adds the blocks' partial weight gradients: block x = side (q, k), eight
// warps that take every eighth row, one column a lane.
template <typename T>
__global__ void __launch_bounds__(256) weight_grad_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float sums[8][32];
  const bool is_k = blockIdx.x != 0;
  const RopeSide& sd = is_k ? p.k : p.q;
  if (sd.w == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.y * 32 + lane;
  const int lo = is_k ? p.q_blocks : 0, hi = is_k ? p.blocks : p.q_blocks;
  float t = 0.f;
  if (e < p.d) {
#pragma unroll 8
    for (int r = lo + warp; r < hi; r += 8) t += p.part[(long long)r * p.d + e];
  }
  sums[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && e < p.d) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sums[i][lane];
    if (p.w_f32)
      static_cast<float*>(sd.dw)[e] = t;
    else
      static_cast<T*>(sd.dw)[e] = static_cast<T>(t);
  }
}

// fp32 with any d <= 128, any even rot and any strides: one warp a row, lane
// l holding the values l, l + 32, ...; the row passes through shared memory for
// the partners' values. kBackward adds the gradients as above (dw: lane sums,
// then the warps' in order). Rows of a block: eight warps, strided over the grid.
template <bool kBackward>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_any_f32_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float buf[8][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = p.d, h = p.rot >> 1;
  const bool is_k = blockIdx.x >= (unsigned)p.q_blocks;
  const RopeSide& sd = is_k ? p.k : p.q;
  const int blk = blockIdx.x - (is_k ? p.q_blocks : 0), blks = is_k ? gridDim.x - p.q_blocks : p.q_blocks;
  const long long rows = (long long)p.B * p.N * sd.H;
  const float* wv = static_cast<const float*>(sd.w);
  float dw[4] = {0.f, 0.f, 0.f, 0.f};
  for (long long row = (long long)blk * 8 + warp; row < rows; row += (long long)blks * 8) {
    const RowAt a(row, p.N, sd.H);
    const float* x = static_cast<const float*>(sd.x) + a.offset(sd.x_st);
    const long long at = p.rot ? table_row(p, a) : 0;
    float xv[4], gv[4], ss = 0.f;
    const float* go = kBackward ? static_cast<const float*>(sd.dout) + a.offset(sd.out_st) : nullptr;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = lane + 32 * j;
      xv[j] = e < d ? x[e] : 0.f;
      gv[j] = kBackward && e < d ? go[e] : 0.f;
      ss = fmaf(xv[j], xv[j], ss);
    }
    ss = row_sum<32>(ss);
    const float r = rsqrtf(ss / d + p.eps);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = lane + 32 * j;
      if (e < d) buf[warp][e] = kBackward ? gv[j] : xv[j] * r * (wv ? wv[e] : 1.f);
    }
    __syncwarp();
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = lane + 32 * j;
      y[j] = 0.f;
      if (e >= d) continue;
      y[j] = buf[warp][e];
      if (e < p.rot) {
        const int pair = p.neighbours ? e >> 1 : (e < h ? e : e - h);
        const int other = p.neighbours ? e ^ 1 : (e < h ? e + h : e - h);
        const bool low = p.neighbours ? (e & 1) == 0 : e < h;
        const float c = p.cos[at + pair], s = low == kBackward ? p.sin[at + pair] : -p.sin[at + pair];
        y[j] = fmaf(y[j], c, buf[warp][other] * s);
      }
    }
    __syncwarp();
    if (!kBackward) {
      float* o = static_cast<float*>(sd.out) + a.offset(sd.out_st);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < d) o[lane + 32 * j] = y[j];
    } else {
      float gx = 0.f, g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = lane + 32 * j;
        g[j] = e < d ? y[j] * (wv ? wv[e] : 1.f) : 0.f;
        gx = fmaf(g[j], xv[j], gx);
      }
      gx = row_sum<32>(gx);
      const float k1 = gx / d * r;
      float* o = static_cast<float*>(sd.dx) + a.offset(sd.dx_st);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float xn = xv[j] * r;
        dw[j] = fmaf(y[j], xn, dw[j]);
        if (lane + 32 * j < d) o[lane + 32 * j] = r * fmaf(-xn, k1, g[j]);
      }
    }
  }
  if (!kBackward || wv == nullptr) return;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) buf[warp][lane + 32 * j] = dw[j];
  __syncthreads();
  if (threadIdx.x < d) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < 8; ++g) t += buf[g][threadIdx.x];
    p.part[(long long)blockIdx.x * d + threadIdx.x] = t;
  }
}

// Whether the vector kernels cover the call: eight-value lanes need d in {64, 128}, rot a
// multiple of 16 and rows that start on 16 bytes (16-bit calls always meet this, the entry
// points see to it).
bool vector_rows(const RopeParams& p, int dtype, bool backward) {
  if (dtype != FA_F32) return true;
  if ((p.d != 64 && p.d != 128) || (p.rot & 15)) return false;
  for (const RopeSide* s : {&p.q, &p.k}) {
    const fa_strides st[3] = {s->x_st, s->out_st, backward ? s->dx_st : s->x_st};
    for (const fa_strides& t : st)
      if ((t.b | t.n | t.h) & 3) return false;
  }
  return true;
}

template <typename T>
cudaError_t launch_fwd(const RopeParams& p, unsigned grid, cudaStream_t st) {
  if (p.d == 64) {
    if (p.neighbours)
      norm_rope_fwd_kernel<T, 64, true><<<grid, kRopeThreads, 0, st>>>(p);
    else
      norm_rope_fwd_kernel<T, 64, false><<<grid, kRopeThreads, 0, st>>>(p);
  } else {
    if (p.neighbours)
      norm_rope_fwd_kernel<T, 128, true><<<grid, kRopeThreads, 0, st>>>(p);
    else
      norm_rope_fwd_kernel<T, 128, false><<<grid, kRopeThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const RopeParams& p, unsigned grid, cudaStream_t st) {
  if (p.d == 64) {
    if (p.neighbours)
      norm_rope_bwd_kernel<T, 64, true><<<grid, kRopeThreads, 0, st>>>(p);
    else
      norm_rope_bwd_kernel<T, 64, false><<<grid, kRopeThreads, 0, st>>>(p);
  } else {
    if (p.neighbours)
      norm_rope_bwd_kernel<T, 128, true><<<grid, kRopeThreads, 0, st>>>(p);
    else
      norm_rope_bwd_kernel<T, 128, false><<<grid, kRopeThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

long long blocks_for(long long rows, int per_block) { return (rows + per_block - 1) / per_block; }

}  // namespace

int rope_bwd_max_blocks() { return kBwdBlocks + 2; }

cudaError_t launch_norm_rope_fwd(RopeParams& p, int dtype, cudaStream_t st) {
  const long long rq = (long long)p.B * p.N * p.q.H, rk = (long long)p.B * p.N * p.k.H;
  if (!vector_rows(p, dtype, false)) {
    // enough blocks of eight rows to fill the GPU twice; longer inputs loop
    p.q_blocks = (int)std::min<long long>(blocks_for(rq, 8), 152 * 8);
    const int kb = (int)std::min<long long>(blocks_for(rk, 8), 152 * 8);
    norm_rope_any_f32_kernel<false><<<p.q_blocks + kb, kRopeThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  const int per = kRopeThreads / (p.d / 8) * kFwdRows;
  const long long qb = blocks_for(rq, per), kb = blocks_for(rk, per);
  if (qb + kb > 0x7fffffffll) return cudaErrorInvalidValue;
  p.q_blocks = (int)qb;
  const unsigned grid = (unsigned)(qb + kb);
  if (dtype == FA_F32) return launch_fwd<float>(p, grid, st);
  return dtype == FA_BF16 ? launch_fwd<__nv_bfloat16>(p, grid, st) : launch_fwd<__half>(p, grid, st);
}

cudaError_t launch_norm_rope_bwd(RopeParams& p, int dtype, cudaStream_t st) {
  const bool vec = vector_rows(p, dtype, true);
  const int per = vec ? kRopeThreads / (p.d / 8) * kBwdRows : 8;
  const long long rq = (long long)p.B * p.N * p.q.H, rk = (long long)p.B * p.N * p.k.H;
  // one resident set of blocks, shared between q and k by their rows
  const long long want = std::min<long long>(blocks_for(rq, per) + blocks_for(rk, per), kBwdBlocks);
  const long long qb = std::min<long long>(std::max<long long>(1, want * rq / (rq + rk)), blocks_for(rq, per));
  const long long kb = std::min<long long>(std::max<long long>(1, want - qb), blocks_for(rk, per));
  p.q_blocks = (int)qb;
  p.blocks = (int)(qb + kb);
  cudaError_t e;
  if (!vec) {
    norm_rope_any_f32_kernel<true><<<p.blocks, kRopeThreads, 0, st>>>(p);
    e = cudaGetLastError();
  } else if (dtype == FA_F32) {
    e = launch_bwd<float>(p, p.blocks, st);
  } else {
    e = dtype == FA_BF16 ? launch_bwd<__nv_bfloat16>(p, p.blocks, st) : launch_bwd<__half>(p, p.blocks, st);
  }
  if (e != cudaSuccess || (p.q.w == nullptr && p.k.w == nullptr)) return e;
  const dim3 grid(2, (p.d + 31) / 32);
  if (dtype == FA_F32 || p.w_f32)
    weight_grad_kernel<float><<<grid, 256, 0, st>>>(p);
  else if (dtype == FA_BF16)
    weight_grad_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
  else
    weight_grad_kernel<__half><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
