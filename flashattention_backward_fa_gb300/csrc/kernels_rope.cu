// Per-head RMS norm of queries and keys with their position rotation, forward
// and backward (the formulas and the lane layout: rope_common.cuh).
//
// Backward, with dy = R(pos)^T dout, xn = x r, g = w o dy:
//   dx = r (g - xn mean(g o xn));  dw = sum over rows of dy o xn
// r is formed again from x, which the backward reads anyway, so nothing but
// the inputs is kept between the two passes. dw: every lane keeps the sums of
// its 16 columns over its rows, a block adds its lanes' sums in a fixed
// order into one row of the workspace, and a second kernel adds the blocks'
// rows in a fixed order, so the gradients are the same bits on every run.
//
// Both are bound by memory: 4 bytes an element (forward) and 6 (backward, 16-bit
// types), against about 13 and 18 thread instructions. A row is in registers
// between its one load and its one store, and the next rows are on their way to
// shared memory. Measured, bf16: forward 1x32x8192x128 (q and k) 44.2 us a call
// (91% of the copy rate), backward 4x16x2048x128 35 us (86%).
#include <algorithm>

#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kFwdDepth = 3;          // rows a row group of the forward has on their way, and the one at hand
constexpr int kBwdDepth = 2;          // the same of the backward (x and dout each)
constexpr int kFwdBlocks = 152 * 12;  // four resident sets of blocks: ragged ends even out
constexpr int kBwdBlocks = 152 * 2;   // one resident set: every block adds a row of partial sums

// The token's rows in the tables: its position, clamped into them.
__device__ __forceinline__ long long table_row(const RopeParams& p, long long b, int n) {
  const int pos = p.positions ? p.positions[b * p.pos_stride + n] : n;
  return (long long)min(max(pos, 0), p.max_pos - 1) * (p.rot >> 1);
}

template <typename T, int D, bool kNeighbours>
__global__ void __launch_bounds__(kRopeThreads, 3) norm_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ __align__(16) float w[D];
  let_next_begin();
  wait_for_previous();
  const bool is_k = blockIdx.x >= (unsigned)p.q_blocks;
  const RopeSide& sd = is_k ? p.k : p.q;
  const long long group =
      (long long)(blockIdx.x - (is_k ? p.q_blocks : 0)) * (kRopeThreads / (D / 16)) + threadIdx.x / (D / 16);
  norm_rope_rows<T, D, kNeighbours, kFwdDepth>(
      ring, static_cast<const T*>(sd.x), static_cast<T*>(sd.out), sd.x_st, sd.out_st, (long long)p.B * p.N * sd.H, p.N,
      sd.H, group * sd.span, sd.span, sd.w, p.w_f32, w, p.cos, p.sin, p.rot, p.eps,
      [&](long long b, int n) { return p.rot ? table_row(p, b, n) : 0ll; });
}

// Each row group takes sd.span consecutive rows, as in the forward; its lanes
// keep the weight gradients of their columns.
template <typename T, int D, bool kNeighbours, bool kPartial>
__global__ void __launch_bounds__(kRopeThreads, 2) norm_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int G = D / 16, kGroups = kRopeThreads / G;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float w[D];
  let_next_begin();
  wait_for_previous();
  RowRing<T, 4, kBwdDepth> ring(smem);
  const int group = threadIdx.x / G;
  const bool is_k = blockIdx.x >= (unsigned)p.q_blocks;
  const RopeSide& sd = is_k ? p.k : p.q;
  const long long rows = (long long)p.B * p.N * sd.H;
  const long long first = ((long long)(blockIdx.x - (is_k ? p.q_blocks : 0)) * kGroups + group) * sd.span;
  const int live = (int)min((long long)sd.span, max(rows - first, 0ll));
  const LanePlace at = lane_place<D, kNeighbours, kPartial>(threadIdx.x % G, p.rot);
  RowWalk wx;
  wx.start(first, p.N, sd.H, sd.x_st);
  RowWalk wg = wx.in(sd.out_st), wo = wx.in(sd.dx_st);
  uint64_t dwa[4], dwb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dwa[i] = dwb[i] = 0ull;
  float c[8], s[8];
  int loaded = 0;
  const T* x_in = static_cast<const T*>(sd.x) + at.a;
  const T* g_in = static_cast<const T*>(sd.dout) + at.a;
  T* dx_out = static_cast<T*>(sd.dx) + at.a;
  const int hop = at.b - at.a;
  auto fetch = [&] {
    if (loaded < live) {
      const T* x = x_in + wx.at;
      const T* g = g_in + wg.at;
      ring.fetch(0, x);
      ring.fetch(1, x + hop);
      ring.fetch(2, g);
      ring.fetch(3, g + hop);
    } else if (loaded < sd.span) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ring.clear(i);
    }
    copies_commit();
    ring.step(ring.put);
    wx.next(p.N, sd.H, sd.x_st);
    wg.next(p.N, sd.H, sd.out_st);
    ++loaded;
  };
#pragma unroll
  for (int i = 0; i < kBwdDepth - 1; ++i) fetch();
  stage_weights<T>(sd.w, p.w_f32, D, w);
  __syncthreads();
  bool token = true;
  for (int i = 0; i < sd.span; ++i) {
    fetch();
    if (token) {
      const bool ok = i < live;
      const long long row = ok && p.rot ? table_row(p, wo.b, wo.n) : 0;
      load_rotation<kNeighbours>(p.cos + row, p.sin + row, at, ok ? p.rot : 0, c, s);
    }
    copies_wait<kBwdDepth - 1>();
    Raw8<T> raw;
    uint64_t xa[4], xb[4], ga[4], gb[4];
    ring.take(2, raw);
    raw.unpack(ga);
    ring.take(3, raw);
    raw.unpack(gb);
    // dy = R^T dout
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kNeighbours) {
        const uint64_t cj = f2_pack(c[j], c[j]), sj = f2_pack(s[j], -s[j]);
        const uint64_t ck = f2_pack(c[4 + j], c[4 + j]), sk = f2_pack(s[4 + j], -s[4 + j]);
        ga[j] = f2_fma(ga[j], cj, f2_mul(f2_if(at.turn_a, f2_swap(ga[j])), sj));
        gb[j] = f2_fma(gb[j], ck, f2_mul(f2_if(at.turn_b, f2_swap(gb[j])), sk));
      } else {
        const uint64_t cj = f2_pack(c[2 * j], c[2 * j + 1]), sj = f2_pack(s[2 * j], s[2 * j + 1]);
        const uint64_t nj = f2_pack(-s[2 * j], -s[2 * j + 1]);
        const uint64_t da = f2_fma(ga[j], cj, f2_mul(f2_if(at.turn_a, gb[j]), sj));
        gb[j] = f2_fma(gb[j], cj, f2_mul(f2_if(at.turn_a, ga[j]), nj));
        ga[j] = da;
      }
    }
    ring.take(0, raw);
    raw.unpack(xa);
    ring.take(1, raw);
    raw.unpack(xb);
    ring.step(ring.got);
    uint64_t s2 = 0ull, g2 = 0ull, wa[4], wb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = reinterpret_cast<const float2*>(w + at.a)[j], v = reinterpret_cast<const float2*>(w + at.b)[j];
      wa[j] = f2_mul(ga[j], f2_pack(u.x, u.y));  // g = w o dy
      wb[j] = f2_mul(gb[j], f2_pack(v.x, v.y));
      s2 = f2_fma(xa[j], xa[j], f2_fma(xb[j], xb[j], s2));
      g2 = f2_fma(wa[j], xa[j], f2_fma(wb[j], xb[j], g2));
    }
    const float ss = row_sum<G>(f2_sum(s2)), gx = row_sum<G>(f2_sum(g2));
    const float rr = inv_sqrt(fmaf(ss, 1.f / D, p.eps));
    const float k1 = -gx * (1.f / D) * rr;  // -mean(g o xn)
    const uint64_t r2 = f2_pack(rr, rr), k2 = f2_pack(k1, k1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      xa[j] = f2_mul(xa[j], r2);
      xb[j] = f2_mul(xb[j], r2);
      dwa[j] = f2_fma(ga[j], xa[j], dwa[j]);
      dwb[j] = f2_fma(gb[j], xb[j], dwb[j]);
      wa[j] = f2_mul(r2, f2_fma(xa[j], k2, wa[j]));
      wb[j] = f2_mul(r2, f2_fma(xb[j], k2, wb[j]));
    }
    if (i < live) {
      T* dx = dx_out + wo.at;
      raw.pack(wa);
      store8(raw, dx);
      raw.pack(wb);
      store8(raw, dx + hop);
    }
    token = wo.next(p.N, sd.H, sd.dx_st);
  }
  if (sd.w == nullptr) return;
  // the block's sums take the ring's place once every copy into it has landed (none is pending
  // beyond the rows above: the last fetches were of nothing but are waited for all the same)
  copies_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);  // [kGroups][D]
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    f2_unpack(dwa[j], lo, hi);
    reinterpret_cast<float2*>(sums + group * D + at.a)[j] = make_float2(lo, hi);
    f2_unpack(dwb[j], lo, hi);
    reinterpret_cast<float2*>(sums + group * D + at.b)[j] = make_float2(lo, hi);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kRopeThreads) {
    float t = 0.f;
#pragma unroll 8
    for (int g = 0; g < kGroups; ++g) t += sums[g * D + e];
    p.part[(long long)blockIdx.x * D + e] = t;
  }
}

// Adds the blocks' partial weight gradients: block x = side (q, k), 32 warps
// that take every 32nd row, one column a lane.
template <typename T>
__global__ void __launch_bounds__(1024) weight_grad_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float sums[32][33];
  let_next_begin();
  wait_for_previous();
  const bool is_k = blockIdx.x != 0;
  const RopeSide& sd = is_k ? p.k : p.q;
  if (sd.w == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.y * 32 + lane;
  const int lo = is_k ? p.q_blocks : 0, hi = is_k ? p.blocks : p.q_blocks;
  float t = 0.f;
  if (e < p.d) {
#pragma unroll 12
    for (int r = lo + warp; r < hi; r += 32) t += __ldcg(p.part + (long long)r * p.d + e);
  }
  sums[warp][lane] = t;
  __syncthreads();
  t = row_sum<32>(sums[lane][warp]);  // column `warp`
  const int col = blockIdx.y * 32 + warp;
  if (lane == 0 && col < p.d) {
    if (p.w_f32)
      static_cast<float*>(sd.dw)[col] = t;
    else
      static_cast<T*>(sd.dw)[col] = static_cast<T>(t);
  }
}

// fp32 with any d <= 128, any even rot and any strides: one warp a row, lane
// l holding the values l, l + 32, ...; the row passes through shared memory for
// the partners' values. kBackward adds the gradients as above (dw: lane sums,
// then the warps' in order). Rows of a block: eight warps, strided over the grid.
template <bool kBackward>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_any_f32_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float buf[8][128];
  let_next_begin();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = p.d, h = p.rot >> 1;
  const bool is_k = blockIdx.x >= (unsigned)p.q_blocks;
  const RopeSide& sd = is_k ? p.k : p.q;
  const int blk = blockIdx.x - (is_k ? p.q_blocks : 0), blks = is_k ? gridDim.x - p.q_blocks : p.q_blocks;
  const long long rows = (long long)p.B * p.N * sd.H;
  const float* wv = static_cast<const float*>(sd.w);
  float dw[4] = {0.f, 0.f, 0.f, 0.f};
  for (long long row = (long long)blk * 8 + warp; row < rows; row += (long long)blks * 8) {
    RowWalk a;
    a.start(row, p.N, sd.H, sd.x_st);
    const float* x = static_cast<const float*>(sd.x) + a.at;
    const long long at = p.rot ? table_row(p, a.b, a.n) : 0;
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
    const float r = inv_sqrt(ss / d + p.eps);
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

// Whether the vector kernels cover the call: 16-value lanes need d in {64, 128}, rot a
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

template <auto kKernel>
cudaError_t launch_ring(const RopeParams& p, int bytes, cudaStream_t st) {
  const cudaError_t e = allow_smem<kKernel>(bytes);
  if (e != cudaSuccess) return e;
  return launch_chained(kKernel, p.blocks, kRopeThreads, bytes, 1, p, st);
}

template <typename T>
cudaError_t launch_fwd(const RopeParams& p, cudaStream_t st) {
  constexpr int bytes = RowRing<T, 2, kFwdDepth>::bytes(kRopeThreads);
  if (p.d == 64)
    return p.neighbours ? launch_ring<norm_rope_fwd_kernel<T, 64, true>>(p, bytes, st)
                        : launch_ring<norm_rope_fwd_kernel<T, 64, false>>(p, bytes, st);
  return p.neighbours ? launch_ring<norm_rope_fwd_kernel<T, 128, true>>(p, bytes, st)
                      : launch_ring<norm_rope_fwd_kernel<T, 128, false>>(p, bytes, st);
}

template <typename T, int D, bool kPartial>
cudaError_t launch_bwd_d(const RopeParams& p, cudaStream_t st) {
  constexpr int bytes = RowRing<T, 4, kBwdDepth>::bytes(kRopeThreads);
  static_assert(bytes >= kRopeThreads * 16 * 4, "the block's weight gradients fit into the ring");
  return p.neighbours ? launch_ring<norm_rope_bwd_kernel<T, D, true, kPartial>>(p, bytes, st)
                      : launch_ring<norm_rope_bwd_kernel<T, D, false, kPartial>>(p, bytes, st);
}

template <typename T>
cudaError_t launch_bwd(const RopeParams& p, cudaStream_t st) {
  if (p.d == 64) return p.rot < 64 ? launch_bwd_d<T, 64, true>(p, st) : launch_bwd_d<T, 64, false>(p, st);
  return p.rot < 128 ? launch_bwd_d<T, 128, true>(p, st) : launch_bwd_d<T, 128, false>(p, st);
}

long long div_up(long long a, long long b) { return (a + b - 1) / b; }

// Gives every row group its number of consecutive rows, and q and k their blocks:
// blocks of `groups` row groups, at most `most` of them, and no fewer than `fewest`
// (one resident set) for the sake of longer spans: from eight rows on a group's
// prologue (weights, first loads, the row's place) no longer counts. Measured with
// the forward at bf16 4x16x2048x128: 5 rows 26.1 us, 9 rows 24.3 us; at
// 1x32x8192x128: 9 rows 47.2 us, 36 rows 50.1 us (ragged ends).
void share_rows(RopeParams& p, int groups, long long fewest, long long most) {
  const long long rq = (long long)p.B * p.N * p.q.H, rk = (long long)p.B * p.N * p.k.H;
  const long long span = std::max(div_up(rq + rk, most * groups), std::min(8ll, div_up(rq + rk, fewest * groups)));
  for (int side = 0; side < 2; ++side) {
    RopeSide& s = side ? p.k : p.q;
    s.span = (int)std::min<long long>(span, 1 << 30);
    const int n = (int)div_up(side ? rk : rq, groups * (long long)s.span);
    if (side)
      p.blocks = p.q_blocks + n;
    else
      p.q_blocks = n;
  }
}

}  // namespace

int rope_bwd_max_blocks() { return kBwdBlocks + 2; }

cudaError_t launch_norm_rope_fwd(RopeParams& p, int dtype, cudaStream_t st) {
  if (!vector_rows(p, dtype, false)) {
    share_rows(p, 8, 152 * 8, 152 * 8);
    return launch_chained(norm_rope_any_f32_kernel<false>, p.blocks, kRopeThreads, 0, 1, p, st);
  }
  share_rows(p, kRopeThreads / (p.d / 16), kFwdBlocks / 4, kFwdBlocks);
  if (dtype == FA_F32) return launch_fwd<float>(p, st);
  return dtype == FA_BF16 ? launch_fwd<__nv_bfloat16>(p, st) : launch_fwd<__half>(p, st);
}

cudaError_t launch_norm_rope_bwd(RopeParams& p, int dtype, cudaStream_t st) {
  const bool vec = vector_rows(p, dtype, true);
  cudaError_t e;
  if (!vec) {
    share_rows(p, 8, kBwdBlocks, kBwdBlocks);
    e = launch_chained(norm_rope_any_f32_kernel<true>, p.blocks, kRopeThreads, 0, 1, p, st);
  } else {
    share_rows(p, kRopeThreads / (p.d / 16), kBwdBlocks, kBwdBlocks);
    if (dtype == FA_F32)
      e = launch_bwd<float>(p, st);
    else
      e = dtype == FA_BF16 ? launch_bwd<__nv_bfloat16>(p, st) : launch_bwd<__half>(p, st);
  }
  if (e != cudaSuccess || (p.q.w == nullptr && p.k.w == nullptr)) return e;
  const dim3 grid(2, (p.d + 31) / 32);
  if (dtype == FA_F32 || p.w_f32) return launch_chained(weight_grad_kernel<float>, grid, 1024, 0, 1, p, st);
  return dtype == FA_BF16 ? launch_chained(weight_grad_kernel<__nv_bfloat16>, grid, 1024, 0, 1, p, st)
                          : launch_chained(weight_grad_kernel<__half>, grid, 1024, 0, 1, p, st);
}

}  // namespace fa
