// Cross attention of few query rows a key head (new tokens of a decoder over an encoder's
// states): the forward, 16-bit types.
//
//   S = scale q k^T, m = running maximum, P = exp2(S - m), l += sum P, O += P V
//
// Bound by reading K and V once; a 128-row tensor-core tile of the main kernel would be
// nearly empty and its start and end as long as the work. A block takes 16 rows (the
// queries of all heads of a group, one behind the other) and one share of the keys. Its four
// warps take key tiles of 8 KB of K and V (16 or 32 keys) in turn, each with a ring of its
// own in shared memory (cp.async in whole lines, 16-byte pieces swizzled by row so that
// ldmatrix reads without conflicts), so that nothing but the end needs the block together.
// S by m16n8k16 with the queries as the rows: its accumulator is the next product's A
// operand. P enters it rounded and once more as its rounding residual: the products are
// far from the bound, and the outputs are as exact as with fp32 weights.
//
// Rows of keys past the end are copied as zeros. The warps' results meet in shared memory,
// the shares of a sequence in the distributed shared memory of a cluster (up to eight
// blocks); where that leaves the GPU empty (few heads, long states) more shares go through
// the workspace and the joining kernel. Where blocks of unequal lengths come in several
// rounds the longest sequences go first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fa_cross.h"
#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 16, kStages = 3;

template <int D>
constexpr int kKeys = 2048 / D;  // keys of a tile: 4 KB of K, 4 KB of V
constexpr uint32_t kHalf = 4096, kTileBytes = 2 * kHalf;

__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A float of another block's shared memory.
__device__ __forceinline__ float peer_float(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// Grid: x the share (a cluster's blocks, or the splits), y row tile, z batch * key head.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 2) cross_few_kernel(const __grid_constant__ CrossParams p) {
  constexpr int kK = kKeys<D>, kTilesN = kK / 8, kSteps = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  let_next_begin();
  wait_for_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, in_quad = lane & 3;
  const int shares = p.few_cluster ? p.few_cluster : p.plan.k_splits, share = blockIdx.x;
  int b = blockIdx.z / p.Hk;
  const int hk = blockIdx.z - b * p.Hk;
  if (p.plan.few_sorted) {  // the b-th longest sequence (the lower number first)
    __shared__ int lens[kThreads], found;
    if ((int)threadIdx.x < p.B) lens[threadIdx.x] = cross_k_len(p, threadIdx.x);
    __syncthreads();
    if ((int)threadIdx.x < p.B) {
      int before = 0;
      for (int i = 0; i < p.B; ++i)
        before += lens[i] > lens[threadIdx.x] || (lens[i] == lens[threadIdx.x] && i < (int)threadIdx.x);
      if (before == b) found = threadIdx.x;
    }
    __syncthreads();
    b = found;
  }
  const int nk = cross_k_len(p, b), nq = cross_q_len(p, b);
  const int tiles = (nk + kK - 1) / kK, per = (tiles + shares - 1) / shares;
  const int t_end = min(tiles, (share + 1) * per);
  const int rows = p.Nq * p.G, row0 = blockIdx.y * kRows;

  // ring: copies of tile t, kK keys of K and V, whole rows by D / 8 lanes
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes a row, rows a copy instruction
  const uint32_t ring = smem_u32(smem) + warp * (kStages * kTileBytes);
  const int piece = lane % kLanes, row_of = lane / kLanes;
  const uint16_t* k = static_cast<const uint16_t*>(p.k) + b * p.k_st.b + hk * p.k_st.h + 8 * piece;
  const uint16_t* v = static_cast<const uint16_t*>(p.v) + b * p.v_st.b + hk * p.v_st.h + 8 * piece;
  int fetched = share * per + warp, put = 0;
  auto fetch = [&] {
    if (fetched < t_end) {
      const uint32_t to = ring + put * kTileBytes;
#pragma unroll
      for (int r0 = 0; r0 < kK; r0 += kAtOnce) {
        const int r = r0 + row_of, j = fetched * kK + r;
        const uint32_t at = to + r * (2 * D) + ((piece ^ (r & 7)) << 4);
        const bool real = j < nk;
        copy16_or_zero(at, k + (real ? j * p.k_st.n : 0), real);
        copy16_or_zero(at + kHalf, v + (real ? j * p.v_st.n : 0), real);
      }
    }
    copies_commit();
    fetched += kWarps;
    put = put == kStages - 1 ? 0 : put + 1;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  // Q as the A operand of rows quad and quad + 8 (zeros where there is none)
  uint32_t q[kSteps][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = row0 + quad + 8 * half, t = r / p.G, h = hk * p.G + r - t * p.G;
    const bool real = r < rows && t < nq;
    const uint16_t* from = static_cast<const uint16_t*>(p.q) + b * p.q_st.b + (real ? t * p.q_st.n + h * p.q_st.h : 0) +
                           2 * in_quad;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        q[s][half + 2 * x] = real ? *reinterpret_cast<const uint32_t*>(from + 16 * s + 8 * x) : 0u;
  }

  float o[D / 8][4];
#pragma unroll
  for (int c = 0; c < D / 8; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // l: of this lane's columns
  // ldmatrix: lane i gives the address of row i % 8 of matrix i / 8
  const int mat = lane >> 3, mrow = lane & 7;
  int got = 0;
  for (int t = share * per + warp; t < t_end; t += kWarps) {
    fetch();
    copies_wait<kStages - 1>();
    __syncwarp();
    const uint32_t kt = ring + got * kTileBytes, vt = kt + kHalf;
    got = got == kStages - 1 ? 0 : got + 1;
    float s[kTilesN][4];
#pragma unroll
    for (int n = 0; n < kTilesN; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
      // B operands of two k steps at once: keys 8 n .. + 7, pieces 4 st .. + 3 of 8 values
#pragma unroll
      for (int st = 0; st < kSteps / 2; ++st) {
        uint32_t kb[4];
        ldmatrix4(kb, kt + (8 * n + mrow) * (2 * D) + (((4 * st + mat) ^ mrow) << 4));
        mma16816<kBf16>(s[n], q[2 * st], kb[0], kb[1]);
        mma16816<kBf16>(s[n], q[2 * st + 1], kb[2], kb[3]);
      }
    }
    const int left = nk - t * kK;  // real keys
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < kTilesN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = 8 * n + 2 * in_quad + (e & 1) < left ? s[n][e] * p.scale_log2 : -INFINITY;
        top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
      }
    float was[2], base[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
      top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
      const float now = fmaxf(m[x], top[x]);
      base[x] = now == -INFINITY ? 0.f : now;  // (every score so far is -inf)
      was[x] = ex2_approx(m[x] - base[x]);
      m[x] = now;
      l[x] *= was[x];
    }
    if (__any_sync(0xffffffffu, was[0] != 1.f || was[1] != 1.f)) {
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        o[c][0] *= was[0];
        o[c][1] *= was[0];
        o[c][2] *= was[1];
        o[c][3] *= was[1];
      }
    }
#pragma unroll
    for (int n = 0; n < kTilesN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = ex2_approx(s[n][e] - base[e >> 1]);
        l[e >> 1] += s[n][e];
      }
#pragma unroll
    for (int g = 0; g < kK / 16; ++g) {  // 16 keys: one k step of the second product
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = s[2 * g + (e >> 1)][2 * (e & 1)], y = s[2 * g + (e >> 1)][2 * (e & 1) + 1];
        hi[e] = pack2<kBf16>(x, y);
        lo[e] = pack2_residual<kBf16>(x, y, hi[e]);
      }
      // V's rows 16 g .. + 15 as the B operand of columns 8 c .. and 8 (c + 1) ..
#pragma unroll
      for (int c = 0; c < D / 8; c += 2) {
        uint32_t vb[4];
        const int r = 16 * g + (mat & 1) * 8 + mrow;
        ldmatrix4_t(vb, vt + r * (2 * D) + (((c + (mat >> 1)) ^ mrow) << 4));
        mma16816<kBf16>(o[c], hi, vb[0], vb[1]);
        mma16816<kBf16>(o[c + 1], hi, vb[2], vb[3]);
        mma16816<kBf16>(o[c], lo, vb[0], vb[1]);
        mma16816<kBf16>(o[c + 1], lo, vb[2], vb[3]);
      }
    }
    __syncwarp();  // (the next copies go where these tiles were)
  }
  copies_wait<0>();
  __syncthreads();

  // The warps' results, then the block's: [kWarps][kRows] m and l, [kWarps][kRows][D] O; the block's in warp 0's place.
  float* sm_m = reinterpret_cast<float*>(smem);
  float* sm_l = sm_m + kWarps * kRows;
  float* sm_o = sm_l + kWarps * kRows;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    const int r = quad + 8 * x;
    if (in_quad == 0) {
      sm_m[warp * kRows + r] = m[x];
      sm_l[warp * kRows + r] = l[x];
    }
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      *reinterpret_cast<float2*>(sm_o + (warp * kRows + r) * D + 8 * c + 2 * in_quad) =
          make_float2(o[c][2 * x], o[c][2 * x + 1]);
  }
  __syncthreads();
  // thread: one column of D (or half the rows of it)
  constexpr int kPer = kRows * D / kThreads;
  const int col = threadIdx.x % D, r_first = threadIdx.x / D * kPer;
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r_first + i;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w * kRows + r]);
    const float at = mm == -INFINITY ? 0.f : mm;
    acc[i] = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2_approx(sm_m[w * kRows + r] - at);
      acc[i] = fmaf(f, sm_o[(w * kRows + r) * D + col], acc[i]);
      sum = fmaf(f, sm_l[w * kRows + r], sum);
    }
    sm_o[r * D + col] = acc[i];  // (only this thread reads or writes the place)
    if (p.few_cluster <= 1) {
      const int rr = row0 + r, tq = rr / p.G, h = hk * p.G + rr - tq * p.G;
      if (rr >= rows) continue;
      const long long lse_at = ((long long)b * p.Hq + h) * p.Nq + tq, all = (long long)p.B * p.Nq * p.Hq;
      const bool has = tq < nq && sum != 0.f;  // (a NaN sum is there)
      const float lse2 = has ? mm + log2f(sum) : -INFINITY;
      if (p.few_cluster) {
        const float out = has ? acc[i] / sum : 0.f;
        uint16_t* to = static_cast<uint16_t*>(p.out) + b * p.out_st.b + tq * p.out_st.n + h * p.out_st.h + col;
        *to = (uint16_t)pack2<kBf16>(out, 0.f);
        if (col == 0) p.lse_out[lse_at] = has ? lse2 * 0.6931471805599453f : -INFINITY;
      } else {
        if (has) p.part[(share * all + ((long long)b * p.Nq + tq) * p.Hq + h) * D + col] = acc[i] / sum;
        if (col == 0) p.part_lse[share * all + lse_at] = lse2;
      }
    }
  }
  if (p.few_cluster <= 1) return;

  // The cluster's blocks share out the rows.
  __syncthreads();  // (the warps' m and l have been read)
  if (threadIdx.x < kRows) {
    float mm = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w * kRows + threadIdx.x]);
    const float at = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      sum = fmaf(ex2_approx(sm_m[w * kRows + threadIdx.x] - at), sm_l[w * kRows + threadIdx.x], sum);
    sm_m[threadIdx.x] = mm;  // (warp 0's place is this thread's alone)
    sm_l[threadIdx.x] = sum;
  }
  cluster_sync();
  const int in_block = (kRows + p.few_cluster - 1) / p.few_cluster;  // rows a block finishes
  const uint32_t am = smem_u32(sm_m), al = smem_u32(sm_l), ao = smem_u32(sm_o);
  const int my = (int)cluster_rank();
  for (int x = threadIdx.x; x < in_block * D; x += kThreads) {
    const int r = my * in_block + x / D, c = x % D, rr = row0 + r;
    if (r >= kRows || rr >= rows) continue;
    float pm[8], mm = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pm[i] = i < p.few_cluster ? peer_float(am + 4 * r, i) : -INFINITY;
      mm = fmaxf(mm, pm[i]);
    }
    const float at = mm == -INFINITY ? 0.f : mm;
    float sum = 0.f, out = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= p.few_cluster) continue;
      const float f = ex2_approx(pm[i] - at);
      sum = fmaf(f, peer_float(al + 4 * r, i), sum);
      out = fmaf(f, peer_float(ao + 4 * (r * D + c), i), out);
    }
    const int tq = rr / p.G, h = hk * p.G + rr - tq * p.G;
    const bool has = tq < nq && sum != 0.f;
    out = has ? out / sum : 0.f;
    uint16_t* to = static_cast<uint16_t*>(p.out) + b * p.out_st.b + tq * p.out_st.n + h * p.out_st.h + c;
    *to = (uint16_t)pack2<kBf16>(out, 0.f);
    if (c == 0)
      p.lse_out[((long long)b * p.Hq + h) * p.Nq + tq] = has ? (mm + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
  cluster_sync();  // (no block leaves while another reads its shared memory)
}

template <int D, bool kBf16>
cudaError_t launch_t(const CrossParams& p, cudaStream_t st) {
  constexpr int bytes = kWarps * kStages * kTileBytes;
  static_assert(bytes >= kWarps * kRows * (D + 2) * 4, "the warps' results fit into the rings");
  constexpr auto kKernel = cross_few_kernel<D, kBf16>;
  const cudaError_t e = allow_smem<kKernel>(bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.few_cluster ? p.few_cluster : p.plan.k_splits, (p.Nq * p.G + kRows - 1) / kRows, p.B * p.Hk);
  return launch_chained(kKernel, grid, kThreads, bytes, std::max(p.few_cluster, 1), p, st);
}

}  // namespace

cudaError_t launch_cross_few(const CrossParams& p, bool bf16, cudaStream_t st) {
  if (p.d == 128) return bf16 ? launch_t<128, true>(p, st) : launch_t<128, false>(p, st);
  return bf16 ? launch_t<64, true>(p, st) : launch_t<64, false>(p, st);
}

}  // namespace fa
