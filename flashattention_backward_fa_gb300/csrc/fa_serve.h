// Parameters and launchers of the norm-and-rotation operators and of the 8-bit
// key/value cache, shared by their C entry points (fa_serve.cu) and kernels.
#pragma once

#include <atomic>

#include "fa_host.h"
#include "fa_internal.h"

namespace fa {

// Raises a kernel's limit of dynamic shared memory to `bytes`, once per kernel and device (the
// default limit, 48 KB, includes the kernel's static part).
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0ull};
  if (bytes <= 32 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev > 63) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  if (done.load(std::memory_order_relaxed) >> dev & 1ull) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

// Launches a kernel whose blocks may take their places while the kernel before it in the stream
// ends (sooner where that one calls let_next_begin). Each of them waits for that kernel's end
// (wait_for_previous) before it touches memory; towards other kernels this is an ordinary launch.
// What such a kernel reads may have been written while its first blocks were already there, so it is
// not read-only for the kernel's lifetime: no __ldg (ld.global.nc) and no const __restrict__ there,
// but ordinary loads or cp.async, at the same times (with __ldcg, which the compiler does not move,
// for the rows the append took 33.1 us instead of 30.5 us).
// Between two of these kernels it saves 1 to 3 us: bf16 norm and rotation 1x32x8192x128 46.9 ->
// 44.2 us, append 32.8 -> 30.6 us, 100 tokens of attention 6.2 -> 5.5 us. cluster > 1: blocks of a
// cluster along x.
template <typename Params>
cudaError_t launch_chained(void (*kernel)(Params), dim3 grid, int threads, int smem, int cluster, const Params& p,
                           cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// One of q and k: x [B, N, H, d], forward output (backward: the gradient that
// comes in, `dout`, with out_st its strides) and the backward's outputs.
struct RopeSide {
  const void* x;
  const void* dout;
  void* out;
  void* dx;
  const void* w;  // weight vector [d] or null (ones)
  void* dw;
  fa_strides x_st, out_st, dx_st;
  int H;
  int span;  // set by the launcher: consecutive rows of a row group
};

// Positions with several axes: pair i of the rotated values takes the table row of the position on its
// axis, 2 bits a pair (axes <= 4, pairs <= 64). axes = 0: one position a token, the call's own way.
struct RopeAxes {
  int axes;
  uint32_t pair_axis[4];
  const int* positions;  // [B, N, axes] by its strides
  int64_t sb, sn, sa;
};

struct RopeParams {
  RopeSide q, k;
  RopeAxes ax;
  const float* cos;  // [max_pos, rot / 2]
  const float* sin;
  const int* positions;  // [B, N], rows pos_stride apart, or null: 0 .. N - 1
  int64_t pos_stride;
  int B, N, d, rot, max_pos;
  int neighbours;  // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
  int w_f32;       // weights (and their gradients) are fp32 whatever the tensors' type
  float eps;
  float* part;          // backward: a row of d partial weight gradients per block
  int q_blocks, blocks;  // set by the launcher: blocks [0, q_blocks) take q's rows
};

// Most rows of `part` that a backward launch writes.
int rope_bwd_max_blocks();
cudaError_t launch_norm_rope_fwd(RopeParams& p, int dtype, cudaStream_t st);
cudaError_t launch_norm_rope_bwd(RopeParams& p, int dtype, cudaStream_t st);

// Device status bit: a block table names a page outside the cache (the page's
// tokens are skipped).
constexpr unsigned int kStatusBadPage = 4u;

// A paged cache of e4m3 codes and its sequences (fa.h, fa_kv8_cache and fa_kv8_seqs).
struct Kv8Cache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;  // [num_pages, H]
  float* v_scale;
  int num_pages, page_shift, H;
  int64_t sp, sn, sh;  // element strides of a page, a token and a head (k and v alike)
  const int* table;    // [B, max_pages], rows table_stride apart
  int64_t table_stride;
  int max_pages;
  const int* seq_lens;  // [B], the call's new tokens counted
  const int* new_lens;  // [B] or null: T each
  unsigned int* status;
};

struct Kv8AppendParams {
  Kv8Cache c;
  const void* k;
  const void* v;
  fa_strides k_st, v_st;
  int B, T, d;
  int pages;  // most pages that T tokens reach
  // norm and rotation (null q: the append alone)
  const void* q;
  void* q_out;
  fa_strides q_st, q_out_st;
  int Hq;
  const void* q_w;
  const void* k_w;
  const float* cos;
  const float* sin;
  int rot, max_pos, neighbours, w_f32;
  float eps;
  RopeAxes ax;  // axes = 0: positions are places in the sequences
  int kv_heads, q_heads;  // set by the launcher: heads of k and v, and of q, that a block takes
};
cudaError_t launch_kv8_append(Kv8AppendParams& p, bool bf16, cudaStream_t st);

struct Kv8AttnParams {
  Kv8Cache c;
  const void* q;
  void* o;
  float* lse;  // [B, Hq, T]
  fa_strides q_st, o_st;
  int B, T, Hq, G, d;  // G = Hq / H query heads share a key head
  float scale_log2;
  int causal, window;
  const float* alibi;
  int64_t alibi_sb;
  int key_limit;  // keys past it are never attended: min(max_seqlen, max_pages * page size)
  int chunk;      // keys of a split (a multiple of 128)
  int splits;     // most splits of a sequence
  int cluster;    // the splits are the blocks of a cluster, which joins them (chunk does not apply)
  int row_tiles;
  int longest_first;  // blocks take the sequences in the order of falling lengths
  float* part_o;   // [B, H, T * G, splits, d]: normalised outputs of the splits
  float* part_lse;  // [B, H, T * G, splits]: their log2-sum-exp2
};

struct Kv8AttnPlan {
  int tiles;      // 8-row query tiles of a block (1 or 2)
  int row_tiles;  // blocks that share the T * G rows of a key head
  int chunk, splits, cluster, longest_first;
  size_t workspace;
};
Kv8AttnPlan kv8_attn_plan(int B, int T, int Hq, int H, int d, int key_limit, int causal, int window);
cudaError_t launch_kv8_attn(Kv8AttnParams& p, const Kv8AttnPlan& plan, bool bf16, cudaStream_t st);

}  // namespace fa
