// Parameters, plan and launchers of cross attention, shared by its C entry
// points (fa_cross.cu) and kernels.
#pragma once

#include "fa_host.h"
#include "fa_internal.h"

namespace fa {

// How a call's work is cut: the forward's and dQ's key axis, and dK/dV's query
// axis, into splits whose partial results a second kernel joins (1: written directly).
struct CrossPlan {
  int k_splits, k_chunk;  // keys of a split (a multiple of the kernel's key step)
  int q_splits, q_chunk;  // query steps of a split (steps run over the group's heads and its queries)
};

struct CrossParams {
  int B, Nq, Nk, Hq, Hk, G, d;  // G = Hq / Hk query heads share a key head
  const int* q_lens;            // [B] or null: Nq each
  const int* k_lens;            // [B] or null: Nk each
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;  // [B, Hq, Nq] natural-log log-sum-exp
  void* out;         // forward: O; backward: dQ
  void* dk;
  void* dv;
  float* lse_out;
  fa_strides q_st, k_st, v_st, o_st, do_st, out_st, dk_st, dv_st;
  float scale, scale_log2;
  // Backward: -L * log2(e) and -D of every query row, [B * Hq, nq_pad], -inf and 0
  // where a row is not there (padding, past its sequence, without keys).
  float* nL2;
  float* nD;
  int nq_pad;
  // Split results in fp32: the forward's normalised outputs [k_splits][B, Nq, Hq, d]
  // and their log2-sum-exp2 [k_splits][B, Hq, Nq] (-inf: the split has no key of the
  // row, and no output is there); dQ [k_splits][B, Nq, Hq, d]; dK and dV
  // [q_splits][2][B, Nk, Hk, d], of the rows of real keys.
  float* part;
  float* part_lse;
  float* part_kv;
  CrossPlan plan;
  unsigned int* status;
};

__device__ __forceinline__ int cross_q_len(const CrossParams& p, int b) {
  return p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
}
__device__ __forceinline__ int cross_k_len(const CrossParams& p, int b) {
  return p.k_lens ? min(max(p.k_lens[b], 0), p.Nk) : p.Nk;
}

// Splits of an axis of `len` in steps of `step`, for `units` independent blocks on
// `places`: as many as fill the places once, `least` steps a split at least.
inline void cross_splits(int len, int step, long long units, int places, int least, int* splits, int* chunk) {
  const int steps = (len + step - 1) / step;
  long long want = units < places ? places / units : 1;
  if (want > steps / least) want = steps / least;
  if (want < 1) want = 1;
  const int per = (int)((steps + want - 1) / want);
  *splits = (steps + per - 1) / per;
  *chunk = per * step;
}

CrossPlan cross_plan(int B, int Nq, int Nk, int Hq, int Hk, int d, int dtype);

cudaError_t launch_cross_preprocess(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_join_fwd(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_join_dq(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_join_dkdv(const CrossParams& p, int dtype, cudaStream_t st);

cudaError_t launch_cross_fwd_simple(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_dq_simple(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_dkdv_simple(const CrossParams& p, int dtype, cudaStream_t st);

}  // namespace fa
