// Parameters, plan and launchers of cross attention, shared by its C entry
// points (fa_cross.cu) and kernels.
#pragma once

#include "fa_host.h"
#include "fa_internal.h"

namespace fa {

// How a call's work is cut: the forward's and dQ's key axis, and dK/dV's query
// axis, into splits whose partial results a second kernel joins (1: written directly).
//
// Query rows of a key head's group are taken in tiles of `rows` = 2^q_log queries of
// 2^h_log heads each (tensor-core kernels): one TMA box, in which a tile of few
// queries is filled up with further heads of the group, as long as their number
// divides it (so that no row of another group is ever in a tile).
struct CrossTile {
  int q_log, h_log;
  __host__ __device__ int queries() const { return 1 << q_log; }
  __host__ __device__ int heads() const { return 1 << h_log; }
  __host__ __device__ int chunks(int Nq) const { return (Nq + queries() - 1) >> q_log; }   // of a head's queries
  __host__ __device__ int count(int Nq, int G) const { return chunks(Nq) * (G >> h_log); }  // of a group's rows
};
// The tile of at most 2^most rows for Nq queries and groups of G heads; no fewer than
// 2^least queries.
inline CrossTile cross_tile(int Nq, int G, int most, int least) {
  CrossTile t;
  t.q_log = least;
  while (t.q_log < most && (1 << t.q_log) < Nq) ++t.q_log;
  t.h_log = 0;
  while (t.q_log + t.h_log < most && G % (2 << t.h_log) == 0) ++t.h_log;
  return t;
}

struct CrossPlan {
  int k_splits;  // each takes an even share of a sequence's key blocks
  int q_splits;  // of its query steps (steps run over the group's heads and its queries)
  CrossTile q_tile;  // of the forward and dQ (128 rows)
  CrossTile step;    // of the dK/dV kernel's query steps (64 rows)
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

// One (batch, key head), a split of the keys, and up to kTiles consecutive row tiles of
// the group: what a block of the forward (two tiles) or of dQ (one) works on at a time.
struct CrossUnit {
  int b, hk, split, nq, first;  // first: the first tile
  int j_begin, j_end, blocks;   // keys, and their blocks of 128 (0: nothing to compute)
};
// A row tile of a unit.
struct CrossRows {
  int q0, h0;        // first query and head (of all heads)
  bool there, live;  // the tile exists, and has a real query (where its unit has blocks)
};

template <int kTiles>
__device__ __forceinline__ int cross_units(const CrossParams& p) {
  return p.B * p.Hk * ((p.plan.q_tile.count(p.Nq, p.G) + kTiles - 1) / kTiles) * p.plan.k_splits;
}

__device__ __forceinline__ CrossRows cross_rows(const CrossParams& p, const CrossUnit& u, int tile) {
  const CrossTile& t = p.plan.q_tile;
  const int chunks = t.chunks(p.Nq), group = tile / chunks;
  CrossRows r;
  r.q0 = (tile - group * chunks) << t.q_log;
  r.h0 = u.hk * p.G + (group << t.h_log);
  r.there = (group << t.h_log) < p.G;
  r.live = r.there && r.q0 < u.nq;
  return r;
}

// idx: split fastest, then the tiles of a (batch, key head), which share its keys through L2.
template <int kTiles>
__device__ __forceinline__ void cross_unit(const CrossParams& p, int idx, CrossUnit& u) {
  const int sets = (p.plan.q_tile.count(p.Nq, p.G) + kTiles - 1) / kTiles;
  const int rest = idx / p.plan.k_splits;
  u.split = idx - rest * p.plan.k_splits;
  const int bh = rest / sets;
  u.first = (rest - bh * sets) * kTiles;
  u.b = bh / p.Hk;
  u.hk = bh - u.b * p.Hk;
  u.nq = cross_q_len(p, u.b);
  // the sequence's blocks in even shares
  const int nk = cross_k_len(p, u.b), per = ((nk + 127) / 128 + p.plan.k_splits - 1) / p.plan.k_splits * 128;
  u.j_begin = u.split * per;
  u.j_end = min(nk, u.j_begin + per);
  bool any = false;
#pragma unroll
  for (int x = 0; x < kTiles; ++x) any |= cross_rows(p, u, u.first + x).live;
  u.blocks = any ? max(u.j_end - u.j_begin + 127, 0) >> 7 : 0;
}

// The same number, opaque to the compiler: what is computed from it is computed anew instead of being kept
// in registers since the first time (the row-math loops have none to spare, and their spills miss L1).
__device__ __forceinline__ int again(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// 16 fp32 values of the accumulators, times mul as 16-bit values, or as they are, to consecutive places.
template <bool kBf16>
__device__ __forceinline__ void store16_h(uint16_t* to, const uint32_t* r, float mul) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack2<kBf16>(__uint_as_float(r[8 * t + 2 * e]) * mul, __uint_as_float(r[8 * t + 2 * e + 1]) * mul);
    reinterpret_cast<uint4*>(to)[t] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void store16_f(float* to, const uint32_t* r, float mul = 1.f) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
    reinterpret_cast<float4*>(to)[t] =
        make_float4(__uint_as_float(r[4 * t]) * mul, __uint_as_float(r[4 * t + 1]) * mul,
                    __uint_as_float(r[4 * t + 2]) * mul, __uint_as_float(r[4 * t + 3]) * mul);
}

// Zeros to rows [from, to) of a tile of 128-byte rows in kPanels panels in shared memory, by one
// converged warp, ordered before the MMAs that it issues next (swizzles permute within a row).
template <int kPanels>
__device__ __forceinline__ void zero_rows(uint32_t tile, uint32_t panel, int from, int to) {
  for (int c = (threadIdx.x & 31) + 8 * from; c < 8 * to; c += 32)
#pragma unroll
    for (int pn = 0; pn < kPanels; ++pn) st_shared_v4(tile + pn * panel + 16 * c, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

cudaError_t launch_cross_preprocess(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_join_fwd(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_join_dq(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_join_dkdv(const CrossParams& p, int dtype, cudaStream_t st);

// maps: Q (boxes of the tile's queries x heads), K, V (boxes of 128 rows), all of 64 head-dim
// elements, 128-byte swizzle.
cudaError_t launch_cross_fwd_tc(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st);

// maps: Q (boxes of the query step's rows), K, V (boxes of 128 rows), dO (as Q).
cudaError_t launch_cross_dkdv_tc(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st);
// maps: Q (boxes of the tile's rows), K, V (boxes of 128 rows), dO (as Q).
cudaError_t launch_cross_dq_tc(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st);

cudaError_t launch_cross_fwd_f32(const CrossParams& p, cudaStream_t st);
cudaError_t launch_cross_dq_f32(const CrossParams& p, cudaStream_t st);
cudaError_t launch_cross_dkdv_f32(const CrossParams& p, cudaStream_t st);

}  // namespace fa
