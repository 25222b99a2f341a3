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

// fp16 has no normal values below 2^-14, where P is over more than 2^14 keys: the dV product takes P * 2^15 (at most
// 2^15), with 2^-15 on the sums; -L * log2(e) is kept with the 15 added. Without, over 40000 even keys dV was 3.4
// times as far off as its own rounding (1.0 so).
template <bool kBf16>
constexpr float kCrossPLog2 = kBf16 ? 0.f : 15.f;
template <bool kBf16>
constexpr float kCrossPUnit = kBf16 ? 1.f : 32768.f;

// dS in fp16. |dP_ij - D_i| <= bound_i = 2 |dO_i| max_j |V_j| (2-norms, the sequence's real keys; D is a mean of
// dP): above 65504 dS is infinite and below 2^-14 loses its bits and its residual, both within the range of ordinary
// calls (loss scaling; upstream gradients of 1e-3 over 4096 keys). So dS enters dQ's product times 2^e of its row, and
// dK's times 2^e of its key head (by the largest bound of the group's rows), 2^e bound in [2^14, 2^15), and the sums
// are multiplied by 2^-e. dQ of 200 queries over 4096 keys with dO of 1e-3 6.2 -> 1.0 times its own rounding, dK 2.3
// -> 1.0.
__device__ __forceinline__ int cross_exponent(float dout_norm, float v_norm) {
  const int bits = __float_as_int(2.f * dout_norm * v_norm);
  return min(max(14 + 127 - (bits >> 23 & 255), -64), 100);  // (0, infinity, NaN: any will do)
}
__device__ __forceinline__ float power_of_2(int e) { return __int_as_float((e + 127) << 23); }
constexpr int kMostNorms = 64;  // partial maxima of |V_j|^2 of a (batch, key head)

struct CrossPlan {
  int k_splits;  // each takes an even share of a sequence's key blocks
  int q_splits;  // of its query steps (steps run over the group's heads and its queries)
  CrossTile q_tile;  // of the forward and dQ (128 rows)
  CrossTile step;    // of the dK/dV kernel's query steps (64 rows)
  int kv_blocks, q_blocks;  // the backward's blocks for dK/dV and for dQ, which share out the units
  bool few;                 // the forward's kernel of few rows
  int few_cluster;
  bool few_sorted;          // its blocks take the sequences in the order of falling lengths
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
  // Backward: -L * log2(e) (+ kCrossPLog2) and -D of every query row, [B * Hq, nq_pad], -inf and 0
  // where a row is not there (padding, past its sequence, without keys).
  float* nL2;
  float* nD;
  int nq_pad;
  // fp16 (cross_exponent): |dO_i| of every query row, [B * Hq, nq_pad], and of every (batch, key head) the largest
  // (bits of a float that is not negative) and partial maxima of |V_j|^2, [B * Hk, v_norms].
  float* dout_norm;
  unsigned int* dout_most;
  float* v_norm;
  int v_norms;
  // Split results in fp32: the forward's normalised outputs [k_splits][B, Nq, Hq, d]
  // and their log2-sum-exp2 [k_splits][B, Hq, Nq] (-inf: the split has no key of the
  // row, and no output is there); dQ [k_splits][B, Nq, Hq, d]; dK and dV
  // [q_splits][2][B, Nk, Hk, d], of the rows of real keys.
  float* part;
  float* part_lse;
  float* part_kv;
  CrossPlan plan;
  int few_cluster;  // few rows: blocks of a cluster that share a sequence's keys (0: k_splits through the workspace)
  unsigned int* status;
};

__device__ __forceinline__ int cross_q_len(const CrossParams& p, int b) {
  return p.q_lens ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
}
__device__ __forceinline__ int cross_k_len(const CrossParams& p, int b) {
  return p.k_lens ? min(max(p.k_lens[b], 0), p.Nk) : p.Nk;
}

// One (batch, key head), a split of the keys, and up to two consecutive row tiles of the
// group: what a block of the forward (two tiles) or of dQ (one) works on at a time. A
// block's units are decoded once, side by side, into records in shared memory: the lengths
// in memory and the divisions, about 2000 cycles, were as much as two key blocks' work
// where every warp decoded its next unit by itself.
struct CrossUnit {
  int b, hk, split, nq;
  int j_begin, j_end, blocks;  // keys, and their blocks of 128 (0: nothing to compute)
  int q0[2], h0[2];            // first query and head (of all heads) of a tile
  float v_norm;                // fp16, dQ: the largest |V_j| (cross_v_norm)
  int has;                     // bit x: tile x exists; bit 2 + x: it has a real query
  __device__ __forceinline__ bool there(int x) const { return has >> x & 1; }
  __device__ __forceinline__ bool live(int x) const { return has >> (2 + x) & 1; }
};
constexpr int kMostUnits = 32;  // of a block

template <int kTiles>
__device__ __forceinline__ int cross_units(const CrossParams& p) {
  return p.B * p.Hk * ((p.plan.q_tile.count(p.Nq, p.G) + kTiles - 1) / kTiles) * p.plan.k_splits;
}

// idx: split fastest, then the tiles of a (batch, key head), which share its keys through L2.
template <int kTiles>
__device__ __forceinline__ void cross_unit(const CrossParams& p, int idx, CrossUnit& u) {
  const CrossTile& t = p.plan.q_tile;
  const int sets = (t.count(p.Nq, p.G) + kTiles - 1) / kTiles, chunks = t.chunks(p.Nq);
  const int rest = idx / p.plan.k_splits;
  u.split = idx - rest * p.plan.k_splits;
  const int bh = rest / sets, set = rest - bh * sets;
  u.b = bh / p.Hk;
  u.hk = bh - u.b * p.Hk;
  u.nq = cross_q_len(p, u.b);
  // the sequence's blocks in even shares
  const int nk = cross_k_len(p, u.b), per = ((nk + 127) / 128 + p.plan.k_splits - 1) / p.plan.k_splits * 128;
  u.j_begin = u.split * per;
  u.j_end = min(nk, u.j_begin + per);
  u.has = 0;
#pragma unroll
  for (int x = 0; x < kTiles; ++x) {
    const int tile = set * kTiles + x, group = tile / chunks;
    u.q0[x] = (tile - group * chunks) << t.q_log;
    u.h0[x] = u.hk * p.G + (group << t.h_log);
    if ((group << t.h_log) < p.G) u.has |= (1 << x) | (u.q0[x] < u.nq ? 4 << x : 0);
  }
  u.blocks = u.has >> 2 ? max(u.j_end - u.j_begin + 127, 0) >> 7 : 0;
}

// A value that every lane of a converged warp holds alike, as one that the compiler knows to be uniform.
// The MMA-issuing warps' loops run over units that are decoded from lengths in memory; with trip counts
// and stages that were not known to be uniform an MMA took about 100 cycles to issue instead of 25.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Four 16-byte pieces of a lane's row, u[0 .. 3], to the quad's four lanes: lane q of a quad gets piece q of
// row r (of the quad's four rows) in u[r]. The stores behind it then cover 64 consecutive bytes of a row with
// four lanes instead of 16 with one (a warp's store instruction touches 8 lines instead of 32; the epilogue
// of a 128-row tile was bound by that, 3300 cycles).
__device__ __forceinline__ void quad_transpose(uint4 (&u)[4]) {
  const int q = threadIdx.x & 3;
  // hi lanes give a and get b's place, the others the reverse
  const auto swap = [](uint4& a, uint4& b, bool hi, int o) {
    uint4 give = hi ? a : b;
    give.x = __shfl_xor_sync(0xffffffffu, give.x, o);
    give.y = __shfl_xor_sync(0xffffffffu, give.y, o);
    give.z = __shfl_xor_sync(0xffffffffu, give.z, o);
    give.w = __shfl_xor_sync(0xffffffffu, give.w, o);
    if (hi)
      a = give;
    else
      b = give;
  };
  swap(u[0], u[1], q & 1, 1);
  swap(u[2], u[3], q & 1, 1);
  swap(u[0], u[2], q & 2, 2);
  swap(u[1], u[3], q & 2, 2);
}

// Stores of a converged warp's 32 rows, 64 bytes of each: u holds the lane's own row's, `to` the place of
// the lane's own row, or null where the row is not stored.
__device__ __forceinline__ void store_rows64(uint4 (&u)[4], char* to) {
  quad_transpose(u);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const auto whole = reinterpret_cast<unsigned long long>(to);
    char* at = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, whole, (lane & ~3) + r));
    if (at != nullptr) reinterpret_cast<uint4*>(at)[lane & 3] = u[r];
  }
}

// The same with 32 bytes of each row, by pairs of lanes.
__device__ __forceinline__ void store_rows32(uint4 (&u)[2], char* to) {
  const int lane = threadIdx.x & 31;
  uint4 give = lane & 1 ? u[0] : u[1];
  give.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
  give.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
  give.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
  give.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
  if (lane & 1)
    u[0] = give;
  else
    u[1] = give;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const auto whole = reinterpret_cast<unsigned long long>(to);
    char* at = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, whole, (lane & ~1) + r));
    if (at != nullptr) reinterpret_cast<uint4*>(at)[lane & 1] = u[r];
  }
}

// 32 fp32 values of a row as 16-bit ones times mul, 16 as they are (times mul).
template <bool kBf16>
__device__ __forceinline__ void pack64(uint4 (&u)[4], const uint32_t (&r)[32], float mul) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack2<kBf16>(__uint_as_float(r[8 * t + 2 * e]) * mul, __uint_as_float(r[8 * t + 2 * e + 1]) * mul);
    u[t] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void pack64(uint4 (&u)[4], const uint32_t* r, float mul) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(r[4 * t + e]) * mul);
    u[t] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 32 columns of a converged warp's 32 accumulator rows to memory: as 16-bit values at `out`, or as fp32 at
// `part`, times mul; both null where the row is not stored.
template <bool kBf16>
__device__ __forceinline__ void store_columns32(const uint32_t (&r)[32], float mul, bool parts, float* part,
                                                uint16_t* out) {
  uint4 u[4];
  if (parts) {
    pack64(u, r, mul);
    store_rows64(u, reinterpret_cast<char*>(part));
    pack64(u, r + 16, mul);
    store_rows64(u, reinterpret_cast<char*>(part != nullptr ? part + 16 : nullptr));
  } else {
    pack64<kBf16>(u, r, mul);
    store_rows64(u, reinterpret_cast<char*>(out));
  }
}

// The same with the first 16 columns of r.
template <bool kBf16>
__device__ __forceinline__ void store_columns16(const uint32_t (&r)[32], float mul, bool parts, float* part,
                                                uint16_t* out) {
  uint4 u[4];
  if (parts) {
    pack64(u, r, mul);
    store_rows64(u, reinterpret_cast<char*>(part));
  } else {
    uint4 v[2];
    pack64<kBf16>(u, r, mul);
    v[0] = u[0];
    v[1] = u[1];
    store_rows32(v, reinterpret_cast<char*>(out));
  }
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

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += a b of 16 x 8 x 16, one warp.
template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// max_j |V_j| of a (batch, key head).
__device__ __forceinline__ float cross_v_norm(const CrossParams& p, int bh) {
  float top = 0.f;
#pragma unroll 8
  for (int i = 0; i < p.v_norms; ++i) top = fmaxf(top, p.v_norm[(long long)bh * p.v_norms + i]);
  return sqrtf(top);
}

cudaError_t launch_cross_preprocess_f32(const CrossParams& p, cudaStream_t st);
cudaError_t launch_cross_join_fwd(const CrossParams& p, int dtype, cudaStream_t st);
cudaError_t launch_cross_join_bwd(const CrossParams& p, int dtype, cudaStream_t st);

// launch_chained (fa_serve.h) for the kernels that take tensor maps beside their parameters.
template <typename... Args>
cudaError_t launch_chained_maps(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t st,
                                const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// maps: Q (boxes of the tile's queries x heads), K, V (boxes of 128 rows), all of 64 head-dim
// elements, 128-byte swizzle.
cudaError_t launch_cross_fwd_tc(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st);

// -L * log2(e) and -D of the query rows, 16-bit types. maps: Q and dO of the query tiles, K, V (boxes of 128 rows).
cudaError_t launch_cross_dot(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st);

// dK, dV and dQ. maps: Q and dO of the query steps, Q and dO of the query tiles, K, V (boxes of 128 rows).
cudaError_t launch_cross_bwd_tc(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st);

// Forward of few rows a key head (16-bit types).
cudaError_t launch_cross_few(const CrossParams& p, bool bf16, cudaStream_t st);

cudaError_t launch_cross_fwd_f32(const CrossParams& p, cudaStream_t st);
cudaError_t launch_cross_bwd_f32(const CrossParams& p, cudaStream_t st);

}  // namespace fa
