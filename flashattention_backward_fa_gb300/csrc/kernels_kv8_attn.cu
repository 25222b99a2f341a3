// Attention of the newest tokens of each sequence over its 8-bit paged cache.
//
//   S_rj = scale * q_r . k_j (- m |i_r - j|), masked;  O_r = sum_j softmax(S_r)_j v_j
//
// for the rows r = (token t, query head) that share a key head, with k_j, v_j =
// code * scale of the page. It is bound by reading the cache once (2 bytes per
// head value of a token), so everything serves keeping loads in flight:
//
// * Queries are the narrow side of the products: S^T = K Q^T and O^T = V^T P^T,
//   16 keys x 8 rows an instruction (mma.sync, fp32 sums). A tcgen05 tile has at
//   least 64 rows of M from shared memory; with one to a few dozen rows, V would
//   have to be widened and P written to shared memory and read again, while here
//   codes and weights go from registers to the instruction. Its rate is not what
//   bounds the kernel up to 16 rows.
// * Any order of the head dimension serves S, and any order of the output
//   columns serves O: a lane takes 16 consecutive codes of a key (K) or of a
//   key's values (V) and uses them in place.
// * K's codes enter the e4m3 instruction (k32, measured at 0.94 a clock and SM,
//   four times the f16 rate, sums exact to fp32) as they are. The queries are
//   divided by a power of two of each row and written as two (bf16) or three (f16)
//   e4m3 pieces, each the rounding error of those before it times 16. The largest
//   value of a row is brought to [2^7, 2^8) and the pieces end at 2^-13 (2^-17), so a
//   query is exact where its bits end at 2^-20 (2^-24) of the row's largest value, and
//   else off by at most 2^-21 (2^-25) of it. Widening K to f16 instead took 48 more ALU
//   operations a step, at 2 a clock and SM.
// * V's codes are widened to f16 (exact) for the f16 instruction, because the
//   weights P need its range: an e4m3 piece ends 2^-18 below the largest weight,
//   and a long sequence can hold most of its mass below that.
// * Running maximum and sum per row in fp32, kept per lane. A row has two references
//   in the exponent: m for the sum of its weights 2^(s - m), and mv for its outputs,
//   whose factors are P = 2^(s - mv) times the page's V scale. P is what enters f16, so
//   what counts there is a key's weight times the size of its page's values: pages
//   with values of any two sizes may lie in one step, and a page that a row does not
//   attend to has no say in its mv. A reference moves only when it is exceeded by 2^15
//   (P is then at most 2^15, inside f16), and is set so that the largest P is 2^7, so
//   warps agree on new ones a few times a sequence and vote otherwise. P is rounded to
//   f16 (2^-11 of itself, or 2^-32 of the row's largest below 2^-21 of it), and its
//   rounding residual is multiplied too (then 2^-22). bf16 outputs with two row tiles go
//   without the residual: their own rounding is 2^-8, the error against 64 bits the same
//   to two digits (1.6e-3), and the products bound that form (16 sequences of 8192 tokens
//   with 16 rows a key head 75.3 us with it, 66.8 us without). With one row tile, which
//   the cache's bytes bound, it costs 1 to 5% (32 sequences of up to 16384 tokens 100.5 us
//   against 98.7 us, 128 of up to 500 tokens 26.6 us against 25.2 us) and brings the
//   outputs to those of 32-bit weights but for 1e-5 to 7e-5 (5e-4 to 9e-4 without).
// * Four warps take steps of 32 keys (two tiles, whose chains of instructions
//   overlap) in turn. The next step is on its way to the warp's own part of shared
//   memory (cp.async), so a warp waits for itself alone, and 96 KB an SM are in
//   flight without a register. Eight lanes copy one 128-byte line: copied in the
//   order in which lanes use them, the codes of eight lanes lie in two (K) or four
//   (V) lines, and the lines a clock of L1, not DRAM, bounded the kernel at 61% of
//   the copy rate whatever else it did. Lines are swizzled so that neither the
//   copies nor the reads in the instructions' order meet in a bank.
// * A sequence's keys are split over blocks: up to eight blocks of a cluster join
//   their outputs through distributed shared memory; where few sequences and
//   heads leave the GPU empty otherwise, more blocks write normalised outputs
//   that a second kernel joins.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;
constexpr int kTile = 16;       // keys of an instruction
constexpr int U = 2;            // tiles of a step
constexpr int kHopKeys = kTile * U * kWarps;  // keys of a step of all warps; splits are multiples of it
constexpr float kNoMax = -3.0e38f;  // m and mv before any score
constexpr float kHead = 7.f;    // a new reference is set that far below the maximum, whose P is then 2^7
constexpr float kTop = 15.f;    // scores may pass a reference by this much before it moves (log2): P stays within 2^15
constexpr float kLeastScale = 7.888609052210118e-31f;  // 2^-100: V scales below it count as it for mv

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two fp32 values to a pair of e4m3 codes, lo in the low byte, and what the rounding leaves, times 16.
__device__ __forceinline__ uint32_t e4m3_piece(float& lo, float& hi) {
  uint16_t r;
  uint32_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(r));
  float a, b;
  unpack2<false>(h, a, b);
  lo = (lo - a) * 16.f;
  hi = (hi - b) * 16.f;
  return r;
}

// Four codes to two f16 pairs (exact).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 8 x 8 matrix of 16-bit values, two a lane, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLn2 = 0.6931471805599453f;

// All threads of the cluster: shared-memory writes before it are seen behind it by the other blocks.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
// A word of block `rank`'s shared memory at the place of this block's p.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float read_cluster_f32(const void* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 read_cluster_f32x4(const void* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(p, rank))
               : "memory");
  return v;
}

// What a block needs to know of its sequence: keys [lo, hi) are those that some
// row of the row tile attends to, lo rounded down to a tile.
struct Range {
  int len, count;  // tokens of the sequence; how many of them are new
  int keys;        // keys that exist for attention
  int lo, hi;
};

__device__ __forceinline__ Range key_range(const Kv8AttnParams& p, int b, int row_lo, int row_hi) {
  Range r;
  r.len = max(p.c.seq_lens[b], 0);
  r.count = p.c.new_lens ? min(max(p.c.new_lens[b], 0), p.T) : p.T;
  r.keys = min(r.len, p.key_limit);
  // rows [row_lo, row_hi) hold tokens t_lo .. t_hi at positions len - count + t
  const int t_lo = max(row_lo / p.G, r.count - r.len), t_hi = min((row_hi - 1) / p.G, r.count - 1);
  r.lo = r.hi = 0;
  if (t_lo <= t_hi) {
    const int i_lo = r.len - r.count + t_lo, i_hi = r.len - r.count + t_hi;
    r.hi = p.causal ? min(r.keys, i_hi + 1) : r.keys;
    r.lo = p.window > 0 ? max(0, i_lo - p.window + 1) & ~(kTile - 1) : 0;
    if (r.lo >= r.hi) r.lo = r.hi = 0;
  }
  return r;
}

// The sequence that comes at `place` in the order of falling lengths (up to 2^24 - 1), equal ones
// by their number. `ranks` is shared memory for kThreads numbers.
__device__ __forceinline__ int sequence_of(const Kv8AttnParams& p, int place, int* ranks) {
  static_assert(kThreads == 128, "a number takes 7 bits");
  __shared__ int found;
  const int me = threadIdx.x;
  const int mine = me < p.B ? min(max(p.c.seq_lens[me], 0), (1 << 24) - 1) * kThreads + kThreads - 1 - me : -1;
  ranks[me] = mine;
  __syncthreads();
  int before = 0;
#pragma unroll 4
  for (int i = 0; i < p.B; i += 4) {
    const int4 x = *reinterpret_cast<const int4*>(ranks + i);  // (those past the last are behind all)
    before += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
  }
  if (me < p.B && before == place) found = me;
  __syncthreads();
  return found;
}

// Keys of a split: the plan's, or, in a cluster, the sequence's own keys shared out evenly.
__device__ __forceinline__ int split_keys(const Kv8AttnParams& p, const Range& r) {
  if (!p.cluster) return p.chunk;
  const int n = r.hi - r.lo, per = p.splits * kHopKeys;
  return max(1, (n + per - 1) / per) * kHopKeys;
}

// Shared memory of the steps under way: a stage holds U tiles a warp, a tile 16
// keys of K and of V in 128-byte lines (a key, or two with D = 64). Sixteen-byte
// chunk x of line y lies at x ^ swizzle(y).
template <int D>
struct Ring {
  static constexpr int kLines = D / 8;             // lines of a tile of K, and of V
  static constexpr int kHalf = kLines * 128;       // bytes of K (then V) of a tile
  static constexpr int kStages = (D == 128 ? 4 : 8) / U;
  static constexpr int kWarpBytes = U * 2 * kHalf;
  static constexpr int kStageBytes = kWarps * kWarpBytes;
  static constexpr int kScales = kStages * kStageBytes;  // then (K scale, V scale) a stage, warp and tile
  static constexpr int kBytes = kScales + kStages * kWarps * U * 8;
};

__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 read_slot16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 read_slot8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// What a lane keeps to start its copies: its place in page 0 of the head, its rows' stride (a
// page's offsets fit into 31 bits, the entry point sees to it) and its slots. Lane l copies
// chunk l % 8 of lines l / 8, l / 8 + 4, ... of a tile.
template <int D>
struct Fetch {
  using G = Ring<D>;
  const uint8_t* k;
  const uint8_t* v;
  const float* scale;  // lane 0: K's, lane 1: V's
  uint32_t slot_k, slot_v, slot_scale;
  __device__ __forceinline__ Fetch(const Kv8Cache& c, uint32_t ring, int h) {
    const int lane = threadIdx.x & 31, line = lane >> 3, x = lane & 7;
    const long long at = (long long)h * c.sh +
                         (D == 128 ? line * (int)c.sn + 16 * x : (2 * line + (x >> 2)) * (int)c.sn + 16 * (x & 3));
    k = c.k + at;
    v = c.v + at;
    scale = (lane ? c.v_scale : c.k_scale) + h;
    const uint32_t base = ring + (threadIdx.x >> 5) * G::kWarpBytes + line * 128;
    slot_k = base + (D == 128 ? x ^ ((line & 1) * 4) : x) * 16;
    slot_v = base + G::kHalf + (D == 128 ? x ^ (line & 2) : x ^ (line * 2)) * 16;
    slot_scale = ring + G::kScales + (threadIdx.x >> 5) * (U * 8) + (lane & 1) * 4;
  }
  // V's slot of the lane's i-th line (with D = 128 the swizzle has a bit of the line past the fourth).
  __device__ __forceinline__ uint32_t v_slot(uint32_t to, int i) const {
    return ((slot_v + to) ^ (D == 128 && (i & 1) ? 64u : 0u)) + i * 512;
  }
  // Tile u of a step, at token `slot` of a page, into a stage. A page outside the cache leaves zeros.
  __device__ __forceinline__ void operator()(const Kv8Cache& c, int stage, int u, int page, int slot,
                                             bool page_ok) const {
    const uint32_t to = stage * G::kStageBytes + u * 2 * G::kHalf;
    if (!page_ok) {
#pragma unroll
      for (int i = 0; i < G::kLines / 4; ++i) {
        st_shared_v4(slot_k + to + i * 512, 0u, 0u, 0u, 0u);
        st_shared_v4(v_slot(to, i), 0u, 0u, 0u, 0u);
      }
      return;
    }
    const int sn = (int)c.sn;
    const long long at = (long long)page * c.sp + slot * sn;
    const uint8_t* kp = k + at;
    const uint8_t* vp = v + at;
    constexpr int kTokens = D == 128 ? 4 : 8;  // tokens of four lines
#pragma unroll
    for (int i = 0; i < G::kLines / 4; ++i) copy16_async(slot_k + to + i * 512, kp + i * kTokens * sn);
#pragma unroll
    for (int i = 0; i < G::kLines / 4; ++i) copy16_async(v_slot(to, i), vp + i * kTokens * sn);
    if ((threadIdx.x & 31) < 2)
      copy4_async(slot_scale + stage * (kWarps * U * 8) + u * 8, scale + (long long)page * c.H);
  }
};

// Bytes of w that hold an e4m3 NaN (0x7F, 0xFF), as 0x80 flags.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) kv8_attn_kernel(const __grid_constant__ Kv8AttnParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kResidual = !kBf16 || NT == 1;  // see the head of the file
  constexpr int NP = kBf16 ? 2 : 3;    // e4m3 pieces of a query
  constexpr int KS = D / 16;           // row tiles of O^T
  constexpr int KQ = D / 32;           // instructions over the head dimension (S)
  constexpr int kRows = 8 * NT;
  __shared__ __align__(16) uint2 q_frag[KQ][NT][NP][32];
  __shared__ float q_factor[kRows];
  __shared__ float w_m[kWarps][kRows], w_l[kWarps][kRows];
  __shared__ float block_lse[kRows];
  extern __shared__ __align__(128) unsigned char dyn[];
  using G = Ring<D>;
  static_assert(G::kScales >= kWarps * kRows * D * 4, "merging reuses the ring");
  const uint32_t ring = smem_u32(dyn);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  // blocks: splits fastest, then heads, then row tiles (x has room for any number of them), then sequences
  const int split = blockIdx.x % p.splits, unit = blockIdx.x / p.splits;
  const int h = unit % p.c.H, rt = unit / p.c.H, R = p.T * p.G;
  const int row0 = rt * kRows;
  // (and no let_next_begin here: blocks of the next call would take the places of this one's; the
  // call at 131071 tokens took 57 us with it at the start, 51.4 us at the end, 51.2 us without)
  wait_for_previous();
  static_assert(sizeof(q_frag) >= kThreads * sizeof(int), "sequence_of uses its place");
  const int b = p.longest_first ? sequence_of(p, blockIdx.z, reinterpret_cast<int*>(q_frag)) : blockIdx.z;
  const Range kr = key_range(p, b, row0, min(row0 + kRows, R));
  const int chunk = split_keys(p, kr);
  const int begin = kr.lo + split * chunk, end = min(kr.hi, begin + chunk);
  // (the joining kernel counts splits the same way; the blocks of a cluster all come along)
  if (begin >= end && p.splits > 1 && !p.cluster) return;

  // Steps of this warp: begin + 16 U warp, + 64 U, ...; kStages - 1 of them are under way while
  // one is computed, their page numbers read one step earlier still.
  constexpr int kStep = kTile * U, kHop = kStep * kWarps;
  const int* table = p.c.table + b * p.c.table_stride;
  const int shift = p.c.page_shift, mask = (1 << shift) - 1;
  const int first = begin + kStep * warp;
  int ahead = first;          // key of the next step to fetch
  uint32_t bad_tiles = 0u;    // bit n U + u: tile u of stage n is in a page outside the cache
  bool bad = false;
  int into = 0;               // stage of the next fetch
  const Fetch<D> copy(p.c, ring, h);
  struct Pages {
    int id[U];
  };
  auto pages_of = [&](int key) {
    Pages pg;
#pragma unroll
    for (int u = 0; u < U; ++u) pg.id[u] = key + kTile * u < end ? table[(key + kTile * u) >> shift] : -1;
    return pg;
  };
  auto fetch = [&](const Pages& pg) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int key = ahead + kTile * u;
      const bool inside = key < end;  // (a tile past the end counts as one outside the cache)
      const bool ok = inside && (unsigned)pg.id[u] < (unsigned)p.c.num_pages;
      if (!ok) {
        bad |= inside;
        bad_tiles |= 1u << (into * U + u);
      }
      if (ahead < end) copy(p.c, into, u, pg.id[u], key & mask, ok);
    }
    copies_commit();
    into = into + 1 == G::kStages ? 0 : into + 1;
    ahead += kHop;
  };
  Pages pages[G::kStages];
#pragma unroll
  for (int i = 0; i < G::kStages; ++i) pages[i] = pages_of(first + i * kHop);
#pragma unroll
  for (int i = 0; i < G::kStages - 1; ++i) fetch(pages[i]);
  Pages next_pages = pages[G::kStages - 1];

  // Queries: row tile nt of this warp's share as e4m3 operand registers in shared memory.
  for (int nt = warp; nt < NT; nt += kWarps) {
    const int row = row0 + 8 * nt + r, t = row / p.G, hq = h * p.G + row % p.G;
    const bool live = row < R && t < kr.count && kr.len - kr.count + t >= 0;
    const T* qp = static_cast<const T*>(p.q) + b * p.q_st.b + (long long)t * p.q_st.n + (long long)hq * p.q_st.h;
    float x[KQ][8], top = 0.f;
#pragma unroll
    for (int i = 0; i < KQ; ++i) {
      const uint4 raw = live ? *reinterpret_cast<const uint4*>(qp + 64 * (i >> 1) + 16 * c + 8 * (i & 1))
                             : make_uint4(0u, 0u, 0u, 0u);
      unpack2<kBf16>(raw.x, x[i][0], x[i][1]);
      unpack2<kBf16>(raw.y, x[i][2], x[i][3]);
      unpack2<kBf16>(raw.z, x[i][4], x[i][5]);
      unpack2<kBf16>(raw.w, x[i][6], x[i][7]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (fabsf(x[i][e]) == INFINITY) x[i][e] = __int_as_float(0x7FC00000);  // (its row becomes NaN)
        top = fmaxf(top, fabsf(x[i][e]));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // largest magnitude of the row to [2^7, 2^8): a division by a power of two
    const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127 - 7, -110), 120);
    const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
    for (int i = 0; i < KQ; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= down;
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const uint32_t w0 = e4m3_piece(x[i][0], x[i][1]), w1 = e4m3_piece(x[i][2], x[i][3]);
        const uint32_t w2 = e4m3_piece(x[i][4], x[i][5]), w3 = e4m3_piece(x[i][6], x[i][7]);
        q_frag[i][nt][n][lane] = make_uint2(w0 | (w1 << 16), w2 | (w3 << 16));
      }
    }
    if (c == 0) q_factor[8 * nt + r] = p.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
  }

  // This lane's rows are 2c and 2c + 1 of every tile: scale, position, slope.
  float m[NT][2], mv[NT][2], l[NT][2], slope[NT][2];
  int pos[NT][2];
  int all_lo = 0, all_hi = kr.hi;  // keys [all_lo, all_hi) are attended by every live row of the block
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = row0 + 8 * nt + 2 * c + e, t = row / p.G;
      pos[nt][e] = kr.len - kr.count + t;
      const bool live = row < R && t < kr.count && pos[nt][e] >= 0;
      if (!live) pos[nt][e] = -1;
      slope[nt][e] = live && p.alibi ? p.alibi[b * p.alibi_sb + h * p.G + row % p.G] * 1.4426950408889634f : 0.f;
      m[nt][e] = mv[nt][e] = kNoMax;
      l[nt][e] = 0.f;
    }
  {
    const int t_lo = max(row0 / p.G, kr.count - kr.len), t_hi = min((min(row0 + kRows, R) - 1) / p.G, kr.count - 1);
    if (p.causal) all_hi = min(all_hi, kr.len - kr.count + t_lo + 1);
    if (p.window > 0) all_lo = max(0, kr.len - kr.count + t_hi - p.window + 1);
  }
  float acc[KS][NT][4];
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
  __syncthreads();
  // One row tile: two pieces of the queries stay in registers, f16's third one is read from shared
  // memory at its use. With all three held the f16 form spilled more in the loop (d = 128, 32
  // sequences of up to 4096 tokens, 32 heads: 132 us against 103 us), with one of bf16's two in
  // shared memory 32 sequences of up to 16384 tokens took 102 us against 100 us. Two row tiles have
  // no register to spare. (At d = 128 f16 still spills 20 bytes at 168 registers and, with two row
  // tiles, 48 bytes at 255; bf16 with two row tiles 16.)
  constexpr int kHeld = NT == 1 ? 2 : 0;
  uint2 q_reg[NT == 1 ? KQ : 1][NP];
#pragma unroll
  for (int i = 0; i < KQ; ++i)
#pragma unroll
    for (int n = 0; n < kHeld; ++n) q_reg[NT == 1 ? i : 0][n] = q_frag[i][0][n][lane];
  float fac[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) fac[nt][e] = q_factor[8 * nt + 2 * c + e];

  // where in a tile the lane reads (key r and value row 2c, each first chunk)
  const uint32_t k_read = D == 128 ? r * 128 + (c ^ ((r & 1) * 4)) * 16 : (r >> 1) * 128 + ((r & 1) * 4 + c) * 16;
  const uint32_t v_read = D == 128 ? 2 * c * 128 + (r ^ (2 * c)) * 16 : c * 128 + ((r >> 1) ^ (2 * c)) * 16 + (r & 1) * 8;

  auto compute = [&](int stage, int at) {
    const uint32_t step_bad = bad_tiles >> (stage * U) & ((1u << U) - 1u);
    if (step_bad) bad_tiles &= ~(((1u << U) - 1u) << (stage * U));
    const uint32_t slot = ring + stage * G::kStageBytes + warp * G::kWarpBytes;
    float ks[U], vs[U], sc[U][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                   : "=f"(ks[u]), "=f"(vs[u])
                   : "r"(ring + G::kScales + ((stage * kWarps + warp) * U + u) * 8)
                   : "memory");
      // codes [64 x + 16 c, + 16) of keys r and r + 8
      uint4 kv[2 * (D / 64)];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          kv[i * (D / 64) + x] = read_slot16(((slot + k_read) ^ (64u * x)) + u * 2 * G::kHalf + i * (G::kHalf / 2));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float part[NP][4];
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[n][e] = 0.f;
#pragma unroll
        for (int i = 0; i < KQ; ++i) {
          const uint4 k0 = kv[i >> 1], k1 = kv[(D / 64) + (i >> 1)];
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            const uint2 f = n < kHeld ? q_reg[NT == 1 ? i : 0][n] : q_frag[i][nt][n][lane];
            mma_e4m3(part[n], i & 1 ? k0.z : k0.x, i & 1 ? k1.z : k1.x, i & 1 ? k0.w : k0.y, i & 1 ? k1.w : k1.y, f.x, f.y);
          }
        }
        const float f[2] = {ks[u] * fac[nt][0], ks[u] * fac[nt][1]};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = part[NP - 1][e];
#pragma unroll
          for (int n = NP - 2; n >= 0; --n) x = fmaf(x, 0.0625f, part[n][e]);
          sc[u][nt][e] = x * f[e & 1];
        }
      }
    }
    const bool whole = at >= all_lo && at + kStep <= all_hi && step_bad == 0u;
    auto attends = [&](int u, int nt, int e) {
      const int j = at + kTile * u + r + 8 * (e >> 1), i = pos[nt][e & 1];
      return !(step_bad >> u & 1u) && j < kr.keys && i >= 0 && (!p.causal || j <= i) && (p.window <= 0 || j > i - p.window);
    };
    if (p.alibi) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[u][nt][e] = fmaf(-slope[nt][e & 1], fabsf((float)(pos[nt][e & 1] - (at + kTile * u + r + 8 * (e >> 1)))),
                                sc[u][nt][e]);
    }
    if (!whole) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!attends(u, nt, e)) sc[u][nt][e] = -INFINITY;
    }
    float lv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (step_bad >> u & 1u) vs[u] = 0.f;  // (was not fetched)
      lv[u] = lg2_approx(fmaxf(fabsf(vs[u]), kLeastScale));
    }
    bool over = false;
    float top[NT][2], top_v[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[nt][e] = top_v[nt][e] = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float x = fmaxf(sc[u][nt][e], sc[u][nt][e + 2]);
          top[nt][e] = fmaxf(top[nt][e], x);
          top_v[nt][e] = fmaxf(top_v[nt][e], x + lv[u]);
        }
        over |= top[nt][e] > m[nt][e] + kTop || top_v[nt][e] > mv[nt][e] + kTop;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = top[nt][e], y = top_v[nt][e];
#pragma unroll
          for (int lanes = 4; lanes <= 16; lanes *= 2) {
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, lanes));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, lanes));
          }
          if (x > m[nt][e] + kTop) {
            l[nt][e] *= ex2_approx(m[nt][e] - (x - kHead));
            m[nt][e] = x - kHead;
          }
          if (y > mv[nt][e] + kTop) {
            const float to = y - kHead, f = ex2_approx(mv[nt][e] - to);
            mv[nt][e] = to;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              acc[i][nt][e] *= f;
              acc[i][nt][e + 2] *= f;
            }
          }
        }
    }
    // 2^(m - mv), which takes a weight of the sum to its P: in two factors, because with V scales up to
    // 2^120 and down to 2^-100 it alone may leave fp32's range
    float to_p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) to_p[nt][e] = ex2_approx(m[nt][e] - mv[nt][e] + 10.f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t b0[NT], b1[NT], d0[NT], d1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = ex2_approx(sc[u][nt][e] - m[nt][e & 1]);
          l[nt][e & 1] += x[e];
          x[e] *= vs[u] * 0.0009765625f * to_p[nt][e & 1];
        }
        const uint32_t lo = pack2<false>(x[0], x[1]), hi = pack2<false>(x[2], x[3]);
        if (kResidual) {
          d0[nt] = transpose8x8(pack2_residual<false>(x[0], x[1], lo));
          d1[nt] = transpose8x8(pack2_residual<false>(x[2], x[3], hi));
        }
        b0[nt] = transpose8x8(lo);
        b1[nt] = transpose8x8(hi);
      }
      // values [(D / 8) r, + D / 8) of keys 2c, 2c + 1, 2c + 8, 2c + 9
      uint32_t v[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t far = u * 2 * G::kHalf + G::kHalf + (i >> 1) * (G::kHalf / 2);
        if (D == 128) {
          const uint4 x = read_slot16(slot + v_read + far + (i & 1) * 128);
          v[i][0] = x.x, v[i][1] = x.y, v[i][D / 32 - 2] = x.z, v[i][D / 32 - 1] = x.w;
        } else {
          const uint2 x = read_slot8(((slot + v_read) ^ (64u * (i & 1))) + far);
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
      if (!whole) {
        // Values behind the last key are whatever the page holds: zeros for the
        // product. A NaN among the others belongs to the rows that attend to its
        // key and to no other row, but the product would give it to all (0 * NaN):
        // it is taken out here, and rows that attend to it get their NaN by a
        // product of where the NaNs are with who attends.
        bool has = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool dead = at + kTile * u + 2 * c + (i & 1) + 8 * (i >> 1) >= kr.keys;
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            if (dead) v[i][w] = 0u;
            has |= nan_bytes(v[i][w]) != 0u;
          }
        }
        if (__any_sync(0xffffffffu, has)) {
          uint32_t i0[NT], i1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            i0[nt] = transpose8x8((attends(u, nt, 0) ? 0x3C00u : 0u) | (attends(u, nt, 1) ? 0x3C000000u : 0u));
            i1[nt] = transpose8x8((attends(u, nt, 2) ? 0x3C00u : 0u) | (attends(u, nt, 3) ? 0x3C000000u : 0u));
          }
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            const int w = mt >> 1, sh = 16 * (mt & 1);
            uint32_t f[4];  // NaN flags of the two values of this tile for the four keys
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = nan_bytes(v[i][w]) >> sh;
            auto pair = [](uint32_t x, uint32_t y, uint32_t bit) {
              return ((x & bit) ? 0x3C00u : 0u) | ((y & bit) ? 0x3C000000u : 0u);
            };
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float hit[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(hit, pair(f[0], f[1], 0x80u), pair(f[0], f[1], 0x8000u), pair(f[2], f[3], 0x80u),
                      pair(f[2], f[3], 0x8000u), i0[nt], i1[nt]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (hit[e] > 0.f) acc[mt][nt][e] = __int_as_float(0x7FC00000);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[i][w] &= ~((nan_bytes(v[i][w]) >> 7) * 0xFFu);
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        // codes of two keys side by side: bytes (k0.0, k1.0, k0.1, k1.1) and (k0.2, k1.2, k0.3, k1.3)
        const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
        uint32_t a[2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          widen4(half ? x1 : x0, a[half][0], a[half][1]);
          widen4(half ? y1 : y0, a[half][2], a[half][3]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            mma_f16(acc[2 * w + half][nt], a[half][0], a[half][1], a[half][2], a[half][3], b0[nt], b1[nt]);
        if (kResidual) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              mma_f16(acc[2 * w + half][nt], a[half][0], a[half][1], a[half][2], a[half][3], d0[nt], d1[nt]);
        }
      }
    }
  };

  int stage = 0;
  for (int base = first; base < end; base += kHop) {
    const Pages pg = next_pages;
    next_pages = pages_of(base + G::kStages * kHop);
    __syncwarp();  // (every lane has read what the next copies overwrite)
    fetch(pg);
    copies_wait<G::kStages - 1>();
    __syncwarp();  // every lane's copies have landed
    compute(stage, base);
    stage = stage + 1 == G::kStages ? 0 : stage + 1;
  }
  if (bad && lane == 0) atomicOr(p.c.status, kStatusBadPage);
  copies_wait<0>();

  // The warps' sums become one: row sums over the lanes of a row, then every
  // warp's share scaled to the block's maximum and to normalised outputs.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
      l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
      l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
      if (r == 0) {
        w_m[warp][8 * nt + 2 * c + e] = m[nt][e];
        w_l[warp][8 * nt + 2 * c + e] = l[nt][e];
      }
    }
  __syncthreads();
  float lse2[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * nt + 2 * c + e;
      float top = w_m[0][row], sum = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, w_m[w][row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += w_l[w][row] * ex2_approx(w_m[w][row] - top);
      if (pos[nt][e] < 0) sum = 0.f;  // a padding row (unmasked in whole steps)
      lse2[nt][e] = sum == 0.f ? -INFINITY : top + lg2_approx(sum);
      const bool none = sum == 0.f;  // (its sums may hold NaN all the same: a padding row's)
      const float f = 1024.f / sum, g = ex2_approx(mv[nt][e] - top - 10.f);  // (in two factors as above)
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        acc[i][nt][e] = none ? 0.f : acc[i][nt][e] * f * g;
        acc[i][nt][e + 2] = none ? 0.f : acc[i][nt][e + 2] * f * g;
      }
    }
  // Every warp's outputs in shared memory, summed there by (row, four values). Lane (r, c) holds
  // values [(D / 8) r, + D / 8) of rows 2c and 2c + 1 of every tile; chunk x of a row lies at
  // x ^ turn(row), so that eight lanes' stores meet in no bank.
  const auto turn = [](int row) { return D == 128 ? (row >> 1) & 3 : ((row >> 1) & 1) | (row & 4); };
  float* sums = reinterpret_cast<float*>(dyn);  // [kWarps][kRows][D], then in [0] the block's
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * nt + 2 * c + e;
#pragma unroll
      for (int x = 0; x < D / 32; ++x)
        *reinterpret_cast<float4*>(sums + (warp * kRows + row) * D + (((D / 32) * r + x) ^ turn(row)) * 4) =
            make_float4(acc[2 * x][nt][e], acc[2 * x][nt][e + 2], acc[2 * x + 1][nt][e], acc[2 * x + 1][nt][e + 2]);
      if (warp == 0 && r == 0) block_lse[row] = lse2[nt][e];
    }
  __syncthreads();
  const int items = min(kRows, R - row0) * (D / 4);
  const auto out = [&](int row, int x) {
    const int t = (row0 + row) / p.G, hq = h * p.G + (row0 + row) % p.G;
    return static_cast<T*>(p.o) + b * p.o_st.b + (long long)t * p.o_st.n + (long long)hq * p.o_st.h + 4 * x;
  };
  const auto out_lse = [&](int row, float lse) {
    const int t = (row0 + row) / p.G, hq = h * p.G + (row0 + row) % p.G;
    p.lse[((long long)b * p.Hq + hq) * p.T + t] = lse * kLn2;
  };
  for (int item = threadIdx.x; item < items; item += kThreads) {
    const int row = item / (D / 4), x = item % (D / 4);
    float4* at = reinterpret_cast<float4*>(sums + row * D + (x ^ turn(row)) * 4);
    float4 v = at[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 o = at[w * kRows * (D / 4)];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    if (p.cluster) {
      at[0] = v;
    } else if (p.splits == 1) {
      *reinterpret_cast<uint2*>(out(row, x)) = make_uint2(pack2<kBf16>(v.x, v.y), pack2<kBf16>(v.z, v.w));
      if (x == 0) out_lse(row, block_lse[row]);
    } else {
      const long long to = (((long long)b * p.c.H + h) * R + row0 + row) * p.splits + split;
      *reinterpret_cast<float4*>(p.part_o + to * D + 4 * x) = v;
      if (x == 0) p.part_lse[to] = block_lse[row];
    }
  }
  if (!p.cluster) return;
  // Each block of the cluster joins its share of the items from all of them.
  cluster_sync();
  const int n = p.splits;
  for (int item = split * kThreads + threadIdx.x; item < items; item += n * kThreads) {
    const int row = item / (D / 4), x = item % (D / 4);
    float part[kMaxCluster], top = -INFINITY;
    float4 o[kMaxCluster];
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s)
      if (s < n) {
        part[s] = read_cluster_f32(&block_lse[row], s);
        o[s] = read_cluster_f32x4(sums + row * D + (x ^ turn(row)) * 4, s);
        top = fmaxf(top, part[s]);
      }
    float sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s)
      if (s < n) {
        const float w = part[s] == -INFINITY ? 0.f : ex2_approx(part[s] - top);  // (no key for this row there)
        sum += w;
        v[0] = fmaf(w, o[s].x, v[0]), v[1] = fmaf(w, o[s].y, v[1]);
        v[2] = fmaf(w, o[s].z, v[2]), v[3] = fmaf(w, o[s].w, v[3]);
      }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(out(row, x)) =
        make_uint2(pack2<kBf16>(v[0] * inv, v[1] * inv), pack2<kBf16>(v[2] * inv, v[3] * inv));
    if (x == 0) out_lse(row, sum == 0.f ? -INFINITY : top + lg2_approx(sum));
  }
  cluster_sync();  // (no block leaves while another reads its shared memory)
}

// Joins the splits of one row (a block): O = sum_s w_s O_s / sum_s w_s with
// w_s = 2^(lse_s - max). Eight warps take every eighth split.
constexpr int kJoinWarps = 8;

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) kv8_join_kernel(const __grid_constant__ Kv8AttnParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kPer = D / 32;
  __shared__ float acc_s[kJoinWarps][D];
  __shared__ float top_s[kJoinWarps], sum_s[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, h = blockIdx.y, b = blockIdx.z, R = p.T * p.G;
  const int rt = row / (8 * NT);
  wait_for_previous();
  const Range kr = key_range(p, b, rt * 8 * NT, min((rt + 1) * 8 * NT, R));
  const int n = (kr.hi - kr.lo + p.chunk - 1) / p.chunk;
  const long long at = (((long long)b * p.c.H + h) * R + row) * p.splits;
  // every warp on its own, eight of its splits at a time with all their loads under way at once
  float top = -INFINITY, acc[kPer], sum = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int base = warp; base < n; base += 8 * kJoinWarps) {
    float x[8], v[8][kPer];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = base + i * kJoinWarps;
      x[i] = -INFINITY;
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[i][e] = 0.f;
      if (s < n) {
        x[i] = __ldcg(p.part_lse + at + s);
        const float* o = p.part_o + (at + s) * D + kPer * lane;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
          const float2 two = __ldcg(reinterpret_cast<const float2*>(o + e));
          v[i][e] = two.x, v[i][e + 1] = two.y;
        }
      }
    }
    float t = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = fmaxf(t, x[i]);
    const float f = top == t ? 1.f : ex2_approx(top - t);
    sum *= f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = x[i] == -INFINITY ? 0.f : ex2_approx(x[i] - t);  // (a split without a key for this row)
      sum += w;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, v[i][e], acc[e]);
    }
    top = t;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc_s[warp][kPer * lane + e] = acc[e];
  if (lane == 0) {
    sum_s[warp] = sum;
    top_s[warp] = top;
  }
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  top = top_s[0];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, top_s[w]);
  float v[2] = {0.f, 0.f};
  const int e = 2 * threadIdx.x;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = sum_s[w] == 0.f ? 0.f : ex2_approx(top_s[w] - top);
    sum = fmaf(f, sum_s[w], sum);
    v[0] = fmaf(f, acc_s[w][e], v[0]);
    v[1] = fmaf(f, acc_s[w][e + 1], v[1]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int t = row / p.G, hq = h * p.G + row % p.G;
  T* o = static_cast<T*>(p.o) + b * p.o_st.b + (long long)t * p.o_st.n + (long long)hq * p.o_st.h + e;
  *reinterpret_cast<uint32_t*>(o) = pack2<kBf16>(v[0] * inv, v[1] * inv);
  if (threadIdx.x == 0)
    p.lse[((long long)b * p.Hq + hq) * p.T + t] = sum == 0.f ? -INFINITY : (top + lg2_approx(sum)) * kLn2;
}

template <typename T, int D, int NT>
cudaError_t launch_nt(const Kv8AttnParams& p, cudaStream_t st) {
  constexpr auto kKernel = kv8_attn_kernel<T, D, NT>;
  constexpr int kBytes = Ring<D>::kBytes;
  cudaError_t e = allow_smem<kKernel>(kBytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.splits * p.c.H * p.row_tiles, 1, p.B);
  e = launch_chained(kKernel, grid, kThreads, kBytes, p.cluster ? p.splits : 1, p, st);
  if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
  return launch_chained(kv8_join_kernel<T, D, NT>, dim3(p.T * p.G, p.c.H, p.B), 32 * kJoinWarps, 0, 1, p, st);
}

template <typename T, int D>
cudaError_t launch_tiles(const Kv8AttnParams& p, int tiles, cudaStream_t st) {
  return tiles == 1 ? launch_nt<T, D, 1>(p, st) : launch_nt<T, D, 2>(p, st);
}

}  // namespace

// Splits (times: bf16, d = 128, eight key heads where nothing else is said).
// * Up to eight blocks a sequence and row tile join within a cluster, each
//   sequence sharing out its own keys: no workspace, no second kernel. One
//   sequence of 1000 tokens takes 6.95 us so, 7.6 us with the second kernel.
// * Where eight splits leave the GPU empty and a block's share is more than
//   kClusterKeys keys, one resident set of blocks and the joining kernel: one
//   sequence of 4096 tokens 8.3 us against 9.9 us in a cluster; twice as many
//   blocks at 131071 tokens 55 us against 49 us.
// * Where the units alone fill the GPU (kSplitBlocks sets of slots) a split has at
//   least kSplitKeys keys: its start and its merge cost about 4 us. 16 sequences
//   with 5 queries and a window of 1024 (f16, d = 64, 16 heads) 14.2 us against
//   22.9 us with two sets; 32 sequences of up to 16384 tokens 100 us, 140 us
//   unsplit (unequal lengths) and 118 us with splits from 2048 keys on.
// * Where the blocks come in several rounds, the longest sequences come first: a
//   round's free places go to shorter ones (same batch 100 us against 107 us in the
//   given order; 8 sequences of up to 32768 tokens with 64 heads 59 us against 69 us).
//   Each block ranks the lengths for itself, which it can up to its number of threads,
//   in up to a microsecond: worth it where a block may have more than kOrderKeys keys
//   (128 sequences of up to 2048 tokens 56.3 us against 57.7 us, of up to 1024 tokens
//   36.8 us against 36.0 us, of up to 500 tokens 27.1 us against 25.1 us). Where all
//   lengths are equal it costs 1% (32 of 4096 tokens, 32 key heads, 173.6 us against
//   172.5 us).
Kv8AttnPlan kv8_attn_plan(int B, int T, int Hq, int H, int d, int key_limit, int causal, int window) {
  constexpr long long kClusterKeys = 256, hop = kHopKeys;
  constexpr long long kSplitBlocks = 1, kSplitKeys = 4096, kOrderKeys = 1024;
  Kv8AttnPlan plan;
  const long long R = (long long)T * (Hq / H);
  // More than eight rows: 16 a block, further ones in blocks of their own that find the cache in
  // L2. (Blocks of 32 rows spill registers and hold eight warps an SM: 153 us against 126 us for
  // 16 sequences of 4096 tokens with 64 rows a key head; blocks of eight rows 90 us against 69 us
  // for 8192 tokens with 16.)
  plan.tiles = R <= 8 ? 1 : 2;
  plan.row_tiles = (int)((R + 8 * plan.tiles - 1) / (8 * plan.tiles));
  // keys that one block's rows can reach
  long long range = key_limit;
  if (causal && window > 0) range = std::min<long long>(range, (long long)window + T + kTile);
  const long long units = (long long)B * H * plan.row_tiles, slots = 152 * (plan.tiles == 1 ? 3 : 2);
  const auto round_hop = [&](long long x) { return std::max(hop, (x + hop - 1) / hop * hop); };
  long long splits = std::min<long long>(kMaxCluster, (range + hop - 1) / hop);
  while (splits > 1 && units * splits > kSplitBlocks * slots && range / splits < kSplitKeys) splits >>= 1;
  plan.cluster = 1;
  if (units * kMaxCluster < slots && round_hop((range + splits - 1) / splits) > kClusterKeys) {
    plan.cluster = 0;
    splits = std::max<long long>(1, slots / units);
  }
  plan.chunk = (int)round_hop((range + splits - 1) / splits);
  plan.splits = (int)((range + plan.chunk - 1) / plan.chunk);
  if (plan.splits == 1) plan.cluster = 0;
  plan.longest_first = B > 1 && B <= kThreads && units * plan.splits > slots && plan.chunk > kOrderKeys;
  plan.workspace = 0;
  if (plan.splits > 1 && !plan.cluster)
    plan.workspace = ((size_t)B * Hq * T * plan.splits * (d + 1) * 4 + 255) / 256 * 256;
  return plan;
}

cudaError_t launch_kv8_attn(Kv8AttnParams& p, const Kv8AttnPlan& plan, bool bf16, cudaStream_t st) {
  if (p.d == 64)
    return bf16 ? launch_tiles<__nv_bfloat16, 64>(p, plan.tiles, st) : launch_tiles<__half, 64>(p, plan.tiles, st);
  return bf16 ? launch_tiles<__nv_bfloat16, 128>(p, plan.tiles, st) : launch_tiles<__half, 128>(p, plan.tiles, st);
}

}  // namespace fa
