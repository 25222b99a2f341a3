// Attention of the newest tokens of each sequence over its 8-bit paged cache.
//
//   S_rj = scale * q_r . k_j (- m |i_r - j|), masked;  O_r = sum_j softmax(S_r)_j v_j
//
// for the rows r = (token t, query head) that share a key head, with k_j, v_j =
// code * scale of the page. It is bound by reading the cache once (2 bytes per
// head value of a token), so everything serves keeping loads in flight:
//
// * Queries are the narrow side of the products: S^T = K Q^T and O^T = V^T P^T,
//   16 keys x 8 rows an instruction (mma.sync m16n8k16, f16 operands, fp32
//   sums). A tcgen05 tile has at least 64 rows of M from shared memory and its
//   smallest useful N; with one to a few dozen rows the codes would have to be
//   widened into shared memory first (2 bytes a value written and read again),
//   while here they go from global memory straight into the registers that the
//   instruction reads. Its rate is not what bounds the kernel up to 32 rows.
// * Any order of the head dimension serves S, and any order of the output
//   columns serves O: a lane takes 16 consecutive codes of a key (K) or of a
//   key's values (V) with one load and uses them in place. A warp's loads cover
//   whole 64-byte (K) and 128-byte (V) pieces of rows.
// * e4m3 is exact in f16, so codes enter the products unrounded; the page's key
//   scale multiplies S in fp32. V's codes are summed in units of their scale;
//   the sums are rescaled on the rare page whose scale differs (exact for
//   powers of two). bf16 queries become f16 after division by a power of two of
//   each row (exact down to 2^-28 of the row's largest value).
// * Running maximum and sum per row in fp32, kept per lane; the reference m
//   moves only when a score exceeds it by 2^15 (P is then at most 2^15, inside
//   f16), starting 2^7 above the first maximum, so warps agree on a new m a few
//   times a sequence and vote otherwise. P is rounded to f16 (2^-12 of itself);
//   for f16 outputs, whose own rounding is no larger, its rounding residual is
//   multiplied too.
// * Four warps take steps of 16 keys in turn. A lane's pieces of the next steps
//   are on their way to shared memory (cp.async) in slots that it alone reads
//   back, so a warp waits for its own copies and for nothing else, and about 48
//   KB a block are in flight without a register. The warps are merged once, at
//   the end.
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
constexpr int kStep = 16;       // keys of a step
constexpr float kNoMax = -3.0e38f;  // m before any score
constexpr float kHead = 7.f;    // m starts that far below 2^15: P of the first maximum is 2^7
constexpr float kTop = 15.f;    // scores may pass m by this much (in log2)

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
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
// row of the row tile attends to, lo rounded down to a step.
struct Range {
  int len, count;  // tokens of the sequence; how many of them are new
  int keys;        // keys that exist for attention
  int lo, hi;
};

__device__ __forceinline__ Range key_range(const Kv8AttnParams& p, int b, int row_lo, int row_hi) {
  Range r;
  r.len = max(__ldg(p.c.seq_lens + b), 0);
  r.count = p.c.new_lens ? min(max(__ldg(p.c.new_lens + b), 0), p.T) : p.T;
  r.keys = min(r.len, p.key_limit);
  // rows [row_lo, row_hi) hold tokens t_lo .. t_hi at positions len - count + t
  const int t_lo = max(row_lo / p.G, r.count - r.len), t_hi = min((row_hi - 1) / p.G, r.count - 1);
  r.lo = r.hi = 0;
  if (t_lo <= t_hi) {
    const int i_lo = r.len - r.count + t_lo, i_hi = r.len - r.count + t_hi;
    r.hi = p.causal ? min(r.keys, i_hi + 1) : r.keys;
    r.lo = p.window > 0 ? max(0, i_lo - p.window + 1) & ~(kStep - 1) : 0;
    if (r.lo >= r.hi) r.lo = r.hi = 0;
  }
  return r;
}

// Keys of a split: the plan's, or, in a cluster, the sequence's own keys shared out evenly.
__device__ __forceinline__ int split_keys(const Kv8AttnParams& p, const Range& r) {
  if (!p.cluster) return p.chunk;
  const int hop = kStep * kWarps, n = r.hi - r.lo, per = p.splits * hop;
  return max(1, (n + per - 1) / per) * hop;
}

// A lane's pieces of one step: lane (r = lane / 4, c = lane % 4) takes codes
// [64 x + 16 c, + 16) of keys r and r + 8 (K) and codes [(D / 8) r, + D / 8) of
// keys 2c, 2c + 1, 2c + 8, 2c + 9 (V). Slots of a piece are a thread apart.
template <int D>
struct Ring {
  static constexpr int kK = 2 * (D / 64);          // 16-byte pieces of K
  static constexpr int kVBytes = D / 8;            // bytes of a piece of V (four of them)
  static constexpr int kStages = D == 128 ? 4 : 6;
  static constexpr int kStageBytes = (kK * 16 + 4 * kVBytes) * kThreads;
  static constexpr int kScales = kStages * kStageBytes;  // then (K scale, V scale) a warp and stage
  static constexpr int kBytes = kScales + kStages * kWarps * 8;
};

__device__ __forceinline__ void copy8_async(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(valid ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
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

// Starts the copies of the step at `slot` of a page into a stage (zeros for a page outside the cache).
template <int D>
__device__ __forceinline__ void fetch_step(const Kv8Cache& c, uint32_t ring, int stage, int page, int slot, int h,
                                           bool page_ok) {
  using G = Ring<D>;
  const int lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  const long long at = page_ok ? (long long)page * c.sp + (long long)h * c.sh + (long long)slot * c.sn : 0;
  const uint32_t base = ring + stage * G::kStageBytes + threadIdx.x * 16;
  const uint8_t* kp = c.k + at + (page_ok ? r * c.sn + 16 * q : 0);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
      copy16_async(base + (i * (D / 64) + x) * (kThreads * 16), kp + (page_ok ? (long long)(8 * i) * c.sn + 64 * x : 0), page_ok);
  const uint8_t* vp = c.v + at + (page_ok ? (long long)(2 * q) * c.sn + G::kVBytes * r : 0);
  const uint32_t vbase = ring + stage * G::kStageBytes + G::kK * 16 * kThreads + threadIdx.x * G::kVBytes;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* row = vp + (page_ok ? (long long)((i & 1) + 8 * (i >> 1)) * c.sn : 0);
    if (D == 128)
      copy16_async(vbase + i * (kThreads * G::kVBytes), row, page_ok);
    else
      copy8_async(vbase + i * (kThreads * G::kVBytes), row, page_ok);
  }
  if (lane < 2) {
    const float* s = (lane ? c.v_scale : c.k_scale) + (page_ok ? (long long)page * c.H + h : 0);
    copy4_async(ring + G::kScales + (stage * kWarps + (threadIdx.x >> 5)) * 8 + lane * 4, s, page_ok);
  }
}

// Bytes of w that hold an e4m3 NaN (0x7F, 0xFF), as 0x80 flags.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : NT == 2 ? 3 : 2) kv8_attn_kernel(const __grid_constant__ Kv8AttnParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kResidual = !kBf16;  // see the head of the file
  constexpr int KS = D / 16;          // instructions' depth steps over the head dimension (S), row tiles of O^T
  constexpr int kRows = 8 * NT;
  constexpr int kAcc = KS * NT * 4;
  __shared__ uint2 q_frag[KS][NT][32];
  __shared__ float q_factor[kRows];
  __shared__ float w_m[kWarps][kRows], w_l[kWarps][kRows];
  __shared__ float block_lse[kRows];
  extern __shared__ __align__(16) unsigned char dyn[];
  using G = Ring<D>;
  static_assert(G::kScales >= (kWarps / 2) * kAcc * 32 * 4 && G::kScales >= kRows * D * 4, "merging reuses the ring");
  float (*merge)[kAcc][32] = reinterpret_cast<float (*)[kAcc][32]>(dyn);
  const uint32_t ring = smem_u32(dyn);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y % p.c.H, rt = blockIdx.y / p.c.H, R = p.T * p.G;
  const int row0 = rt * kRows;
  const Range kr = key_range(p, b, row0, min(row0 + kRows, R));
  const int chunk = split_keys(p, kr);
  const int begin = kr.lo + blockIdx.x * chunk, end = min(kr.hi, begin + chunk);
  // (the joining kernel counts splits the same way; the blocks of a cluster all come along)
  if (begin >= end && p.splits > 1 && !p.cluster) return;

  // Steps of this warp: begin + 16 warp, + 64, ...; kStages - 1 of them are under way while one is
  // computed, their page numbers read one step earlier still.
  constexpr int kHop = kStep * kWarps;
  const int* table = p.c.table + b * p.c.table_stride;
  const int shift = p.c.page_shift, mask = (1 << shift) - 1;
  const int first = begin + kStep * warp;
  int ahead = first;          // key of the next step to fetch
  uint32_t page_bits = 0u;    // bit n % 32: step n's page is in the cache
  int fetched = 0;
  bool bad = false;
  auto page_of = [&](int key) { return key < end ? __ldg(table + (key >> shift)) : -1; };
  auto fetch = [&](int page) {
    if (ahead < end) {
      const bool ok = (unsigned)page < (unsigned)p.c.num_pages;
      bad |= !ok;
      page_bits = (page_bits & ~(1u << (fetched & 31))) | ((ok ? 1u : 0u) << (fetched & 31));
      fetch_step<D>(p.c, ring, fetched % G::kStages, page, ahead & mask, h, ok);
    }
    copies_commit();
    ++fetched;
    ahead += kHop;
  };
  int pages[G::kStages];
#pragma unroll
  for (int i = 0; i < G::kStages; ++i) pages[i] = page_of(first + i * kHop);
#pragma unroll
  for (int i = 0; i < G::kStages - 1; ++i) fetch(pages[i]);
  int next_page = pages[G::kStages - 1];

  // Queries: row tile nt of this warp's share as f16 operand registers in shared memory.
  for (int nt = warp; nt < NT; nt += kWarps) {
    const int row = row0 + 8 * nt + r, t = row / p.G, hq = h * p.G + row % p.G;
    const bool live = row < R && t < kr.count && kr.len - kr.count + t >= 0;
    const T* qp = static_cast<const T*>(p.q) + b * p.q_st.b + (long long)t * p.q_st.n + (long long)hq * p.q_st.h;
    uint2 raw[KS];
    uint32_t top = 0u;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      raw[ks] = live ? __ldg(reinterpret_cast<const uint2*>(qp + 64 * (ks >> 2) + 16 * c + 4 * (ks & 3)))
                     : make_uint2(0u, 0u);
      const uint32_t a = raw[ks].x & 0x7FFF7FFFu, e = raw[ks].y & 0x7FFF7FFFu;
      top = max(top, max(max(a & 0xFFFFu, a >> 16), max(e & 0xFFFFu, e >> 16)));
    }
    float factor = p.scale_log2;
    if (kBf16) {
      // largest magnitude of the row to [2^14, 2^15): a division by a power of two
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = min(max((int)(top >> 7) - 127 - 14, -110), 113);
      const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
      factor *= __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        float x0, x1, x2, x3;
        unpack2<true>(raw[ks].x, x0, x1);
        unpack2<true>(raw[ks].y, x2, x3);
        raw[ks] = make_uint2(pack2<false>(x0 * down, x1 * down), pack2<false>(x2 * down, x3 * down));
      }
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q_frag[ks][nt][lane] = raw[ks];
    if (c == 0) q_factor[8 * nt + r] = factor;
  }

  // This lane's rows are 2c and 2c + 1 of every tile: scale, key limits, slope.
  float m[NT][2], l[NT][2], slope[NT][2];
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
      slope[nt][e] = live && p.alibi ? __ldg(p.alibi + b * p.alibi_sb + h * p.G + row % p.G) * 1.4426950408889634f : 0.f;
      m[nt][e] = kNoMax;
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
  float unit = 1.f, unit_top = 0.f;  // acc is in units of `unit`
  __syncthreads();
  uint2 q_reg[NT == 1 ? KS : 1];
  if (NT == 1) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q_reg[NT == 1 ? ks : 0] = q_frag[ks][0][lane];
  }
  float fac[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) fac[nt][e] = q_factor[8 * nt + 2 * c + e];

  auto compute = [&](int stage, bool page_ok, int at) {
    const uint32_t slot = ring + stage * G::kStageBytes + threadIdx.x * 16;
    float2 scales;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                 : "=f"(scales.x), "=f"(scales.y)
                 : "r"(ring + G::kScales + (stage * kWarps + warp) * 8)
                 : "memory");
    uint4 kv[G::kK];
#pragma unroll
    for (int i = 0; i < G::kK; ++i) kv[i] = read_slot16(slot + i * (kThreads * 16));
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint4 k0 = kv[ks >> 2], k1 = kv[(D / 64) + (ks >> 2)];
      const uint32_t w0 = (ks & 3) == 0 ? k0.x : (ks & 3) == 1 ? k0.y : (ks & 3) == 2 ? k0.z : k0.w;
      const uint32_t w1 = (ks & 3) == 0 ? k1.x : (ks & 3) == 1 ? k1.y : (ks & 3) == 2 ? k1.z : k1.w;
      uint32_t a0, a1, a2, a3;
      widen4(w0, a0, a2);
      widen4(w1, a1, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint2 f = NT == 1 ? q_reg[NT == 1 ? ks : 0] : q_frag[ks][nt][lane];
        mma_f16(sc[nt], a0, a1, a2, a3, f.x, f.y);
      }
    }
    const float vs = page_ok ? scales.y : unit;
    const bool whole = at >= all_lo && at + kStep <= all_hi && page_ok;
    bool over = false;
    bool keep[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = at + r + 8 * (e >> 1), i = pos[nt][e & 1];
        float x = sc[nt][e] * (scales.x * fac[nt][e & 1]);
        if (p.alibi) x = fmaf(-slope[nt][e & 1], fabsf((float)(i - j)), x);
        keep[nt][e] = true;
        if (!whole) {
          keep[nt][e] = page_ok && j < kr.keys && i >= 0 && (!p.causal || j <= i) && (p.window <= 0 || j > i - p.window);
          if (!keep[nt][e]) x = -INFINITY;
        }
        sc[nt][e] = x;
        over |= x > m[nt][e & 1] + kTop;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[nt][e], sc[nt][e + 2]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          if (x > m[nt][e] + kTop) {
            const float to = x - kHead, f = ex2_approx(m[nt][e] - to);
            m[nt][e] = to;
            l[nt][e] *= f;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              acc[i][nt][e] *= f;
              acc[i][nt][e + 2] *= f;
            }
          }
        }
    }
    float pv = 1.f;
    if (vs != unit) {
      // another V scale: the sums go over to its unit, but not below 2^-64 of
      // the largest so far (P takes the rest), so that they stay in range
      unit_top = fmaxf(unit_top, vs);
      const float to = fmaxf(fmaxf(vs, unit_top * 5.421010862427522e-20f), 1.1754944e-38f);
      const float f = unit / to;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] *= f;
      unit = to;
      pv = vs / to;
    }
    uint32_t b0[NT], b1[NT], d0[NT], d1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = ex2_approx(sc[nt][e] - m[nt][e & 1]);
        l[nt][e & 1] += x[e];
        x[e] *= pv;
      }
      const uint32_t lo = pack2<false>(x[0], x[1]), hi = pack2<false>(x[2], x[3]);
      if (kResidual) {
        d0[nt] = transpose8x8(pack2_residual<false>(x[0], x[1], lo));
        d1[nt] = transpose8x8(pack2_residual<false>(x[2], x[3], hi));
      }
      b0[nt] = transpose8x8(lo);
      b1[nt] = transpose8x8(hi);
    }
    uint32_t v[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = ring + stage * G::kStageBytes + G::kK * 16 * kThreads + (i * kThreads + threadIdx.x) * G::kVBytes;
      if (D == 128) {
        const uint4 x = read_slot16(a);
        v[i][0] = x.x, v[i][1] = x.y, v[i][D / 32 - 2] = x.z, v[i][D / 32 - 1] = x.w;
      } else {
        const uint2 x = read_slot8(a);
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
        const bool dead = at + 2 * c + (i & 1) + 8 * (i >> 1) >= kr.keys;
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
          i0[nt] = transpose8x8((keep[nt][0] ? 0x3C00u : 0u) | (keep[nt][1] ? 0x3C000000u : 0u));
          i1[nt] = transpose8x8((keep[nt][2] ? 0x3C00u : 0u) | (keep[nt][3] ? 0x3C000000u : 0u));
        }
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int w = mt >> 1, sh = 16 * (mt & 1);
          uint32_t f[4];  // flags (f16 one or zero) of the two values of this tile for the four keys
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = nan_bytes(v[i][w]) >> sh;
          auto pair = [](uint32_t a, uint32_t b2, uint32_t bit) {
            return ((a & bit) ? 0x3C00u : 0u) | ((b2 & bit) ? 0x3C000000u : 0u);
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
      uint32_t a0, a1, a2, a3;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        widen4(half ? x1 : x0, a0, a1);
        widen4(half ? y1 : y0, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(acc[2 * w + half][nt], a0, a1, a2, a3, b0[nt], b1[nt]);
          if (kResidual) mma_f16(acc[2 * w + half][nt], a0, a1, a2, a3, d0[nt], d1[nt]);
        }
      }
    }
  };

  int stage = 0, step = 0;
  for (int base = first; base < end; base += kHop) {
    const int page = next_page;
    next_page = page_of(base + G::kStages * kHop);
    fetch(page);
    copies_wait<G::kStages - 1>();
    __syncwarp();  // (the scales' copies are lanes 0's and 1's)
    compute(stage, (page_bits >> (step & 31)) & 1u, base);
    stage = stage + 1 == G::kStages ? 0 : stage + 1;
    ++step;
  }
  if (bad && lane == 0) atomicOr(p.c.status, kStatusBadPage);
  copies_wait<0>();
  let_next_begin();

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
      const float f = sum == 0.f ? 0.f : ex2_approx(m[nt][e] - top) / sum * unit;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        acc[i][nt][e] *= f;
        acc[i][nt][e + 2] *= f;
      }
    }
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) merge[warp - half][(i * NT + nt) * 4 + e][lane] = acc[i][nt][e];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] += merge[warp][(i * NT + nt) * 4 + e][lane];
    }
    __syncthreads();
  }
  // Lane (r, c) of warp 0 holds values [(D / 8) r, + D / 8) of rows 2c and 2c + 1 of every tile.
  if (p.cluster) {
    // every block's normalised outputs and log-sum-exp in its shared memory, then each block
    // joins its share of the (row, four values) items from all of them
    float* mine = reinterpret_cast<float*>(dyn);  // [kRows][D]; the merge is over
    if (warp == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * nt + 2 * c + e;
          float4* o = reinterpret_cast<float4*>(mine + row * D + (D / 8) * r);
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            o[x] = make_float4(acc[2 * x][nt][e], acc[2 * x][nt][e + 2], acc[2 * x + 1][nt][e], acc[2 * x + 1][nt][e + 2]);
          if (r == 0) block_lse[row] = lse2[nt][e];
        }
    }
    cluster_sync();
    const int n = p.splits, rows = min(kRows, R - row0);
    for (int item = blockIdx.x * kThreads + threadIdx.x; item < rows * (D / 4); item += n * kThreads) {
      const int row = item / (D / 4), e = (item % (D / 4)) * 4;
      float part[kMaxCluster], top = -INFINITY;
      float4 o[kMaxCluster];
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s)
        if (s < n) {
          part[s] = read_cluster_f32(&block_lse[row], s);
          o[s] = read_cluster_f32x4(mine + row * D + e, s);
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
      const int t = (row0 + row) / p.G, hq = h * p.G + (row0 + row) % p.G;
      T* to = static_cast<T*>(p.o) + b * p.o_st.b + (long long)t * p.o_st.n + (long long)hq * p.o_st.h + e;
      *reinterpret_cast<uint2*>(to) = make_uint2(pack2<kBf16>(v[0] * inv, v[1] * inv), pack2<kBf16>(v[2] * inv, v[3] * inv));
      if (e == 0)
        p.lse[((long long)b * p.Hq + hq) * p.T + t] = sum == 0.f ? -INFINITY : (top + lg2_approx(sum)) * kLn2;
    }
    cluster_sync();  // (no block leaves while another reads its shared memory)
    return;
  }
  if (warp != 0) return;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = row0 + 8 * nt + 2 * c + e;
      if (row >= R) continue;
      const int t = row / p.G, hq = h * p.G + row % p.G;
      if (p.splits == 1) {
        T* o = static_cast<T*>(p.o) + b * p.o_st.b + (long long)t * p.o_st.n + (long long)hq * p.o_st.h + (D / 8) * r;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack2<kBf16>(acc[4 * x + i][nt][e], acc[4 * x + i][nt][e + 2]);
          reinterpret_cast<uint4*>(o)[x] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (r == 0) p.lse[((long long)b * p.Hq + hq) * p.T + t] = lse2[nt][e] * kLn2;
      } else {
        const long long at = (((long long)b * p.c.H + h) * R + row) * p.splits + blockIdx.x;
        float4* o = reinterpret_cast<float4*>(p.part_o + at * D + (D / 8) * r);
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
          o[x] = make_float4(acc[2 * x][nt][e], acc[2 * x][nt][e + 2], acc[2 * x + 1][nt][e], acc[2 * x + 1][nt][e + 2]);
        if (r == 0) p.part_lse[at] = lse2[nt][e];
      }
    }
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
  const Range kr = key_range(p, b, rt * 8 * NT, min((rt + 1) * 8 * NT, R));
  const int n = (kr.hi - kr.lo + p.chunk - 1) / p.chunk;
  const long long at = (((long long)b * p.c.H + h) * R + row) * p.splits;
  wait_for_previous();
  // every warp on its own: its splits' maximum, weights and sums, joined at the end
  float top = -INFINITY, acc[kPer], sum = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int s = warp + kJoinWarps * lane; s < n; s += kJoinWarps * 32) top = fmaxf(top, __ldcg(p.part_lse + at + s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 8
  for (int s = warp; s < n; s += kJoinWarps) {
    const float x = __ldcg(p.part_lse + at + s);
    const float w = x == -INFINITY ? 0.f : ex2_approx(x - top);  // (a split without a key for this row)
    sum += w;
    const float* o = p.part_o + (at + s) * D + kPer * lane;
    if (kPer == 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(o));
      acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
      acc[kPer - 2] = fmaf(w, v.z, acc[kPer - 2]), acc[kPer - 1] = fmaf(w, v.w, acc[kPer - 1]);
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(o));
      acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
    }
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
  cudaError_t e = allow_smem<kKernel>(Ring<D>::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.splits, p.c.H * p.row_tiles, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<D>::kBytes;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = p.cluster ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kKernel, p);
  if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
  return launch_behind(kv8_join_kernel<T, D, NT>, dim3(p.T * p.G, p.c.H, p.B), 32 * kJoinWarps, p, st);
}

template <typename T, int D>
cudaError_t launch_tiles(const Kv8AttnParams& p, int tiles, cudaStream_t st) {
  if (tiles == 1) return launch_nt<T, D, 1>(p, st);
  return tiles == 2 ? launch_nt<T, D, 2>(p, st) : launch_nt<T, D, 4>(p, st);
}

}  // namespace

// Splits. Up to eight blocks a sequence and row tile join within a cluster, each
// sequence sharing out its own keys. That is taken where eight splits fill the
// GPU's resident slots, and where a block's share is at most kClusterKeys keys, so
// that more blocks would gain less than the joining kernel's launch costs. What is
// left, few sequences with long contexts, gets one resident set of blocks.
Kv8AttnPlan kv8_attn_plan(int B, int T, int Hq, int H, int d, int key_limit, int causal, int window) {
  constexpr long long kClusterKeys = 512, hop = kStep * kWarps;
  Kv8AttnPlan plan;
  const long long R = (long long)T * (Hq / H);
  plan.tiles = R <= 8 ? 1 : R <= 16 ? 2 : 4;
  plan.row_tiles = (int)((R + 8 * plan.tiles - 1) / (8 * plan.tiles));
  // keys that one block's rows can reach
  long long range = key_limit;
  if (causal && window > 0) range = std::min<long long>(range, (long long)window + T + kStep);
  const long long units = (long long)B * H * plan.row_tiles, slots = 152 * (plan.tiles == 4 ? 2 : 3);
  const auto round_hop = [&](long long x) { return std::max(hop, (x + hop - 1) / hop * hop); };
  long long splits = std::min<long long>(kMaxCluster, (range + hop - 1) / hop);
  // (with more units than slots several rounds of blocks run anyway: splits of at least 1024 keys then)
  while (splits > 1 && units * splits > 8 * slots && range / splits < 1024) splits >>= 1;
  plan.cluster = 1;
  if (units * kMaxCluster < slots && round_hop((range + splits - 1) / splits) > kClusterKeys) {
    plan.cluster = 0;
    splits = std::max<long long>(1, slots / units);
  }
  plan.chunk = (int)round_hop((range + splits - 1) / splits);
  plan.splits = (int)((range + plan.chunk - 1) / plan.chunk);
  if (plan.splits == 1) plan.cluster = 0;
  plan.workspace = 256;
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
