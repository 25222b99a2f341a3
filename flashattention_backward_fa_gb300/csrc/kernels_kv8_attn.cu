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
// * Four warps take steps of 16 keys in turn, each with its next step's loads
//   issued before it computes; they are merged once, at the end. Long sequences
//   are split over blocks, whose normalised outputs a second kernel joins.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fa_serve.h"

namespace fa {

namespace {

constexpr int kWarps = 4;
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

// One step's keys and values in registers. Lane (r = lane / 4, c = lane % 4)
// holds codes [64 h + 16 c, + 16) of keys r and r + 8 (K), and codes
// [kVBytes r, + kVBytes) of keys 2c, 2c + 1, 2c + 8, 2c + 9 (V).
template <int D>
struct Step {
  static constexpr int kHalves = D / 64;
  uint4 k[2 * kHalves];
  uint32_t v[4][D / 32];
  float ks, vs;
  bool page_ok;
};

template <int D>
__device__ __forceinline__ void load_step(const Kv8Cache& c, int page, int slot, int h, int lane, Step<D>& s) {
  const int r = lane >> 2, q = lane & 3;
  s.page_ok = (unsigned)page < (unsigned)c.num_pages;
  if (!s.page_ok) {
#pragma unroll
    for (int i = 0; i < 2 * (D / 64); ++i) s.k[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 0; w < D / 32; ++w) s.v[i][w] = 0u;
    s.ks = s.vs = 1.f;
    return;
  }
  const long long at = (long long)page * c.sp + (long long)h * c.sh + (long long)slot * c.sn;
  const uint8_t* kp = c.k + at + r * c.sn + 16 * q;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
      s.k[i * (D / 64) + x] = __ldg(reinterpret_cast<const uint4*>(kp + (long long)(8 * i) * c.sn + 64 * x));
  const uint8_t* vp = c.v + at + (long long)(2 * q) * c.sn + (D / 8) * r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* row = vp + (long long)((i & 1) + 8 * (i >> 1)) * c.sn;
    if (D == 128) {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(row));
      s.v[i][0] = t.x, s.v[i][1] = t.y, s.v[i][D / 32 - 2] = t.z, s.v[i][D / 32 - 1] = t.w;
    } else {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(row));
      s.v[i][0] = t.x, s.v[i][1] = t.y;
    }
  }
  const long long sc = (long long)page * c.H + h;
  s.ks = __ldg(c.k_scale + sc);
  s.vs = __ldg(c.v_scale + sc);
}

// Bytes of w that hold an e4m3 NaN (0x7F, 0xFF), as 0x80 flags.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kWarps) kv8_attn_kernel(const __grid_constant__ Kv8AttnParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kResidual = !kBf16;  // see the head of the file
  constexpr int KS = D / 16;          // instructions' depth steps over the head dimension (S), row tiles of O^T
  constexpr int kRows = 8 * NT;
  constexpr int kAcc = KS * NT * 4;
  __shared__ uint2 q_frag[KS][NT][32];
  __shared__ float q_factor[kRows];
  __shared__ float w_m[kWarps][kRows], w_l[kWarps][kRows];
  __shared__ float merge[kWarps / 2][kAcc][32];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y % p.c.H, rt = blockIdx.y / p.c.H, R = p.T * p.G;
  const int row0 = rt * kRows;
  const Range kr = key_range(p, b, row0, min(row0 + kRows, R));
  const int begin = kr.lo + blockIdx.x * p.chunk, end = min(kr.hi, begin + p.chunk);
  if (begin >= end && (p.splits > 1 || blockIdx.x > 0)) return;  // (the joining kernel counts splits the same way)

  const int* table = p.c.table + b * p.c.table_stride;
  const int shift = p.c.page_shift, mask = (1 << shift) - 1;
  int base = begin + kStep * warp;
  int page = base < end ? __ldg(table + (base >> shift)) : -1;

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

  auto compute = [&](Step<D>& s, int at) {
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint4 k0 = s.k[ks >> 2], k1 = s.k[(D / 64) + (ks >> 2)];
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
    const bool whole = at >= all_lo && at + kStep <= all_hi && s.page_ok;
    bool over = false;
    bool keep[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = at + r + 8 * (e >> 1), i = pos[nt][e & 1];
        float x = sc[nt][e] * (s.ks * fac[nt][e & 1]);
        if (p.alibi) x = fmaf(-slope[nt][e & 1], fabsf((float)(i - j)), x);
        keep[nt][e] = true;
        if (!whole) {
          keep[nt][e] = s.page_ok && j < kr.keys && i >= 0 && (!p.causal || j <= i) && (p.window <= 0 || j > i - p.window);
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
    if (s.vs != unit) {
      // another V scale: the sums go over to its unit, but not below 2^-64 of
      // the largest so far (P takes the rest), so that they stay in range
      unit_top = fmaxf(unit_top, s.vs);
      const float to = fmaxf(fmaxf(s.vs, unit_top * 5.421010862427522e-20f), 1.1754944e-38f);
      const float f = unit / to;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] *= f;
      unit = to;
      pv = s.vs / to;
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
          if (dead) s.v[i][w] = 0u;
          has |= nan_bytes(s.v[i][w]) != 0u;
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
          for (int i = 0; i < 4; ++i) f[i] = nan_bytes(s.v[i][w]) >> sh;
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
          for (int w = 0; w < D / 32; ++w) s.v[i][w] &= ~((nan_bytes(s.v[i][w]) >> 7) * 0xFFu);
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      // codes of two keys side by side: bytes (k0.0, k1.0, k0.1, k1.1) and (k0.2, k1.2, k0.3, k1.3)
      const uint32_t x0 = __byte_perm(s.v[0][w], s.v[1][w], 0x5140), x1 = __byte_perm(s.v[0][w], s.v[1][w], 0x7362);
      const uint32_t y0 = __byte_perm(s.v[2][w], s.v[3][w], 0x5140), y1 = __byte_perm(s.v[2][w], s.v[3][w], 0x7362);
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

  // Steps of this warp: base, base + 64, ...; the next step's page number and
  // then its loads are under way while a step is computed.
  constexpr int kHop = kStep * kWarps;
  bool bad = false;
  {
    Step<D> s0, s1;
    if (base < end) load_step<D>(p.c, page, base & mask, h, lane, s0);
    int next = base + kHop < end ? __ldg(table + ((base + kHop) >> shift)) : -1;
    while (base < end) {
      if (base + kHop < end) load_step<D>(p.c, next, (base + kHop) & mask, h, lane, s1);
      next = base + 2 * kHop < end ? __ldg(table + ((base + 2 * kHop) >> shift)) : -1;
      bad |= !s0.page_ok;
      compute(s0, base);
      base += kHop;
      if (base >= end) break;
      if (base + kHop < end) load_step<D>(p.c, next, (base + kHop) & mask, h, lane, s0);
      next = base + 2 * kHop < end ? __ldg(table + ((base + 2 * kHop) >> shift)) : -1;
      bad |= !s1.page_ok;
      compute(s1, base);
      base += kHop;
    }
  }
  if (bad && lane == 0) atomicOr(p.c.status, kStatusBadPage);

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
  if (warp != 0) return;
  // Lane (r, c) holds values [(D / 8) r, + D / 8) of rows 2c and 2c + 1 of every tile.
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
        if (r == 0) p.lse[((long long)b * p.Hq + hq) * p.T + t] = lse2[nt][e] * 0.6931471805599453f;
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
// w_s = 2^(lse_s - max). Four warps take every fourth split.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(128) kv8_join_kernel(const __grid_constant__ Kv8AttnParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kPer = D / 32;
  __shared__ float acc_s[4][D];
  __shared__ float top_s[4], sum_s[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, h = blockIdx.y, b = blockIdx.z, R = p.T * p.G;
  const int rt = row / (8 * NT);
  const Range kr = key_range(p, b, rt * 8 * NT, min((rt + 1) * 8 * NT, R));
  const int n = (kr.hi - kr.lo + p.chunk - 1) / p.chunk;
  const long long at = (((long long)b * p.c.H + h) * R + row) * p.splits;
  float top = -INFINITY;
  for (int s = threadIdx.x; s < n; s += 128) top = fmaxf(top, p.part_lse[at + s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) top_s[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(top_s[0], top_s[1]), fmaxf(top_s[2], top_s[3]));
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int s = warp; s < n; s += 4) {
    const float x = p.part_lse[at + s];
    const float w = x == -INFINITY ? 0.f : ex2_approx(x - top);  // (a split without a key for this row)
    sum += w;
    const float* o = p.part_o + (at + s) * D + kPer * lane;
    if (kPer == 4) {
      const float4 v = *reinterpret_cast<const float4*>(o);
      acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
      acc[kPer - 2] = fmaf(w, v.z, acc[kPer - 2]), acc[kPer - 1] = fmaf(w, v.w, acc[kPer - 1]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(o);
      acc[0] = fmaf(w, v.x, acc[0]), acc[1] = fmaf(w, v.y, acc[1]);
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc_s[warp][kPer * lane + e] = acc[e];
  if (lane == 0) sum_s[warp] = sum;
  __syncthreads();
  sum = sum_s[0] + sum_s[1] + sum_s[2] + sum_s[3];
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int t = row / p.G, hq = h * p.G + row % p.G;
  if (threadIdx.x < D / 2) {
    const int e = 2 * threadIdx.x;
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = (acc_s[0][e + i] + acc_s[1][e + i] + acc_s[2][e + i] + acc_s[3][e + i]) * inv;
    T* o = static_cast<T*>(p.o) + b * p.o_st.b + (long long)t * p.o_st.n + (long long)hq * p.o_st.h + e;
    *reinterpret_cast<uint32_t*>(o) = pack2<kBf16>(v[0], v[1]);
  }
  if (threadIdx.x == 0)
    p.lse[((long long)b * p.Hq + hq) * p.T + t] =
        sum == 0.f ? -INFINITY : (top + lg2_approx(sum)) * 0.6931471805599453f;
}

template <typename T, int D, int NT>
cudaError_t launch_nt(const Kv8AttnParams& p, cudaStream_t st) {
  const dim3 grid(p.splits, p.c.H * p.row_tiles, p.B);
  kv8_attn_kernel<T, D, NT><<<grid, 32 * kWarps, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  kv8_join_kernel<T, D, NT><<<dim3(p.T * p.G, p.c.H, p.B), 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_tiles(const Kv8AttnParams& p, int tiles, cudaStream_t st) {
  if (tiles == 1) return launch_nt<T, D, 1>(p, st);
  return tiles == 2 ? launch_nt<T, D, 2>(p, st) : launch_nt<T, D, 4>(p, st);
}

}  // namespace

// Splits: enough blocks to fill the GPU's resident slots once, of at least one
// step a warp; no more than 1024 keys a block where there are many sequences,
// so that unequal lengths even out over several rounds of blocks.
Kv8AttnPlan kv8_attn_plan(int B, int T, int Hq, int H, int d, int key_limit, int causal, int window) {
  Kv8AttnPlan plan;
  const long long R = (long long)T * (Hq / H);
  plan.tiles = R <= 8 ? 1 : R <= 16 ? 2 : 4;
  plan.row_tiles = (int)((R + 8 * plan.tiles - 1) / (8 * plan.tiles));
  // keys that one block's rows can reach
  long long range = key_limit;
  if (causal && window > 0) range = std::min<long long>(range, (long long)window + T + kStep);
  const long long units = (long long)B * H * plan.row_tiles, slots = 152 * (plan.tiles == 4 ? 2 : 3);
  const long long hop = kStep * kWarps;
  long long chunk = (units * range + slots - 1) / slots;
  chunk = std::min<long long>(std::max<long long>((chunk + hop - 1) / hop * hop, hop), 1024);
  plan.chunk = (int)chunk;
  plan.splits = (int)((range + chunk - 1) / chunk);
  plan.workspace = 256;
  if (plan.splits > 1) plan.workspace = ((size_t)B * Hq * T * plan.splits * (d + 1) * 4 + 255) / 256 * 256;
  return plan;
}

cudaError_t launch_kv8_attn(Kv8AttnParams& p, const Kv8AttnPlan& plan, bool bf16, cudaStream_t st) {
  if (p.d == 64)
    return bf16 ? launch_tiles<__nv_bfloat16, 64>(p, plan.tiles, st) : launch_tiles<__half, 64>(p, plan.tiles, st);
  return bf16 ? launch_tiles<__nv_bfloat16, 128>(p, plan.tiles, st) : launch_tiles<__half, 128>(p, plan.tiles, st);
}

}  // namespace fa
