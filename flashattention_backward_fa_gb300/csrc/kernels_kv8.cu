// New keys and values into the paged 8-bit cache, alone (kv8_append) or behind
// the per-head norm and rotation of queries and keys (kv8_norm_rope_append).
//
// A page holds page-size tokens of every head as e4m3 codes of x / s, with one
// scale s per (page, head), a power of two: s = 2^e, e the least integer with
// amax <= 448 * 2^e (448 is the largest e4m3 value). A power of two costs
// e4m3 nothing but range (its precision is relative), and it makes every step
// exact but the one rounding: x / s is a change of exponent, and when a page
// that already holds tokens needs a larger scale, its codes are divided by a
// power of two, which moves only those that reach e4m3's subnormals.
//
// One block takes one (page, head) of the new keys or of the new values: it
// loads the page's new rows once, keeps them in registers while the block
// agrees on their largest magnitude, and writes the codes. With norm and
// rotation the keys' rows are normed, rotated and rounded to their type in
// registers in between, so the cache holds the same codes as after the two
// operators one by one; further blocks take q's rows. Nothing but the inputs
// and the outputs moves through memory. Bound by memory (2 bytes in and 1 byte
// out an element of k and v, 2 and 2 of q); for single tokens by the launch and
// two dependent loads (length, then rows and page number side by side). Measured,
// bf16: 1x32x8192x128 32.7 us (91% of the copy rate; eight blocks an SM at 32
// registers, five at 40 took 35 us); 4x16x2048x128 with norm and rotation 45.2 us
// (56%: at 80 registers three blocks an SM, bound by the instructions they issue).
#include <algorithm>

#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kQDepth = 3;    // rows of q a row group has on their way, and the one at hand
constexpr int kQRows = 32;    // most rows of q that a row group takes
constexpr int kMinExp = -100;  // least scale exponent: blocks of zeros (or below 2^-91) get it

// The scale's bits for a largest finite magnitude: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = max((int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0), kMinExp);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two fp32 values to a pair of e4m3 codes, lo in the low byte (round to nearest even).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack_e4m3x2(uint32_t two, float& lo, float& hi) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
  unpack2<false>(h, lo, hi);
}

// Bits of an infinity of the type, sign cleared: magnitudes from it up are not finite.
template <typename T>
__device__ __forceinline__ constexpr uint32_t inf_bits() {
  return std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
}

// Largest magnitude of eight values as bits of their type (kFinite: of the finite ones).
template <typename T, bool kFinite>
__device__ __forceinline__ uint32_t amax_bits(const uint4& a) {
  const uint32_t wv[4] = {a.x, a.y, a.z, a.w};
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = wv[i] & 0x7FFF7FFFu;
    if (kFinite) {
      if ((v & 0xFFFFu) >= inf_bits<T>()) v &= 0xFFFF0000u;
      if ((v >> 16) >= inf_bits<T>()) v &= 0x0000FFFFu;
    }
    m = max_u16x2(m, v);
  }
  return max(m & 0xFFFFu, m >> 16);
}

// Largest value over the block (every thread gets it); red: one word a warp.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = red[0];
  for (int i = 1; i < warps; ++i) m = max(m, red[i]);
  __syncthreads();
  return m;
}

// Eight values to eight codes. kAny: infinities become NaN codes as NaN do (a
// finite value is never beyond 448 times the scale).
template <typename T, bool kAny>
__device__ __forceinline__ uint2 quantise8(const Raw8<T>& raw, float inv) {
  uint64_t v[4];
  raw.unpack(v);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f2_mul(v[i], f2_pack(inv, inv)), lo, hi);
    if (kAny) {
      if (fabsf(lo) == INFINITY) lo = __int_as_float(0x7FC00000);
      if (fabsf(hi) == INFINITY) hi = __int_as_float(0x7FC00000);
    }
    c[i] = e4m3x2(lo, hi);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

struct NewTokens {
  int start, len, count;  // position of the first, tokens of the sequence with them, how many
};

__device__ __forceinline__ NewTokens new_tokens(const Kv8Cache& c, int b, int T) {
  NewTokens n;
  n.count = c.new_lens ? min(max(__ldg(c.new_lens + b), 0), T) : T;
  n.len = max(__ldg(c.seq_lens + b), 0);
  n.start = n.len - n.count;
  return n;
}

// Grid: x the heads of k, then of v, then (kNorm) blocks that share q's rows of
// the page's tokens; y the page among those that T tokens reach; z the sequence.
// kRows rows of a page a thread; blockDim.x * kRows * 16 values hold a page's new
// rows. kNorm: 0 append alone, 1 / 2 norm and rotation with partners rot / 2
// apart / neighbours.
template <typename T, int D, int kRows, int kNorm>
__global__ void __launch_bounds__(256, kNorm == 0 ? (kRows == 4 ? 4 : 8) : (kRows == 4 ? 2 : 3)) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p) {
  extern __shared__ __align__(16) unsigned char ring[];  // (q's rows only)
  constexpr int G = D / 16;
  constexpr bool kNeighbours = kNorm != 1;
  __shared__ uint32_t red[8];
  const Kv8Cache& c = p.c;
  __shared__ __align__(16) float w[D];
  const int b = blockIdx.z;
  const NewTokens n = new_tokens(c, b, p.T);
  if (kNorm != 0 && blockIdx.x >= 2u * c.H) {
    // q: rows (t, head) of the tokens whose positions fall into the page (the positions of padding
    // rows run on past the sequence, or before it), q_span a row group; padding rows become zeros
    const long long lo = ((long long)(n.start >> c.page_shift) + blockIdx.y) << c.page_shift;
    const int t_lo = (int)max(lo - n.start, 0ll);
    const int t_hi = (int)min(lo + (1 << c.page_shift) - n.start, (long long)p.T);
    if (t_lo >= t_hi) return;
    fa_strides in = p.q_st, out = p.q_out_st;
    const long long group = (long long)(blockIdx.x - 2u * c.H) * (blockDim.x / G) + threadIdx.x / G;
    norm_rope_rows<T, D, kNeighbours, true, kQDepth>(
        ring, static_cast<const T*>(p.q) + b * in.b + t_lo * in.n, static_cast<T*>(p.q_out) + b * out.b + t_lo * out.n,
        in, out, (long long)(t_hi - t_lo) * p.Hq, t_hi - t_lo, p.Hq, group * p.q_span, p.q_span, p.q_w, p.w_f32, w,
        p.cos, p.sin, p.rot, p.eps, [&](long long, int i) {
          const int t = t_lo + i;
          return t < n.count && n.start + t >= 0 ? (long long)min(n.start + t, max(p.max_pos - 1, 0)) * (p.rot >> 1)
                                                 : -1ll;
        });
    return;
  }
  const bool is_v = blockIdx.x >= (unsigned)c.H;
  const int h = blockIdx.x - (is_v ? c.H : 0);
  const int size = 1 << c.page_shift;
  const int pg = (max(n.start, 0) >> c.page_shift) + blockIdx.y;
  if (pg >= c.max_pages) return;  // (and positions below stay in 31 bits)
  const int t_lo = max(max(n.start, 0), pg << c.page_shift);
  const int t_hi = min(n.len, (pg + 1) << c.page_shift);  // positions [t_lo, t_hi)
  if (t_lo >= t_hi) return;
  const int id = __ldg(c.table + b * c.table_stride + pg);  // (checked once the rows' loads are under way)
  const int rows = t_hi - t_lo, slot0 = t_lo & (size - 1);
  const fa_strides& st = is_v ? p.v_st : p.k_st;
  const T* src = static_cast<const T*>(is_v ? p.v : p.k) + b * st.b + (long long)(t_lo - n.start) * st.n + h * st.h;
  const int groups = blockDim.x / G, row0 = threadIdx.x / G;
  const LanePlace at = lane_place<D, kNeighbours>(threadIdx.x % G, p.rot);
  Raw8<T> ra[kRows], rb[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i * groups;
    zero8(ra[i]);
    zero8(rb[i]);
    if (r < rows) {
      load8(ra[i], src + r * st.n + at.a);
      load8(rb[i], src + r * st.n + at.b);
    }
  }
  if (id < 0 || id >= c.num_pages) {
    if (threadIdx.x == 0) atomicOr(c.status, kStatusBadPage);
    return;
  }
  uint8_t* page = (is_v ? c.v : c.k) + id * c.sp + h * c.sh;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + (long long)id * c.H + h;
  const float was = slot0 > 0 ? *scale_at : 0.f;  // a page without earlier tokens has no former scale
  if (kNorm != 0 && !is_v) {
    // every load of the rows, the weights and the tables is under way before the first is used
    constexpr int kAhead = kRows < 2 ? kRows : 2;
    float cc[kAhead][8], ss[kAhead][8];
    auto rotation = [&](int i, float (&cr)[8], float (&sr)[8]) {
      const int r = row0 + i * groups;
      const long long row = r < rows ? (long long)min(t_lo + r, max(p.max_pos - 1, 0)) * (p.rot >> 1) : 0;
      load_rotation<kNeighbours>(p.cos + row, p.sin + row, at, r < rows ? p.rot : 0, cr, sr);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) rotation(i, cc[i], ss[i]);
    stage_weights<T>(p.k_w, p.w_f32, D, w);
    __syncthreads();
    LaneWeights lw;
    lw.read(w, at);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      norm_rope_lane<T, D, kNeighbours>(ra[i], rb[i], lw, cc[i % kAhead], ss[i % kAhead], p.eps);
      if (i + kAhead < kRows) rotation(i + kAhead, cc[i % kAhead], ss[i % kAhead]);
    }
  }
  // (places without a row: zeros, also where a NaN among the weights has reached them)
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (kNorm != 0 && row0 + i * groups >= rows) {
      zero8(ra[i]);
      zero8(rb[i]);
    }
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < kRows; ++i) m = max(m, max(amax_bits<T, false>(ra[i].q[0]), amax_bits<T, false>(rb[i].q[0])));
  m = block_max(m, red);
  const bool any = m >= inf_bits<T>();  // infinities or NaN among the new values
  if (any) {
    m = 0u;
#pragma unroll
    for (int i = 0; i < kRows; ++i) m = max(m, max(amax_bits<T, true>(ra[i].q[0]), amax_bits<T, true>(rb[i].q[0])));
    m = block_max(m, red);
  }
  const float scale = fmaxf(scale_for(h16_bits_to_f32<std::is_same<T, __nv_bfloat16>::value>(m)), was);
  const float inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i * groups;
    if (r >= rows) continue;
    uint8_t* to = page + (slot0 + r) * c.sn;
    *reinterpret_cast<uint2*>(to + at.a) = any ? quantise8<T, true>(ra[i], inv) : quantise8<T, false>(ra[i], inv);
    *reinterpret_cast<uint2*>(to + at.b) = any ? quantise8<T, true>(rb[i], inv) : quantise8<T, false>(rb[i], inv);
  }
  if (slot0 > 0 && scale != was) {  // earlier tokens to the larger scale, 16 codes a thread
    const float ratio = was * inv;
    for (int r = row0; r < slot0; r += groups) {
      uint4* to = reinterpret_cast<uint4*>(page + r * c.sn) + threadIdx.x % G;
      const uint4 q = *to;
      uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
        unpack_e4m3x2(v[i] & 0xFFFFu, f[0], f[1]);
        unpack_e4m3x2(v[i] >> 16, f[2], f[3]);
        v[i] = e4m3x2(f[0] * ratio, f[1] * ratio) | (e4m3x2(f[2] * ratio, f[3] * ratio) << 16);
      }
      *to = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  // (every thread has read the former scale: block_max synchronised since)
  if (threadIdx.x == 0) *scale_at = scale;
}

template <typename T, int D, int kRows>
cudaError_t launch_rows(const Kv8AppendParams& p, dim3 grid, int threads, cudaStream_t st) {
  const int ring = RowRing<T, 2, kQDepth>::bytes(threads);
  if (p.q == nullptr)
    kv8_append_kernel<T, D, kRows, 0><<<grid, threads, 0, st>>>(p);
  else if (!p.neighbours)
    kv8_append_kernel<T, D, kRows, 1><<<grid, threads, ring, st>>>(p);
  else
    kv8_append_kernel<T, D, kRows, 2><<<grid, threads, ring, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(Kv8AppendParams& p, cudaStream_t st) {
  constexpr int G = D / 16;
  const int rows = std::min(1 << p.c.page_shift, p.T);  // most new rows of one page
  // up to 256 threads, then more rows a thread; at least two warps, so that a
  // single token still shares out the rescaling of its page
  const int lanes = rows * G;
  const int per = lanes <= 256 ? 1 : lanes <= 512 ? 2 : 4;
  const int threads = std::max(64, ((lanes + per - 1) / per + 31) / 32 * 32);
  int q_blocks = 0;
  if (p.q) {
    // q's rows of a page's tokens: kQRows a row group where there are that many, so that a token's
    // factors serve several heads, and one where that leaves the GPU empty
    const long long q_rows = (long long)rows * p.Hq, groups = threads / G;
    p.q_span = (int)std::max<long long>(1, std::min<long long>(kQRows, q_rows * p.pages * p.B / (groups * 152 * 4)));
    q_blocks = (int)((q_rows + groups * p.q_span - 1) / (groups * p.q_span));
  }
  const dim3 grid(2 * p.c.H + q_blocks, p.pages, p.B);
  if (per == 1) return launch_rows<T, D, 1>(p, grid, threads, st);
  return per == 2 ? launch_rows<T, D, 2>(p, grid, threads, st) : launch_rows<T, D, 4>(p, grid, threads, st);
}

}  // namespace

cudaError_t launch_kv8_append(Kv8AppendParams& p, bool bf16, cudaStream_t st) {
  if (p.d == 64) return bf16 ? launch_d<__nv_bfloat16, 64>(p, st) : launch_d<__half, 64>(p, st);
  return bf16 ? launch_d<__nv_bfloat16, 128>(p, st) : launch_d<__half, 128>(p, st);
}

}  // namespace fa
