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
// A block takes one page's new keys or new values of one head: it loads the
// page's new rows once, keeps them in registers while the block agrees on their
// largest magnitude, and writes the codes. With norm and rotation a block takes
// several heads one after the other (or several heads of q): a thread keeps its
// tokens, so the tables' values and the weights are read once for all of them,
// and the next head's rows are on their way to shared memory while one is
// finished. The keys' rows are normed, rotated and rounded to their type in
// registers, so the cache holds the same codes as after the two operators one by
// one. Nothing but the inputs and the outputs moves through memory. Bound by
// memory (2 bytes in and 1 byte out an element of k and v, 2 and 2 of q); for
// single tokens by the launch and two dependent loads (length, then rows and page
// number side by side). Measured, bf16: 1x32x8192x128 30.6 us (97% of the copy
// rate; eight blocks an SM at 32 registers, five at 40 took 2 us more); 4x16x2048x128
// with norm and rotation 38.0 us (67%: two blocks an SM at 120 registers; one head
// a block, with the tables read for each, took 5 us more).
#include <algorithm>

#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kAhead = 2;        // heads in a block with norm: one on its way, one at hand (three and four ran alike)
constexpr int kMaxHeads = 8;     // most heads that a block of the form with norm takes
constexpr int kBlocks = 152 * 2;  // blocks of k, of v and of q that are kept where there is work for them
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
  n.count = c.new_lens ? min(max(c.new_lens[b], 0), T) : T;
  n.len = max(c.seq_lens[b], 0);
  n.start = n.len - n.count;
  return n;
}

// Grid: x a group of heads of k, then of v, then (kNorm) of q; y the page among
// those that T tokens reach; z the sequence. A block takes the heads of its group
// one after the other: a thread keeps its tokens, so the tables' values and the
// weights are loaded once for all heads, and the next head's rows are on their way
// while one is finished. kRows rows of a page a thread; blockDim.x * kRows * 16
// values hold a page's new rows. kNorm: 0 append alone, 1 / 2 norm and rotation
// with partners rot / 2 apart / neighbours; kPartial: rot < D; kAxes: positions are
// given (on one axis or several), not places in the sequences.
template <typename T, int D, int kRows, int kNorm, bool kPartial, bool kAxes>
__global__ void __launch_bounds__(kNorm == 0 ? 256 : 512, kNorm == 0 ? (kRows == 4 ? 4 : 8) : 1)
    kv8_append_kernel(const __grid_constant__ Kv8AppendParams p) {
  constexpr int G = D / 16;
  constexpr bool kNeighbours = kNorm != 1;
  extern __shared__ __align__(16) unsigned char smem[];  // (kNorm) rows of the next heads
  __shared__ uint32_t red[16];
  __shared__ __align__(16) float w[D];
  let_next_begin();
  wait_for_previous();
  const Kv8Cache& c = p.c;
  const int b = blockIdx.z;
  const NewTokens n = new_tokens(c, b, p.T);
  const int kv_groups = kNorm == 0 ? c.H : (c.H + p.kv_heads - 1) / p.kv_heads;
  const bool is_q = kNorm != 0 && blockIdx.x >= 2u * kv_groups;
  const bool is_v = !is_q && blockIdx.x >= (unsigned)kv_groups;
  int first, rows;  // the block's tokens: t = first .. first + rows - 1
  const int size = 1 << c.page_shift;
  const int pg = (max(n.start, 0) >> c.page_shift) + blockIdx.y;
  if (is_q) {
    // tokens whose positions fall into the page; those of padding rows run on past the sequence, or
    // before it
    const long long lo = ((long long)(n.start >> c.page_shift) + blockIdx.y) << c.page_shift;
    first = (int)max(lo - n.start, 0ll);
    rows = (int)min(lo + size - n.start, (long long)p.T) - first;
  } else {
    if (pg >= c.max_pages) return;  // (and positions below stay in 31 bits)
    const int lo = max(max(n.start, 0), pg << c.page_shift);
    first = lo - n.start;
    rows = min(n.len, (pg + 1) << c.page_shift) - lo;
  }
  if (rows <= 0) return;
  // (checked once the rows' loads are under way)
  const int id = is_q ? 0 : c.table[b * c.table_stride + pg];
  // Row groups beside each other: rows of the page, or, with few tokens, q's further heads.
  const int groups = blockDim.x / G;
  int row0 = threadIdx.x / G, beside = 1, head = 0;
  if (kRows == 1 && is_q && groups >= 2 * rows) {
    beside = groups / rows;
    head = row0 / rows;
    row0 -= head * rows;
    if (head >= beside) row0 = rows;  // (left over)
  }
  const int H = is_q ? p.Hq : c.H, span = kNorm == 0 ? 1 : is_q ? p.q_heads : p.kv_heads;
  const int group = blockIdx.x - (is_q ? 2 * kv_groups : is_v ? kv_groups : 0);
  const int heads = min(span, H - group * span);
  head += group * span;
  const int turns = kNorm == 0 ? 1 : (heads + beside - 1) / beside, head_end = group * span + heads;
  const fa_strides& st = is_q ? p.q_st : is_v ? p.v_st : p.k_st;
  const LanePlace at = lane_place<D, kNeighbours, kPartial>(threadIdx.x % G, p.rot);
  const T* src = static_cast<const T*>(is_q ? p.q : is_v ? p.v : p.k) + b * st.b + (long long)(first + row0) * st.n +
                 at.a;
  const int hop = at.b - at.a;
  bool live[kRows];  // the row has a token (q: padding rows have none)
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i * groups, t = first + r;
    live[i] = r < rows && (!is_q || (t < n.count && n.start + t >= 0));
  }
  const int head0 = head;
  Raw8<T> ra[kRows], rb[kRows];
  RowRing<T, 2 * kRows, kAhead> ring(smem);
  int fetched = 0;
  auto fetch = [&] {  // the rows of one more head, on their way to shared memory
    const int h = head0 + fetched * beside;
    if (fetched < turns) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (live[i] && h < head_end) {
          const T* x = src + (long long)(i * groups) * st.n + h * st.h;
          ring.fetch(2 * i, x);
          ring.fetch(2 * i + 1, x + hop);
        } else {
          ring.clear(2 * i);
          ring.clear(2 * i + 1);
        }
      }
    }
    copies_commit();
    ring.step(ring.put);
    ++fetched;
  };
  if (kNorm != 0) {
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) fetch();
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      zero8(ra[i]);
      zero8(rb[i]);
      if (live[i]) {
        const T* x = src + (long long)(i * groups) * st.n + head * st.h;
        load8(ra[i], x);
        load8(rb[i], x + hop);
      }
    }
  }
  float cc[kRows][8], ss[kRows][8];
  LaneWeights lw;
  if (kNorm != 0 && !is_v) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int t = first + row0 + i * groups;
      if constexpr (kAxes) {
        load_rotation_axes<kNeighbours>(p.ax, p.cos, p.sin, p.max_pos, b, t, at, live[i] ? p.rot : 0, cc[i], ss[i]);
      } else {
        const long long row = live[i] ? (long long)min(n.start + t, max(p.max_pos - 1, 0)) * (p.rot >> 1) : 0;
        load_rotation<kNeighbours>(p.cos + row, p.sin + row, at, live[i] ? p.rot : 0, cc[i], ss[i]);
      }
    }
    stage_weights<T>(is_q ? p.q_w : p.k_w, p.w_f32, D, w);
    __syncthreads();
    lw.read(w, at);
  }
  if (!is_q && (id < 0 || id >= c.num_pages)) {
    if (threadIdx.x == 0) atomicOr(c.status, kStatusBadPage);
    if (kNorm != 0) copies_wait<0>();
    return;
  }
  const int slot0 = (n.start + first) & (size - 1);
  for (int turn = 0; turn < turns; ++turn) {
    if (kNorm != 0) {
      fetch();
      head = head0 + turn * beside;
      copies_wait<kAhead - 1>();
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        ring.take(2 * i, ra[i]);
        ring.take(2 * i + 1, rb[i]);
      }
      ring.step(ring.got);
    }
    if (kNorm != 0 && !is_v) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        norm_rope_lane<T, D, kNeighbours>(ra[i], rb[i], at, lw, cc[i], ss[i], p.eps);
        if (!live[i]) {  // zeros, also where a NaN among the weights has reached them
          zero8(ra[i]);
          zero8(rb[i]);
        }
      }
    }
    if (is_q) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = row0 + i * groups;
        if (r >= rows || head >= head_end) continue;
        T* to = static_cast<T*>(p.q_out) + b * p.q_out_st.b + (long long)(first + r) * p.q_out_st.n +
                head * p.q_out_st.h + at.a;
        store8(ra[i], to);
        store8(rb[i], to + hop);
      }
      continue;
    }
    uint8_t* page = (is_v ? c.v : c.k) + id * c.sp + head * c.sh;
    float* scale_at = (is_v ? c.v_scale : c.k_scale) + (long long)id * c.H + head;
    const float was = slot0 > 0 ? *scale_at : 0.f;  // a page without earlier tokens has no former scale
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
      uint8_t* to = page + (slot0 + r) * c.sn + at.a;
      *reinterpret_cast<uint2*>(to) = any ? quantise8<T, true>(ra[i], inv) : quantise8<T, false>(ra[i], inv);
      *reinterpret_cast<uint2*>(to + hop) = any ? quantise8<T, true>(rb[i], inv) : quantise8<T, false>(rb[i], inv);
    }
    if (slot0 > 0 && scale != was) {  // earlier tokens to the larger scale, 16 codes a thread
      const float ratio = was * inv;
      for (int r = threadIdx.x / G; r < slot0; r += groups) {
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
  if (kNorm != 0) copies_wait<0>();
}

template <typename T, int D, int kRows, int kNorm, bool kPartial, bool kAxes = false>
cudaError_t launch_norm(const Kv8AppendParams& p, dim3 grid, int threads, cudaStream_t st) {
  constexpr auto kKernel = kv8_append_kernel<T, D, kRows, kNorm, kPartial, kAxes>;
  const cudaError_t e = allow_smem<kKernel>(RowRing<T, 2 * kRows, kAhead>::bytes(512));
  if (e != cudaSuccess) return e;
  return launch_chained(kKernel, grid, threads, RowRing<T, 2 * kRows, kAhead>::bytes(threads), 1, p, st);
}

template <typename T, int D, int kRows>
cudaError_t launch_rows(const Kv8AppendParams& p, dim3 grid, int threads, cudaStream_t st) {
  if constexpr (kRows <= 2) {
    if (p.q != nullptr) {
      // (whole heads have no form of their own here: 43.7 us with one, 44.0 without, at bf16 4x16x2048x128)
      if (p.ax.axes)
        return p.neighbours ? launch_norm<T, D, kRows, 2, true, true>(p, grid, threads, st)
                            : launch_norm<T, D, kRows, 1, true, true>(p, grid, threads, st);
      if (p.rot < D)
        return p.neighbours ? launch_norm<T, D, kRows, 2, true>(p, grid, threads, st)
                            : launch_norm<T, D, kRows, 1, true>(p, grid, threads, st);
      return p.neighbours ? launch_norm<T, D, kRows, 2, false>(p, grid, threads, st)
                          : launch_norm<T, D, kRows, 1, false>(p, grid, threads, st);
    }
  }
  return launch_chained(kv8_append_kernel<T, D, kRows, 0, true, false>, grid, threads, 0, 1, p, st);
}

template <typename T, int D>
cudaError_t launch_d(Kv8AppendParams& p, cudaStream_t st) {
  constexpr int G = D / 16;
  const int rows = std::min(1 << p.c.page_shift, p.T);  // most new rows of one page
  // up to 256 threads, then more rows a thread (with norm, whose rows keep their tables' values
  // in registers, two at most); at least two warps, so that a single token still shares out the
  // rescaling of its page
  const int lanes = rows * G;
  const int per = lanes <= 256 ? 1 : lanes <= 512 || p.q ? 2 : 4;
  const int threads = std::max(64, ((lanes + per - 1) / per + 31) / 32 * 32);
  int x = 2 * p.c.H;
  if (p.q) {
    // Heads a block: up to kMaxHeads where kBlocks blocks remain, else one (q, with few tokens: one a
    // row group). At bf16 4x16x2048x128: one head a block 45.2 us, up to eight 40.2 us; 152 or 608 for
    // kBlocks 50 and 43 us.
    const long long places = (long long)p.pages * p.B;
    const auto share = [&](int heads, int least) {
      const long long most = places * heads / kBlocks;
      return std::min(heads, (int)std::max<long long>(least, std::min<long long>(kMaxHeads, most)));
    };
    p.kv_heads = share(p.c.H, 1);
    p.q_heads = share(p.Hq, per == 1 ? std::max(1, threads / G / rows) : 1);
    x = 2 * ((p.c.H + p.kv_heads - 1) / p.kv_heads) + (p.Hq + p.q_heads - 1) / p.q_heads;
  }
  const dim3 grid(x, p.pages, p.B);
  if (per == 1) return launch_rows<T, D, 1>(p, grid, threads, st);
  return per == 2 ? launch_rows<T, D, 2>(p, grid, threads, st) : launch_rows<T, D, 4>(p, grid, threads, st);
}

}  // namespace

cudaError_t launch_kv8_append(Kv8AppendParams& p, bool bf16, cudaStream_t st) {
  if (p.d == 64) return bf16 ? launch_d<__nv_bfloat16, 64>(p, st) : launch_d<__half, 64>(p, st);
  return bf16 ? launch_d<__nv_bfloat16, 128>(p, st) : launch_d<__half, 128>(p, st);
}

}  // namespace fa
