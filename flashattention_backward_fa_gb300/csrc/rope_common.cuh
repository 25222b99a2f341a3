// Per-head RMS norm and position rotation of one head row, shared by the
// training kernels and the cache-append kernels.
//
//   xn = x / sqrt(mean(x^2) + eps);  y = w o xn
//   out = R(pos) y: the pairs (a, b) of the first rot values become
//         (a cos - b sin, b cos + a sin)
//
// A row of D values is held by D/16 lanes, two chunks of eight consecutive
// values each, so that a load is 16 bytes (16-bit types) and both values of
// every pair are in one lane: with partners rot / 2 apart the second chunk is
// the first one's partners (rot is a multiple of 16; what is not rotated goes
// to the remaining lanes), with neighbouring partners the second chunk is D / 2
// further on. Only the sum of squares crosses lanes, and everything else is packed
// (two-wide) arithmetic. A layout with one chunk a lane, which exchanges partners
// by shuffles, ran at 70% of the copy rate, bound by its instructions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "device_common.cuh"
#include "fa.h"

namespace fa {

// Waits until the kernel before this one in the stream has ended and its writes are there (see
// launch_chained). Every block calls it before it touches memory.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the blocks of the next kernel take their places once all of this one's have called it or ended.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Eight consecutive values of a row as they lie in memory.
template <typename T>
struct Raw8 {
  static constexpr int kQuads = 1;  // 16-byte pieces
  uint4 q[1];
  __device__ __forceinline__ void unpack(uint64_t (&f)[4]) const {
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack2<bf>(w[i], lo, hi);
      f[i] = f2_pack(lo, hi);
    }
  }
  __device__ __forceinline__ void pack(const uint64_t (&f)[4]) {
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      f2_unpack(f[i], lo, hi);
      w[i] = pack2<bf>(lo, hi);
    }
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Raw8<float> {
  static constexpr int kQuads = 2;
  uint4 q[2];
  __device__ __forceinline__ void unpack(uint64_t (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = f2_pack(__uint_as_float(q[i].x), __uint_as_float(q[i].y));
      f[2 * i + 1] = f2_pack(__uint_as_float(q[i].z), __uint_as_float(q[i].w));
    }
  }
  __device__ __forceinline__ void pack(const uint64_t (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, b, c, d;
      f2_unpack(f[2 * i], a, b);
      f2_unpack(f[2 * i + 1], c, d);
      q[i] = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
  }
};

template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& v, const T* p) {
#pragma unroll
  for (int i = 0; i < Raw8<T>::kQuads; ++i) v.q[i] = reinterpret_cast<const uint4*>(p)[i];
}
template <typename T>
__device__ __forceinline__ void store8(const Raw8<T>& v, T* p) {
#pragma unroll
  for (int i = 0; i < Raw8<T>::kQuads; ++i) reinterpret_cast<uint4*>(p)[i] = v.q[i];
}
template <typename T>
__device__ __forceinline__ void zero8(Raw8<T>& v) {
#pragma unroll
  for (int i = 0; i < Raw8<T>::kQuads; ++i) v.q[i] = make_uint4(0u, 0u, 0u, 0u);
}

// 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Sum over the kLanes lanes of a row (kLanes a power of two, rows aligned in the warp).
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A weight vector to shared memory as fp32 (fp32 or T in memory; ones where there is none).
template <typename T>
__device__ __forceinline__ void stage_weights(const void* w, bool w_f32, int d, float* to) {
  for (int e = threadIdx.x; e < d; e += blockDim.x)
    to[e] = w == nullptr ? 1.f : w_f32 ? static_cast<const float*>(w)[e] : static_cast<float>(static_cast<const T*>(w)[e]);
}

__device__ __forceinline__ void read4(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
}

// First values of the two chunks of lane j of a row, and which of them are rotated (both or none
// where one chunk holds the other's partners). The others go through the same arithmetic with
// cos = 1, sin = 0, and with 0 in the partner's place: an infinity or NaN times sin would reach a
// value that it has nothing to do with. kPartial false: rot = D, all are rotated and nothing is
// put in place. (Zeros by selects where needed or not took the backward at bf16 4x16x2048x128
// 0.5 us and the append with norm 0.8 us more; a branch around the rotation 2.7 us more there.)
struct LanePlace {
  int a, b;
  bool turn_a, turn_b;
};
template <int D, bool kNeighbours, bool kPartial>
__device__ __forceinline__ LanePlace lane_place(int j, int rot) {
  if (kNeighbours) return {8 * j, 8 * j + D / 2, !kPartial || 8 * j < rot, !kPartial || 8 * j + D / 2 < rot};
  const int pairs = rot >> 4;  // lanes that hold rotated values
  if (!kPartial || j < pairs) return {8 * j, 8 * j + (rot >> 1), true, true};
  return {rot + 16 * (j - pairs), rot + 16 * (j - pairs) + 8, false, false};
}

// cos and sin of a lane's eight pairs (a token's table rows hold rot / 2 values each): pairs
// (a_i, b_i) of the two chunks, or, with neighbours, four pairs of each chunk.
template <bool kNeighbours>
__device__ __forceinline__ void load_rotation(const float* cos_row, const float* sin_row, const LanePlace& at, int rot,
                                              float (&c)[8], float (&s)[8]) {
  // neighbours: pair indices of the chunks; else both halves are the chunk's one run
  const int lo = kNeighbours ? at.a >> 1 : at.a, hi = kNeighbours ? at.b >> 1 : at.a + 4;
  const bool has_lo = at.a < rot, has_hi = (kNeighbours ? at.b : at.a) < rot;
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (has_lo) {
    read4(cos_row + lo, c);
    read4(sin_row + lo, s);
  }
  if (has_hi) {
    read4(cos_row + hi, c + 4);
    read4(sin_row + hi, s + 4);
  }
}

__device__ __forceinline__ uint64_t f2_swap(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return f2_pack(hi, lo);
}

// v, or zeros.
__device__ __forceinline__ uint64_t f2_if(bool yes, uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return f2_pack(yes ? lo : 0.f, yes ? hi : 0.f);
}

__device__ __forceinline__ void read_pairs(const float* p, uint64_t (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 a = reinterpret_cast<const float4*>(p)[i];
    f[2 * i] = f2_pack(a.x, a.y);
    f[2 * i + 1] = f2_pack(a.z, a.w);
  }
}

// The weights of a lane's two chunks.
struct LaneWeights {
  uint64_t a[4], b[4];
  __device__ __forceinline__ void read(const float* w, const LanePlace& at) {
    read_pairs(w + at.a, a);
    read_pairs(w + at.b, b);
  }
};

__device__ __forceinline__ float f2_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}

// 1 / sqrt(x). rsqrtf is off by up to two units in the last place, which all values of a row
// would share; a Newton step leaves about half a unit. (x past the fp32 range: 0.)
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return x < INFINITY ? fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r) : r;
}

// Forward of a lane's 16 values, in place; every lane of the warp calls it (shuffles).
template <typename T, int D, bool kNeighbours>
__device__ __forceinline__ void norm_rope_lane(Raw8<T>& ra, Raw8<T>& rb, const LanePlace& at, const LaneWeights& w,
                                               const float (&c)[8], const float (&s)[8], float eps) {
  uint64_t a[4], b[4];
  ra.unpack(a);
  rb.unpack(b);
  uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s0 = f2_fma(a[i], a[i], s0);
    s1 = f2_fma(b[i], b[i], s1);
  }
  const float ss = row_sum<D / 16>(f2_sum(f2_add(s0, s1)));
  const float r1 = inv_sqrt(fmaf(ss, 1.f / D, eps));
  const uint64_t r = f2_pack(r1, r1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = f2_mul(a[i], f2_mul(r, w.a[i]));
    b[i] = f2_mul(b[i], f2_mul(r, w.b[i]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kNeighbours) {
      a[i] = f2_fma(a[i], f2_pack(c[i], c[i]), f2_mul(f2_if(at.turn_a, f2_swap(a[i])), f2_pack(-s[i], s[i])));
      b[i] = f2_fma(b[i], f2_pack(c[4 + i], c[4 + i]),
                    f2_mul(f2_if(at.turn_b, f2_swap(b[i])), f2_pack(-s[4 + i], s[4 + i])));
    } else {
      const uint64_t ci = f2_pack(c[2 * i], c[2 * i + 1]), si = f2_pack(s[2 * i], s[2 * i + 1]);
      const uint64_t ni = f2_pack(-s[2 * i], -s[2 * i + 1]);
      const uint64_t oa = f2_fma(a[i], ci, f2_mul(f2_if(at.turn_a, b[i]), ni));
      b[i] = f2_fma(b[i], ci, f2_mul(f2_if(at.turn_a, a[i]), si));
      a[i] = oa;
    }
  }
  ra.pack(a);
  rb.pack(b);
}

// A walk over the rows (b, n, head) of [B, N, H, *], heads fastest, with the
// offset of the row in one tensor. The one decomposition of a row number is in
// 32 bits where it fits (a 64-bit division costs as much as a row's arithmetic).
struct RowWalk {
  long long b, at;
  int n, head;
  __device__ __forceinline__ void start(long long row, int N, int H, const fa_strides& st) {
    long long token;
    if (row >> 32) {
      token = row / H;
      b = token / N;
    } else {
      token = (unsigned)row / (unsigned)H;
      b = (unsigned)token / (unsigned)N;
    }
    head = (int)(row - token * H);
    n = (int)(token - b * N);
    at = offset(st);
  }
  __device__ __forceinline__ long long offset(const fa_strides& st) const {
    return b * st.b + (long long)n * st.n + (long long)head * st.h;
  }
  // The same row in another tensor.
  __device__ __forceinline__ RowWalk in(const fa_strides& st) const {
    RowWalk w = *this;
    w.at = offset(st);
    return w;
  }
  // To the next row; true when it is another token's.
  __device__ __forceinline__ bool next(int N, int H, const fa_strides& st) {
    at += st.h;
    if (++head < H) return false;
    head = 0;
    if (++n == N) {
      n = 0;
      ++b;
    }
    at = b * st.b + (long long)n * st.n;
    return true;
  }
};

// A lane's slots for rows on their way: kDepth rows of kChunks chunks, each lane reading back
// only what it copied itself, so waiting for its own copies is all the synchronisation needed.
// Slots of a chunk are 16 bytes a thread apart (no bank conflicts).
template <typename T, int kChunks, int kDepth>
struct RowRing {
  static constexpr int kPieces = kChunks * Raw8<T>::kQuads;
  static constexpr int bytes(int threads) { return kDepth * kPieces * threads * 16; }
  uint32_t base, apart, put, got;  // slots of this thread, bytes between pieces, of the next row to come and to take
  __device__ __forceinline__ RowRing(void* smem)
      : base(smem_u32(smem) + threadIdx.x * 16), apart(blockDim.x * 16), put(base), got(base) {}
  __device__ __forceinline__ void step(uint32_t& at) const {
    at += kPieces * apart;
    if (at == base + kDepth * kPieces * apart) at = base;
  }
  __device__ __forceinline__ void fetch(int chunk, const T* p) const {
#pragma unroll
    for (int i = 0; i < Raw8<T>::kQuads; ++i)
      copy16_async(put + (chunk * Raw8<T>::kQuads + i) * apart, reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void clear(int chunk) const {
#pragma unroll
    for (int i = 0; i < Raw8<T>::kQuads; ++i)
      st_shared_v4(put + (chunk * Raw8<T>::kQuads + i) * apart, 0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void take(int chunk, Raw8<T>& v) const {
#pragma unroll
    for (int i = 0; i < Raw8<T>::kQuads; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.q[i].x), "=r"(v.q[i].y), "=r"(v.q[i].z), "=r"(v.q[i].w)
                   : "r"(got + (chunk * Raw8<T>::kQuads + i) * apart)
                   : "memory");
  }
};

// Rows [first, first + count) of one tensor by one row group (D / 16 lanes; the
// groups of a warp call it together, each with its own rows and all with the same
// count). kDepth - 1 rows are on their way while a row is computed.
// table_at(b, n): offset of the token's table rows. The weights are staged into w (a
// block-wide step) once the first copies are under way.
template <typename T, int D, bool kNeighbours, int kDepth, typename TableAt>
__device__ __forceinline__ void norm_rope_rows(void* smem, const T* x, T* out, const fa_strides& x_st,
                                               const fa_strides& out_st, long long rows, int N, int H, long long first,
                                               int count, const void* weights, bool w_f32, float* w,
                                               const float* cos, const float* sin, int rot, float eps,
                                               const TableAt& table_at) {
  RowRing<T, 2, kDepth> ring(smem);
  const LanePlace at = lane_place<D, kNeighbours, true>(threadIdx.x % (D / 16), rot);  // (costs nothing here)
  const int live = (int)min((long long)count, max(rows - first, 0ll));
  RowWalk in;
  in.start(first, N, H, x_st);
  RowWalk to = in.in(out_st);
  x += at.a;
  out += at.a;
  const int hop = at.b - at.a;
  int loaded = 0;
  auto fetch = [&] {
    if (loaded < live) {
      const T* p = x + in.at;
      ring.fetch(0, p);
      ring.fetch(1, p + hop);
    } else if (loaded < count) {
      ring.clear(0);
      ring.clear(1);
    }
    copies_commit();
    ring.step(ring.put);
    in.next(N, H, x_st);
    ++loaded;
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch();
  stage_weights<T>(weights, w_f32, D, w);
  __syncthreads();
  LaneWeights lw;
  lw.read(w, at);
  float c[8], s[8];
  bool token = true;
  for (int i = 0; i < count; ++i) {
    fetch();
    if (token) {
      const bool ok = i < live;
      const long long row = ok ? table_at(to.b, to.n) : 0;
      load_rotation<kNeighbours>(cos + row, sin + row, at, ok ? rot : 0, c, s);
    }
    copies_wait<kDepth - 1>();
    Raw8<T> a, b;
    ring.take(0, a);
    ring.take(1, b);
    ring.step(ring.got);
    norm_rope_lane<T, D, kNeighbours>(a, b, at, lw, c, s, eps);
    if (i < live) {
      T* p = out + to.at;
      store8(a, p);
      store8(b, p + hop);
    }
    token = to.next(N, H, out_st);
  }
}

}  // namespace fa
