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
// further on. Only the sum of squares crosses lanes. With the weights folded
// into the token's factors, out = r (x C + partner S) is three packed (two-wide)
// operations for two values; a layout with one chunk a lane, which exchanges
// partners by shuffles, took 238 instructions for 16 values against about 90
// and ran at 70% of the copy rate.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "device_common.cuh"
#include "fa.h"

namespace fa {

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
  for (int i = 0; i < Raw8<T>::kQuads; ++i) v.q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
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

// 16 bytes from global to shared memory, asynchronously; zeros where !valid (nothing is read then).
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
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

// First values of the two chunks of lane j of a row.
struct LanePlace {
  int a, b;
};
template <int D, bool kNeighbours>
__device__ __forceinline__ LanePlace lane_place(int j, int rot) {
  if (kNeighbours) return {8 * j, 8 * j + D / 2};
  const int pairs = rot >> 4;  // lanes that hold rotated values
  if (j < pairs) return {8 * j, 8 * j + (rot >> 1)};
  return {rot + 16 * (j - pairs), rot + 16 * (j - pairs) + 8};
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

// A token's factors with the weights folded in: out_a = r (a ca + pa sa), pa the partners of a
// (b, or a with neighbours swapped), and alike for b.
struct Factors {
  uint64_t ca[4], sa[4], cb[4], sb[4];
};
template <bool kNeighbours>
__device__ __forceinline__ void fold_weights(const float* w, const LanePlace& at, const float (&c)[8],
                                             const float (&s)[8], Factors& f) {
  float wa[8], wb[8];
  read4(w + at.a, wa);
  read4(w + at.a + 4, wa + 4);
  read4(w + at.b, wb);
  read4(w + at.b + 4, wb + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = 2 * i, y = 2 * i + 1;
    if (kNeighbours) {
      f.ca[i] = f2_pack(c[i] * wa[x], c[i] * wa[y]);
      f.sa[i] = f2_pack(-s[i] * wa[y], s[i] * wa[x]);
      f.cb[i] = f2_pack(c[4 + i] * wb[x], c[4 + i] * wb[y]);
      f.sb[i] = f2_pack(-s[4 + i] * wb[y], s[4 + i] * wb[x]);
    } else {
      f.ca[i] = f2_pack(c[x] * wa[x], c[y] * wa[y]);
      f.sa[i] = f2_pack(-s[x] * wb[x], -s[y] * wb[y]);
      f.cb[i] = f2_pack(c[x] * wb[x], c[y] * wb[y]);
      f.sb[i] = f2_pack(s[x] * wa[x], s[y] * wa[y]);
    }
  }
}

__device__ __forceinline__ uint64_t f2_swap(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return f2_pack(hi, lo);
}

__device__ __forceinline__ float f2_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}

// Forward of a lane's 16 values, in place; every lane of the warp calls it (shuffles).
template <typename T, int D, bool kNeighbours>
__device__ __forceinline__ void norm_rope_lane(Raw8<T>& ra, Raw8<T>& rb, const Factors& f, float eps) {
  uint64_t a[4], b[4], oa[4], ob[4];
  ra.unpack(a);
  rb.unpack(b);
  uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s0 = f2_fma(a[i], a[i], s0);
    s1 = f2_fma(b[i], b[i], s1);
  }
  const float ss = row_sum<D / 16>(f2_sum(f2_add(s0, s1)));
  const float r1 = rsqrtf(fmaf(ss, 1.f / D, eps));
  const uint64_t r = f2_pack(r1, r1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    oa[i] = f2_mul(r, f2_fma(a[i], f.ca[i], f2_mul(kNeighbours ? f2_swap(a[i]) : b[i], f.sa[i])));
    ob[i] = f2_mul(r, f2_fma(b[i], f.cb[i], f2_mul(kNeighbours ? f2_swap(b[i]) : a[i], f.sb[i])));
  }
  ra.pack(oa);
  rb.pack(ob);
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
    at = b * st.b + (long long)n * st.n + (long long)head * st.h;
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
  uint32_t base;
  int threads;
  __device__ __forceinline__ RowRing(void* smem) : base(smem_u32(smem) + threadIdx.x * 16), threads(blockDim.x) {}
  __device__ __forceinline__ uint32_t slot(int row, int chunk, int piece) const {
    return base + (uint32_t)(((row % kDepth) * kPieces + chunk * Raw8<T>::kQuads + piece) * threads) * 16u;
  }
  __device__ __forceinline__ void fetch(int row, int chunk, const T* p, bool valid) const {
#pragma unroll
    for (int i = 0; i < Raw8<T>::kQuads; ++i)
      copy16_async(slot(row, chunk, i), reinterpret_cast<const uint4*>(p) + i, valid);
  }
  __device__ __forceinline__ void take(int row, int chunk, Raw8<T>& v) const {
#pragma unroll
    for (int i = 0; i < Raw8<T>::kQuads; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.q[i].x), "=r"(v.q[i].y), "=r"(v.q[i].z), "=r"(v.q[i].w)
                   : "r"(slot(row, chunk, i))
                   : "memory");
  }
};

// The launch that follows a kernel in the stream may begin (its own prologue) while the
// kernel ends; what reads the kernel's outputs waits for all of it first. Both are no-ops
// in launches without the attribute.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Rows [first, first + count) of one tensor by one row group (D / 16 lanes; the
// groups of a warp call it together, each with its own rows and all with the same
// count). kDepth - 1 rows are on their way while a row is computed.
// table_at(b, n): offset of the token's table rows, or -1 for a padding row, which
// becomes zeros (kPadding) and is not read. The weights are staged into w (a block-wide step)
// once the first copies are under way.
template <typename T, int D, bool kNeighbours, bool kPadding, int kDepth, typename TableAt>
__device__ __forceinline__ void norm_rope_rows(void* smem, const T* x, T* out, const fa_strides& x_st,
                                               const fa_strides& out_st, long long rows, int N, int H, long long first,
                                               int count, const void* weights, bool w_f32, float* w,
                                               const float* cos, const float* sin, int rot, float eps,
                                               const TableAt& table_at) {
  const RowRing<T, 2, kDepth> ring(smem);
  const LanePlace at = lane_place<D, kNeighbours>(threadIdx.x % (D / 16), rot);
  const int live = (int)min((long long)count, max(rows - first, 0ll));
  RowWalk in, to;
  in.start(first, N, H, x_st);
  to.start(first, N, H, out_st);
  int loaded = 0;
  auto fetch = [&] {
    const bool ok = loaded < live && (!kPadding || table_at(in.b, in.n) >= 0);
    const T* p = x + (ok ? in.at : 0);
    ring.fetch(loaded, 0, p + at.a, ok);
    ring.fetch(loaded, 1, p + at.b, ok);
    copies_commit();
    in.next(N, H, x_st);
    ++loaded;
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch();
  stage_weights<T>(weights, w_f32, D, w);
  __syncthreads();
  Factors f;
  bool token = true;
  for (int i = 0; i < count; ++i) {
    fetch();
    if (token) {
      const bool ok = i < live;
      const long long row = ok ? max(table_at(to.b, to.n), 0ll) : 0;
      float c[8], s[8];
      load_rotation<kNeighbours>(cos + row, sin + row, at, ok ? rot : 0, c, s);
      fold_weights<kNeighbours>(w, at, c, s, f);
    }
    copies_wait<kDepth - 1>();
    Raw8<T> a, b;
    ring.take(i, 0, a);
    ring.take(i, 1, b);
    norm_rope_lane<T, D, kNeighbours>(a, b, f, eps);  // (zeros stay zeros)
    if (i < live) {
      store8(a, out + to.at + at.a);
      store8(b, out + to.at + at.b);
    }
    token = to.next(N, H, out_st);
  }
}

}  // namespace fa
