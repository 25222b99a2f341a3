// Per-head RMS norm and position rotation of one head row, shared by the
// training kernels and the cache-append kernels.
//
//   xn = x / sqrt(mean(x^2) + eps);  y = w o xn
//   out = R(pos) y: the pairs (a, b) of the first rot values become
//         (a cos - b sin, b cos + a sin)
//
// A row of D values is held by D/8 lanes, eight consecutive values each, so a
// lane's load is 16 bytes (16-bit types) and a warp moves whole rows. The
// rotation is written element-wise, out_i = y_i c_i + y_partner(i) s_i, with the
// sign of the pair folded into s_i: partners rot/2 apart sit in another lane of
// the row at the same place in its eight (rot is a multiple of 16), so the raw
// words are exchanged by shuffles before they are unpacked; neighbouring
// partners sit in the same lane. Values past rot have c = 1, s = 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"

namespace fa {

// Eight consecutive values of a row as loaded.
template <typename T>
struct Raw8 {
  uint4 a;
  __device__ __forceinline__ void load(const T* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    unpack2<bf>(a.x, f[0], f[1]);
    unpack2<bf>(a.y, f[2], f[3]);
    unpack2<bf>(a.z, f[4], f[5]);
    unpack2<bf>(a.w, f[6], f[7]);
  }
  __device__ __forceinline__ void pack(const float (&f)[8]) {
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    a = make_uint4(pack2<bf>(f[0], f[1]), pack2<bf>(f[2], f[3]), pack2<bf>(f[4], f[5]), pack2<bf>(f[6], f[7]));
  }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ Raw8 from_lane(int src) const {
    Raw8 r;
    r.a.x = __shfl_sync(0xffffffffu, a.x, src);
    r.a.y = __shfl_sync(0xffffffffu, a.y, src);
    r.a.z = __shfl_sync(0xffffffffu, a.z, src);
    r.a.w = __shfl_sync(0xffffffffu, a.w, src);
    return r;
  }
};

template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void pack(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ Raw8 from_lane(int src) const {
    float f[8];
    unpack(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __shfl_sync(0xffffffffu, f[i], src);
    Raw8 r;
    r.pack(f);
    return r;
  }
};

// Sum over the kLanes lanes of a row (kLanes a power of two, rows aligned in the warp).
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's eight weights (fp32 or T in memory; ones without a weight vector).
template <typename T>
__device__ __forceinline__ void load_weight8(const void* w, bool w_f32, int e0, float (&f)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (w_f32) {
    const float* p = static_cast<const float*>(w) + e0;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __ldg(p + i);
  } else {
    const T* p = static_cast<const T*>(w) + e0;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(p[i]);
  }
}

// Which lane of the warp holds the rotation partners of a lane's eight values
// (itself where there are none or where partners are neighbours).
template <bool kNeighbours>
__device__ __forceinline__ int partner_lane(int lane, int e0, int rot) {
  if (kNeighbours || e0 >= rot) return lane;
  const int hop = rot >> 4;  // lanes between partners: (rot / 2) / 8
  return e0 < (rot >> 1) ? lane + hop : lane - hop;
}

// c_i and signed s_i of a lane's eight values from the token's table rows (rot / 2 values each).
template <bool kNeighbours>
__device__ __forceinline__ void load_rotation(const float* cos_row, const float* sin_row, int e0, int rot,
                                              float (&c)[8], float (&s)[8]) {
  if (e0 >= rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    return;
  }
  if (kNeighbours) {
    const float4 cc = __ldg(reinterpret_cast<const float4*>(cos_row + (e0 >> 1)));
    const float4 ss = __ldg(reinterpret_cast<const float4*>(sin_row + (e0 >> 1)));
    const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[2 * j] = c[2 * j + 1] = cv[j];
      s[2 * j] = -sv[j];
      s[2 * j + 1] = sv[j];
    }
  } else {
    const int h = rot >> 1;
    const bool low = e0 < h;
    const int at = low ? e0 : e0 - h;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(cos_row + at));
    const float4 c1 = __ldg(reinterpret_cast<const float4*>(cos_row + at) + 1);
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(sin_row + at));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(sin_row + at) + 1);
    const float sg = low ? -1.f : 1.f;
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = sg * s0.x, s[1] = sg * s0.y, s[2] = sg * s0.z, s[3] = sg * s0.w;
    s[4] = sg * s1.x, s[5] = sg * s1.y, s[6] = sg * s1.z, s[7] = sg * s1.w;
  }
}

// Forward of one row chunk: every lane of the warp calls it (shuffles). w_p are
// the partners' weights (equal to w where the partner lane is the lane itself
// and partners are neighbours, where they are not used).
template <typename T, int D, bool kNeighbours>
__device__ __forceinline__ void norm_rope_chunk(const Raw8<T>& raw, int partner, const float (&w)[8],
                                                const float (&w_p)[8], const float (&c)[8], const float (&s)[8],
                                                float eps, float (&out)[8]) {
  float x[8];
  raw.unpack(x);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = row_sum<D / 8>(ss);
  const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
  if (kNeighbours) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = fmaf(x[i], c[i], x[i ^ 1] * s[i]);
  } else {
    float xp[8];
    raw.from_lane(partner).unpack(xp);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = fmaf(x[i] * r * w[i], c[i], xp[i] * r * w_p[i] * s[i]);
  }
}

}  // namespace fa
