// Rows of [rows, D] arrays held in the registers of the threads that share
// them: vectors of adjacent elements, and sums over a row's threads.
#pragma once
#include "elem.cuh"

namespace cat {

// Threads of a CTA that the helpers below are written for, unless given.
constexpr int kRowThreads = 256;

// VEC adjacent elements, aligned to their total size: as loaded, and as fp32.
template <typename T, int VEC>
struct Vec;
template <>
struct Vec<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ Raw ldr(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ void widen(Raw x, float* v) { v[0] = x; }
  static __device__ __forceinline__ void st(float* p, const float* v) { p[0] = v[0]; }
};
template <>
struct Vec<float, 2> {
  using Raw = float2;
  static __device__ __forceinline__ Raw ldr(const float* p) { return ld_pair(p); }
  static __device__ __forceinline__ void widen(Raw x, float* v) { v[0] = x.x; v[1] = x.y; }
  static __device__ __forceinline__ void st(float* p, const float* v) {
    st_pair(p, make_float2(v[0], v[1]));
  }
};
template <>
struct Vec<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ Raw ldr(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
  }
  static __device__ __forceinline__ void widen(Raw x, float* v) {
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
  static __device__ __forceinline__ void st(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  using Raw = unsigned short;
  static __device__ __forceinline__ Raw ldr(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const unsigned short*>(p));
  }
  static __device__ __forceinline__ void widen(Raw x, float* v) {
    v[0] = __uint_as_float((unsigned int)x << 16);
  }
  static __device__ __forceinline__ void st(__nv_bfloat16* p, const float* v) {
    st_elem(p, v[0]);
  }
};
template <>
struct Vec<__nv_bfloat16, 2> {
  using Raw = unsigned int;
  static __device__ __forceinline__ Raw ldr(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const unsigned int*>(p));
  }
  static __device__ __forceinline__ void widen(Raw x, float* v) {
    v[0] = __uint_as_float(x << 16);
    v[1] = __uint_as_float(x & 0xffff0000u);
  }
  static __device__ __forceinline__ void st(__nv_bfloat16* p, const float* v) {
    st_pair(p, make_float2(v[0], v[1]));
  }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw ldr(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  }
  static __device__ __forceinline__ void widen(Raw x, float* v) {
    const unsigned int w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void st(__nv_bfloat16* p, const float* v) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(h);
  }
};
template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float* v) {
  Vec<T, VEC>::widen(Vec<T, VEC>::ldr(p), v);
}

// Sum over the threads of a row: a warp, or the CTA (TPR = 256) through
// `red` (one float a warp; two barriers, so `red` can be used again at once).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += red[i];
    __syncthreads();
  }
  return v;
}

// Two sums at once over the TPR threads of row group `sub` of a CTA of BT threads;
// `red` holds two floats a warp for each use in turn (`use`), so that one barrier
// a call (the group's own) is enough.
template <int TPR, int BT = kRowThreads>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* red, int sub, int use) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (TPR > 32) {
    red += use * (BT / 32);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "n"(TPR) : "memory");
    red += sub * (TPR / 32);
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      a += red[i].x;
      b += red[i].y;
    }
  }
}

}  // namespace cat
