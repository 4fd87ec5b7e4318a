// The residual stream between two blocks, with its norms (resnorm_fwd.cu,
// resnorm_bwd.cu):
//   u = post ? LN(B)·pg + pb : B,  H = R + scale·gate·u,  Y = LN(H)·gamma + beta.
#pragma once
#include "cat_internal.h"
#include "rows.cuh"
#include "../../include/cat.h"

namespace cat {

enum { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_ROW = 2 };

// Arithmetic on the elements of a vector, two at a time where it has an even number
// (packed fp32 instructions, each half rounded as the single one is).  The kernels
// of the residual stream were bound by instructions before memory.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0,
                                     float b1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0,
                                     float b1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// d = a·b + c, a·b, a + b; a plain float stands for itself in every element.
struct Each {
  const float* p;
  float s;
  __device__ __forceinline__ Each(const float* q) : p(q), s(0.f) {}
  __device__ __forceinline__ Each(float v) : p(nullptr), s(v) {}
  __device__ __forceinline__ float operator[](int e) const { return p ? p[e] : s; }
};
template <int VEC>
__device__ __forceinline__ void v_fma(float* d, Each a, Each b, Each c) {
  if (VEC == 1) d[0] = fmaf(a[0], b[0], c[0]);
#pragma unroll
  for (int e = 0; e + 1 < VEC; e += 2)
    fma2(d[e], d[e + 1], a[e], a[e + 1], b[e], b[e + 1], c[e], c[e + 1]);
}
template <int VEC>
__device__ __forceinline__ void v_mul(float* d, Each a, Each b) {
  if (VEC == 1) d[0] = a[0] * b[0];
#pragma unroll
  for (int e = 0; e + 1 < VEC; e += 2) mul2(d[e], d[e + 1], a[e], a[e + 1], b[e], b[e + 1]);
}
template <int VEC>
__device__ __forceinline__ void v_add(float* d, Each a, Each b) {
  if (VEC == 1) d[0] = a[0] + b[0];
#pragma unroll
  for (int e = 0; e + 1 < VEC; e += 2) add2(d[e], d[e + 1], a[e], a[e + 1], b[e], b[e + 1]);
}
// A running sum of two halves (of a single one where VEC is 1).
template <int VEC>
struct Sum2 {
  float x = 0.f, y = 0.f;
  __device__ __forceinline__ void add(const float* v) {
    if (VEC == 1) x += v[0];
#pragma unroll
    for (int e = 0; e + 1 < VEC; e += 2) add2(x, y, x, y, v[e], v[e + 1]);
  }
  __device__ __forceinline__ void dot(const float* a, const float* b) {
    if (VEC == 1) x = fmaf(a[0], b[0], x);
#pragma unroll
    for (int e = 0; e + 1 < VEC; e += 2) fma2(x, y, a[e], a[e + 1], b[e], b[e + 1], x, y);
  }
  __device__ __forceinline__ float total() const { return x + y; }
};

// fp32 values of a vector at p, or `fill` where there is none.
template <typename T, int VEC>
__device__ __forceinline__ void load_or(const T* p, int c, float fill, float* v) {
  if (p) {
    load<T, VEC>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = fill;
  }
}

}  // namespace cat
