// What the tensor-core attention kernels share: packed fp32 arithmetic, the
// exponential, bf16 packing and the care for values that are not finite.
#pragma once
#include <cuda_bf16.h>

#include "attn.cuh"
#include "tc.cuh"

namespace cat {

constexpr int kTile = 128;                 // rows of a query tile, keys of a block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// a·b + c on two fp32 values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Whether either bf16 half of w is an infinity or NaN.
__device__ __forceinline__ bool odd2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t drop_odd(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// A [kTile][DP] tile in shared memory, by one warp: values that are not
// finite become zero.  True if one of them lay in a row below `rows`.
template <int DP>
__device__ __forceinline__ bool clean_tile(unsigned char* tile, int rows) {
  uint4* v = reinterpret_cast<uint4*>(tile);
  bool found = false;
#pragma unroll 8
  for (int i = threadIdx.x & 31; i < kTile * DP * 2 / 16; i += 32) {
    uint4 x = v[i];
    if (odd2(x.x) || odd2(x.y) || odd2(x.z) || odd2(x.w)) {
      // 8 pieces a row, kTile rows a box of 64 columns.
      if ((i / 8) % kTile < rows) found = true;
      v[i] = make_uint4(drop_odd(x.x), drop_odd(x.y), drop_odd(x.z), drop_odd(x.w));
    }
  }
  return __any_sync(0xffffffffu, found);
}

}  // namespace cat
