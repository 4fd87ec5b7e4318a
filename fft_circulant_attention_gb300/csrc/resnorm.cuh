// The residual stream between two blocks, with its norms (resnorm_fwd.cu,
// resnorm_bwd.cu):
//   u = post ? LN(B)·pg + pb : B,  H = R + scale·gate·u,  Y = LN(H)·gamma + beta.
#pragma once
#include "cat_internal.h"
#include "rows.cuh"
#include "../../include/cat.h"

namespace cat {

enum { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_ROW = 2 };

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
