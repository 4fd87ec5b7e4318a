// Residual addition with gate, scale and the norms before and after a block,
// forward:
//   u = post ? (B - mean_B)·rstd_B·pg + pb : B   (each row of D)
//   H = R + scale·gate·u,   Y = (H - mean_H)·rstd_H·gamma + beta.
// Y and the statistics are those of H before its rounding to the storage type.
//
// Bound by memory: R and B (and a gate of rows) are read once, H and Y written
// once; a row stays in the registers of the threads that share it, a warp up to
// D = 1024, a CTA above.  All sums are fp32, of centred values.
//
// Measured: 65536 fp32 rows of 1024 with a gate of rows 196 us (6.85 TB/s, the copy
// rate), bf16 without gate 81 us (6.6 TB/s); 16384 bf16 rows of 768 with both norms
// 21.8 us (4.6 TB/s, half of the issue slots busy).
#include "resnorm.cuh"

namespace cat {

namespace {

constexpr int kThreads = kRowThreads;

// Mean and 1/sqrt(variance + eps) of the row whose vectors are v (elements
// from D on are 0); v is centred.
template <int VEC, int TPR, int NV, bool FULL>
__device__ __forceinline__ void centre(float (&v)[NV][VEC], int t, int D, float eps, float* red,
                                       float* mean, float* rstd) {
  Sum2<VEC> s, q;
#pragma unroll
  for (int k = 0; k < NV; ++k) s.add(v[k]);
  const float mu = row_sum<TPR>(s.total(), red) / (float)D;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (FULL || (k * TPR + t) * VEC < D) {
      v_add<VEC>(v[k], v[k], -mu);
      q.dot(v[k], v[k]);
    }
  *mean = mu;
  *rstd = 1.f / sqrtf(row_sum<TPR>(q.total(), red) / (float)D + eps);
}

// FULL: the threads' vectors are the row, none lies behind it.
template <typename T, int VEC, int TPR, int E, int POST, bool FULL>
__global__ void __launch_bounds__(kThreads) resnorm_fwd_kernel(ResNormArgs a) {
  constexpr int NV = E / VEC;
  using V = Vec<T, VEC>;
  __shared__ float red[kThreads / 32];
  const int t = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x, D = a.D;
  const int row = TPR == 32 ? blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.rows) return;
  const size_t off = (size_t)row * D;
  const T* B = static_cast<const T*>(a.b) + off;
  const T* R = static_cast<const T*>(a.r) + off;
  const T* G = static_cast<const T*>(a.gate);
  if (a.gate_kind == GATE_ROW) G += off;
  typename V::Raw rr[NV];
  float u[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (FULL || c < D) {
      load<T, VEC>(B + c, u[k]);
      rr[k] = V::ldr(R + c);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[k][e] = 0.f;
    }
  }
  float mb = 0.f, rb = 0.f;
  if (POST) centre<VEC, TPR, NV, FULL>(u, t, D, a.eps, red, &mb, &rb);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (!FULL && c >= D) continue;
    float w[VEC], r[VEC];
    if (POST) {
      float p[VEC];
      load_or<T, VEC>(static_cast<const T*>(a.pg), c, 1.f, w);
      load_or<T, VEC>(static_cast<const T*>(a.pb), c, 0.f, p);
      v_mul<VEC>(u[k], u[k], rb);
      v_fma<VEC>(u[k], u[k], w, p);
    }
    load_or<T, VEC>(G, c, 1.f, w);
    V::widen(rr[k], r);
    v_mul<VEC>(w, w, a.scale);
    v_fma<VEC>(u[k], u[k], w, r);
    V::st(static_cast<T*>(a.h) + off + c, u[k]);
  }
  float mh, rh;
  centre<VEC, TPR, NV, FULL>(u, t, D, a.eps, red, &mh, &rh);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (!FULL && c >= D) continue;
    float w[VEC], p[VEC];
    load_or<T, VEC>(static_cast<const T*>(a.gamma), c, 1.f, w);
    load_or<T, VEC>(static_cast<const T*>(a.beta), c, 0.f, p);
    v_mul<VEC>(u[k], u[k], rh);
    v_fma<VEC>(p, u[k], w, p);
    V::st(static_cast<T*>(a.y) + off + c, p);
  }
  if (t == 0) {
    float* s = a.stats + row;
    s[0] = mh;
    s[(size_t)a.rows] = rh;
    if (POST) {
      s[2 * (size_t)a.rows] = mb;
      s[3 * (size_t)a.rows] = rb;
    }
  }
}

template <typename T, int VEC, int TPR, int E, bool FULL>
cudaError_t go(const ResNormArgs& a, cudaStream_t st) {
  const int per = kThreads / TPR, grid = (a.rows + per - 1) / per;
  if (a.post)
    resnorm_fwd_kernel<T, VEC, TPR, E, 1, FULL><<<grid, kThreads, 0, st>>>(a);
  else
    resnorm_fwd_kernel<T, VEC, TPR, E, 0, FULL><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int VEC, int TPR, int E>
cudaError_t fwd(const ResNormArgs& a, cudaStream_t st) {
  if (VEC > 1 && a.D == TPR * E) return go<T, VEC, TPR, E, VEC != 1>(a, st);
  return go<T, VEC, TPR, E, false>(a, st);
}

// A warp a row while its lanes hold the row in at most 32 registers each (by
// eighths), else the CTA.
template <typename T, int VEC>
cudaError_t pick(const ResNormArgs& a, cudaStream_t st) {
  const int D = a.D;
  if (D <= 32 * 8) return fwd<T, VEC, 32, 8>(a, st);
  if (D <= 32 * 16) return fwd<T, VEC, 32, 16>(a, st);
  if (D <= 32 * 24) return fwd<T, VEC, 32, 24>(a, st);
  if (D <= 32 * 32) return fwd<T, VEC, 32, 32>(a, st);
  if (D <= 256 * 8) return fwd<T, VEC, 256, 8>(a, st);
  if (D <= 256 * 16) return fwd<T, VEC, 256, 16>(a, st);
  return fwd<T, VEC, 256, 32>(a, st);
}

}  // namespace

cudaError_t launch_resnorm_forward(const ResNormArgs& a, int dtype, cudaStream_t st) {
  // Full vectors where they divide the rows (every row start aligned).
  if (dtype == CAT_BF16)
    return a.D % 8 == 0 ? pick<__nv_bfloat16, 8>(a, st) : pick<__nv_bfloat16, 1>(a, st);
  return a.D % 4 == 0 ? pick<float, 4>(a, st) : pick<float, 1>(a, st);
}

}  // namespace cat
