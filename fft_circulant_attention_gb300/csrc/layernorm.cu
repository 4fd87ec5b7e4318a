// Layer norm over the rows of a [rows, D] array, forward and backward.
//   mean = Σ x / D, rstd = 1 / sqrt(Σ (x - mean)² / D + eps),
//   x̂ = (x - mean)·rstd, y = x̂·gamma + beta;
//   g = dy·gamma, dx = rstd·(g - mean(g) - x̂·mean(g·x̂)),
//   dgamma = Σ_rows dy·x̂, dbeta = Σ_rows dy.
//
// Bound by memory: the forward reads x and writes y, the backward reads x
// and dy and writes dx, each element once.  A row stays in the registers of
// the threads that share it (a warp up to D = 1024, a CTA of 256 threads
// above), so the mean is subtracted before the squares are summed (no
// cancellation) and nothing is read twice.  All sums are fp32.
//
// The backward keeps each thread's columns of Σ dy·x̂ and Σ dy in registers
// over all the rows its persistent CTA takes, adds the CTA's warps in shared
// memory and writes one partial row a CTA; a second kernel adds the partial
// rows in a fixed order.  No atomics: results repeat bit for bit.
//
// Measured: 65536 fp32 rows of 1024, forward 79 us (6.8 TB/s, the measured copy
// rate), backward 131 us (6.1 TB/s, 91 %) and 4 us for the partial rows; 16384
// bf16 rows of 768, forward 10.6 us, backward 17.4 and 3.5 us, where a launch's
// start and end are a third of it.
#include "cat_internal.h"
#include "rows.cuh"
#include "../../include/cat.h"

namespace cat {

namespace {

constexpr int kThreads = kRowThreads;

// E elements a thread in vectors of VEC: vector k of thread t covers columns
// (k·TPR + t)·VEC ..
template <typename T, int VEC, int TPR, int E>
__global__ void __launch_bounds__(kThreads)
ln_fwd_kernel(const T* __restrict__ X, const T* __restrict__ gamma, const T* __restrict__ beta,
              T* __restrict__ Y, float* __restrict__ mean, float* __restrict__ rstd, int rows,
              int D, float eps) {
  constexpr int NV = E / VEC;
  __shared__ float red[kThreads / 32];
  const int t = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int row = TPR == 32 ? blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= rows) return;
  const T* x = X + (size_t)row * D;
  T* y = Y + (size_t)row * D;
  float v[NV][VEC];
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (c < D) {
      load<T, VEC>(x + c, v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) s += v[k][e];
  }
  const float mu = row_sum<TPR>(s, red) / (float)D;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (c < D) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[k][e] -= mu;
        q = fmaf(v[k][e], v[k][e], q);
      }
    }
  }
  const float r = 1.f / sqrtf(row_sum<TPR>(q, red) / (float)D + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (c < D) {
      float w[VEC], b[VEC];
      if (gamma) load<T, VEC>(gamma + c, w);
      if (beta) load<T, VEC>(beta + c, b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float u = v[k][e] * r;
        if (gamma) u *= w[e];
        if (beta) u += b[e];
        w[e] = u;
      }
      Vec<T, VEC>::st(y + c, w);
    }
  }
  if (t == 0) {
    mean[row] = mu;
    rstd[row] = r;
  }
}

// CTAs of the backward that an SM holds: its persistent grid is that many an
// SM, so that none waits for another to end.
template <typename T, int VEC, int E>
constexpr int bwd_per_sm() {
  return E == 8 ? (sizeof(T) == 2 && VEC == 8 ? 4 : 3) : E == 16 ? 2 : 1;
}

// part: [gridDim.x][2][D] sums of dy·x̂ and dy over the CTA's rows (null: none).
template <typename T, int VEC, int TPR, int E>
__global__ void __launch_bounds__(kThreads, bwd_per_sm<T, VEC, E>())
ln_bwd_kernel(const T* __restrict__ X, const T* __restrict__ gamma, const float* __restrict__ mean,
              const float* __restrict__ rstd, const T* __restrict__ dY, T* __restrict__ dX,
              float* __restrict__ part, int rows, int D) {
  using V = Vec<T, VEC>;
  using Raw = typename V::Raw;
  constexpr int NV = E / VEC;
  constexpr int kRows = kThreads / TPR;         // rows a CTA works on at once
  extern __shared__ float sm[];                 // [2][D] sums of the CTA's row groups
  __shared__ float2 red[2 * (kThreads / 32)];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float sg[NV][VEC], sb[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sg[k][e] = sb[k][e] = 0.f;
  const float inv = 1.f / (float)D;
  // The next row is on its way while this one is worked on.
  Raw nx[NV], ng[NV];
  float nmu = 0.f, nr = 0.f;
  auto fetch = [&](int row) {
    if (row >= rows) return;
    const T* x = X + (size_t)row * D;
    const T* dy = dY + (size_t)row * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (c < D) {
        nx[k] = V::ldr(x + c);
        ng[k] = V::ldr(dy + c);
      }
    }
    nmu = __ldg(mean + row);
    nr = __ldg(rstd + row);
  };
  int row = blockIdx.x * kRows + sub;
  fetch(row);
  for (int use = 0; row < rows; row += gridDim.x * kRows, use ^= 1) {
    float xh[NV][VEC], g[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      V::widen(nx[k], xh[k]);
      V::widen(ng[k], g[k]);
    }
    const float mu = nmu, r = nr;
    fetch(row + gridDim.x * kRows);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (c < D) {
        float w[VEC];
        if (gamma) load<T, VEC>(gamma + c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xh[k][e] = (xh[k][e] - mu) * r;
          sg[k][e] = fmaf(g[k][e], xh[k][e], sg[k][e]);
          sb[k][e] += g[k][e];
          if (gamma) g[k][e] *= w[e];
          s1 += g[k][e];
          s2 = fmaf(g[k][e], xh[k][e], s2);
        }
      }
    }
    row_sum2<TPR>(s1, s2, red, sub, use);
    s1 *= inv;
    s2 *= inv;
    T* dx = dX + (size_t)row * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (c < D) {
        float u[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[e] = r * (g[k][e] - s1 - xh[k][e] * s2);
        V::st(dx + c, u);
      }
    }
  }
  if (!part) return;
  float* pg = part + (size_t)blockIdx.x * 2 * D;
  if (kRows > 1) {
    // The CTA's row groups one after another.
    for (int w = 0; w < kRows; ++w) {
      if (sub == w) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = (k * TPR + t) * VEC;
          if (c < D) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              sm[c + e] = (w ? sm[c + e] : 0.f) + sg[k][e];
              sm[D + c + e] = (w ? sm[D + c + e] : 0.f) + sb[k][e];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * D; c += kThreads) pg[c] = sm[c];
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (c < D) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          pg[c + e] = sg[k][e];
          pg[D + c + e] = sb[k][e];
        }
      }
    }
  }
}

// dgamma and dbeta (either may be null) from the partial rows: a CTA takes 32
// of the 2·D columns, its 32 warps every 32nd partial row each.
constexpr int kRedWarps = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kRedWarps)
ln_reduce_kernel(const float* part, int nparts, T* __restrict__ dgamma, T* __restrict__ dbeta,
                 int D) {
  __shared__ float s[kRedWarps][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  pdl_wait();
  float v = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int i = w; i < nparts; i += kRedWarps) v += __ldcg(part + (size_t)i * 2 * D + c);
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < 2 * D) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kRedWarps; ++i) v += s[i][lane];
    if (c < D) {
      if (dgamma) st_elem(dgamma + c, v);
    } else {
      if (dbeta) st_elem(dbeta + c - D, v);
    }
  }
}

template <typename T, int VEC, int TPR, int E>
cudaError_t fwd(const NormArgs& a, cudaStream_t st) {
  const int per = kThreads / TPR;
  ln_fwd_kernel<T, VEC, TPR, E><<<(a.rows + per - 1) / per, kThreads, 0, st>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.gamma), static_cast<const T*>(a.beta),
      static_cast<T*>(a.y), a.mean, a.rstd, a.rows, a.D, a.eps);
  return cudaGetLastError();
}

template <typename T, int VEC, int TPR, int E>
cudaError_t bwd(const NormArgs& a, cudaStream_t st) {
  const int per = kThreads / TPR;
  const int need = (a.rows + per - 1) / per;
  const int most = a.max_parts / 4 * bwd_per_sm<T, VEC, E>();
  const int grid = need < most ? need : most;
  const bool weights = a.dgamma || a.dbeta;
  const size_t smem = per > 1 && weights ? (size_t)2 * a.D * sizeof(float) : 0;
  ln_bwd_kernel<T, VEC, TPR, E><<<grid, kThreads, smem, st>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.gamma), a.mean, a.rstd,
      static_cast<const T*>(a.dy), static_cast<T*>(a.dx), weights ? a.part : nullptr, a.rows, a.D);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !weights) return e;
  return launch_dependent(ln_reduce_kernel<T>, dim3((2 * a.D + 31) / 32), dim3(32 * kRedWarps), 0,
                          st, (const float*)a.part, grid, static_cast<T*>(a.dgamma),
                          static_cast<T*>(a.dbeta), a.D);
}

// Threads a row and elements a thread.  Forward: a warp while its lanes hold
// the row in at most 32 registers each (by eighths), else the CTA.  Backward:
// as many threads as leave 8 elements each (up to the CTA): it holds four
// values an element (x̂, dy and the two column sums), and rows in flight are
// what it needs (16384 x 768 bf16: 39.6 us with a warp a row, 163 registers
// and 8 warps an SM, against 16.7 with 128 threads a row).
template <typename T, int VEC>
cudaError_t pick(const NormArgs& a, bool backward, cudaStream_t st) {
  const int D = a.D;
  if (backward) {
    if (D <= 32 * 8) return bwd<T, VEC, 32, 8>(a, st);
    if (D <= 64 * 8) return bwd<T, VEC, 64, 8>(a, st);
    if (D <= 128 * 8) return bwd<T, VEC, 128, 8>(a, st);
    if (D <= 256 * 8) return bwd<T, VEC, 256, 8>(a, st);
    if (D <= 256 * 16) return bwd<T, VEC, 256, 16>(a, st);
    return bwd<T, VEC, 256, 32>(a, st);
  }
  if (D <= 32 * 8) return fwd<T, VEC, 32, 8>(a, st);
  if (D <= 32 * 16) return fwd<T, VEC, 32, 16>(a, st);
  if (D <= 32 * 24) return fwd<T, VEC, 32, 24>(a, st);
  if (D <= 32 * 32) return fwd<T, VEC, 32, 32>(a, st);
  if (D <= 256 * 8) return fwd<T, VEC, 256, 8>(a, st);
  if (D <= 256 * 16) return fwd<T, VEC, 256, 16>(a, st);
  return fwd<T, VEC, 256, 32>(a, st);
}

template <typename T, int FULL>
cudaError_t by_width(const NormArgs& a, bool backward, cudaStream_t st) {
  // The widest vector that divides the rows keeps every row start aligned.
  if (a.D % FULL == 0) return pick<T, FULL>(a, backward, st);
  if (a.D % 2 == 0) return pick<T, 2>(a, backward, st);
  return pick<T, 1>(a, backward, st);
}

}  // namespace

int layernorm_parts(int sms) { return 4 * sms; }

cudaError_t launch_layernorm(const NormArgs& a, int dtype, bool backward, cudaStream_t st) {
  return dtype == CAT_BF16 ? by_width<__nv_bfloat16, 8>(a, backward, st)
                           : by_width<float, 4>(a, backward, st);
}

}  // namespace cat
