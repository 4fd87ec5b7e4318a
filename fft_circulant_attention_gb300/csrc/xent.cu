// Softmax cross entropy over a vocabulary, from hidden states X [T, D] and the
// output weights W [V, D]:
//   l_iv = x_i·w_v,  lse_i = log Σ_v exp(l_iv),  loss_i = lse_i - l_{i,t_i};
//   d_iv = g_i·(exp(l_iv - lse_i) - [v = t_i]),  dX = d·W,  dW = dᵀ·X.
// The logits are never kept: the forward keeps the maximum and the sum of
// exponentials of each row, the backward makes them again, a piece of the
// vocabulary at a time.  Tokens without a target (a negative one) take no part:
// the others' rows are worked on as one dense list.
#include "cat_internal.h"
#include "elem.cuh"
#include "ids.cuh"
#include "../../include/cat.h"

namespace cat {

namespace {

constexpr int kPrep = 1024;
constexpr float kLog2e = 1.4426950408889634f;

// The list of the tokens that have a target (rows, tgt; count: how many), with
// their statistics for the backward (stat: lse·log2(e) and the upstream
// gradient).  A CTA takes kPrep tokens and counts those before them itself.
// loss, lse: forward, zero for the tokens without a target.
__global__ void __launch_bounds__(kPrep)
xent_prepare_kernel(Ids targets, int tokens, int V, int* __restrict__ rows, int* __restrict__ tgt,
                    int* __restrict__ count, float* loss, float* lse_out, const float* lse,
                    const float* dloss, int dloss_each, float2* __restrict__ stat,
                    unsigned int* status) {
  __shared__ int red[kPrep / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * kPrep, t = t0 + threadIdx.x;
  int before = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < t0; i += kPrep) before += id_at(targets, i, V) >= 0;
  const int id = t < tokens ? id_at(targets, t, V) : -1;
  if (id == -2) report(status, 0x801);
  const unsigned held = __ballot_sync(0xffffffffu, id >= 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (lane == 0) red[warp] = before;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kPrep / 32; ++w) base += red[w];
  __syncthreads();
  if (lane == 0) red[warp] = __popc(held);
  __syncthreads();
  int mine = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPrep / 32; ++w) {
    if (w < warp) mine += red[w];
    all += red[w];
  }
  const int pos = base + mine + __popc(held & ((1u << lane) - 1));
  if (id >= 0) {
    rows[pos] = t;
    tgt[pos] = id;
    if (stat) stat[pos] = make_float2(__ldg(lse + t) * kLog2e, __ldg(dloss + (dloss_each ? t : 0)));
  } else if (t < tokens && loss) {
    loss[t] = 0.f;
    lse_out[t] = 0.f;
  }
  if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) *count = base + all;
}

constexpr int kTile = 64, kStep = 16, kThreads = 256;

// One 64 x 64 tile of A·Bᵀ: 256 threads, 4 x 4 values each (rows 4·ty .., columns
// 4·tx ..).  A(m, k), B(n, k): elements, zero outside; *_mn: their rows run along
// m (n) in memory.
template <bool A_MN, bool B_MN, typename FA, typename FB>
__device__ __forceinline__ void tile_product(FA A, FB B, int K, float (&c)[4][4],
                                             float (*sa)[kTile + 4], float (*sb)[kTile + 4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
  for (int k0 = 0; k0 < K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      const int m = A_MN ? i % kTile : i / kStep, k = A_MN ? i / kTile : i % kStep;
      sa[k][m] = A(m, k0 + k);
    }
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      const int n = B_MN ? i % kTile : i / kStep, k = B_MN ? i / kTile : i % kStep;
      sb[k][n] = B(n, k0 + k);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sa[k][4 * ty + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = sb[k][4 * tx + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(x[i], y[j], c[i][j]);
    }
    __syncthreads();
  }
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// part[run][pos]: maximum and sum of exponentials of 64·run_tiles logits.
template <typename T>
__global__ void __launch_bounds__(kThreads)
xent_lse_kernel(XentArgs a, int run_tiles) {
  __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
  const T* X = static_cast<const T*>(a.x);
  const T* W = static_cast<const T*>(a.w);
  const int n = __ldg(a.count), m0 = blockIdx.x * kTile;
  if (m0 >= n) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float mx[4], sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mx[i] = -INFINITY;
    sum[i] = 0.f;
  }
  for (int r = 0; r < run_tiles; ++r) {
    const int v0 = (blockIdx.y * run_tiles + r) * kTile;
    if (v0 >= a.V) break;
    float c[4][4];
    tile_product<false, false>(
        [&](int m, int k) {
          return m0 + m < n && k < a.D ? ld_elem(X + (size_t)a.rows[m0 + m] * a.D + k) : 0.f;
        },
        [&](int v, int k) {
          return v0 + v < a.V && k < a.D ? ld_elem(W + (size_t)(v0 + v) * a.D + k) : 0.f;
        },
        a.D, c, sa, sb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = m0 + 4 * ty + i;
      const int t = pos < n ? a.tgt[pos] : -1;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = v0 + 4 * tx + j;
        if (v >= a.V) c[i][j] = -INFINITY;
        if (v == t) a.hit[pos] = c[i][j];
        top = fmaxf(top, c[i][j]);
      }
      top = fmaxf(mx[i], half_warp_max(top));
      const float sh = top == -INFINITY ? 0.f : top;
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s += exp2f((c[i][j] - sh) * kLog2e);
      sum[i] = sum[i] * exp2f((mx[i] - sh) * kLog2e) + half_warp_sum(s);
      mx[i] = top;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = m0 + 4 * ty + i;
    if (tx == 0 && pos < n) a.part[(size_t)blockIdx.y * a.ld + pos] = make_float2(mx[i], sum[i]);
  }
}

__global__ void __launch_bounds__(256)
xent_finish_kernel(XentArgs a, int nparts) {
  const int pos = blockIdx.x * 256 + threadIdx.x;
  if (pos >= __ldg(a.count)) return;
  float top = -INFINITY, s = 0.f;
  for (int i = 0; i < nparts; ++i) top = fmaxf(top, a.part[(size_t)i * a.ld + pos].x);
  const float sh = top == -INFINITY ? 0.f : top;
  for (int i = 0; i < nparts; ++i) {
    const float2 q = a.part[(size_t)i * a.ld + pos];
    s += q.y * exp2f((q.x - sh) * kLog2e);
  }
  const float z = top + logf(s);
  const int t = a.rows[pos];
  a.lse[t] = z;
  a.loss[t] = z - a.hit[pos];
}

// d of a piece of the vocabulary: fp32 [pos][piece].
template <typename T>
__global__ void __launch_bounds__(kThreads)
xent_dlog_kernel(XentArgs a, float* __restrict__ d, int v0p, int width) {
  __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
  const T* X = static_cast<const T*>(a.x);
  const T* W = static_cast<const T*>(a.w);
  const int n = __ldg(a.count), m0 = blockIdx.x * kTile, v0 = v0p + blockIdx.y * kTile;
  if (m0 >= n) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float c[4][4];
  tile_product<false, false>(
      [&](int m, int k) {
        return m0 + m < n && k < a.D ? ld_elem(X + (size_t)a.rows[m0 + m] * a.D + k) : 0.f;
      },
      [&](int v, int k) {
        return v0 + v < a.V && k < a.D ? ld_elem(W + (size_t)(v0 + v) * a.D + k) : 0.f;
      },
      a.D, c, sa, sb);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = m0 + 4 * ty + i;
    if (pos >= n) continue;
    const int t = a.tgt[pos];
    const float2 st = a.stat[pos];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + 4 * tx + j;
      float p = 0.f;
      if (v < a.V) p = st.y * (exp2f(c[i][j] * kLog2e - st.x) - (v == t ? 1.f : 0.f));
      d[(size_t)pos * width + v - v0p] = p;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
xent_dx_kernel(XentArgs a, const float* __restrict__ d, float* __restrict__ acc, int v0p,
               int width, int first, int last) {
  __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
  const T* W = static_cast<const T*>(a.w);
  const int n = __ldg(a.count), m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
  if (m0 >= n) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float c[4][4];
  tile_product<false, true>(
      [&](int m, int k) { return m0 + m < n ? d[(size_t)(m0 + m) * width + k] : 0.f; },
      [&](int j, int k) {
        return n0 + j < a.D && v0p + k < a.V ? ld_elem(W + (size_t)(v0p + k) * a.D + n0 + j) : 0.f;
      },
      width, c, sa, sb);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = m0 + 4 * ty + i;
    if (pos >= n) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = n0 + 4 * tx + j;
      if (q >= a.D) continue;
      float* to = acc + (size_t)pos * a.D + q;
      const float v = first ? c[i][j] : *to + c[i][j];
      if (last)
        st_elem(static_cast<T*>(a.dx) + (size_t)a.rows[pos] * a.D + q, v);
      else
        *to = v;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
xent_dw_kernel(XentArgs a, const float* __restrict__ d, int v0p, int width) {
  __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
  const T* X = static_cast<const T*>(a.x);
  const int n = __ldg(a.count), m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float c[4][4];
  tile_product<true, true>(
      [&](int m, int k) { return k < n ? d[(size_t)k * width + m0 + m] : 0.f; },
      [&](int j, int k) {
        return n0 + j < a.D && k < n ? ld_elem(X + (size_t)a.rows[k] * a.D + n0 + j) : 0.f;
      },
      n, c, sa, sb);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = v0p + m0 + 4 * ty + i;
    if (v >= a.V) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = n0 + 4 * tx + j;
      if (q < a.D) st_elem(static_cast<T*>(a.dw) + (size_t)v * a.D + q, c[i][j]);
    }
  }
}

template <typename T>
cudaError_t forward(const XentCfg& c, const XentArgs& a, int T_, cudaStream_t st) {
  const int tiles = (c.V + kTile - 1) / kTile, run = 16, runs = (tiles + run - 1) / run;
  xent_lse_kernel<T><<<dim3((T_ + kTile - 1) / kTile, runs), kThreads, 0, st>>>(a, run);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  xent_finish_kernel<<<(T_ + 255) / 256, 256, 0, st>>>(a, runs);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const XentCfg& c, const XentArgs& a, int T_, cudaStream_t st) {
  const int mt = (T_ + kTile - 1) / kTile, nt = (a.D + kTile - 1) / kTile;
  if (a.dx) {
    const cudaError_t e = cudaMemsetAsync(a.dx, 0, (size_t)T_ * a.D * sizeof(T), st);
    if (e != cudaSuccess) return e;
  }
  for (int v0 = 0; v0 < c.V; v0 += c.piece) {
    const int last = v0 + c.piece >= c.V;
    xent_dlog_kernel<T><<<dim3(mt, c.piece / kTile), kThreads, 0, st>>>(a, c.d, v0, c.piece);
    if (a.dx)
      xent_dx_kernel<T><<<dim3(mt, nt), kThreads, 0, st>>>(a, c.d, c.dxacc, v0, c.piece, v0 == 0,
                                                           last);
    if (a.dw)
      xent_dw_kernel<T><<<dim3(c.piece / kTile, nt), kThreads, 0, st>>>(a, c.d, v0, c.piece);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

int xent_piece(int max_tokens, int V) {
  const int most = (V + kTile - 1) / kTile * kTile;
  return most < 4096 ? most : 4096;
}
size_t xent_part_count(int max_tokens, int V) {
  return (size_t)((V + 16 * kTile - 1) / (16 * kTile)) * max_tokens;
}

cudaError_t launch_xent(const cat_plan_s* p, XentArgs a, Ids targets, int tokens, bool back) {
  const XentCfg& c = p->xe;
  cudaStream_t st = p->stream;
  a.V = c.V;
  a.D = p->D;
  a.ld = c.max_tokens;
  a.count = c.count; a.rows = c.rows; a.tgt = c.tgt; a.stat = c.stat; a.hit = c.hit;
  a.part = c.part;
  xent_prepare_kernel<<<(tokens + kPrep - 1) / kPrep, kPrep, 0, st>>>(
      targets, tokens, c.V, c.rows, c.tgt, c.count, back ? nullptr : a.loss,
      back ? nullptr : a.lse, a.lse, a.dloss, a.dloss_each, back ? c.stat : nullptr, p->status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p->dtype == CAT_BF16)
    return back ? backward<__nv_bfloat16>(c, a, tokens, st)
                : forward<__nv_bfloat16>(c, a, tokens, st);
  return back ? backward<float>(c, a, tokens, st) : forward<float>(c, a, tokens, st);
}

}  // namespace cat
