// Softmax attention over packed sequences on the FP32 pipe: what the
// tensor-core kernels do not take.  That is bf16 whose rows or heads do not
// all start on 16-byte boundaries (any head width up to 128), and the
// backward of fp32 heads wider than 64.  Also the choice between the kernels.
//
// Per sequence and query head h (key head g = h / (Hq/Hkv)), with rows i, j:
//   s_ij = scale·q_i·k_j (j <= i if causal), lse_i = log Σ_j exp s_ij,
//   p_ij = exp(s_ij - lse_i), o_i = Σ_j p_ij v_j;
//   delta_i = dO_i·o_i, ds_ij = p_ij (dO_i·v_j - delta_i),
//   dq_i = scale Σ_j ds_ij k_j, dk_j = scale Σ_i ds_ij q_i, dv_j = Σ_i p_ij dO_i,
// dk and dv summed over the query heads of a key head.
//
// 64 x 64 blocks of scores, 256 threads.  Operands sit in shared memory as
// fp32 rows of DP + 4 floats (DP: the head width rounded up); a thread's 4 x 4
// scores take rows ty + 16·i and tx + 16·j, so that the 8 lanes of a
// quarter-warp read 8 distinct bank groups.  The softmax runs in one pass
// over the keys with a running maximum and sum.  The probabilities go back
// through shared memory as the second product's operand, read 4 rows at a
// time as a broadcast.  The backward is two kernels, one over key blocks
// (dk, dv) and one over query blocks (dq): 7 products instead of 5, no
// atomics, results that repeat bit for bit.
//
// A masked pair contributes nothing even where the masked row holds an
// infinity or NaN: blocks that the mask cuts take the guarded product loops.
//
// Bound by shared-memory reads beside the FP32 pipe.  Measured, 12 heads of 64,
// 16 documents of 57 .. 1024 tokens: forward 444 us and backward 1413 us in bf16
// at odd addresses, where the tensor-core kernels take 25 and 84 us; backward of
// fp32 heads of 128 3139 us (of 64, on the tensor cores, 425).
#include "attn.cuh"
#include "../../include/cat.h"
#include "cat_internal.h"

namespace cat {

namespace {

constexpr int kBlk = 64;           // query rows and keys of a block
constexpr int kThr = 256;
constexpr int kPs = kBlk + 4;      // row stride of the probability block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* v);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float* v) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
}

// Rows 0 .. kBlk - 1 of a [.., dh] operand into dst [kBlk][DP + 4], zeros
// from row `rows` and column dh on.
template <typename T, int DP>
__device__ __forceinline__ void stage(float* dst, const T* src, long long ld, int rows, int dh,
                                      int vec) {
  constexpr int kLd = DP + 4;
  for (int i = threadIdx.x; i < kBlk * (DP / 4); i += kThr) {
    const int r = i / (DP / 4), c = 4 * (i % (DP / 4));
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < rows) {
      const T* p = src + (long long)r * ld + c;
      if (vec) {
        if (c < dh) load4(p, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < dh) v[e] = ld_elem(p + e);
      }
    }
    *reinterpret_cast<float4*>(dst + r * kLd + c) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// acc[i][j] = Σ_d A[ty + 16 i][d] · B[tx + 16 j][d].
template <int DP>
__device__ __forceinline__ void scores(const float* A, const float* B, int ty, int tx,
                                       float acc[4][4]) {
  constexpr int kLd = DP + 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
  for (int d = 0; d < DP; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * kLd + d);
      y[i] = *reinterpret_cast<const float4*>(B + (tx + 16 * i) * kLd + d);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
      }
  }
}

// Columns of an accumulator that one thread owns: 4·G of DP, G groups of 4
// columns 64 apart (one group of 2 columns at DP = 32).
template <int DP>
struct Cols {
  static constexpr int kW = DP >= 64 ? 4 : 2;
  static constexpr int kG = DP >= 64 ? DP / 64 : 1;
};

// acc[i][g][c] += Σ_n P[n][4 ty + i] · B[n][col].  kGuard: pair (4 ty + i, n)
// counts only if n >= lo[i] and n <= hi[i].
template <int DP, bool kGuard>
__device__ __forceinline__ void product(const float* P, const float* B, int ty, int tx,
                                        float (&acc)[4][Cols<DP>::kG][Cols<DP>::kW],
                                        const int* lo, const int* hi) {
  constexpr int kLd = DP + 4, kG = Cols<DP>::kG, kW = Cols<DP>::kW;
#pragma unroll 4
  for (int n = 0; n < kBlk; ++n) {
    const float4 p4 = *reinterpret_cast<const float4*>(P + n * kPs + 4 * ty);
    const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      float b[kW];
      if constexpr (kW == 4) {
        const float4 x = *reinterpret_cast<const float4*>(B + n * kLd + 64 * g + 4 * tx);
        b[0] = x.x; b[1] = x.y; b[2] = x.z; b[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(B + n * kLd + 2 * tx);
        b[0] = x.x; b[1] = x.y;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kGuard && (n < lo[i] || n > hi[i])) continue;
#pragma unroll
        for (int c = 0; c < kW; ++c) acc[i][g][c] = fmaf(p[i], b[c], acc[i][g][c]);
      }
    }
  }
}

// f · accumulator rows 4 ty + i (< rows) to a [.., dh] output.
template <typename T, int DP>
__device__ __forceinline__ void store_rows(T* dst, long long ld, int rows, int dh, int vec, int ty,
                                           int tx,
                                           const float (&acc)[4][Cols<DP>::kG][Cols<DP>::kW],
                                           const float* f) {
  constexpr int kG = Cols<DP>::kG, kW = Cols<DP>::kW;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= rows) continue;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int c0 = 64 * g + kW * tx;
      T* p = dst + (long long)r * ld + c0;
#pragma unroll
      for (int c = 0; c < kW; c += 2) {
        const float a = acc[i][g][c] * f[i], b = acc[i][g][c + 1] * f[i];
        if (vec) {
          if (c0 + c < dh) st_pair(p + c, make_float2(a, b));
        } else {
          if (c0 + c < dh) st_elem(p + c, a);
          if (c0 + c + 1 < dh) st_elem(p + c + 1, b);
        }
      }
    }
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThr)
attn_fwd_kernel(const AttnArgs a) {
  constexpr int kLd = DP + 4, kG = Cols<DP>::kG, kW = Cols<DP>::kW;
  extern __shared__ float sm[];
  float* Q = sm;
  float* K = Q + kBlk * kLd;
  float* V = K + kBlk * kLd;
  float* P = V + kBlk * kLd;        // [key][query row]
  float* R = P + kBlk * kPs;        // per query row: rescale factor, then 1 / sum
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int h = blockIdx.x % a.Hq;
  const int slot = (int)(gridDim.x / a.Hq) - 1 - (int)(blockIdx.x / a.Hq);
  if (blockIdx.x == 0) attn_check_sequences(a, threadIdx.x, kThr);
  AttnBlock b;
  if (!attn_find_block(a, slot, 6, &b)) return;
  const int g = h / (a.Hq / a.Hkv);
  const T* q = static_cast<const T*>(a.q) + (b.start + b.row0) * a.ldq + (long long)h * a.dh;
  const T* k = static_cast<const T*>(a.k) + b.start * a.ldk + (long long)g * a.dh;
  const T* v = static_cast<const T*>(a.v) + b.start * a.ldv + (long long)g * a.dh;
  const int rows = min(kBlk, b.len - b.row0);
  stage<T, DP>(Q, q, a.ldq, rows, a.dh, a.vec);
  const float sc = a.scale * kLog2e;       // scores in units of log 2
  float m[4], l[4], acc[4][kG][kW];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int gg = 0; gg < kG; ++gg)
#pragma unroll
      for (int c = 0; c < kW; ++c) acc[i][gg][c] = 0.f;
  }
  const int keys = a.causal ? min(b.len, b.row0 + kBlk) : b.len;
  for (int j0 = 0; j0 < keys; j0 += kBlk) {
    const int nk = min(kBlk, b.len - j0);
    __syncthreads();
    stage<T, DP>(K, k + j0 * a.ldk, a.ldk, nk, a.dh, a.vec);
    stage<T, DP>(V, v + j0 * a.ldv, a.ldv, nk, a.dh, a.vec);
    __syncthreads();
    float s[4][4];
    scores<DP>(Q, K, ty, tx, s);
    const bool cut = nk < kBlk || (a.causal && j0 + kBlk > b.row0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = b.row0 + ty + 16 * i;
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j;
        s[i][j] *= sc;
        if (cut && (c >= nk || (a.causal && j0 + c > r))) s[i][j] = -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float base = mx == -INFINITY ? 0.f : mx;
      const float f = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - base);
        sum += s[i][j];
        P[(tx + 16 * j) * kPs + ty + 16 * i] = s[i][j];
      }
      l[i] = l[i] * f + sum;
      m[i] = mx;
      if (tx == 0) R[ty + 16 * i] = f;
    }
    __syncthreads();
    int lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = R[4 * ty + i];
#pragma unroll
      for (int gg = 0; gg < kG; ++gg)
#pragma unroll
        for (int c = 0; c < kW; ++c) acc[i][gg][c] *= f;
      lo[i] = 0;
      hi[i] = a.causal ? min(nk - 1, b.row0 + 4 * ty + i - j0) : nk - 1;
    }
    if (cut)
      product<DP, true>(P, V, ty, tx, acc, lo, hi);
    else
      product<DP, false>(P, V, ty, tx, acc, lo, hi);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t = l[i];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (tx == 0) {
      const int r = ty + 16 * i;
      R[r] = 1.f / t;
      if (r < rows)
        a.lse[(long long)h * a.T + b.start + b.row0 + r] = (m[i] + log2f(t)) * kLn2;
    }
  }
  __syncthreads();
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = R[4 * ty + i];
  const long long ldo = (long long)a.Hq * a.dh;
  store_rows<T, DP>(static_cast<T*>(a.out) + (b.start + b.row0) * ldo + (long long)h * a.dh, ldo,
                    rows, a.dh, a.vec, ty, tx, acc, f);
}

// delta[h][t] = Σ_c dO[t, h, c] · O[t, h, c], one warp a (t, h).
template <typename T>
__global__ void __launch_bounds__(kThr)
attn_delta_kernel(const AttnArgs a) {
  const long long i = (long long)blockIdx.x * (kThr / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) attn_check_sequences(a, threadIdx.x, kThr);
  if (i >= (long long)a.T * a.Hq) return;
  const T* o = static_cast<const T*>(a.o) + i * a.dh;
  const T* d = static_cast<const T*>(a.dO) + i * a.dh;
  float s = 0.f;
  for (int c = lane; c < a.dh; c += 32) s = fmaf(ld_elem(o + c), ld_elem(d + c), s);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
  if (lane == 0) a.delta[(i % a.Hq) * a.T + i / a.Hq] = s;
}

// dq of one query block: s and dO·v^T per key block, dq += ds·k.
template <typename T, int DP>
__global__ void __launch_bounds__(kThr)
attn_dq_kernel(const AttnArgs a) {
  constexpr int kLd = DP + 4, kG = Cols<DP>::kG, kW = Cols<DP>::kW;
  extern __shared__ float sm[];
  float* Q = sm;
  float* G = Q + kBlk * kLd;
  float* K = G + kBlk * kLd;
  float* V = K + kBlk * kLd;
  float* P = V + kBlk * kLd;        // ds as [key][query row]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int h = blockIdx.x % a.Hq;
  const int slot = (int)(gridDim.x / a.Hq) - 1 - (int)(blockIdx.x / a.Hq);
  AttnBlock b;
  if (!attn_find_block(a, slot, 6, &b)) return;
  const int g = h / (a.Hq / a.Hkv);
  const long long ldo = (long long)a.Hq * a.dh;
  const long long t0 = b.start + b.row0;
  const int rows = min(kBlk, b.len - b.row0);
  stage<T, DP>(Q, static_cast<const T*>(a.q) + t0 * a.ldq + (long long)h * a.dh, a.ldq, rows, a.dh,
               a.vec);
  stage<T, DP>(G, static_cast<const T*>(a.dO) + t0 * ldo + (long long)h * a.dh, ldo, rows, a.dh,
               a.vec);
  const T* k = static_cast<const T*>(a.k) + b.start * a.ldk + (long long)g * a.dh;
  const T* v = static_cast<const T*>(a.v) + b.start * a.ldv + (long long)g * a.dh;
  const float sc = a.scale * kLog2e;
  float ls[4], de[4], acc[4][kG][kW];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    ls[i] = r < rows ? a.lse[(long long)h * a.T + t0 + r] * kLog2e : 0.f;
    de[i] = r < rows ? a.delta[(long long)h * a.T + t0 + r] : 0.f;
#pragma unroll
    for (int gg = 0; gg < kG; ++gg)
#pragma unroll
      for (int c = 0; c < kW; ++c) acc[i][gg][c] = 0.f;
  }
  const int keys = a.causal ? min(b.len, b.row0 + kBlk) : b.len;
  for (int j0 = 0; j0 < keys; j0 += kBlk) {
    const int nk = min(kBlk, b.len - j0);
    __syncthreads();
    stage<T, DP>(K, k + j0 * a.ldk, a.ldk, nk, a.dh, a.vec);
    stage<T, DP>(V, v + j0 * a.ldv, a.ldv, nk, a.dh, a.vec);
    __syncthreads();
    float s[4][4], dp[4][4];
    scores<DP>(Q, K, ty, tx, s);
    scores<DP>(G, V, ty, tx, dp);
    const bool cut = nk < kBlk || (a.causal && j0 + kBlk > b.row0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j;
        float ds = exp2f(fmaf(s[i][j], sc, -ls[i])) * (dp[i][j] - de[i]);
        if (cut && (c >= nk || (a.causal && j0 + c > b.row0 + ty + 16 * i))) ds = 0.f;
        P[c * kPs + ty + 16 * i] = ds;
      }
    __syncthreads();
    int lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = 0;
      hi[i] = a.causal ? min(nk - 1, b.row0 + 4 * ty + i - j0) : nk - 1;
    }
    if (cut)
      product<DP, true>(P, K, ty, tx, acc, lo, hi);
    else
      product<DP, false>(P, K, ty, tx, acc, lo, hi);
  }
  const float f[4] = {a.scale, a.scale, a.scale, a.scale};
  store_rows<T, DP>(static_cast<T*>(a.dq) + t0 * a.lddq + (long long)h * a.dh, a.lddq, rows, a.dh,
                    a.vec, ty, tx, acc, f);
}

// dk and dv of one key block: over the query heads of the key head and the
// query blocks that see it.  Scores are held transposed, s[key][query].
template <typename T, int DP>
__global__ void __launch_bounds__(kThr)
attn_dkv_kernel(const AttnArgs a) {
  constexpr int kLd = DP + 4, kG = Cols<DP>::kG, kW = Cols<DP>::kW;
  extern __shared__ float sm[];
  float* Q = sm;
  float* G = Q + kBlk * kLd;
  float* K = G + kBlk * kLd;
  float* V = K + kBlk * kLd;
  float* P = V + kBlk * kLd;        // p, then ds, as [query row][key]
  float* D = P + kBlk * kPs;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int g = blockIdx.x % a.Hkv;
  const int slot = (int)(blockIdx.x / a.Hkv);
  AttnBlock b;
  if (!attn_find_block(a, slot, 6, &b)) return;
  const long long ldo = (long long)a.Hq * a.dh;
  const long long t0 = b.start + b.row0;
  const int keys = min(kBlk, b.len - b.row0);
  stage<T, DP>(K, static_cast<const T*>(a.k) + t0 * a.ldk + (long long)g * a.dh, a.ldk, keys, a.dh,
               a.vec);
  stage<T, DP>(V, static_cast<const T*>(a.v) + t0 * a.ldv + (long long)g * a.dh, a.ldv, keys, a.dh,
               a.vec);
  const float sc = a.scale * kLog2e;
  float ak[4][kG][kW], av[4][kG][kW];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int gg = 0; gg < kG; ++gg)
#pragma unroll
      for (int c = 0; c < kW; ++c) ak[i][gg][c] = av[i][gg][c] = 0.f;
  const int rep = a.Hq / a.Hkv;
  for (int h = g * rep; h < (g + 1) * rep; ++h) {
    const T* q = static_cast<const T*>(a.q) + b.start * a.ldq + (long long)h * a.dh;
    const T* go = static_cast<const T*>(a.dO) + b.start * ldo + (long long)h * a.dh;
    const float* lse = a.lse + (long long)h * a.T + b.start;
    const float* del = a.delta + (long long)h * a.T + b.start;
    for (int i0 = a.causal ? b.row0 : 0; i0 < b.len; i0 += kBlk) {
      const int nq = min(kBlk, b.len - i0);
      __syncthreads();
      stage<T, DP>(Q, q + i0 * a.ldq, a.ldq, nq, a.dh, a.vec);
      stage<T, DP>(G, go + i0 * ldo, ldo, nq, a.dh, a.vec);
      __syncthreads();
      float s[4][4], dp[4][4];
      scores<DP>(K, Q, ty, tx, s);
      scores<DP>(V, G, ty, tx, dp);
      // The block is cut where queries or keys run out or the diagonal passes.
      const bool cut = nq < kBlk || keys < kBlk || (a.causal && i0 < b.row0 + kBlk);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j;
        const float ls = c < nq ? lse[i0 + c] * kLog2e : 0.f;
        const float de = c < nq ? del[i0 + c] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = ty + 16 * i;
          float p = exp2f(fmaf(s[i][j], sc, -ls));
          float ds = p * (dp[i][j] - de);
          if (cut && (c >= nq || r >= keys || (a.causal && b.row0 + r > i0 + c))) p = ds = 0.f;
          P[c * kPs + r] = p;
          D[c * kPs + r] = ds;
        }
      }
      __syncthreads();
      int lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = a.causal ? max(0, b.row0 + 4 * ty + i - i0) : 0;
        hi[i] = nq - 1;
      }
      if (cut) {
        product<DP, true>(P, G, ty, tx, av, lo, hi);
        product<DP, true>(D, Q, ty, tx, ak, lo, hi);
      } else {
        product<DP, false>(P, G, ty, tx, av, lo, hi);
        product<DP, false>(D, Q, ty, tx, ak, lo, hi);
      }
    }
  }
  const float one[4] = {1.f, 1.f, 1.f, 1.f};
  const float f[4] = {a.scale, a.scale, a.scale, a.scale};
  store_rows<T, DP>(static_cast<T*>(a.dv) + t0 * a.lddv + (long long)g * a.dh, a.lddv, keys, a.dh,
                    a.vec, ty, tx, av, one);
  store_rows<T, DP>(static_cast<T*>(a.dk) + t0 * a.lddk + (long long)g * a.dh, a.lddk, keys, a.dh,
                    a.vec, ty, tx, ak, f);
}

constexpr size_t fwd_smem(int DP) {
  return ((size_t)3 * kBlk * (DP + 4) + kBlk * kPs + kBlk) * sizeof(float);
}
constexpr size_t dq_smem(int DP) {
  return ((size_t)4 * kBlk * (DP + 4) + kBlk * kPs) * sizeof(float);
}
constexpr size_t dkv_smem(int DP) {
  return ((size_t)4 * kBlk * (DP + 4) + 2 * kBlk * kPs) * sizeof(float);
}

template <int DP>
cudaError_t setup_one() {
  cudaError_t e = allow_max_smem(attn_fwd_kernel<__nv_bfloat16, DP>);
  if (e == cudaSuccess) e = allow_max_smem(attn_dq_kernel<__nv_bfloat16, DP>);
  if (e == cudaSuccess) e = allow_max_smem(attn_dkv_kernel<__nv_bfloat16, DP>);
  return e;
}

template <int DP>
cudaError_t fwd(const AttnArgs& a, cudaStream_t st) {
  attn_fwd_kernel<__nv_bfloat16, DP>
      <<<(unsigned)(attn_slots(a.T, a.S, 6) * a.Hq), kThr, fwd_smem(DP), st>>>(a);
  return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t bwd(const AttnArgs& a, cudaStream_t st) {
  const long long slots = attn_slots(a.T, a.S, 6);
  attn_dkv_kernel<T, DP><<<(unsigned)(slots * a.Hkv), kThr, dkv_smem(DP), st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attn_dq_kernel<T, DP><<<(unsigned)(slots * a.Hq), kThr, dq_smem(DP), st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t setup_attn() {
  cudaError_t e = setup_one<32>();
  if (e == cudaSuccess) e = setup_one<64>();
  if (e == cudaSuccess) e = setup_one<128>();
  if (e == cudaSuccess) e = allow_max_smem(attn_dq_kernel<float, 128>);
  if (e == cudaSuccess) e = allow_max_smem(attn_dkv_kernel<float, 128>);
  return e;
}

cudaError_t launch_attn_forward(const cat_plan_s* p, const AttnArgs& a) {
  if (p->dtype == CAT_F32) return launch_attn_tc32_forward(a, p->stream);
  if (a.tc) return launch_attn_tc_forward(a, p->stream);
  return a.dh <= 32   ? fwd<32>(a, p->stream)
         : a.dh <= 64 ? fwd<64>(a, p->stream)
                      : fwd<128>(a, p->stream);
}

cudaError_t launch_attn_backward(const cat_plan_s* p, const AttnArgs& a) {
  if (a.tc) return launch_attn_tc_backward(a, p->stream);
  const long long rows = (long long)a.T * a.Hq;
  const unsigned grid = (unsigned)((rows + kThr / 32 - 1) / (kThr / 32));
  if (p->dtype == CAT_BF16)
    attn_delta_kernel<__nv_bfloat16><<<grid, kThr, 0, p->stream>>>(a);
  else
    attn_delta_kernel<float><<<grid, kThr, 0, p->stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p->dtype == CAT_F32)
    return a.dh <= 64 ? launch_attn_tc32_backward(a, p->stream) : bwd<float, 128>(a, p->stream);
  return a.dh <= 32   ? bwd<__nv_bfloat16, 32>(a, p->stream)
         : a.dh <= 64 ? bwd<__nv_bfloat16, 64>(a, p->stream)
                      : bwd<__nv_bfloat16, 128>(a, p->stream);
}

}  // namespace cat
