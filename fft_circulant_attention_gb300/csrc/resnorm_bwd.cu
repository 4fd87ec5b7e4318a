// Residual addition with gate, scale and the norms before and after a block,
// backward.  With x̂ = (H - mean_H)·rstd_H, g = dY·gamma, b̂ = (B - mean_B)·rstd_B:
//   dh = dH + rstd_H·(g - mean(g) - x̂·mean(g·x̂)),   dR = dh,
//   u = post ? b̂·pg + pb : B,   dgate = scale·u·dh,   du = scale·gate·dh,
//   dB = post ? rstd_B·(w - mean(w) - b̂·mean(w·b̂)) with w = du·pg : du,
//   dgamma = Σ dY·x̂, dbeta = Σ dY, dpg = Σ du·b̂, dpb = Σ du over the rows, and
//   dgate too where the gate is one of channels.
// H is read as stored, with the statistics of H before its rounding: for bf16 x̂ is
// off by H's half step, which dgamma shows beside its own rounding (16384 rows of
// 768, a few channels large: 0.0020 of the norm instead of 0.0014; the other gradients
// stay at their own rounding).
//
// Bound by memory: H, B, dH, dY (and a gate of rows) are read once, dR, dB (and
// its gradient) written once.  A row is spread over as many threads as leave 8
// elements each, so that a thread's columns of the five sums over the rows stay
// in registers while its persistent CTA goes through its rows; above D = 2048
// the sums are in shared memory, each column its thread's own.  A CTA writes one
// partial row of each sum, a second kernel adds those in a fixed order: no
// atomics, results repeat bit for bit.
//
// Measured: 65536 fp32 rows of 1024 with a gate of rows 338 us (6.35 TB/s, 94 % of the
// copy rate), 16384 bf16 rows of 768 with both norms 41.5 us (3.6 TB/s), the second
// kernel included: five rows of 96 threads an SM at 128 registers, half of the issue
// slots busy; the next row is fetched while one is worked on (58 us without).
#include "resnorm.cuh"

namespace cat {

namespace {

// The sums over the rows, as they lie in a partial row.
enum { S_GAMMA = 0, S_BETA = 1, S_GATE = 2, S_PG = 3, S_PB = 4, kSums = 5 };

constexpr int kPerSm = 2;                // most CTAs of an SM

template <int TPR>
constexpr int block_threads() {
  return TPR > 256 ? TPR : TPR == 96 ? 480 : 256;
}
template <int TPR>
constexpr int per_sm() {
  return TPR > 256 || TPR == 96 ? 1 : 2;
}

// part: [gridDim.x][kSums][D].
// GATE: GATE_ROW, or any other kind (a.gate_kind).  FULL: the threads' vectors are
// the row, none lies behind it.
template <typename T, int VEC, int TPR, int E, int POST, int GATE, bool FULL>
__global__ void __launch_bounds__(block_threads<TPR>(), per_sm<TPR>())
resnorm_bwd_kernel(ResNormArgs a) {
  using V = Vec<T, VEC>;
  using Raw = typename V::Raw;
  constexpr int NV = E / VEC, BT = block_threads<TPR>(), kRows = BT / TPR;
  constexpr bool kShared = TPR > 256;           // sums in shared memory
  extern __shared__ float sm[];                 // [kSums][D]
  __shared__ float2 red[4 * (BT / 32)];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, D = a.D;
  float acc[kSums][kShared ? 1 : NV][VEC];
  if (kShared) {
    for (int c = threadIdx.x; c < kSums * D; c += BT) sm[c] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int s = 0; s < kSums; ++s)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[s][kShared ? 0 : k][e] = 0.f;
  }
  // Sum s, vector k (at column c): plus a·b, plus a.
  auto sum_dot = [&](int s, int k, int c, const float* x, const float* y) {
    float* to = kShared ? sm + s * D + c : acc[s][kShared ? 0 : k];
    v_fma<VEC>(to, x, y, to);
  };
  auto sum_add = [&](int s, int k, int c, const float* x) {
    float* to = kShared ? sm + s * D + c : acc[s][kShared ? 0 : k];
    v_add<VEC>(to, to, x);
  };
  const float inv = 1.f / (float)D, scale = a.scale;
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* pg = static_cast<const T*>(a.pg);
  const T* pb = static_cast<const T*>(a.pb);
  const T* gate = static_cast<const T*>(a.gate);
  // The next row is on its way while this one is worked on.
  Raw nh[NV], ny[NV], nb[NV], nd[NV], ng[NV];
  float4 nst;
  auto fetch = [&](int row) {
    if (row >= a.rows) return;
    const size_t off = (size_t)row * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (FULL || c < D) {
        nh[k] = V::ldr(static_cast<const T*>(a.hin) + off + c);
        ny[k] = V::ldr(static_cast<const T*>(a.dy) + off + c);
        nb[k] = V::ldr(static_cast<const T*>(a.b) + off + c);
        if (a.dh) nd[k] = V::ldr(static_cast<const T*>(a.dh) + off + c);
        if (GATE == GATE_ROW) ng[k] = V::ldr(static_cast<const T*>(a.gate) + off + c);
      }
    }
    const float* st = a.stats + row;
    nst.x = __ldg(st);
    nst.y = __ldg(st + (size_t)a.rows);
    if (POST) {
      nst.z = __ldg(st + 2 * (size_t)a.rows);
      nst.w = __ldg(st + 3 * (size_t)a.rows);
    }
  };
  int use = 0, row = blockIdx.x * kRows + sub;
  fetch(row);
  for (; row < a.rows; row += gridDim.x * kRows, use ^= 2) {
    const size_t off = (size_t)row * D;
    const bool has_dh = a.dh;
    Raw rb[NV], rh[NV], rg[NV];
    float xh[NV][VEC], g[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      V::widen(nh[k], xh[k]);
      V::widen(ny[k], g[k]);
      rb[k] = nb[k];
      rh[k] = nd[k];
      if (GATE == GATE_ROW) rg[k] = ng[k];
    }
    const float mh = nst.x, rsh = nst.y, mb = nst.z, rsb = nst.w;
    fetch(row + gridDim.x * kRows);
    Sum2<VEC> p1, p2;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (FULL || c < D) {
        float w[VEC];
        load_or<T, VEC>(gamma, c, 1.f, w);
        v_add<VEC>(xh[k], xh[k], -mh);
        v_mul<VEC>(xh[k], xh[k], rsh);
        sum_dot(S_GAMMA, k, c, g[k], xh[k]);
        sum_add(S_BETA, k, c, g[k]);
        v_mul<VEC>(g[k], g[k], w);
        p1.add(g[k]);
        p2.dot(g[k], xh[k]);
      }
    }
    float s1 = p1.total(), s2 = p2.total();
    row_sum2<TPR, BT>(s1, s2, red, sub, use);
    s1 *= inv;
    s2 *= inv;
    // g becomes dh, then du·pg; xh becomes b̂.
    Sum2<VEC> q1, q2;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (FULL || c < D) {
        float w[VEC], b[VEC], u[VEC];
        // dh = dH + rstd·((g - s1) - x̂·s2)
        v_add<VEC>(g[k], g[k], -s1);
        v_fma<VEC>(g[k], xh[k], -s2, g[k]);
        if (has_dh) {
          V::widen(rh[k], w);
          v_fma<VEC>(g[k], g[k], rsh, w);
        } else {
          v_mul<VEC>(g[k], g[k], rsh);
        }
        V::st(static_cast<T*>(a.dr) + off + c, g[k]);
        V::widen(rb[k], b);
        if (POST) {
          load_or<T, VEC>(pg, c, 1.f, w);
          load_or<T, VEC>(pb, c, 0.f, u);
          v_add<VEC>(b, b, -mb);
          v_mul<VEC>(b, b, rsb);
          v_fma<VEC>(u, b, w, u);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) u[e] = b[e];
        }
        // g: scale·dh from here on.
        v_mul<VEC>(g[k], g[k], scale);
        if (GATE == GATE_ROW) {
          v_mul<VEC>(u, u, g[k]);
          if (a.dgate) V::st(static_cast<T*>(a.dgate) + off + c, u);
        } else if (a.gate_kind == GATE_CHANNEL) {
          sum_dot(S_GATE, k, c, u, g[k]);
        }
        if (GATE == GATE_ROW) {
          V::widen(rg[k], u);
          v_mul<VEC>(g[k], g[k], u);
        } else if (a.gate_kind == GATE_CHANNEL) {
          load<T, VEC>(gate + c, u);
          v_mul<VEC>(g[k], g[k], u);
        }
        if (POST) {
          sum_dot(S_PG, k, c, g[k], b);
          sum_add(S_PB, k, c, g[k]);
          v_mul<VEC>(g[k], g[k], w);
          q1.add(g[k]);
          q2.dot(g[k], b);
#pragma unroll
          for (int e = 0; e < VEC; ++e) xh[k][e] = b[e];
        }
      }
    }
    float t1 = 0.f, t2 = 0.f;
    if (POST) {
      t1 = q1.total();
      t2 = q2.total();
      row_sum2<TPR, BT>(t1, t2, red, sub, use + 1);
      t1 *= inv;
      t2 *= inv;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (FULL || c < D) {
        if (POST) {
          v_add<VEC>(g[k], g[k], -t1);
          v_fma<VEC>(g[k], xh[k], -t2, g[k]);
          v_mul<VEC>(g[k], g[k], rsb);
        }
        V::st(static_cast<T*>(a.db) + off + c, g[k]);
      }
    }
  }
  float* to = a.part + (size_t)blockIdx.x * kSums * D;
  if (!kShared) {
    // The CTA's row groups one after another.
    for (int w = 0; w < kRows; ++w) {
      if (sub == w) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = (k * TPR + t) * VEC;
          if (c < D) {
#pragma unroll
            for (int s = 0; s < kSums; ++s)
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                float* q = sm + s * D + c + e;
                *q = (w ? *q : 0.f) + acc[s][kShared ? 0 : k][e];
              }
          }
        }
      }
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  for (int c = threadIdx.x; c < kSums * D; c += BT) to[c] = sm[c];
}

// The sums from the partial rows: a CTA takes 32 columns of one sum, its 32
// warps every 32nd partial row each.
constexpr int kRedWarps = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kRedWarps)
resnorm_reduce_kernel(const float* part, int nparts, ResNormArgs a) {
  __shared__ float s[kRedWarps][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, D = a.D;
  const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
  void* const outs[kSums] = {a.dgamma, a.dbeta, a.gate_kind == GATE_CHANNEL ? a.dgate : nullptr,
                             a.dpg, a.dpb};
  T* out = static_cast<T*>(outs[which]);
  pdl_wait();
  if (!out) return;
  float v = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int i = w; i < nparts; i += kRedWarps)
      v += __ldcg(part + ((size_t)i * kSums + which) * D + c);
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < D) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kRedWarps; ++i) v += s[i][lane];
    st_elem(out + c, v);
  }
}

template <typename T, int VEC, int TPR, int E, int POST, int GATE, bool FULL>
cudaError_t go(const ResNormArgs& a, cudaStream_t st, bool setup) {
  constexpr int BT = block_threads<TPR>();
  const int per = BT / TPR, need = (a.rows + per - 1) / per;
  const int most = a.max_parts / kPerSm * per_sm<TPR>();
  const int grid = need < most ? need : most;
  const size_t smem = (size_t)kSums * a.D * sizeof(float);
  if (setup)
    return smem > 40 * 1024 ? allow_max_smem(resnorm_bwd_kernel<T, VEC, TPR, E, POST, GATE, FULL>)
                            : cudaSuccess;
  resnorm_bwd_kernel<T, VEC, TPR, E, POST, GATE, FULL><<<grid, BT, smem, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(resnorm_reduce_kernel<T>, dim3((a.D + 31) / 32, kSums),
                          dim3(32 * kRedWarps), 0, st, (const float*)a.part, grid, a);
}
template <typename T, int VEC, int TPR, int E, int POST, int GATE>
cudaError_t bwd(const ResNormArgs& a, cudaStream_t st, bool setup) {
  // (bf16 is 4 % slower so, 16384 rows of 768.)
  constexpr bool kFull = VEC > 1 && sizeof(T) == 4;
  if (kFull && a.D == TPR * E) return go<T, VEC, TPR, E, POST, GATE, kFull>(a, st, setup);
  return go<T, VEC, TPR, E, POST, GATE, false>(a, st, setup);
}

template <typename T, int VEC, int POST, int GATE>
cudaError_t pick(const ResNormArgs& a, cudaStream_t st, bool setup) {
  const int D = a.D;
  if (D <= 32 * 8) return bwd<T, VEC, 32, 8, POST, GATE>(a, st, setup);
  if (D <= 64 * 8) return bwd<T, VEC, 64, 8, POST, GATE>(a, st, setup);
  if (VEC > 1 && D <= 96 * 8) return bwd<T, VEC, 96, 8, POST, GATE>(a, st, setup);
  if (D <= 128 * 8) return bwd<T, VEC, 128, 8, POST, GATE>(a, st, setup);
  if (D <= 256 * 8) return bwd<T, VEC, 256, 8, POST, GATE>(a, st, setup);
  if (D <= 512 * 8) return bwd<T, VEC, 512, 8, POST, GATE>(a, st, setup);
  return bwd<T, VEC, 512, 16, POST, GATE>(a, st, setup);
}

template <typename T, int VEC>
cudaError_t by_post(const ResNormArgs& a, cudaStream_t st, bool setup) {
  if (a.gate_kind == GATE_ROW)
    return a.post ? pick<T, VEC, 1, GATE_ROW>(a, st, setup)
                  : pick<T, VEC, 0, GATE_ROW>(a, st, setup);
  return a.post ? pick<T, VEC, 1, GATE_NONE>(a, st, setup)
                : pick<T, VEC, 0, GATE_NONE>(a, st, setup);
}

}  // namespace

int resnorm_parts(int sms) { return kPerSm * sms; }
size_t resnorm_part_count(int sms, int D) { return (size_t)resnorm_parts(sms) * kSums * D; }

// One call's launches; setup: only raises its kernel's shared-memory limit.
static cudaError_t dispatch(const ResNormArgs& a, int dtype, cudaStream_t st, bool setup) {
  // Full vectors where they divide the rows (every row start aligned).
  if (dtype == CAT_BF16)
    return a.D % 8 == 0 ? by_post<__nv_bfloat16, 8>(a, st, setup)
                        : by_post<__nv_bfloat16, 1>(a, st, setup);
  return a.D % 4 == 0 ? by_post<float, 4>(a, st, setup) : by_post<float, 1>(a, st, setup);
}

cudaError_t launch_resnorm_backward(const ResNormArgs& a, int dtype, cudaStream_t st) {
  return dispatch(a, dtype, st, false);
}

cudaError_t setup_resnorm(int D, int dtype, int post) {
  ResNormArgs a = {};
  a.D = D;
  a.post = post;
  for (a.gate_kind = GATE_NONE; a.gate_kind <= GATE_ROW; a.gate_kind += GATE_ROW) {
    const cudaError_t e = dispatch(a, dtype, nullptr, true);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace cat
