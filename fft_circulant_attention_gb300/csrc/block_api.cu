// C ABI of the operators around a CAT layer (include/cat.h): softmax
// attention over packed sequences, layer norm, gradient norm and clipping.
// Plans are cat_plan_t; the kernels are in attn*.cu, layernorm.cu and
// gradclip.cu.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <new>
#include <vector>

#include "../../include/cat.h"
#include "attn.cuh"
#include "cat_internal.h"
#include "op_api.cuh"

namespace {

using cat::DeviceGuard;
using cat::Span2;
using cat::alloc;
using cat::alloc_status;
using cat::aliased;
using cat::elem_size;
using cat::fail;
using cat::flat;
using cat::new_plan;
using cat::overlap;
using cat::status_of;

}  // namespace

namespace cat {

void free_op(cat_plan_s* p) {
  cudaFree(p->at.delta);
  cudaFree(p->at.stats);
  cudaFree(p->at.link);
  cudaFree(p->ln.part);
  cudaFree(p->cl.chunks);
  cudaFree(p->cl.part);
  cudaFree(p->em.tok);
  cudaFree(p->em.key);
  cudaFree(p->em.off);
  cudaFree(p->em.first);
  cudaFree(p->em.order);
  cudaFree(p->em.sid);
  cudaFree(p->em.part);
  cudaFree(p->rn.part);
  cudaFree(p->xe.count);
  cudaFree(p->xe.rows);
  cudaFree(p->xe.tgt);
  cudaFree(p->xe.hit);
  cudaFree(p->xe.part);
  cudaFree(p->xe.stat);
  cudaFree(p->xe.inv);
  cudaFree(p->xe.xp);
  cudaFree(p->xe.wp);
  cudaFree(p->xe.d);
  cudaFree(p->xe.dxacc);
  delete[] p->cl.first_chunk;
  delete[] p->cl.sizes;
  delete[] p->cl.dtypes;
}

}  // namespace cat

extern "C" {

int cat_plan_create_attn(cat_plan_t* out, int max_tokens, int max_seqs, int Hq, int Hkv, int dh,
                         int dtype, int causal, float scale, void* stream) {
  if (!out) return CAT_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_tokens < 0 || max_tokens > CAT_ATTN_MAX_TOKENS || max_seqs < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || dh < 1 ||
      dh > CAT_ATTN_MAX_DH || (long long)Hq * dh > (1 << 20))
    return CAT_ERR_INVALID_ARG;
  if (dtype != CAT_F32 && dtype != CAT_BF16) return CAT_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return CAT_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return CAT_ERR_INVALID_ARG;
  // Blocks are counted in int (at most one a 64-row slot and head).
  if (cat::attn_slots(max_tokens, max_seqs, 6) * Hq > INT_MAX ||
      (long long)max_tokens * Hq > INT_MAX)
    return CAT_ERR_INVALID_ARG;
  int st;
  cat_plan_s* p = new_plan(cat::OP_ATTN, dtype, stream, &st);
  if (!p) return st;
  p->at.max_tokens = max_tokens;
  p->at.max_seqs = max_seqs;
  p->at.Hq = Hq;
  p->at.Hkv = Hkv;
  p->at.dh = dh;
  p->at.causal = causal;
  // CAT_ATTN_POLLS: a shorter limit of the fp32 kernels' waits (256 or more).
  p->at.polls = cat::kWaitPolls;
  if (const char* e = std::getenv("CAT_ATTN_POLLS")) {
    const long v = std::atol(e);
    if (v >= 256 && v < (long)cat::kWaitPolls) p->at.polls = (unsigned int)v;
  }
  p->at.scale = scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)dh));
  if (!alloc_status(p) || !alloc(p, &p->at.delta, (size_t)Hq * max_tokens))
    return fail(p, CAT_ERR_ALLOC);
  if (dtype == CAT_BF16 && dh % 8 == 0 &&
      !alloc(p, &p->at.stats, cat::attn_tc_stats_count(max_tokens, max_seqs, Hq)))
    return fail(p, CAT_ERR_ALLOC);
  if (dtype == CAT_F32 &&
      !alloc(p, &p->at.link, (size_t)cat::attn_slots(max_tokens, max_seqs, 7) * Hq))
    return fail(p, CAT_ERR_ALLOC);
  if (cat::setup_attn() != cudaSuccess || cat::setup_attn_tc() != cudaSuccess ||
      cat::setup_attn_tc_bwd() != cudaSuccess || cat::setup_attn_tc32() != cudaSuccess) return fail(p, CAT_ERR_CUDA);
  std::snprintf(p->desc, sizeof(p->desc),
                "op=attn max_tokens=%d max_seqs=%d Hq=%d Hkv=%d dh=%d causal=%d scale=%g "
                "workspace=%zu",
                max_tokens, max_seqs, Hq, Hkv, dh, causal, (double)p->at.scale,
                p->workspace_bytes);
  *out = p;
  return CAT_OK;
}

namespace {

// Checks that both attention calls share; fills the arguments.  *run = false
// for a call with nothing to do.
int attn_prepare(cat_plan_s* p, const void* Q, const void* K, const void* V, const int* cu, int T,
                 int S, long long ldq, long long ldk, long long ldv, cat::AttnArgs* a, bool* run) {
  *run = false;
  if (!p) return CAT_ERR_INVALID_ARG;
  if (p->op != cat::OP_ATTN) return CAT_ERR_PLAN_MISMATCH;
  const cat::AttnCfg& c = p->at;
  if (T < 0 || S < 0) return CAT_ERR_INVALID_ARG;
  if (T > c.max_tokens || S > c.max_seqs) return CAT_ERR_PLAN_MISMATCH;
  const long long wq = (long long)c.Hq * c.dh, wk = (long long)c.Hkv * c.dh;
  if (ldq < wq || ldk < wk || ldv < wk) return CAT_ERR_INVALID_ARG;
  const long long most = LLONG_MAX / 8 / (T > 0 ? T : 1);
  if (ldq > most || ldk > most || ldv > most) return CAT_ERR_INVALID_ARG;
  if (T == 0 || S == 0) return CAT_OK;
  if (!Q || !K || !V || !cu) return CAT_ERR_INVALID_ARG;
  const uintptr_t es1 = elem_size(p->dtype) - 1;
  if ((((uintptr_t)Q | (uintptr_t)K | (uintptr_t)V) & es1) || ((uintptr_t)cu & 3))
    return CAT_ERR_MISALIGNED;
  std::memset(a, 0, sizeof(*a));
  a->q = Q; a->k = K; a->v = V;
  a->cu = cu;
  a->ldq = ldq; a->ldk = ldk; a->ldv = ldv;
  a->T = T; a->S = S;
  a->Hq = c.Hq; a->Hkv = c.Hkv; a->dh = c.dh;
  a->causal = c.causal;
  a->scale = c.scale;
  a->delta = c.delta;
  a->stats = c.stats;
  a->status = p->status;
  a->link = c.link;
  a->polls = c.polls;
  *run = true;
  return CAT_OK;
}

// Whether rows of these operands start on `bytes`-byte boundaries, heads too.
bool rows_aligned(const cat_plan_s* p, std::initializer_list<const void*> ptrs,
                  std::initializer_list<long long> lds, size_t bytes) {
  const size_t es = elem_size(p->dtype);
  if ((size_t)p->at.dh * es % bytes) return false;
  for (const void* q : ptrs)
    if ((uintptr_t)q % bytes) return false;
  for (long long l : lds)
    if ((size_t)l * es % bytes) return false;
  return true;
}

// Whether bf16 rows this far apart fit a tensor map (strides below 2^40 bytes).
bool mappable(std::initializer_list<long long> lds) {
  for (long long l : lds)
    if (l >= (1ll << 39)) return false;
  return true;
}

}  // namespace

int cat_attn_forward(cat_plan_t p, const void* Q, const void* K, const void* V, void* O,
                     float* lse, const int* cu_seqlens, int T, int S, long long ldq, long long ldk,
                     long long ldv) {
  cat::AttnArgs a;
  bool run;
  const int st = attn_prepare(p, Q, K, V, cu_seqlens, T, S, ldq, ldk, ldv, &a, &run);
  if (st != CAT_OK || !run) return st;
  if (!O || !lse) return CAT_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype);
  if (((uintptr_t)O & (es - 1)) || ((uintptr_t)lse & 3)) return CAT_ERR_MISALIGNED;
  const size_t wq = (size_t)p->at.Hq * p->at.dh * es, wk = (size_t)p->at.Hkv * p->at.dh * es;
  const Span2 in[4] = {{Q, (size_t)T, wq, (size_t)ldq * es},
                       {K, (size_t)T, wk, (size_t)ldk * es},
                       {V, (size_t)T, wk, (size_t)ldv * es},
                       flat(cu_seqlens, ((size_t)S + 1) * sizeof(int))};
  const Span2 outs[2] = {flat(O, wq * T), flat(lse, (size_t)p->at.Hq * T * sizeof(float))};
  if (aliased(in, 4, outs, 2)) return CAT_ERR_ALIAS;
  a.out = O;
  a.lse = lse;
  a.vec = rows_aligned(p, {Q, K, V, O}, {ldq, ldk, ldv}, 4 * es);
  a.tc = es == 2 && rows_aligned(p, {Q, K, V, O}, {ldq, ldk, ldv}, 16) &&
         mappable({ldq, ldk, ldv});
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_attn_forward(p, a));
}

int cat_attn_backward(cat_plan_t p, const void* Q, const void* K, const void* V, const void* O,
                      const float* lse, const void* dO, void* dQ, void* dK, void* dV,
                      const int* cu_seqlens, int T, int S, long long ldq, long long ldk,
                      long long ldv, long long lddq, long long lddk, long long lddv) {
  cat::AttnArgs a;
  bool run;
  const int st = attn_prepare(p, Q, K, V, cu_seqlens, T, S, ldq, ldk, ldv, &a, &run);
  if (st != CAT_OK) return st;
  const long long nq = (long long)p->at.Hq * p->at.dh, nk = (long long)p->at.Hkv * p->at.dh;
  const long long most = LLONG_MAX / 8 / (T > 0 ? T : 1);
  if (lddq < nq || lddk < nk || lddv < nk || lddq > most || lddk > most || lddv > most)
    return CAT_ERR_INVALID_ARG;
  if (!run) return CAT_OK;
  if (!O || !lse || !dO || !dQ || !dK || !dV) return CAT_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype);
  if ((((uintptr_t)O | (uintptr_t)dO | (uintptr_t)dQ | (uintptr_t)dK | (uintptr_t)dV) & (es - 1)) ||
      ((uintptr_t)lse & 3))
    return CAT_ERR_MISALIGNED;
  const size_t wq = nq * es, wk = nk * es;
  const Span2 in[7] = {{Q, (size_t)T, wq, (size_t)ldq * es},
                       {K, (size_t)T, wk, (size_t)ldk * es},
                       {V, (size_t)T, wk, (size_t)ldv * es},
                       flat(O, wq * T),
                       flat(dO, wq * T),
                       flat(lse, (size_t)p->at.Hq * T * sizeof(float)),
                       flat(cu_seqlens, ((size_t)S + 1) * sizeof(int))};
  const Span2 outs[3] = {{dQ, (size_t)T, wq, (size_t)lddq * es},
                         {dK, (size_t)T, wk, (size_t)lddk * es},
                         {dV, (size_t)T, wk, (size_t)lddv * es}};
  if (aliased(in, 7, outs, 3)) return CAT_ERR_ALIAS;
  a.o = O;
  a.dO = dO;
  a.lse = const_cast<float*>(lse);
  a.dq = dQ; a.dk = dK; a.dv = dV;
  a.lddq = lddq; a.lddk = lddk; a.lddv = lddv;
  a.vec = rows_aligned(p, {Q, K, V, O, dO, dQ, dK, dV}, {ldq, ldk, ldv, lddq, lddk, lddv}, 4 * es);
  a.tc = es == 2 &&
         rows_aligned(p, {Q, K, V, O, dO, dQ, dK, dV}, {ldq, ldk, ldv, lddq, lddk, lddv}, 16) &&
         mappable({ldq, ldk, ldv});
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_attn_backward(p, a));
}

int cat_plan_create_layernorm(cat_plan_t* out, int max_rows, int D, int dtype, float eps,
                              void* stream) {
  if (!out) return CAT_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_rows < 0 || max_rows > CAT_NORM_MAX_ROWS || D < 1 || D > CAT_MAX_D)
    return CAT_ERR_INVALID_ARG;
  if (dtype != CAT_F32 && dtype != CAT_BF16) return CAT_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return CAT_ERR_INVALID_ARG;
  int st;
  cat_plan_s* p = new_plan(cat::OP_LAYERNORM, dtype, stream, &st);
  if (!p) return st;
  p->D = D;
  p->ln.max_rows = max_rows;
  p->ln.eps = eps;
  p->ln.max_parts = cat::layernorm_parts(p->sms);
  if (!alloc_status(p) || !alloc(p, &p->ln.part, (size_t)p->ln.max_parts * 2 * D))
    return fail(p, CAT_ERR_ALLOC);
  std::snprintf(p->desc, sizeof(p->desc), "op=layernorm max_rows=%d D=%d eps=%g workspace=%zu",
                max_rows, D, (double)eps, p->workspace_bytes);
  *out = p;
  return CAT_OK;
}

namespace {
int norm_prepare(cat_plan_s* p, int rows) {
  if (!p) return CAT_ERR_INVALID_ARG;
  if (p->op != cat::OP_LAYERNORM) return CAT_ERR_PLAN_MISMATCH;
  if (rows < 0) return CAT_ERR_INVALID_ARG;
  return rows > p->ln.max_rows ? CAT_ERR_PLAN_MISMATCH : CAT_OK;
}
}  // namespace

int cat_layernorm_forward(cat_plan_t p, const void* X, const void* gamma, const void* beta,
                          void* Y, float* mean, float* rstd, int rows) {
  const int st = norm_prepare(p, rows);
  if (st != CAT_OK || rows == 0) return st;
  if (!X || !Y || !mean || !rstd) return CAT_ERR_INVALID_ARG;
  if (((uintptr_t)X | (uintptr_t)gamma | (uintptr_t)beta | (uintptr_t)Y) & 15)
    return CAT_ERR_MISALIGNED;
  if (((uintptr_t)mean | (uintptr_t)rstd) & 3) return CAT_ERR_MISALIGNED;
  const size_t es = elem_size(p->dtype), nx = (size_t)rows * p->D * es, nw = (size_t)p->D * es;
  const size_t ns = (size_t)rows * sizeof(float);
  const Span2 in[3] = {flat(X, nx), flat(gamma, nw), flat(beta, nw)};
  const Span2 outs[3] = {flat(Y, nx), flat(mean, ns), flat(rstd, ns)};
  if (aliased(in, 3, outs, 3)) return CAT_ERR_ALIAS;
  cat::NormArgs a = {};
  a.x = X; a.gamma = gamma; a.beta = beta;
  a.y = Y; a.mean = mean; a.rstd = rstd;
  a.rows = rows; a.D = p->D; a.eps = p->ln.eps;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_layernorm(a, p->dtype, false, p->stream));
}

int cat_layernorm_backward(cat_plan_t p, const void* X, const void* gamma, const float* mean,
                           const float* rstd, const void* dY, void* dX, void* dgamma, void* dbeta,
                           int rows) {
  const int st = norm_prepare(p, rows);
  if (st != CAT_OK) return st;
  const size_t es = elem_size(p->dtype), nx = (size_t)rows * p->D * es, nw = (size_t)p->D * es;
  const size_t ns = (size_t)rows * sizeof(float);
  if (rows > 0 && (!X || !mean || !rstd || !dY || !dX)) return CAT_ERR_INVALID_ARG;
  if (((uintptr_t)X | (uintptr_t)gamma | (uintptr_t)dY | (uintptr_t)dX | (uintptr_t)dgamma |
       (uintptr_t)dbeta) & 15)
    return CAT_ERR_MISALIGNED;
  if (((uintptr_t)mean | (uintptr_t)rstd) & 3) return CAT_ERR_MISALIGNED;
  const Span2 in[5] = {flat(X, nx), flat(gamma, nw), flat(mean, ns), flat(rstd, ns), flat(dY, nx)};
  const Span2 outs[3] = {flat(dX, nx), flat(dgamma, nw), flat(dbeta, nw)};
  if (aliased(in, 5, outs, 3)) return CAT_ERR_ALIAS;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  if (rows == 0) {
    // Sums over no rows.
    cudaError_t e = dgamma ? cudaMemsetAsync(dgamma, 0, nw, p->stream) : cudaSuccess;
    if (e == cudaSuccess && dbeta) e = cudaMemsetAsync(dbeta, 0, nw, p->stream);
    return status_of(e);
  }
  cat::NormArgs a = {};
  a.x = X; a.gamma = gamma; a.dy = dY;
  a.dx = dX; a.dgamma = dgamma; a.dbeta = dbeta;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.part = p->ln.part; a.max_parts = p->ln.max_parts;
  a.rows = rows; a.D = p->D; a.eps = p->ln.eps;
  return status_of(cat::launch_layernorm(a, p->dtype, true, p->stream));
}

int cat_plan_create_clip(cat_plan_t* out, int count, const long long* sizes, const int* dtypes,
                         void* stream) {
  if (!out) return CAT_ERR_INVALID_ARG;
  *out = nullptr;
  if (count < 0 || count > CAT_CLIP_MAX_TENSORS || (count > 0 && (!sizes || !dtypes)))
    return CAT_ERR_INVALID_ARG;
  long long nchunks = 0;
  for (int i = 0; i < count; ++i) {
    if (dtypes[i] != CAT_F32 && dtypes[i] != CAT_BF16) return CAT_ERR_INVALID_ARG;
    if (sizes[i] < 0 || sizes[i] > (1ll << 40)) return CAT_ERR_INVALID_ARG;
    const int e = cat::clip_chunk_elems(dtypes[i]);
    nchunks += (sizes[i] + e - 1) / e;
    if (nchunks > INT_MAX / 2) return CAT_ERR_INVALID_ARG;
  }
  int st;
  cat_plan_s* p = new_plan(cat::OP_CLIP, CAT_F32, stream, &st);
  if (!p) return st;
  cat::ClipCfg& c = p->cl;
  c.count = count;
  c.grid = cat::clip_grid(p->sms);
  int* first = new (std::nothrow) int[count + 1];
  long long* sz = new (std::nothrow) long long[count + 1];
  int* dt = new (std::nothrow) int[count + 1];
  cat::ClipChunk* host = new (std::nothrow) cat::ClipChunk[(size_t)nchunks + 1];
  c.first_chunk = first;
  c.sizes = sz;
  c.dtypes = dt;
  if (!first || !sz || !dt || !host) {
    delete[] host;
    return fail(p, CAT_ERR_ALLOC);
  }
  int n = 0;
  for (int i = 0; i < count; ++i) {
    first[i] = n;
    sz[i] = sizes[i];
    dt[i] = dtypes[i];
    const int e = cat::clip_chunk_elems(dtypes[i]);
    for (long long o = 0; o < sizes[i]; o += e)
      host[n++] = cat::ClipChunk{i, dtypes[i] == CAT_BF16, (int)std::min<long long>(e, sizes[i] - o), o};
  }
  first[count] = n;
  bool ok = alloc_status(p) && alloc(p, &c.chunks, (size_t)n) &&
            alloc(p, &c.part, (size_t)cat::clip_max_parts(count, p->sms));
  if (!ok) {
    delete[] host;
    return fail(p, CAT_ERR_ALLOC);
  }
  const cudaError_t e = cat::settled([&](cudaStream_t s) {
    return cudaMemcpyAsync(c.chunks, host, (size_t)n * sizeof(cat::ClipChunk),
                           cudaMemcpyHostToDevice, s);
  });
  delete[] host;
  if (e != cudaSuccess) return fail(p, CAT_ERR_CUDA);
  std::snprintf(p->desc, sizeof(p->desc), "op=clip tensors=%d chunks=%d workspace=%zu", count, n,
                p->workspace_bytes);
  *out = p;
  return CAT_OK;
}

namespace {

int clip_prepare(cat_plan_s* p, const void* const* grads, const float* norm) {
  if (!p) return CAT_ERR_INVALID_ARG;
  if (p->op != cat::OP_CLIP) return CAT_ERR_PLAN_MISMATCH;
  const cat::ClipCfg& c = p->cl;
  if (!norm || (c.count > 0 && !grads)) return CAT_ERR_INVALID_ARG;
  if ((uintptr_t)norm & 3) return CAT_ERR_MISALIGNED;
  for (int i = 0; i < c.count; ++i) {
    if (c.sizes[i] == 0) continue;
    if (!grads[i]) return CAT_ERR_INVALID_ARG;
    if ((uintptr_t)grads[i] & (elem_size(c.dtypes[i]) - 1)) return CAT_ERR_MISALIGNED;
  }
  return CAT_OK;
}

}  // namespace

int cat_grad_norm(cat_plan_t p, const void* const* grads, float* norm) {
  const int st = clip_prepare(p, grads, norm);
  if (st != CAT_OK) return st;
  const Span2 to = flat(norm, sizeof(float));
  for (int i = 0; i < p->cl.count; ++i)
    if (overlap(to, flat(grads[i], (size_t)p->cl.sizes[i] * elem_size(p->cl.dtypes[i]))))
      return CAT_ERR_ALIAS;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_clip(p->cl, grads, nullptr, 0.f, norm, false, p->stream));
}

int cat_grad_clip(cat_plan_t p, const void* const* grads, void* const* outs, float max_norm,
                  float* norm) {
  int st = clip_prepare(p, grads, norm);
  if (st != CAT_OK) return st;
  if (!(max_norm >= 0.f)) return CAT_ERR_INVALID_ARG;
  const cat::ClipCfg& c = p->cl;
  if (c.count > 0 && !outs) return CAT_ERR_INVALID_ARG;
  // An output may be its own gradient (in place); apart from that no output
  // may meet a gradient, another output or the norm: sorted by address, a
  // written range may not reach the next one.
  struct Range {
    uintptr_t a, b;
    int kind;            // 0 read, 1 written
  };
  std::vector<Range> r;
  try {
    r.reserve(2 * (size_t)c.count + 1);
  } catch (const std::bad_alloc&) {
    return CAT_ERR_ALLOC;
  }
  for (int i = 0; i < c.count; ++i) {
    if (c.sizes[i] == 0) continue;
    const size_t es = elem_size(c.dtypes[i]), n = (size_t)c.sizes[i] * es;
    if (!outs[i]) return CAT_ERR_INVALID_ARG;
    if ((uintptr_t)outs[i] & (es - 1)) return CAT_ERR_MISALIGNED;
    if (outs[i] != grads[i]) r.push_back(Range{(uintptr_t)grads[i], (uintptr_t)grads[i] + n, 0});
    r.push_back(Range{(uintptr_t)outs[i], (uintptr_t)outs[i] + n, 1});
  }
  r.push_back(Range{(uintptr_t)norm, (uintptr_t)norm + sizeof(float), 1});
  std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
  uintptr_t end_any = 0, end_out = 0;
  for (const Range& x : r) {
    if (x.a < end_out || (x.kind && x.a < end_any)) return CAT_ERR_ALIAS;
    end_any = std::max(end_any, x.b);
    if (x.kind) end_out = std::max(end_out, x.b);
  }
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_clip(c, grads, outs, max_norm, norm, true, p->stream));
}

}  // extern "C"
