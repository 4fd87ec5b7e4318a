// C ABI of the rest of a language model's training step (include/cat.h): the
// embedding, the residual stream with its norms, and the cross entropy over the
// vocabulary.  Plans are cat_plan_t; the kernels are in embed.cu, resnorm_*.cu
// and xent*.cu.
#include <cmath>
#include <cstdint>
#include <cstdio>

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
using cat::status_of;

bool bad_ids(int id_type) { return id_type != CAT_I32 && id_type != CAT_I64; }
size_t id_size(int id_type) { return id_type == CAT_I64 ? 8 : 4; }

// Whether a pointer is off a 16-byte boundary (rows are read in vectors).
bool off16(std::initializer_list<const void*> ptrs) {
  uintptr_t any = 0;
  for (const void* q : ptrs) any |= (uintptr_t)q;
  return any & 15;
}

}  // namespace

extern "C" {

int cat_plan_create_embed(cat_plan_t* out, int max_tokens, int V, int D, int dtype, float scale,
                          void* stream) {
  if (!out) return CAT_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_tokens < 0 || max_tokens > CAT_STEP_MAX_TOKENS || V < 1 || V > CAT_MAX_VOCAB || D < 1 ||
      D > CAT_MAX_D)
    return CAT_ERR_INVALID_ARG;
  if (dtype != CAT_F32 && dtype != CAT_BF16) return CAT_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return CAT_ERR_INVALID_ARG;
  int st;
  cat_plan_s* p = new_plan(cat::OP_EMBED, dtype, stream, &st);
  if (!p) return st;
  p->D = D;
  cat::EmbedCfg& c = p->em;
  c.max_tokens = max_tokens;
  c.V = V;
  c.scale = scale;
  c.range = cat::embed_range(V, p->sms);
  const size_t split = cat::embed_split_count(max_tokens);
  if (!alloc_status(p) || !alloc(p, &c.tok, split) || !alloc(p, &c.key, split) ||
      !alloc(p, &c.off, cat::embed_off_count(max_tokens, V, p->sms)) || !alloc(p, &c.first, (size_t)V + 1) ||
      !alloc(p, &c.order, (size_t)max_tokens) || !alloc(p, &c.sid, (size_t)max_tokens) ||
      !alloc(p, &c.part, cat::embed_part_count(max_tokens, D)))
    return fail(p, CAT_ERR_ALLOC);
  if (cat::setup_embed() != cudaSuccess) return fail(p, CAT_ERR_CUDA);
  std::snprintf(p->desc, sizeof(p->desc),
                "op=embed max_tokens=%d V=%d D=%d scale=%g workspace=%zu", max_tokens, V, D,
                (double)scale, p->workspace_bytes);
  *out = p;
  return CAT_OK;
}

namespace {
// Checks that calls over tokens share.
int tokens_prepare(cat_plan_s* p, int op, int max_tokens, const void* ids, int id_type, int T) {
  if (p->op != op) return CAT_ERR_PLAN_MISMATCH;
  if (T < 0 || bad_ids(id_type)) return CAT_ERR_INVALID_ARG;
  if (T > max_tokens) return CAT_ERR_PLAN_MISMATCH;
  if (T > 0 && !ids) return CAT_ERR_INVALID_ARG;
  return (uintptr_t)ids & (id_size(id_type) - 1) ? CAT_ERR_MISALIGNED : CAT_OK;
}
}  // namespace

int cat_embed_forward(cat_plan_t p, const void* ids, int id_type, const void* W, void* Y, int T) {
  if (!p) return CAT_ERR_INVALID_ARG;
  const int st = tokens_prepare(p, cat::OP_EMBED, p->em.max_tokens, ids, id_type, T);
  if (st != CAT_OK || T == 0) return st;
  if (!W || !Y) return CAT_ERR_INVALID_ARG;
  if (off16({W, Y})) return CAT_ERR_MISALIGNED;
  const size_t row = (size_t)p->D * elem_size(p->dtype);
  const Span2 in[2] = {flat(ids, (size_t)T * id_size(id_type)), flat(W, row * p->em.V)};
  const Span2 outs[1] = {flat(Y, row * T)};
  if (aliased(in, 2, outs, 1)) return CAT_ERR_ALIAS;
  cat::EmbedArgs a = {};
  a.ids.p = ids;
  a.ids.wide = id_type == CAT_I64;
  a.x = W;
  a.y = Y;
  a.tokens = T;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_embed(p, a, false));
}

int cat_embed_backward(cat_plan_t p, const void* ids, int id_type, const void* dY, void* dW,
                       int accumulate, int T) {
  if (!p) return CAT_ERR_INVALID_ARG;
  const int st = tokens_prepare(p, cat::OP_EMBED, p->em.max_tokens, ids, id_type, T);
  if (st != CAT_OK) return st;
  if (!dW || (T > 0 && !dY) || (accumulate != 0 && accumulate != 1)) return CAT_ERR_INVALID_ARG;
  if (off16({dY, dW})) return CAT_ERR_MISALIGNED;
  const size_t row = (size_t)p->D * elem_size(p->dtype);
  const Span2 in[2] = {flat(ids, (size_t)T * id_size(id_type)), flat(dY, row * T)};
  const Span2 outs[1] = {flat(dW, row * p->em.V)};
  if (aliased(in, 2, outs, 1)) return CAT_ERR_ALIAS;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  if (T == 0)          // sums over no tokens
    return accumulate ? CAT_OK : status_of(cudaMemsetAsync(dW, 0, row * p->em.V, p->stream));
  cat::EmbedArgs a = {};
  a.ids.p = ids;
  a.ids.wide = id_type == CAT_I64;
  a.x = dY;
  a.y = dW;
  a.tokens = T;
  a.add = accumulate;
  return status_of(cat::launch_embed(p, a, true));
}

int cat_plan_create_resnorm(cat_plan_t* out, int max_rows, int D, int dtype, int post, float eps,
                            float scale, void* stream) {
  if (!out) return CAT_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_rows < 0 || max_rows > CAT_NORM_MAX_ROWS || D < 1 || D > CAT_MAX_D)
    return CAT_ERR_INVALID_ARG;
  if (dtype != CAT_F32 && dtype != CAT_BF16) return CAT_ERR_INVALID_ARG;
  if (post != 0 && post != 1) return CAT_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(scale)) return CAT_ERR_INVALID_ARG;
  int st;
  cat_plan_s* p = new_plan(cat::OP_RESNORM, dtype, stream, &st);
  if (!p) return st;
  p->D = D;
  cat::ResNormCfg& c = p->rn;
  c.max_rows = max_rows;
  c.post = post;
  c.eps = eps;
  c.scale = scale;
  c.max_parts = cat::resnorm_parts(p->sms);
  if (!alloc_status(p) || !alloc(p, &c.part, cat::resnorm_part_count(p->sms, D)))
    return fail(p, CAT_ERR_ALLOC);
  if (cat::setup_resnorm(D, dtype, post) != cudaSuccess) return fail(p, CAT_ERR_CUDA);
  std::snprintf(p->desc, sizeof(p->desc),
                "op=resnorm max_rows=%d D=%d post=%d eps=%g scale=%g workspace=%zu", max_rows, D,
                post, (double)eps, (double)scale, p->workspace_bytes);
  *out = p;
  return CAT_OK;
}

namespace {
int resnorm_prepare(cat_plan_s* p, const void* gate, int gate_rows, int rows) {
  if (!p) return CAT_ERR_INVALID_ARG;
  if (p->op != cat::OP_RESNORM) return CAT_ERR_PLAN_MISMATCH;
  if (rows < 0 || (gate_rows != 0 && gate_rows != 1) || (gate_rows && rows > 0 && !gate))
    return CAT_ERR_INVALID_ARG;
  return rows > p->rn.max_rows ? CAT_ERR_PLAN_MISMATCH : CAT_OK;
}

cat::ResNormArgs resnorm_args(const cat_plan_s* p, const void* B, const void* gate, int gate_rows,
                              const void* post_gamma, const void* post_beta, const void* gamma,
                              int rows) {
  cat::ResNormArgs a = {};
  a.b = B;
  a.gate = gate;
  a.gate_kind = !gate ? 0 : gate_rows ? 2 : 1;
  a.pg = post_gamma;
  a.pb = post_beta;
  a.gamma = gamma;
  a.post = p->rn.post;
  a.rows = rows;
  a.D = p->D;
  a.eps = p->rn.eps;
  a.scale = p->rn.scale;
  a.part = p->rn.part;
  a.max_parts = p->rn.max_parts;
  return a;
}
}  // namespace

int cat_resnorm_forward(cat_plan_t p, const void* R, const void* B, const void* gate,
                        int gate_rows, const void* post_gamma, const void* post_beta,
                        const void* gamma, const void* beta, void* H, void* Y, float* stats,
                        int rows) {
  const int st = resnorm_prepare(p, gate, gate_rows, rows);
  if (st != CAT_OK) return st;
  if (!p->rn.post && (post_gamma || post_beta)) return CAT_ERR_INVALID_ARG;
  if (rows == 0) return CAT_OK;
  if (!R || !B || !H || !Y || !stats) return CAT_ERR_INVALID_ARG;
  if (off16({R, B, gate, post_gamma, post_beta, gamma, beta, H, Y})) return CAT_ERR_MISALIGNED;
  if ((uintptr_t)stats & 3) return CAT_ERR_MISALIGNED;
  const size_t es = elem_size(p->dtype), nw = (size_t)p->D * es, nx = nw * rows;
  const Span2 in[7] = {flat(R, nx), flat(B, nx), flat(gate, gate_rows ? nx : nw),
                       flat(post_gamma, nw), flat(post_beta, nw), flat(gamma, nw), flat(beta, nw)};
  const Span2 outs[3] = {flat(H, nx), flat(Y, nx),
                         flat(stats, (size_t)rows * (p->rn.post ? 4 : 2) * sizeof(float))};
  if (aliased(in, 7, outs, 3)) return CAT_ERR_ALIAS;
  cat::ResNormArgs a = resnorm_args(p, B, gate, gate_rows, post_gamma, post_beta, gamma, rows);
  a.r = R;
  a.beta = beta;
  a.h = H;
  a.y = Y;
  a.stats = stats;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_resnorm_forward(a, p->dtype, p->stream));
}

int cat_resnorm_backward(cat_plan_t p, const void* H, const void* B, const void* gate,
                         int gate_rows, const void* post_gamma, const void* post_beta,
                         const void* gamma, const float* stats, const void* dH, const void* dY,
                         void* dR, void* dB, void* dgate, void* dpost_gamma, void* dpost_beta,
                         void* dgamma, void* dbeta, int rows) {
  const int st = resnorm_prepare(p, gate, gate_rows, rows);
  if (st != CAT_OK) return st;
  if (!p->rn.post && (post_gamma || post_beta || dpost_gamma || dpost_beta))
    return CAT_ERR_INVALID_ARG;
  if (dgate && !gate) return CAT_ERR_INVALID_ARG;
  if (rows > 0 && (!H || !B || !stats || !dY || !dR || !dB)) return CAT_ERR_INVALID_ARG;
  if (off16({H, B, gate, post_gamma, post_beta, gamma, dH, dY, dR, dB, dgate, dpost_gamma,
             dpost_beta, dgamma, dbeta}))
    return CAT_ERR_MISALIGNED;
  if ((uintptr_t)stats & 3) return CAT_ERR_MISALIGNED;
  const size_t es = elem_size(p->dtype), nw = (size_t)p->D * es, nx = nw * rows;
  const size_t ng = gate_rows ? nx : nw;
  const Span2 in[9] = {flat(H, nx), flat(B, nx), flat(gate, ng), flat(post_gamma, nw),
                       flat(post_beta, nw), flat(gamma, nw),
                       flat(stats, (size_t)rows * (p->rn.post ? 4 : 2) * sizeof(float)),
                       flat(dH, nx), flat(dY, nx)};
  const Span2 outs[7] = {flat(dR, nx), flat(dB, nx), flat(dgate, ng), flat(dpost_gamma, nw),
                         flat(dpost_beta, nw), flat(dgamma, nw), flat(dbeta, nw)};
  if (aliased(in, 9, outs, 7)) return CAT_ERR_ALIAS;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  if (rows == 0) {     // sums over no rows
    void* const sums[5] = {gate_rows ? nullptr : dgate, dpost_gamma, dpost_beta, dgamma, dbeta};
    for (void* s : sums)
      if (s && cudaMemsetAsync(s, 0, nw, p->stream) != cudaSuccess) {
        cudaGetLastError();
        return CAT_ERR_CUDA;
      }
    return CAT_OK;
  }
  cat::ResNormArgs a = resnorm_args(p, B, gate, gate_rows, post_gamma, post_beta, gamma, rows);
  a.hin = H;
  a.stats = const_cast<float*>(stats);
  a.dh = dH;
  a.dy = dY;
  a.dr = dR;
  a.db = dB;
  a.dgate = dgate;
  a.dpg = dpost_gamma;
  a.dpb = dpost_beta;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  return status_of(cat::launch_resnorm_backward(a, p->dtype, p->stream));
}

int cat_plan_create_xent(cat_plan_t* out, int max_tokens, int V, int D, int dtype, int grad,
                         void* stream) {
  if (!out) return CAT_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_tokens < 0 || max_tokens > CAT_XENT_MAX_TOKENS || V < 1 || V > CAT_MAX_VOCAB || D < 1 ||
      D > CAT_MAX_D)
    return CAT_ERR_INVALID_ARG;
  if (dtype != CAT_F32 && dtype != CAT_BF16) return CAT_ERR_INVALID_ARG;
  if (grad != 0 && grad != 1) return CAT_ERR_INVALID_ARG;
  int st;
  cat_plan_s* p = new_plan(cat::OP_XENT, dtype, stream, &st);
  if (!p) return st;
  p->D = D;
  cat::XentCfg& c = p->xe;
  c.max_tokens = max_tokens;
  c.V = V;
  c.grad = grad;
  int pairs = 0;
  if (cat::setup_xent_mma(dtype, p->sms, &pairs) != cudaSuccess) return fail(p, CAT_ERR_CUDA);
  cat::xent_shape(&c, D, dtype, pairs);
  const size_t n = (size_t)max_tokens, rows = (size_t)c.rows_alloc;
  const size_t row = (size_t)c.terms * c.pitch * 2;        // bytes of a packed row
  auto bytes = [&](void** q, size_t count) { return alloc(p, (unsigned char**)q, count); };
  bool ok = alloc_status(p) && alloc(p, &c.count, 4) && alloc(p, &c.rows, n) &&
            alloc(p, &c.tgt, n) && alloc(p, &c.hit, n) &&
            alloc(p, &c.part, cat::xent_part_count(c)) && bytes(&c.xp, rows * row);
  if (ok && c.pack) ok = bytes(&c.wp, (size_t)V * row);
  if (ok && grad)
    ok = alloc(p, &c.stat, n) && alloc(p, &c.inv, n) &&
         bytes(&c.d, rows * c.piece * 2 * c.terms * (c.pieces > 1 ? 2 : 1)) &&
         alloc(p, &c.dxacc, (size_t)c.acc_tiles * 256 * c.acc_pitch);
  if (!ok) return fail(p, CAT_ERR_ALLOC);
  std::snprintf(p->desc, sizeof(p->desc), "op=xent max_tokens=%d V=%d D=%d grad=%d piece=%d "
                "workspace=%zu", max_tokens, V, D, grad, c.piece, p->workspace_bytes);
  *out = p;
  return CAT_OK;
}

int cat_xent_forward(cat_plan_t p, const void* X, const void* W, const void* targets, int id_type,
                     float* loss, float* lse, int T) {
  if (!p) return CAT_ERR_INVALID_ARG;
  const int st = tokens_prepare(p, cat::OP_XENT, p->xe.max_tokens, targets, id_type, T);
  if (st != CAT_OK || T == 0) return st;
  if (!X || !W || !loss || !lse) return CAT_ERR_INVALID_ARG;
  if (off16({X, W}) || (((uintptr_t)loss | (uintptr_t)lse) & 3)) return CAT_ERR_MISALIGNED;
  const size_t row = (size_t)p->D * elem_size(p->dtype), ns = (size_t)T * sizeof(float);
  const Span2 in[3] = {flat(X, row * T), flat(W, row * p->xe.V),
                       flat(targets, (size_t)T * id_size(id_type))};
  const Span2 outs[2] = {flat(loss, ns), flat(lse, ns)};
  if (aliased(in, 3, outs, 2)) return CAT_ERR_ALIAS;
  cat::XentArgs a = {};
  a.x = X;
  a.w = W;
  a.loss = loss;
  a.lse = lse;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  return status_of(cat::launch_xent(p, a, cat::Ids{targets, id_type == CAT_I64}, T, false));
}

int cat_xent_backward(cat_plan_t p, const void* X, const void* W, const void* targets, int id_type,
                      const float* lse, const float* dloss, int dloss_each, void* dX, void* dW,
                      int T) {
  if (!p) return CAT_ERR_INVALID_ARG;
  const int st = tokens_prepare(p, cat::OP_XENT, p->xe.max_tokens, targets, id_type, T);
  if (st != CAT_OK) return st;
  if (!p->xe.grad) return CAT_ERR_PLAN_MISMATCH;
  if ((dloss_each != 0 && dloss_each != 1) || (T > 0 && (!X || !W || !lse || !dloss)))
    return CAT_ERR_INVALID_ARG;
  if (off16({X, W, dX, dW}) || (((uintptr_t)lse | (uintptr_t)dloss) & 3))
    return CAT_ERR_MISALIGNED;
  const size_t row = (size_t)p->D * elem_size(p->dtype), ns = (size_t)T * sizeof(float);
  const Span2 in[5] = {flat(X, row * T), flat(W, row * p->xe.V),
                       flat(targets, (size_t)T * id_size(id_type)), flat(lse, ns),
                       flat(dloss, dloss_each ? ns : sizeof(float))};
  const Span2 outs[2] = {flat(dX, row * T), flat(dW, row * p->xe.V)};
  if (aliased(in, 5, outs, 2)) return CAT_ERR_ALIAS;
  if (!dX && !dW) return CAT_OK;
  DeviceGuard dev(p->device);
  if (dev.status != cudaSuccess) return CAT_ERR_CUDA;
  if (T == 0)          // sums over no tokens
    return dW ? status_of(cudaMemsetAsync(dW, 0, row * p->xe.V, p->stream)) : CAT_OK;
  cat::XentArgs a = {};
  a.x = X;
  a.w = W;
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.dloss_each = dloss_each;
  a.dx = dX;
  a.dw = dW;
  return status_of(cat::launch_xent(p, a, cat::Ids{targets, id_type == CAT_I64}, T, true));
}

}  // extern "C"
