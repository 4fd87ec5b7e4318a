// Softmax cross entropy over a vocabulary, from hidden states X [T, D] and the
// output weights W [V, D]:
//   l_iv = x_i·w_v,  lse_i = log Σ_v exp(l_iv),  loss_i = lse_i - l_{i,t_i};
//   d_iv = g_i·(exp(l_iv - lse_i) - [v = t_i]),  dX = d·W,  dW = dᵀ·X.
// The logits are never kept: the forward keeps the maximum and the sum of
// exponentials of each row, the backward makes them again, a piece of the
// vocabulary at a time.  Tokens without a target (a negative one) take no part:
// the others' rows are worked on as one dense list.
#include <cuda_bf16.h>

#include "cat_internal.h"
#include "elem.cuh"
#include "ids.cuh"
#include "xent_mma.cuh"
#include "../../include/cat.h"

namespace cat {

namespace {

constexpr int kThreads = 256;
constexpr int kPrep = 1024;              // threads of the preparing kernel
constexpr int kPer = 128;                // tokens of a CTA of it, at least
constexpr float kLog2e = 1.4426950408889634f;

// What the call's first kernel prepares.
struct Prep {
  Ids targets;
  int tokens, per, V, D, pitch, terms;   // per: tokens of a CTA; pitch: columns of a packed row
  int direct;                            // 1: X itself serves where every token has a target
  int list_ctas;                         // CTAs of the list; the others pack W
  const void* x; const void* w;
  void* xp; void* wp;                    // packed rows: [row][term][pitch] bf16
  int* rows; int* tgt; int* inv; int* count;
  float* loss; float* lse;               // forward: 0 for the tokens without a target
  const float* lse_in; const float* dloss;
  int dloss_each;
  float2* stat;
  unsigned int* status;
};

// Eight columns of a row from c on (zeros from D on; src null: zeros), in vectors
// where rows are whole ones.
__device__ __forceinline__ void load8(const float* src, int c, int D, bool whole, float* v) {
  if (whole && src) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(src + c));
    const float4 b = __ldg(reinterpret_cast<const float4*>(src + c) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = src && c + e < D ? __ldg(src + c + e) : 0.f;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* src, int c, int D, bool whole,
                                      float* v) {
  if (whole && src) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(src + c));
    const unsigned int w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = src && c + e < D ? ld_elem(src + c + e) : 0.f;
}

// `terms` bf16 terms of 8 columns from c on of a row.
template <typename T>
__device__ __forceinline__ void pack8(const T* src, __nv_bfloat16* dst, int c, int D, int pitch,
                                      int terms) {
  float v[8];
  load8(src, c, D, D % 8 == 0 && c < D, v);
  for (int t = 0; t < terms; ++t) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(dst + (size_t)t * pitch + c) = *reinterpret_cast<uint4*>(h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] -= __bfloat162float(h[i].x);
      v[2 * i + 1] -= __bfloat162float(h[i].y);
    }
  }
}

// The list of the tokens that have a target (rows, tgt; inv: a token's place in
// it; count: its length and whether X itself serves as its rows), their
// statistics for the backward (stat: lse and the upstream gradient, 1 where one
// value serves all: results are scaled by that in fp32, so that the target's entry of
// d, near -1, is not rounded off for the factor's sake) and their rows of X, dense
// and, for fp32, as bf16 terms; rows of zeros up to a multiple of 256.  A CTA takes
// `per` tokens and counts the others' itself.  The other CTAs pack W.
template <typename T>
__global__ void __launch_bounds__(kPrep) xent_prepare_kernel(Prep p) {
  const int vecs = p.pitch / 8;
  if ((int)blockIdx.x >= p.list_ctas) {
    const long long n = (long long)p.V * vecs;
    const long long step = (long long)(gridDim.x - p.list_ctas) * kPrep;
    for (long long i = (long long)(blockIdx.x - p.list_ctas) * kPrep + threadIdx.x; i < n;
         i += step) {
      const long long v = i / vecs;
      pack8(static_cast<const T*>(p.w) + v * p.D,
            static_cast<__nv_bfloat16*>(p.wp) + v * p.terms * p.pitch, (int)(i - v * vecs) * 8,
            p.D, p.pitch, p.terms);
    }
    return;
  }
  __shared__ int red[2][kPrep / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * p.per, t1 = min(p.tokens, t0 + p.per);
  int before = 0, all = 0;
  // (8192 ids on their way at once: a CTA has the whole list to look through.)
  for (int i0 = 0; i0 < p.tokens; i0 += 8 * kPrep) {
    unsigned key[8];
    keys_at<8>(p.targets, i0 + threadIdx.x, kPrep, p.tokens, key);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int held = key[u] < (unsigned)p.V;
      all += held;
      before += i0 + u * kPrep + (int)threadIdx.x < t0 ? held : 0;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) {
    red[0][warp] = before;
    red[1][warp] = all;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kPrep / 32; ++w) {
    before += red[0][w];
    all += red[1][w];
  }
  const int direct = p.direct && all == p.tokens;
  int place = before;
  for (int b = t0; b < t1; b += kPrep) {
    const int t = b + threadIdx.x;
    const int id = t < t1 ? id_at(p.targets, t, p.V) : -1;
    if (id == -2) report(p.status, 0x801);
    const unsigned held = __ballot_sync(0xffffffffu, id >= 0);
    __syncthreads();
    if (lane == 0) red[0][warp] = __popc(held);
    __syncthreads();
    int mine = place;
#pragma unroll
    for (int w = 0; w < kPrep / 32; ++w) {
      if (w < warp) mine += red[0][w];
      place += red[0][w];
    }
    const int pos = mine + __popc(held & ((1u << lane) - 1));
    if (id >= 0) {
      p.rows[pos] = t;
      p.tgt[pos] = id;
      if (p.stat)
        p.stat[pos] = make_float2(__ldg(p.lse_in + t), p.dloss_each ? __ldg(p.dloss + t) : 1.f);
    } else if (t < t1 && p.loss) {
      p.loss[t] = 0.f;
      p.lse[t] = 0.f;
    }
    if (p.inv && t < t1) p.inv[t] = id >= 0 ? pos : -1;
  }
  if (threadIdx.x == 0 && blockIdx.x == p.list_ctas - 1) {
    p.count[0] = all;
    p.count[1] = direct;
  }
  if (direct) return;
  __syncthreads();                       // (rows that this CTA's threads wrote)
  // This CTA's rows of the list, the last CTA those behind it too.
  const bool tail = (int)blockIdx.x == p.list_ctas - 1;
  const int end = tail ? (all + 255) / 256 * 256 : place;
  const int n = (end - before) * vecs;
#pragma unroll 2
  for (int i = threadIdx.x; i < n; i += kPrep) {
    const int r = i / vecs, pos = before + r;
    const T* src = pos < all ? static_cast<const T*>(p.x) + (size_t)p.rows[pos] * p.D : nullptr;
    pack8(src, static_cast<__nv_bfloat16*>(p.xp) + (size_t)pos * p.terms * p.pitch,
          (i - r * vecs) * 8, p.D, p.pitch, p.terms);
  }
}

// loss and lse from the parts' maxima and sums: 32 places of the
// list a CTA, its warps every so-many-th part each (1024 tokens, 394 parts: 61 us
// with a thread a place, 5 so).
constexpr int kFinWarps = 16;
__global__ void __launch_bounds__(32 * kFinWarps)
xent_finish_kernel(const float2* part, int nparts, int ld, const int* count, const int* rows,
                   const float* hit, float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 red[kFinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pos = blockIdx.x * 32 + lane;
  pdl_wait();
  const int n = __ldcg(count);
  if (blockIdx.x * 32 >= n) return;
  float top = -INFINITY, s = 0.f;
  auto join = [&](float2 q) {
    const float m = fmaxf(top, q.x), sh = fabsf(m) < INFINITY ? m : 0.f;
    s = s * exp2f((top - sh) * kLog2e) + q.y * exp2f((q.x - sh) * kLog2e);
    top = m;
  };
  if (pos < n) {
#pragma unroll 4
    for (int i = warp; i < nparts; i += kFinWarps) join(__ldcg(part + (size_t)i * ld + pos));
  }
  red[warp][lane] = make_float2(top, s);
  __syncthreads();
  if (warp || pos >= n) return;
  for (int w = 1; w < kFinWarps; ++w) join(red[w][lane]);
  // (Not lse less the target's logit, two large numbers: where the target rules its row
  // the maximum less its logit is 0, and the loss as near as the sum is to 1.)
  const int t = __ldcg(rows + pos);
  const float rest = logf(s);
  lse[t] = top + rest;
  loss[t] = top - __ldcg(hit + pos) + rest;
}

// dX's rows from the sums of the list's (the slices of each, in order), zeros for
// the tokens without a target.  A warp takes kDxRows rows side by side, in vectors of
// four where they divide a row.
constexpr int kDxRows = 4;
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads)
xent_dx_kernel(const float* acc, int pitch, const int* inv, const int* count, T* __restrict__ dX,
               int tokens, int D, int pairs, int piece, int acc_tiles, const float* factor) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int row0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kDxRows;
  if (row0 >= tokens) return;
  const float f = factor ? __ldg(factor) : 1.f;
  const int mt = (__ldcg(count) + kXtM - 1) / kXtM;
  const int slices = mt ? xent_slices(pairs, mt, (D + kXtN - 1) / kXtN, piece, acc_tiles) : 0;
  const size_t apart = (size_t)mt * kXtM * pitch;
  int pos[kDxRows];
#pragma unroll
  for (int r = 0; r < kDxRows; ++r) pos[r] = row0 + r < tokens ? __ldcg(inv + row0 + r) : -1;
  for (int c = lane * VEC; c < D; c += 32 * VEC) {
    float v[kDxRows][4] = {};
    for (int s = 0; s < slices; ++s) {
#pragma unroll
      for (int r = 0; r < kDxRows; ++r) {
        if (pos[r] < 0) continue;
        const float* q = acc + s * apart + (size_t)pos[r] * pitch + c;
        if (VEC == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(q));
          v[r][0] += x.x; v[r][1] += x.y; v[r][2] += x.z; v[r][3] += x.w;
        } else {
          v[r][0] += __ldcg(q);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kDxRows; ++r) {
      if (row0 + r >= tokens) break;
      if (pos[r] >= 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[r][e] *= f;
      }
      T* to = dX + (size_t)(row0 + r) * D + c;
      if (VEC == 4 && sizeof(T) == 4) {
        *reinterpret_cast<float4*>(to) = make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
      } else if (VEC == 4) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[r][0], v[r][1]),
                               __floats2bfloat162_rn(v[r][2], v[r][3])};
        *reinterpret_cast<uint2*>(to) = *reinterpret_cast<uint2*>(h);
      } else {
        st_elem(to, v[r][0]);
      }
    }
  }
}

int tiles(long long n, int m) { return (int)((n + m - 1) / m); }

// Tiles of the vocabulary in a forward part: as many as leave each pair of CTAs
// sixteen parts, at most 32.
int run_length(int V, int tokens, int pairs) {
  const long long all = (long long)tiles(V, kXtN) * tiles(tokens, kXtM);
  const long long r = all / (16ll * pairs);
  return r < 1 ? 1 : r > 32 ? 32 : (int)r;
}

// Parts of a call's rows, and how far apart one part's and the next's lie.
int part_count(const XentCfg& c, int tokens) {
  return 2 * tiles(tiles(c.V, kXtN), run_length(c.V, tokens, c.pairs));
}
int part_pitch(int tokens) { return tiles(tokens, 32) * 32; }

}  // namespace

// Shapes of a plan's workspace.
void xent_shape(XentCfg* c, int D, int dtype, int pairs) {
  c->pairs = pairs;
  c->terms = dtype == CAT_F32 ? 3 : 1;
  c->pitch = (D + 63) / 64 * 64;
  c->acc_pitch = (D + 3) / 4 * 4;
  c->pack = dtype == CAT_F32 || D % 8 != 0;
  c->rows_alloc = tiles(c->max_tokens, kXtM) * kXtM;
  if (c->rows_alloc == 0) c->rows_alloc = kXtM;
  c->acc_tiles = c->rows_alloc / kXtM + pairs / tiles(D, kXtN);
  // A piece of the vocabulary: dW's tiles (of the piece by D) are the longest of a
  // launch, so that their number is a multiple of the pairs, or just below; more
  // of the vocabulary at once where there are few tokens (the pairs then share a
  // piece's ids out among slices of dX, of at most 65536 each), and less where two
  // pieces' d would take more than 2 GB, down to one tile of 256 ids (which takes more by
  // itself from 2^21 rows of terms on: fp32's most tokens, 2 x 1.6 GB).
  const int nt = tiles(D, kXtN), vt = tiles(c->V, kXtN);
  long long w = 32768 / c->rows_alloc;
  if (w < 1) w = 1;
  long long pt = w * pairs / nt;
  const long long tile_bytes = (long long)c->rows_alloc * kXtN * 2 * c->terms;
  const long long most = (2ll << 30) / (2 * tile_bytes);
  if (pt > most) pt = most;
  if (pt < 1) pt = 1;
  if (pt > vt) pt = vt;
  c->piece = (int)pt * kXtN;
  c->pieces = tiles(c->V, c->piece);
}
// Of all calls' parts: the fewer tokens the shorter the runs and the more parts of each,
// so neither the most tokens nor the most parts decide.  (Both at once: 1.05 GB for
// 131072 tokens and 128256 ids, where 34 MB are used.)
size_t xent_part_count(const XentCfg& c) {
  size_t most = 0;
  for (int m = 1; m <= c.rows_alloc / kXtM; ++m) {
    const int tokens = m * kXtM < c.max_tokens ? m * kXtM : c.max_tokens;
    const size_t n = (size_t)part_count(c, tokens) * part_pitch(tokens);
    if (n > most) most = n;
  }
  return most;
}

namespace {

template <typename T>
cudaError_t prepare(const cat_plan_s* p, const XentArgs& a, Ids targets, int tokens, bool back) {
  const XentCfg& c = p->xe;
  Prep q = {};
  q.targets = targets;
  q.tokens = tokens;
  q.per = tokens > 2048 * kPer ? (tokens + 2047) / 2048 : kPer;
  q.V = c.V;
  q.D = p->D;
  q.pitch = c.pitch;
  q.terms = c.terms;
  q.direct = !c.pack;
  q.list_ctas = tiles(tokens, q.per);
  q.x = a.x;
  q.w = a.w;
  q.xp = c.xp;
  q.wp = c.wp;
  q.rows = c.rows;
  q.tgt = c.tgt;
  q.inv = back ? c.inv : nullptr;
  q.count = c.count;
  q.loss = back ? nullptr : a.loss;
  q.lse = back ? nullptr : a.lse;
  q.lse_in = a.lse;
  q.dloss = a.dloss;
  q.dloss_each = a.dloss_each;
  q.stat = back ? c.stat : nullptr;
  q.status = p->status;
  const long long wv = c.pack ? (long long)c.V * (c.pitch / 8) : 0;
  const long long need = (wv + kPrep - 1) / kPrep, most = 8ll * p->sms;
  const int wctas = (int)(need < most ? need : most);
  xent_prepare_kernel<T><<<q.list_ctas + wctas, kPrep, 0, p->stream>>>(q);
  return cudaGetLastError();
}

bool make_maps(const cat_plan_s* p, const XentArgs& a, int tokens, bool back, XentMaps* m) {
  const XentCfg& c = p->xe;
  const int D = p->D;
  const unsigned long long rb = (unsigned long long)c.terms * c.pitch * 2;
  auto both = [](CUtensorMap* by_k, CUtensorMap* by_rows, const void* q, unsigned long long width,
                 unsigned long long planes, unsigned long long rows, unsigned long long bytes) {
    return encode_map_planes_sw128(by_k, q, false, width, planes, rows, bytes, 128) &&
           (width % 64 == 0
                ? encode_map_blocks_sw128(by_rows, q, width, planes, rows, bytes)
                : encode_map_planes_sw128(by_rows, q, false, width, planes, rows, bytes, 64));
  };
  bool ok = both(&m->xp, &m->xpr, c.xp, c.pitch, c.terms, c.rows_alloc, rb);
  if (c.pack) {
    m->x = m->xp;
    m->xr = m->xpr;
    ok = ok && both(&m->w, &m->wr, c.wp, c.pitch, c.terms, c.V, rb);
  } else {
    ok = ok && both(&m->x, &m->xr, a.x, D, 1, tokens, 2ull * D) &&
         both(&m->w, &m->wr, a.w, D, 1, c.V, 2ull * D);
  }
  if (!ok || !back) return ok;
  const unsigned long long db = (unsigned long long)c.terms * c.piece * 2;
  const unsigned long long drows = (unsigned long long)c.rows_alloc * (c.pieces > 1 ? 2 : 1);
  ok = both(&m->d, &m->dr, c.d, c.piece, c.terms, drows, db) &&
       encode_map_planes_sw128(&m->acc, c.dxacc, true, D, 1, (unsigned long long)c.acc_tiles * kXtM,
                               (unsigned long long)c.acc_pitch * 4, 32);
  const bool f32 = p->dtype == CAT_F32;
  if (ok && a.dw && D % (f32 ? 4 : 8) == 0)
    ok = encode_map_planes_sw128(&m->dw, a.dw, f32, D, 1, c.V,
                                 (unsigned long long)D * (f32 ? 4 : 2), 32);
  return ok;
}

template <typename T, int VEC>
cudaError_t finish_dx(const cat_plan_s* p, const XentArgs& a, int tokens) {
  const XentCfg& c = p->xe;
  return launch_dependent(xent_dx_kernel<T, VEC>, dim3(tiles(tokens, kThreads / 32 * kDxRows)),
                          dim3(kThreads), 0, p->stream, (const float*)c.dxacc, c.acc_pitch,
                          (const int*)c.inv, (const int*)c.count, static_cast<T*>(a.dx), tokens,
                          p->D, c.pairs, c.piece, c.acc_tiles, a.dloss_each ? nullptr : a.dloss);
}

}  // namespace

cudaError_t launch_xent(const cat_plan_s* p, XentArgs a, Ids targets, int tokens, bool back) {
  const XentCfg& c = p->xe;
  cudaStream_t st = p->stream;
  const bool f32 = p->dtype == CAT_F32;
  cudaError_t e = f32 ? prepare<float>(p, a, targets, tokens, back)
                      : prepare<__nv_bfloat16>(p, a, targets, tokens, back);
  if (e != cudaSuccess) return e;
  XentMaps maps;
  if (!make_maps(p, a, tokens, back, &maps)) return cudaErrorInvalidValue;
  XentMma k = {};
  k.V = c.V;
  k.D = p->D;
  k.rows = c.rows_alloc;
  k.piece = c.piece;
  k.acc_tiles = c.acc_tiles;
  k.pairs = c.pairs;
  k.ld = part_pitch(tokens);
  k.count = c.count;
  k.tgt = c.tgt;
  k.rows_of = c.rows;
  k.x = a.x;
  k.w = a.w;
  k.stat = c.stat;
  k.hit = c.hit;
  k.factor = back && !a.dloss_each ? a.dloss : nullptr;
  k.part = c.part;
  k.d = c.d;
  k.dw = a.dw;
  k.two_w = !c.pack && p->D % 64;
  k.dw_tma = p->D % (f32 ? 4 : 8) == 0;
  k.status = p->status;
  k.dw_piece = k.dx_piece = k.d_piece = -1;
  // (No more pairs than there is work for.)
  auto go = [&](long long work) {
    const int n = work < c.pairs ? (work < 1 ? 1 : (int)work) : c.pairs;
    return launch_xent_mma(maps, k, p->dtype, n, k.dw_piece >= 0 ? tokens : 0, st);
  };
  const long long mt = tiles(tokens, kXtM), nt = tiles(p->D, kXtN), pt = c.piece / kXtN;
  if (!back) {
    k.lse = 1;
    k.run = run_length(c.V, tokens, c.pairs);
    e = go(mt * tiles(tiles(c.V, kXtN), k.run));
    if (e != cudaSuccess) return e;
    return launch_dependent(xent_finish_kernel, dim3(tiles(tokens, 32)), dim3(32 * kFinWarps), 0,
                            st, (const float2*)c.part, part_count(c, tokens), k.ld,
                            (const int*)c.count, (const int*)c.rows, (const float*)c.hit, a.loss,
                            a.lse);
  }
  // Piece i's products beside d of piece i + 1.
  for (int i = -1; i < c.pieces; ++i) {
    k.dw_piece = i >= 0 && a.dw ? i : -1;
    k.dx_piece = i >= 0 && a.dx ? i : -1;
    k.d_piece = i + 1 < c.pieces ? i + 1 : -1;
    k.first = i == 0;
    e = go((k.dw_piece >= 0 ? pt * nt : 0) + (k.dx_piece >= 0 ? c.acc_tiles * nt : 0) +
           (k.d_piece >= 0 ? pt * mt : 0));
    if (e != cudaSuccess) return e;
  }
  if (!a.dx) return cudaSuccess;
  if (p->D % 4)
    return f32 ? finish_dx<float, 1>(p, a, tokens) : finish_dx<__nv_bfloat16, 1>(p, a, tokens);
  return f32 ? finish_dx<float, 4>(p, a, tokens) : finish_dx<__nv_bfloat16, 4>(p, a, tokens);
}

}  // namespace cat
