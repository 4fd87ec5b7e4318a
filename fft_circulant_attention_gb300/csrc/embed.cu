// Embedding: rows of a table looked up by token, and the table's gradient.
//   Y[i] = scale·W[id_i],   dW[v] = scale·Σ_{i: id_i = v} dY[i],
// tokens without an id (negative) give rows of zeros and no gradient.
//
// Bound by memory: each row is read once and written once.  For the gradient
// the tokens are first sorted by id, so that every row of dW is summed in the
// order of its tokens and written once: no atomics on values, results repeat
// bit for bit.  Four launches:
//   split: blocks of the tokens, each put in the order of ranges of ids;
//   sort:  a CTA for each range takes its tokens from all blocks and puts them in
//          the order of their ids, and clears the rows of ids without tokens.  Both count by warp (a warp has a stretch of
//          the tokens) and keep the tokens' order within an id.  (One kernel whose
//          CTAs each looked through all ids: 15 us for 16384 tokens, 33 for 65536.)
//   sum:   the sorted list in pieces of equal length, a group of threads each; a
//          run of equal ids within a piece, or of at most kLong places, belongs to
//          the piece it starts in and is a finished row, a longer one leaves a
//          partial row (fp32) in each piece it touches;
//   join:  the partial rows of each long run, in a fixed order.
//
// Measured: 16384 tokens of 768 bf16 in a vocabulary of 50257, forward 8.6 us, gradient
// 40.5 (split, sort, sum and join alone 7, 17, 15 and 9: chains of dependent reads, and
// 66 MB of cleared rows); 65536 tokens of 1024 fp32 in 32003, 64 and 108 us (rows at
// 5 TB/s).
#include "cat_internal.h"
#include "ids.cuh"
#include "rows.cuh"
#include "../../include/cat.h"

namespace cat {

namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRange = 1024;        // most ids of a sorting CTA
constexpr int kBlocks = 256;            // most CTAs of the sort's first step
constexpr int kLong = 16;               // places of a run that is not split
constexpr int kSumPerSm = 4;            // CTAs of an SM that sum
constexpr int kFwdPerSm = 6;            // CTAs of an SM that look up
constexpr int kLookup = 1024;           // vectors of a looking-up CTA, about

// A CTA copies `per` rows at a time, its next rows' ids on their way meanwhile.
// COPY: the scale is 1, rows are copied as they are (16384 rows of 768 bf16 took more
// instructions than memory).
template <typename T, int VEC, bool COPY>
__global__ void __launch_bounds__(kThreads)
embed_fwd_kernel(Ids ids, const T* __restrict__ W, T* __restrict__ Y, int tokens, int V, int D,
                 int per, float scale, unsigned int* status) {
  using Vc = Vec<T, VEC>;
  constexpr int U = 4;                          // vectors on their way at once
  const int nv = D / VEC, chunk = per * nv;
  int r[U], c[U];                               // the same place in every chunk of rows
  for (int i0 = threadIdx.x; i0 < chunk; i0 += U * kThreads) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      r[u] = i < chunk ? i / nv : tokens;       // (none)
      c[u] = (i - i / nv * nv) * VEC;
    }
    int id[U], next[U];
    auto fetch_as = [&](auto* p, long long row0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        next[u] = row0 + r[u] < tokens ? id_of(id_key(__ldg(p + row0 + r[u])), V) : -1;
    };
    auto fetch = [&](long long row0) {
      if (ids.wide)
        fetch_as(static_cast<const long long*>(ids.p), row0);
      else
        fetch_as(static_cast<const int*>(ids.p), row0);
    };
    const long long step = (long long)gridDim.x * per;
    long long row0 = (long long)blockIdx.x * per;
    fetch(row0);
    for (; row0 < tokens; row0 += step) {
      typename Vc::Raw raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        id[u] = next[u];
        if (id[u] >= 0) raw[u] = Vc::ldr(W + (size_t)id[u] * D + c[u]);
      }
      fetch(row0 + step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (row0 + r[u] >= tokens) continue;
        T* to = Y + (size_t)(row0 + r[u]) * D + c[u];
        if (COPY && id[u] >= 0) {
          *reinterpret_cast<typename Vc::Raw*>(to) = raw[u];
          continue;
        }
        float v[VEC];
        if (id[u] >= 0) {
          Vc::widen(raw[u], v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] *= scale;
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] = 0.f;
          if (id[u] == -2 && c[u] == 0) report(status, 0x701);
        }
        Vc::st(to, v);
      }
    }
  }
}

// Block-wide exclusive sum over threads 0 .. kSortThreads - 1; *total: of all.
__device__ __forceinline__ int block_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    red[lane] = w;
  }
  __syncthreads();
  *total = red[kSortWarps - 1];
  return x - v + (warp ? red[warp - 1] : 0);
}

// A warp's counts of each class (hist [kSortWarps][classes]) become where its tokens
// of that class start: classes in order from `base` on, within a class the warps.
// Returns the number of all tokens; *start, *own: of class threadIdx.x, where its
// tokens start and how many they are.
__device__ __forceinline__ int class_starts(int* hist, int classes, int base, int* red,
                                            int* start, int* own) {
  const int c = threadIdx.x;
  int count = 0, all;
  if (c < classes) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) count += hist[w * classes + c];
  }
  int at = base + block_scan(count, red, &all);
  *start = at;
  *own = count;
  if (c < classes) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = hist[w * classes + c];
      hist[w * classes + c] = at;
      at += n;
    }
  }
  __syncthreads();
  return all;
}

// The lanes with `mine` of one class each (by `cls`) count (COUNT), or take their
// places, in the order of the lanes; h: the warp's counts or starts.
template <bool COUNT>
__device__ __forceinline__ int warp_class(int* h, bool mine, int cls) {
  const unsigned any = __ballot_sync(0xffffffffu, mine);
  if (!any) return -1;
  int pos = -1;
  if (mine) {
    const int lane = threadIdx.x & 31;
    const unsigned same = __match_any_sync(any, cls);
    const int start = h[cls];
    if (!COUNT) pos = start + __popc(same & ((1u << lane) - 1));
    __syncwarp(any);
    if (lane == __ffs(same) - 1) h[cls] = start + __popc(same);
  }
  __syncwarp();
  return pos;
}

// First step of the sort: a CTA puts its `per` tokens in the order of their ids'
// ranges (`range` ids each; magic: 2^32 / range, rounded up, exact for ids below
// 2^20).  tok, key: [blocks][per]; off: [blocks][ranges + 1].
__global__ void __launch_bounds__(kSortThreads)
embed_split_kernel(Ids ids, int tokens, int V, int per, int ranges, unsigned magic,
                   int* __restrict__ tok, int* __restrict__ key_out, int* __restrict__ off,
                   unsigned int* status) {
  extern __shared__ int hist[];                 // [kSortWarps][ranges]
  __shared__ int red[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b0 = blockIdx.x * per;
  const int steps = per / kSortThreads;
  const int t0 = b0 + warp * steps * 32;
  int* h = hist + warp * ranges;
  for (int i = lane; i < ranges; i += 32) h[i] = 0;
  __syncwarp();
  bool bad = false;
  for (int s = 0; s < steps; ++s) {
    const int t = t0 + 32 * s + lane;
    const int id = t < tokens ? id_at(ids, t, V) : -1;
    bad |= id == -2;
    warp_class<true>(h, id >= 0, id >= 0 ? (int)__umulhi((unsigned)id, magic) : 0);
  }
  if (bad) report(status, 0x702);
  __syncthreads();
  int start, own;
  const int all = class_starts(hist, ranges, 0, red, &start, &own);
  int* o = off + (size_t)blockIdx.x * (ranges + 1);
  if ((int)threadIdx.x < ranges) o[threadIdx.x] = start;
  if (threadIdx.x == 0) o[ranges] = all;
  for (int s = 0; s < steps; ++s) {
    const int t = t0 + 32 * s + lane;
    const int id = t < tokens ? id_at(ids, t, V) : -1;
    const int pos =
        warp_class<false>(h, id >= 0, id >= 0 ? (int)__umulhi((unsigned)id, magic) : 0);
    if (pos >= 0) {
      tok[b0 + pos] = t;
      key_out[b0 + pos] = id;
    }
  }
}

// Second step: a CTA sorts the tokens of one range, which it takes from the blocks
// of the first step in their order.  first[v]: where id v's tokens start in the
// sorted list (first[V]: its length); order: the tokens; sid: their ids.
__global__ void __launch_bounds__(kSortThreads)
embed_sort_kernel(const int* tok, const int* key, const int* off, int blocks, int per, int V,
                  int range, int* __restrict__ first, int* __restrict__ order,
                  int* __restrict__ sid, unsigned char* dW, size_t row_bytes) {
  extern __shared__ int hist[];                 // [kSortWarps][range]
  __shared__ int red[kSortWarps];
  __shared__ unsigned none[kSortRange / 32];    // ids without tokens
  __shared__ int2 part[kBlocks];                // where a block's tokens of this range lie
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ranges = gridDim.x, lo = blockIdx.x * range, n = min(range, V - lo);
  int* h = hist + warp * n;
  for (int i = lane; i < n; i += 32) h[i] = 0;
  pdl_wait();
  int below = 0, own, base, start, count;
  if ((int)threadIdx.x < blocks) {
    const int* o = off + (size_t)threadIdx.x * (ranges + 1) + blockIdx.x;
    below = __ldcg(o);
    const int q = threadIdx.x * per + below;
    part[threadIdx.x] = make_int2(q, q + __ldcg(o + 1) - below);
  }
  block_scan(below, red, &base);
  __syncthreads();
  // A warp takes a stretch of the blocks; f(place, end of the block's) for its
  // tokens, 256 at a time.  (Looking each token's block up cost more than the rest:
  // a range may hold a good part of all tokens.)
  const int each = (blocks + kSortWarps - 1) / kSortWarps;
  const int first_block = warp * each, last_block = min(blocks, first_block + each);
  constexpr int U = 8;
  auto tokens_of = [&](auto f) {
    for (int b = first_block; b < last_block; ++b) {
      const int2 s = part[b];
      for (int q = s.x; q < s.y; q += 32 * U) f(q + lane, s.y);
    }
  };
  tokens_of([&](int q, int end) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = q + 32 * u < end ? __ldcg(key + q + 32 * u) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) warp_class<true>(h, id[u] >= 0, id[u] - lo);
  });
  __syncthreads();
  own = class_starts(hist, n, base, red, &start, &count);
  if ((int)threadIdx.x < n) first[lo + threadIdx.x] = start;
  if (threadIdx.x == 0 && lo + n == V) first[V] = base + own;
  const unsigned empty = __ballot_sync(0xffffffffu, (int)threadIdx.x < n && count == 0);
  if (lane == 0) none[warp] = empty;
  tokens_of([&](int q, int end) {
    int id[U], t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = q + 32 * u < end;
      id[u] = in ? __ldcg(key + q + 32 * u) : -1;
      t[u] = in ? __ldcg(tok + q + 32 * u) : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pos = warp_class<false>(h, id[u] >= 0, id[u] - lo);
      if (pos >= 0) {
        order[pos] = t[u];
        sid[pos] = id[u];
      }
    }
  });
  // Rows of ids without tokens, where the gradient is not added to another's: the
  // ranges with few tokens have most of them, and time while a full one sorts.
  if (!dW) return;
  __syncthreads();
  for (int i = warp; i < n; i += kSortWarps) {
    if (!(none[i >> 5] >> (i & 31) & 1)) continue;
    unsigned char* row = dW + (size_t)(lo + i) * row_bytes;
    if (row_bytes % 16 == 0) {
      for (size_t c = lane * 16; c < row_bytes; c += 512)
        *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
    } else {
      for (size_t c = lane * 2; c < row_bytes; c += 64)
        *reinterpret_cast<unsigned short*>(row + c) = 0;
    }
  }
}

// dst = scale·acc, or dst + scale·acc.
template <typename T, int VEC>
__device__ __forceinline__ void put(T* dst, const float* acc, float scale, bool add) {
  float v[VEC];
  if (add) {
    using Raw = typename Vec<T, VEC>::Raw;
    Vec<T, VEC>::widen(__ldcg(reinterpret_cast<const Raw*>(dst)), v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = fmaf(scale, acc[e], v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = scale * acc[e];
  }
  Vec<T, VEC>::st(dst, v);
}

// Pieces of P places of the sorted list, a group of TPR threads each (gridDim.y
// blocks of TPR vectors cover a row).
template <typename T, int VEC, int TPR>
__global__ void __launch_bounds__(kThreads, kSumPerSm)
embed_sum_kernel(const int* first, const int* order, const int* sid, const T* __restrict__ dY,
                 T* dW, float* __restrict__ part, int V, int D, int P, float scale, int add) {
  constexpr int kGroups = kThreads / TPR;
  using Vc = Vec<T, VEC>;
  const int c = (blockIdx.y * TPR + threadIdx.x % TPR) * VEC;
  const bool in = c < D;
  pdl_wait();
  const int piece = blockIdx.x * kGroups + threadIdx.x / TPR;
  const int total = __ldcg(first + V);
  const long long q0 = (long long)piece * P;
  if (q0 >= total) return;
  int p0 = (int)q0, p1 = (int)min((long long)total, q0 + P);
  // Runs of the ids at both ends of the piece.  A short one that starts ahead is
  // the piece ahead's, one that goes on behind is taken to its end here; of a long
  // one the places of this piece.
  const int ida = __ldcg(sid + p0), idb = __ldcg(sid + p1 - 1);
  const int a0 = __ldcg(first + ida), a1 = __ldcg(first + ida + 1);
  const int b0 = __ldcg(first + idb), b1 = __ldcg(first + idb + 1);
  const bool a_part = a0 < p0 && a1 - a0 > kLong, b_part = b1 > p1 && b1 - b0 > kLong;
  if (a0 < p0 && !a_part) p0 = a1;
  if (b1 > p1 && !b_part) p1 = b1;
  if (p0 >= p1) return;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  int cur = __ldcg(sid + p0);
  // The run of `cur` ends here (or at the piece's end).
  auto flush = [&] {
    if (in) {
      const bool ahead = a_part && cur == ida;
      if (!ahead && !(b_part && cur == idb)) {
        put<T, VEC>(dW + (size_t)cur * D + c, acc, scale, add);
      } else {
        // (A piece's first partial row, or that of a run that starts in it.)
        float* q = part + ((size_t)piece * 2 + !ahead) * D + c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) q[e] = acc[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  };
  constexpr int U = 8;                          // rows on their way at once
  for (int p = p0; p < p1; p += U) {
    typename Vc::Raw raw[U];
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = min(p + u, p1 - 1);
      id[u] = __ldcg(sid + q);
      if (in) raw[u] = Vc::ldr(dY + (size_t)__ldcg(order + q) * D + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p + u >= p1) break;
      if (id[u] != cur) {
        flush();
        cur = id[u];
      }
      float v[VEC];
      if (in) {
        Vc::widen(raw[u], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += v[e];
      }
    }
  }
  flush();
}

// The partial rows of the long runs that go over a piece's end: one in each piece
// they touch.  A CTA looks at kLook pieces, a lane each, for long runs that start in them,
// and joins those one after another: its warps add every so-many-th partial row
// each, the warps' sums in order then.  (A thread adding a column's partial rows one
// after another: 38 us for 16384 tokens, 66 pieces of the most frequent id.)
constexpr int kJoinWarps = kThreads / 32;
constexpr int kLook = 8;                // pieces a CTA looks at
template <typename T>
__global__ void __launch_bounds__(kThreads)
embed_join_kernel(const int* first, const int* sid, const float* part, T* dW, int V, int D, int P,
                  float scale, int add) {
  __shared__ float red[kJoinWarps][4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  const int total = __ldcg(first + V), lo = blockIdx.y * 128;
  const int piece = blockIdx.x * kLook + lane;
  const long long q0 = (long long)piece * P;
  int v = -1, last = 0;
  if (lane < kLook && q0 + P < total) {
    v = __ldcg(sid + q0 + P - 1);
    const int a = __ldcg(first + v), b = __ldcg(first + v + 1);
    if (a < (int)q0 || b <= (int)q0 + P || b - a <= kLong) v = -1;
    last = (b - 1) / P;
  }
  unsigned left = __ballot_sync(0xffffffffu, v >= 0);
  while (left) {
    const int j = __ffs(left) - 1;
    left &= left - 1;
    const int id = __shfl_sync(0xffffffffu, v, j), to = __shfl_sync(0xffffffffu, last, j);
    const int from = blockIdx.x * kLook + j;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = from + warp; i <= to; i += kJoinWarps) {
      const float* q = part + ((size_t)i * 2 + (i == from)) * D + lo + lane;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (lo + 32 * e + lane < D) acc[e] += __ldcg(q + 32 * e);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][e][lane] = acc[e];
    __syncthreads();
    const int e = warp, c = lo + 32 * e + lane;
    if (e < 4 && c < D) {
      float s = red[0][e][lane];
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) s += red[w][e][lane];
      put<T, 1>(dW + (size_t)id * D + c, &s, scale, add);
    }
    __syncthreads();
  }
}

// Places of a piece: one wave of the summing CTAs (`slots` groups of threads), at
// most 1024 pieces, so that a run of them all is joined in a bounded time, and at
// least kLong places, so that a short run lies in two pieces at most.  (With runs as
// long as a piece taken whole the pieces differed by a factor of two: 77 us instead
// of 66 for 65536 rows of 1024 fp32.)
constexpr int kMaxPieces = 1024;
int piece_length(int tokens, int slots) {
  const int n = slots < 1 ? 1 : slots < kMaxPieces ? slots : kMaxPieces;
  const int p = (tokens + n - 1) / n;
  return p < kLong ? kLong : p;
}

// Tokens of a block of the sort's first step: a thread each, more where there would
// be more than kBlocks of them.
int block_tokens(int tokens) {
  const int m = (tokens + kBlocks * kSortThreads - 1) / (kBlocks * kSortThreads);
  return (m < 1 ? 1 : m) * kSortThreads;
}

// Ids of a sorting CTA: an equal share of the vocabulary, at most kSortRange.
int sort_range(int V, int sms) {
  const int r = (V + sms - 1) / sms;
  return r < 32 ? 32 : r > kSortRange ? kSortRange : r;
}

template <typename T, int VEC, int TPR>
cudaError_t sums(const EmbedCfg& c, const EmbedArgs& a, int D, int sms, cudaStream_t st) {
  const int groups = kThreads / TPR;
  const int cols = (D / VEC + TPR - 1) / TPR;
  const int P = piece_length(a.tokens, kSumPerSm * sms * groups / cols);
  const int pieces = (a.tokens + P - 1) / P, ctas = (pieces + groups - 1) / groups;
  cudaError_t e = launch_dependent(
      embed_sum_kernel<T, VEC, TPR>, dim3(ctas, cols), dim3(kThreads), 0, st,
      (const int*)c.first, (const int*)c.order, (const int*)c.sid, static_cast<const T*>(a.x),
      static_cast<T*>(a.y), c.part, c.V, D, P, c.scale, a.add);
  if (e != cudaSuccess || pieces < 2) return e;
  return launch_dependent(embed_join_kernel<T>,
                          dim3((pieces + kLook - 1) / kLook, (D + 127) / 128),
                          dim3(kThreads), 0, st,
                          (const int*)c.first, (const int*)c.sid, (const float*)c.part,
                          static_cast<T*>(a.y), c.V, D, P, c.scale, a.add);
}

template <typename T, int VEC>
cudaError_t run(const EmbedCfg& c, const EmbedArgs& a, int D, bool backward, unsigned int* status,
                int sms, cudaStream_t st) {
  const int nv = D / VEC;
  if (!backward) {
    const int per = nv >= kLookup ? 1 : kLookup / nv;
    const int need = (a.tokens + per - 1) / per, most = kFwdPerSm * sms;
    auto kernel = c.scale == 1.f ? embed_fwd_kernel<T, VEC, true> : embed_fwd_kernel<T, VEC, false>;
    kernel<<<need < most ? need : most, kThreads, 0, st>>>(
        a.ids, static_cast<const T*>(a.x), static_cast<T*>(a.y), a.tokens, c.V, D, per, c.scale,
        status);
    return cudaGetLastError();
  }
  const int per = block_tokens(a.tokens), blocks = (a.tokens + per - 1) / per;
  const int ranges = (c.V + c.range - 1) / c.range;
  embed_split_kernel<<<blocks, kSortThreads, (size_t)kSortWarps * ranges * sizeof(int), st>>>(
      a.ids, a.tokens, c.V, per, ranges,
      (unsigned)(((1ull << 32) + c.range - 1) / c.range), c.tok, c.key, c.off, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(embed_sort_kernel, dim3(ranges), dim3(kSortThreads),
                       (size_t)kSortWarps * c.range * sizeof(int), st, (const int*)c.tok,
                       (const int*)c.key, (const int*)c.off, blocks, per, c.V, c.range, c.first,
                       c.order, c.sid, a.add ? nullptr : static_cast<unsigned char*>(a.y),
                       (size_t)D * sizeof(T));
  if (e != cudaSuccess) return e;
  if (nv <= 8) return sums<T, VEC, 8>(c, a, D, sms, st);
  if (nv <= 32) return sums<T, VEC, 32>(c, a, D, sms, st);
  if (nv <= 64) return sums<T, VEC, 64>(c, a, D, sms, st);
  if (nv <= 128) return sums<T, VEC, 128>(c, a, D, sms, st);
  return sums<T, VEC, 256>(c, a, D, sms, st);
}

template <typename T, int FULL>
cudaError_t by_width(const EmbedCfg& c, const EmbedArgs& a, int D, bool backward,
                     unsigned int* status, int sms, cudaStream_t st) {
  // The widest vector that divides the rows keeps every row start aligned.
  if (D % FULL == 0) return run<T, FULL>(c, a, D, backward, status, sms, st);
  if (D % 2 == 0) return run<T, 2>(c, a, D, backward, status, sms, st);
  return run<T, 1>(c, a, D, backward, status, sms, st);
}

}  // namespace

int embed_range(int V, int sms) { return sort_range(V, sms); }

size_t embed_part_count(int max_tokens, int D) {
  // (Pieces have kLong places at least.)
  const size_t most = ((size_t)max_tokens + kLong - 1) / kLong;
  return (most < kMaxPieces ? most : kMaxPieces) * 2 * D;
}
size_t embed_split_count(int max_tokens) {
  // (Fewer tokens have blocks no longer than these.)
  const size_t per = block_tokens(max_tokens);
  return (max_tokens + per - 1) / per * per;
}
size_t embed_off_count(int max_tokens, int V, int sms) {
  const int per = block_tokens(max_tokens), range = sort_range(V, sms);
  const size_t blocks = max_tokens > kSortThreads * kBlocks ? kBlocks
                                                            : (max_tokens + per - 1) / per;
  return blocks * ((V + range - 1) / range + 1);
}

cudaError_t setup_embed() {
  const cudaError_t e = allow_max_smem(embed_split_kernel);
  return e != cudaSuccess ? e : allow_max_smem(embed_sort_kernel);
}

cudaError_t launch_embed(const cat_plan_s* p, const EmbedArgs& a, bool backward) {
  return p->dtype == CAT_BF16
             ? by_width<__nv_bfloat16, 8>(p->em, a, p->D, backward, p->status, p->sms, p->stream)
             : by_width<float, 4>(p->em, a, p->D, backward, p->status, p->sms, p->stream);
}

}  // namespace cat
