// The products of the cross entropy on the tensor cores (tcgen05), with what
// follows them fused in:
//   LSE  X·Wᵀ, a run of the vocabulary at a time -> maximum and sum of
//        exponentials of each row, and the target's logit;
//   D    X·Wᵀ again, a piece of the vocabulary -> d = g·(exp(l - lse) - [v = t]);
//   DX   d·W over the piece, added to dX in fp32;
//   DW   dᵀ·X over all rows of the list -> the piece's rows of dW.
//
// All four are tiles of 256 x 256 by one pair of CTAs (cta_group::2): each CTA
// holds 128 rows of A and half of B in shared memory, the pair's tensor cores
// read both halves, so that a stage of K = 64 needs 32 KB an SM instead of the
// 48 KB of a tile of one CTA.  What is K in one product is a row in another: an
// operand's rows by K come as one box of 64 columns by 128 rows, its K rows by
// 128 columns as one box of two times 64 columns by 64 rows (a third coordinate
// counts columns by 64), both with 128-byte swizzle, and the matrix descriptors
// say which of the two is K.  Copies of 16 KB matter: with four of 8 KB a stage
// the products waited for copies (tensor pipe 72 % busy, 94 % with two of 16 KB;
// sharing B's copies between two pairs by multicast did not help).
//
// fp32 operands are three bf16 terms each, of whose products the six that matter
// are taken, smallest first; the accumulator, which cuts instead of rounding, is
// read out every two stages of K and added up in registers.  A bf16 sum stays in its
// accumulator for at most 65536 of K (dX's parts are never longer, see xent_shape; dW's
// are read out and added up likewise): what is cut off summands of one sign adds up,
// 0.0004 of the sum at that length, where half a step of the result is 0.004 (all of
// 2^20 tokens in one: 0.0065).
//
// Roles of a CTA: warp 0 issues copies, warp 1 (of the pair's first CTA) the
// MMAs, warp 2 holds the tensor memory (two accumulators of 256 columns), warps
// 4 to 11 read a finished accumulator, four of them its first and four its second
// half of columns, while the next tile's products run.  The pairs are persistent;
// which tiles a pair works on is computed, not handed out: a launch's kinds of
// tiles differ in length, and each pair gets about the same number of K stages.
// Every wait is bounded; a lost one ends its role's loop and is reported.
//
// Measured at 16384 tokens, 50257 ids, width 768, bf16: the forward 597 to 628 us (2.0
// to 2.1 PFLOP/s, the tensor pipe 93 to 95 % busy), d of 12800 ids 201 us (72 %), dW and
// dX of as many beside d of the next 530 us (85 %); 2048 fp32 tokens, 32003 ids, width
// 512: 206, 275 (64 %: d's three terms are written) and 458 us.
#include <cuda_bf16.h>

#include "elem.cuh"
#include "tc.cuh"
#include "xent_mma.cuh"
#include "../../include/cat.h"

namespace cat {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kStages = 5;
constexpr int kBox = 64 * 128;                     // bytes of 64 rows of 64 columns
constexpr int kOperand = 2 * kBox;                 // A's or B's share of a stage
constexpr int kStage = 2 * kOperand;
constexpr int kResult = 32 * 128;                  // a box of results
constexpr int kStaging = 2 * kResult;              // two for each warp
constexpr int kAccCols = 256;
constexpr uint32_t kPolls = 1u << 20;              // of a wait: 4 s (3.8 us each)
constexpr int kChunk = 2;                          // K stages between read-outs (fp32)
constexpr int kLongChunk = 1024;                   // the same (bf16)
constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kEpiWarps * kStaging + 512;
constexpr float kLog2e = 1.4426950408889634f;
enum { LSE = 0, DLOG = 1, DX = 2, DW = 3 };

// ---- pairs of CTAs ----
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Address of the pair's first CTA's copy of a shared-memory variable.
__device__ __forceinline__ uint32_t of_first(uint32_t a) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ void pair_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
               : "memory");
}
// A box into this CTA's shared memory; its bytes are reported to `bar`, which
// may be the pair's first CTA's.
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                          int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                          int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// 64 rows by 128 columns from (row, column) on, the columns by 64: one box, or
// two where the rows of the user's array are not whole blocks of 64.
__device__ __forceinline__ void pair_load_rows(uint32_t dst, const CUtensorMap* map, int col,
                                               int term, int row, int two, uint32_t bar) {
  if (two) {
    pair_load(dst, map, col, term, row, bar);
    pair_load(dst + kBox, map, col + 64, term, row, bar);
  } else {
    pair_load(dst, map, 0, row, col >> 6, term, bar);
  }
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive at both CTAs' `bar` once the MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"((unsigned short)3)
      : "memory");
}

// ---- results ----
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int c0, int c1,
                                          int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void add_box(const CUtensorMap* map, uint32_t src, int c0, int c1,
                                        int c2) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group "
      "[%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void stores_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the last store's box may be written again.
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(x - y).  The difference is taken ahead of the factor: of two logits near each
// other it is exact, while y times log2(e) would be off by half a step of y's size.
__device__ __forceinline__ float exp_less(float x, float y) { return ex2((x - y) * kLog2e); }
// The same of two values at once, two packed instructions as one fma each would be
// (four plain ones cost 1024 tokens' loss half a microsecond of 59).
__device__ __forceinline__ void exp_less(float& x0, float& x1, float y) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tadd.rn.f32x2 a, a, b;\n\t"
      "mov.b64 b, {%3, %3};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(-y), "f"(kLog2e));
  x0 = ex2(x0);
  x1 = ex2(x1);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                            uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// 32 bytes with an L2 policy.
__device__ __forceinline__ void st_global32(void* p, const uint32_t* v, uint64_t policy) {
  asm volatile(
      "st.global.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(p),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "l"(policy)
      : "memory");
}

// One tile of a launch.
struct Tile {
  int kind, m0, n0, N;                             // rows and columns of the result
  int steps;                                       // K stages
  int v0, drow;                                    // its piece's first id, rows of d
  int k0, arow;                                    // DX: first K stage, rows of its slice
  int last;                                        // LSE: the run's last tile
};

// Which tiles this pair works on; the same in all of its threads.
struct Plan {
  int mt, nt, vt;                                  // tiles of rows, of D, of a piece (run)
  int dk, tk, pk;                                  // K stages of D, of the list, of a piece
  int w1, x1, l0, l1;                              // DW and DX (every pairs-th), D tiles
  int pairs, pair;
  int by, rest;                                    // pairs over a row of strided tiles
};

__device__ __forceinline__ int pieces_tiles(const XentMma& a, int piece) {
  const int left = a.V - piece * a.piece;
  return (min(left, a.piece) + kXtN - 1) / kXtN;
}

// (By a warp: a thread's loop over the pairs took 6 us.)
__device__ void make_plan(const XentMma& a, int n, Plan* to) {
  const int lane = threadIdx.x & 31;
  Plan mine, *p = &mine;
  p->pairs = gridDim.x >> 1;
  p->pair = blockIdx.x >> 1;
  p->mt = (n + kXtM - 1) / kXtM;
  p->nt = (a.D + kXtN - 1) / kXtN;
  p->dk = (a.D + kXtK - 1) / kXtK;
  p->tk = (n + kXtK - 1) / kXtK;
  p->w1 = p->x1 = p->l0 = p->l1 = 0;
  p->vt = p->pk = 0;
  if (a.lse) {
    p->vt = ((a.V + kXtN - 1) / kXtN + a.run - 1) / a.run;
    p->by = p->pairs / max(p->mt, 1);
    p->rest = p->pairs % max(p->mt, 1);
    if (lane == 0) *to = mine;
    return;
  }
  p->by = p->pairs / p->nt;
  p->rest = p->pairs % p->nt;
  // Tiles and their lengths in K stages; a tile of D ends in stores that no
  // product of its own hides.
  int nw = 0, nx = 0, nl = 0, cx = 1;
  if (a.dw_piece >= 0) nw = pieces_tiles(a, a.dw_piece) * p->nt;
  if (a.dx_piece >= 0) {
    cx = pieces_tiles(a, a.dx_piece) * (kXtN / kXtK);
    const int slices = xent_slices(a.pairs, p->mt, p->nt, a.piece, a.acc_tiles);
    cx = (cx + slices - 1) / slices;
    nx = p->mt * p->nt * slices;
  }
  p->pk = cx;
  if (a.d_piece >= 0) {
    p->vt = pieces_tiles(a, a.d_piece);
    nl = p->mt * p->vt;
  }
  p->w1 = nw;
  p->x1 = nw + nx;
  // DW's and DX's tiles go round, so that tiles that read the same rows or columns
  // of d run side by side (of tiles one after another a pair read d again from
  // memory for each); of D's each pair takes so many as bring it up to the
  // average.  In integers: pair j's end is pair j + 1's beginning.
  const float cw = (float)max(p->tk, 1), cl = (float)(p->dk + 2);
  const float tl = (nw * cw + (float)nx * cx + nl * cl) / p->pairs;
  auto below = [&](int j, int n) { return n > j ? (n - j - 1) / p->pairs + 1 : 0; };
  auto share = [&](int j) {
    const int w = below(j, nw);
    const float load = w * cw + (float)(below(j, nw + nx) - w) * cx;
    return (long long)(fmaxf(0.f, tl - load) / cl * 65536.f);
  };
  long long before = 0;
  for (int j = lane; j < p->pair; j += 32) before += share(j);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  p->l0 = (int)min((long long)nl, (before + 32768) >> 16);
  p->l1 = p->pair + 1 == p->pairs
              ? nl
              : (int)min((long long)nl, (before + share(p->pair) + 32768) >> 16);
  if (lane == 0) *to = mine;
}

// This pair's tiles, one after another.  A role's next tile costs it a few
// additions: with divisions the MMAs waited for them at every tile.
struct Cursor {
  int i, end, x, y;                                // place in the list of a kind; column, row
  int r;                                           // LSE: tile of the run
  int kind;
  Tile t;

  __device__ __forceinline__ void start(const XentMma& a, const Plan& p) {
    if (a.lse) {
      kind = LSE;
      i = p.pair;
      end = p.mt * p.vt;
      y = p.mt ? i % p.mt : 0;                     // row of tiles, run
      x = p.mt ? i / p.mt : 0;
      r = 0;
    } else {
      kind = DW;
      i = p.pair;
      y = i / p.nt;
      x = i % p.nt;
    }
  }
  __device__ bool next(const XentMma& a, const Plan& p) {
    t.k0 = t.arow = t.v0 = t.drow = 0;
    t.last = 1;
    if (a.lse) {
      if (i >= end) return false;
      t.kind = LSE;
      t.m0 = y * kXtM;
      t.n0 = (x * a.run + r) * kXtN;
      t.N = kXtN;
      t.steps = t.n0 < a.V ? p.dk : 0;             // (the last run may be shorter)
      if (++r == a.run) {
        r = 0;
        i += p.pairs;
        x += p.by;
        y += p.rest;
        if (y >= p.mt) {
          y -= p.mt;
          ++x;
        }
      } else {
        t.last = 0;
      }
      return true;
    }
    if (kind != DLOG && i < p.x1) {
      if (kind == DW && i >= p.w1) {
        kind = DX;
        const int j = i - p.w1, tiles = p.mt * p.nt;
        r = j / tiles;                             // slice
        y = (j - r * tiles) / p.nt;
        x = j - r * tiles - y * p.nt;
      }
      t.kind = kind;
      t.m0 = y * kXtM;
      t.n0 = x * kXtN;
      t.N = a.D - t.n0 > kXtN / 2 ? kXtN : kXtN / 2;
      if (kind == DW) {
        t.v0 = a.dw_piece * a.piece;
        t.drow = (a.dw_piece & 1) * a.rows;
        t.steps = p.tk;
      } else {
        t.v0 = a.dx_piece * a.piece;
        t.drow = (a.dx_piece & 1) * a.rows;
        t.k0 = r * p.pk;
        t.steps = max(0, min(p.pk, pieces_tiles(a, a.dx_piece) * (kXtN / kXtK) - t.k0));
        t.arow = r * p.mt * kXtM;
      }
      i += p.pairs;
      y += p.by;
      x += p.rest;
      if (x >= p.nt) {
        x -= p.nt;
        ++y;
      }
      while (kind == DX && y >= p.mt) {
        y -= p.mt;
        ++r;
      }
      return true;
    }
    if (kind != DLOG) {
      kind = DLOG;
      i = p.l0;
      end = p.l1;
      x = p.mt ? i / p.mt : 0;
      y = p.mt ? i - x * p.mt : 0;
    }
    if (i >= end) return false;
    t.kind = DLOG;
    t.v0 = a.d_piece * a.piece;
    t.drow = (a.d_piece & 1) * a.rows;
    t.m0 = y * kXtM;
    t.n0 = x * kXtN;
    t.steps = p.dk;
    t.N = kXtN;
    ++i;
    if (++y == p.mt) {
      y = 0;
      ++x;
    }
    return true;
  }
};

// The terms of the six products, smallest first.
__device__ __forceinline__ int term_a(int q) { return (0x201100 >> (4 * (5 - q))) & 3; }
__device__ __forceinline__ int term_b(int q) { return (0x021010 >> (4 * (5 - q))) & 3; }

// The stages of a tile in the order of their use: f(first K stage, term of A,
// term of B, how the accumulator goes on: 1 starts anew, 2 is read after it).
template <bool F32, bool SUMS, typename F>
__device__ __forceinline__ void each_stage(int steps, F f) {
  if (!F32) {
    auto first = [](int k) { return SUMS ? k % kLongChunk == 0 : k == 0; };
    for (int k = 0; k < steps; ++k)
      f(k, 0, 0, (first(k) ? 1 : 0) | (k == steps - 1 || (SUMS && first(k + 1)) ? 2 : 0));
  } else {
    for (int k0 = 0; k0 < steps; k0 += kChunk) {
      const int kn = min(kChunk, steps - k0);
      for (int q = 0; q < 6; ++q)
        for (int k = 0; k < kn; ++k)
          f(k0 + k, term_a(q), term_b(q), (q + k == 0 ? 1 : 0) | (q == 5 && k == kn - 1 ? 2 : 0));
    }
  }
}

struct Smem {
  uint32_t stages, staging;                        // addresses
  uint32_t full, empty, tfull, tempty, done;       // barriers, 8 bytes apart
};

template <bool F32>
__device__ void copy_role(const XentMaps& maps, const XentMma& a, const Plan& p, const Smem& s,
                          int direct, uint32_t rank) {
  const CUtensorMap* mx = direct ? &maps.x : &maps.xp;
  const CUtensorMap* mxr = direct ? &maps.xr : &maps.xpr;
  const int two_x = direct && a.D % 64, two_w = a.two_w;
  uint32_t limit = kPolls;
  const uint32_t full0 = of_first(s.full);
  int g = 0, st = 0;
  uint32_t phase = 1;                              // (a fresh barrier's phase ahead is over)
  Cursor cur;
  cur.start(a, p);
  while (limit && cur.next(a, p)) {
    const Tile t = cur.t;
    // This CTA's rows of A and columns of B (a copy of B is always 128 of them,
    // whether the tile has use for all or not).
    const int ar = t.m0 + (int)rank * 128, br = t.n0 + (int)rank * (t.N >> 1);
    each_stage<F32, false>(t.steps, [&](int k, int ta, int tb, int) {
      mbar_poll(s.empty + 8 * st, phase, limit);
      if (!limit) return;
      const uint32_t dst = s.stages + st * kStage, full = full0 + 8 * st;
      if (rank == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                         s.full + 8 * st),
                     "r"(2 * kStage)
                     : "memory");
      const int kk = (t.k0 + k) * kXtK;
      if (t.kind <= DLOG) {
        pair_load(dst, mx, kk, ta, ar, full);
        pair_load(dst + kOperand, &maps.w, kk, tb, t.v0 + br, full);
      } else if (t.kind == DX) {
        pair_load(dst, &maps.d, kk, ta, t.drow + ar, full);
        pair_load_rows(dst + kOperand, &maps.wr, br, tb, t.v0 + kk, two_w, full);
      } else {
        pair_load_rows(dst, &maps.dr, ar, ta, t.drow + kk, 0, full);
        pair_load_rows(dst + kOperand, mxr, br, tb, kk, two_x, full);
      }
      ++g;
      if (++st == kStages) {
        st = 0;
        phase ^= 1;
      }
    });
  }
  if (!limit) {
    // Copies under way land before the pair's memory is given back.
    report(a.status, 0x901);
    if (rank == 0)
      for (int q = g > kStages ? g - kStages : 0; q < g; ++q) {
        uint32_t some = 1u << 16;
        mbar_poll(s.full + 8 * (q % kStages), (q / kStages) & 1, some);
      }
  }
}

template <bool F32, bool SUMS>
__device__ void mma_role(const XentMma& a, const Plan& p, const Smem& s, uint32_t tmem) {
  uint32_t limit = kPolls;
  int st = 0, u = 0;                               // stage; accumulators used
  uint32_t phase = 0;
  const uint64_t base = ((uint64_t)1 << 46) | ((uint64_t)2 << 61) | ((uint64_t)(1024 >> 4) << 32);
  const uint64_t mn = (uint64_t)(kBox >> 4) << 16, km = (uint64_t)1 << 16;
  Cursor cur;
  cur.start(a, p);
  bool more = cur.next(a, p);
  while (limit && more) {
    const Tile t = cur.t;
    more = cur.next(a, p);                         // (while this tile's stages are awaited)
    // Which of the operands' two directions is K: MN-major where it is the rows.
    const uint32_t idesc = idesc_bf16_f32(kXtM, t.N) | (t.kind == DW ? 1u << 15 : 0u) |
                           (t.kind >= DX ? 1u << 16 : 0u);
    each_stage<F32, SUMS>(t.steps, [&](int, int, int, int flags) {
      if (!limit) return;
      const uint32_t b = u & 1;
      if (flags & 1) mbar_poll(s.tempty + 8 * b, ((u >> 1) & 1) ^ 1, limit);
      mbar_poll(s.full + 8 * st, phase, limit);
      if (!limit) return;
      tc_fence_after();
      const uint32_t sa = s.stages + st * kStage, sb = sa + kOperand;
      uint64_t da = base | (t.kind == DW ? mn : km) | ((sa & 0x3FFFFu) >> 4);
      uint64_t db = base | (t.kind >= DX ? mn : km) | ((sb & 0x3FFFFu) >> 4);
      const uint64_t sta = t.kind == DW ? 2048 >> 4 : 32 >> 4;
      const uint64_t stb = t.kind >= DX ? 2048 >> 4 : 32 >> 4;
#pragma unroll
      for (int k = 0; k < kXtK / 16; ++k)
        pair_mma(tmem + b * kAccCols, da + k * sta, db + k * stb, idesc, k > 0 || !(flags & 1));
      pair_commit(s.empty + 8 * st);
      if (++st == kStages) {
        st = 0;
        phase ^= 1;
      }
      if (flags & 2) {
        pair_commit(s.tfull + 8 * b);
        ++u;
      }
    });
  }
  pair_commit(s.done);
  if (!limit) report(a.status, 0x902);
}

// 64 values of a row as 128 bytes (bf16) of the warp's box.
__device__ __forceinline__ void stage_bf16(uint32_t box, int lane, const float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st_shared16(box + lane * 128 + ((j ^ (lane & 7)) << 4), pack2(v[8 * j], v[8 * j + 1]),
                pack2(v[8 * j + 2], v[8 * j + 3]), pack2(v[8 * j + 4], v[8 * j + 5]),
                pack2(v[8 * j + 6], v[8 * j + 7]));
}
// 32 values of a row as 128 bytes (fp32).
__device__ __forceinline__ void stage_f32(uint32_t box, int lane, const float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st_shared16(box + lane * 128 + ((j ^ (lane & 7)) << 4), __float_as_uint(v[4 * j]),
                __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                __float_as_uint(v[4 * j + 3]));
}

// A row's values by a warp, 128 on their way at once: f(value, its place) for each
// that is not finite, in their order, while go_on() (of the whole warp).
template <typename G, typename F>
__device__ __forceinline__ void each_odd(const float* row, int D, G go_on, F f) {
  const int lane = threadIdx.x & 31;
  for (int k0 = 0; k0 < D && go_on(); k0 += 128) {
    float a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      a[u] = k0 + 32 * u + lane < D ? __ldg(row + k0 + 32 * u + lane) : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      for (unsigned at = __ballot_sync(0xffffffffu, !(fabsf(a[u]) < INFINITY)); at && go_on();
           at &= at - 1) {
        const int j = __ffs(at) - 1;
        f(__shfl_sync(0xffffffffu, a[u], j), k0 + 32 * u + j);
      }
  }
}

// Logits that are not finite, again by their definition: an infinity is lost in
// the products of its terms (0 times it, or a difference).  n columns' values of
// each lane's row (v, in local memory); x: the lane's row, w: the first column's.
// Where a row of X or of W holds values that are not finite, the products with those
// alone decide; a sum over all of D is taken, by the warp, one after another, only where
// finite products overflow, or kOdd such values have not decided.  (Such sums for every
// logit: 4 ms a tile of width 512 where X had turned NaN; so 0.15.)  The other roles
// wait meanwhile, for 4096 sums at most: 0.06 s at the largest D, where a wait lasts 4 s
// (kPolls).
constexpr int kOdd = 64;
__device__ __noinline__ void exact_logits(float* v, int n, const float* x, const float* w, int D,
                                          bool live) {
  const unsigned all = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  auto row_of = [&](int src) {
    return reinterpret_cast<const float*>(
        __shfl_sync(all, reinterpret_cast<unsigned long long>(x), src));
  };
  bool wrong = false;
  for (int i = 0; i < n; ++i) wrong = wrong || !(fabsf(v[i]) < INFINITY);
  wrong = wrong && live;
  // Rows of X with such values: 32 columns a step, two of them a lane.
  bool odd = false, full = false;                  // of the lane's row; takes sums
  for (unsigned left = __ballot_sync(all, wrong); left; left &= left - 1) {
    const int src = __ffs(left) - 1;
    float s0 = 0.f, s1 = 0.f;
    int some = 0;
    const float* w0 = w + (size_t)lane * D;
    each_odd(
        row_of(src), D,
        [&] {
          return some < kOdd &&
                 __any_sync(all, (lane < n && s0 == s0) || (lane + 32 < n && s1 == s1));
        },
        [&](float y, int k) {
          ++some;
          if (y != y) {
            s0 = s1 = y;                           // (whatever it meets)
            return;
          }
          if (lane < n) s0 = fmaf(y, __ldg(w0 + k), s0);
          if (lane + 32 < n) s1 = fmaf(y, __ldg(w0 + (size_t)32 * D + k), s1);
        });
    if (!some) continue;
    if (lane == src) {
      odd = true;
      full = some == kOdd;
    }
    for (int i = 0; i < n; ++i) {
      const float s = __shfl_sync(all, i < 32 ? s0 : s1, i & 31);
      if (lane == src) v[i] = s;
    }
  }
  // And rows of W.
  for (int i = 0; i < n; ++i, w += D) {
    bool mine = wrong && (odd ? v[i] == v[i] : !(fabsf(v[i]) < INFINITY));
    if (!__any_sync(all, mine)) continue;
    float s = odd ? v[i] : 0.f;
    int some = 0;
    each_odd(
        w, D, [&] { return some < kOdd && __any_sync(all, mine && s == s); },
        [&](float y, int k) {
          ++some;
          if (mine) s = y != y ? y : fmaf(__ldg(x + k), y, s);
        });
    if (mine && some) v[i] = s;
    mine = mine && s == s && (full || some == kOdd || (!some && !odd));
    for (unsigned left = __ballot_sync(all, mine); left; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const float* row = row_of(src);
      s = 0.f;
      for (int k = lane; k < D; k += 32) s = fmaf(__ldg(row + k), __ldg(w + k), s);
      s = warp_sum(s);
      if (lane == src) v[i] = s;
    }
  }
}

template <bool F32, bool SUMS>
__device__ void result_role(const XentMaps& maps, const XentMma& a, const Plan& p, const Smem& s,
                            uint32_t tmem, int n, uint32_t rank) {
  const int warp = (threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
  const int q = warp & 3, side = warp >> 2;        // tensor-memory lanes, half of the columns
  uint32_t box = s.staging + warp * kStaging;      // the next of the warp's two
  const uint32_t other = 2 * box + kResult;
  const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
  const uint32_t give = of_first(s.tempty);
  uint32_t limit = kPolls;
  int u = 0;
  float mx = -INFINITY, sum = 0.f;                 // LSE: of the run so far
  Cursor cur;
  cur.start(a, p);
  bool more = cur.next(a, p);
  // The other box is free, and holds these values once all lanes have written them.
  auto box_free = [&] {
    box = other - box;
    if (lane == 0) stores_read();
    __syncwarp();
  };
  auto box_full = [&] {
    fence_proxy_async_smem();
    __syncwarp();
  };
  while (limit && more) {
    const Tile t = cur.t;
    more = cur.next(a, p);
    const int chunks = t.N >> 7;                   // of 64 columns, of this half
    const int c0 = t.n0 + side * (t.N >> 1);       // its first column
    const int r0 = t.m0 + (int)rank * 128 + 32 * q, row = r0 + lane;
    const bool live = row < n;
    const int tg = live && t.kind <= DLOG ? a.tgt[row] - t.v0 : -1;
    float2 st = make_float2(0.f, 0.f);
    if (t.kind == DLOG && live) st = a.stat[row];
    float acc[SUMS ? 2 : 1][64];
    int groups = t.steps ? 1 : 0;
    constexpr int kRun = F32 ? kChunk : kLongChunk;
    if (SUMS) groups = (t.steps + kRun - 1) / kRun;
    // Waits for the next accumulator; false if that is lost.
    auto taken = [&] {
      mbar_poll(s.tfull + 8 * (u & 1), (u >> 1) & 1, limit);
      if (!__all_sync(0xffffffffu, limit)) limit = 0;
      if (limit) tc_fence_after();
      return limit != 0;
    };
    auto given = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(give + 8 * (u & 1));
      ++u;
    };
    auto at = [&](int c) {
      return lanes + (uint32_t)((u & 1) * kAccCols + side * (t.N >> 1) + 64 * c);
    };
    auto read64 = [&](int c, float* v) {
      uint32_t r[64];
      tc_ld32(at(c), r);
      tc_ld32(at(c) + 32, r + 32);
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
    };
    if (SUMS) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[SUMS ? c : 0][i] = 0.f;
      for (int g = 0; g < groups && limit; ++g) {
        if (!taken()) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c < chunks) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r[32];
              tc_ld32(at(c) + 32 * h, r);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[SUMS ? c : 0][32 * h + i] += __uint_as_float(r[i]);
            }
          }
        }
        given();
      }
    } else if (groups) {
      taken();
    }
    if (!limit) break;
    // (Sums are in registers, two unrolled chunks; else the code stays small.)
#pragma unroll (SUMS ? 2 : 1)
    for (int c = 0; c < 2; ++c) {
      if (c >= chunks) continue;
      float* v = acc[SUMS ? c : 0];
      if (!SUMS) {
        if (groups) {
          read64(c, v);
          if (c == chunks - 1) given();
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = 0.f;
        }
      }
      const int col = c0 + 64 * c;
      if (t.kind <= DLOG) {
        if (t.steps == 0) continue;                // behind the vocabulary
        const int left = a.V - t.v0 - col;         // ids from this column on
        if (F32) {
          bool fine = true;
#pragma unroll
          for (int i = 0; i < 64; ++i) fine = fine && fabsf(v[i]) < INFINITY;
          if (__any_sync(0xffffffffu, live && !fine)) {
            float apart[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) apart[i] = v[i];
            exact_logits(apart, min(left, 64),
                         static_cast<const float*>(a.x) +
                             (live ? (size_t)a.rows_of[row] * a.D : 0),
                         static_cast<const float*>(a.w) + (size_t)(t.v0 + col) * a.D, a.D, live);
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = apart[i];
          }
        }
        if (left < 64) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= left) v[i] = -INFINITY;
        }
        const int hit = tg - col;
        if (t.kind == LSE) {
          if ((unsigned)hit < 64u) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i == hit) x = v[i];
            a.hit[row] = x;
          }
          float top = mx;
#pragma unroll
          for (int i = 0; i < 64; ++i) top = fmaxf(top, v[i]);
          // (An infinite maximum is no difference to take: exp is 0 or infinite as it is.)
          const float sh = fabsf(top) < INFINITY ? top : 0.f;
          float e0 = 0.f, e1 = 0.f;
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            float x = v[i], y = v[i + 1];
            exp_less(x, y, sh);
            e0 += x;
            e1 += y;
          }
          sum = sum * exp_less(mx, sh) + (e0 + e1);
          mx = top;
          continue;
        }
#pragma unroll
        for (int i = 0; i < 64; i += 2) exp_less(v[i], v[i + 1], st.x);
        if ((unsigned)hit < 64u) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i == hit) v[i] -= 1.f;
        }
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] *= st.y;
        if (!__all_sync(0xffffffffu, live)) {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = live ? v[i] : 0.f;
        }
        // Past shared memory, which the products' operands keep busy: a lane's 64
        // values of its row, 32 bytes at a time, a term after another.  A piece's d is
        // larger than L2: it leaves first, so that the operands stay.
        const uint64_t first_out = policy_evict_first();
        uint32_t* to = static_cast<uint32_t*>(a.d) +
                       ((size_t)(t.drow + row) * (F32 ? 3 : 1) * a.piece + col) / 2;
#pragma unroll
        for (int term = 0; term < (F32 ? 3 : 1); ++term) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float& x = v[16 * j + 2 * i];
              float& y = v[16 * j + 2 * i + 1];
              h[i] = pack2(x, y);
              if (F32 && term < 2) {
                x -= __uint_as_float(h[i] << 16);
                y -= __uint_as_float(h[i] & 0xffff0000u);
              }
            }
            st_global32(to + 8 * j, h, first_out);
          }
          to += a.piece / 2;
        }
      } else if (t.kind == DX) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (col + 32 * h >= a.D || !(groups || a.first)) continue;
          box_free();
          stage_f32(box, lane, v + 32 * h);
          box_full();
          if (lane == 0) {
            if (a.first)
              store_box(&maps.acc, box, col + 32 * h, 0, t.arow + r0);
            else
              add_box(&maps.acc, box, col + 32 * h, 0, t.arow + r0);
            stores_commit();
          }
        }
      } else {
        if (a.factor && groups) {                  // (no tokens: zeros, whatever the factor)
          const float f = __ldg(a.factor);
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] *= f;
        }
        if (a.dw_tma) {
#pragma unroll
          for (int h = 0; h < (F32 ? 2 : 1); ++h) {
            if (col + 32 * h >= a.D) continue;
            box_free();
            if (F32)
              stage_f32(box, lane, v + 32 * h);
            else
              stage_bf16(box, lane, v);
            box_full();
            if (lane == 0) {
              store_box(&maps.dw, box, col + 32 * h, 0, t.v0 + r0);
              stores_commit();
            }
          }
        } else if (t.v0 + row < a.V) {
          const size_t to = (size_t)(t.v0 + row) * a.D + col;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (col + i < a.D) {
              if (F32)
                static_cast<float*>(a.dw)[to + i] = v[i];
              else
                static_cast<__nv_bfloat16*>(a.dw)[to + i] = __float2bfloat16_rn(v[i]);
            }
        }
      }
    }
    if (t.kind == LSE && t.last) {
      const int run = t.n0 / (kXtN * a.run);
      if (live) a.part[(size_t)(2 * run + side) * a.ld + row] = make_float2(mx, sum);
      mx = -INFINITY;
      sum = 0.f;
    }
  }
  if (lane == 0) stores_done();
  __syncwarp();
  if (!limit && lane == 0) report(a.status, 0x903);
}

// SUMS: accumulators are read out and added up in registers (fp32, and bf16 sums that
// are longer than kLongChunk).
template <bool F32, bool SUMS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
xent_mma_kernel(const __grid_constant__ XentMaps maps, const __grid_constant__ XentMma a) {
  extern __shared__ unsigned char raw[];
  __shared__ Plan plan;
  __shared__ uint32_t tslot;
  const uint32_t at = (smem_addr(raw) + 1023u) & ~1023u;
  Smem s;
  s.stages = at;
  s.staging = at + kStages * kStage;
  s.full = s.staging + kEpiWarps * kStaging;
  s.empty = s.full + 8 * kStages;
  s.tfull = s.empty + 8 * kStages;
  s.tempty = s.tfull + 16;
  s.done = s.tempty + 16;
  const uint32_t rank = cta_rank();
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    auto init = [](uint32_t bar, uint32_t count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
    };
    for (int i = 0; i < kStages; ++i) {
      init(s.full + 8 * i, 1);
      init(s.empty + 8 * i, 1);
    }
    for (int b = 0; b < 2; ++b) {
      init(s.tfull + 8 * b, 1);
      init(s.tempty + 8 * b, 2 * kEpiWarps);
    }
    init(s.done, 1);
    mbar_fence_init();
  }
  if (warp == 2) pair_alloc(smem_addr(&tslot), 2 * kAccCols);
  pdl_wait();
  const int n = __ldcg(a.count), direct = __ldcg(a.count + 1);
  if (warp == 3) make_plan(a, n, &plan);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tslot;
  // Sums take 128 registers of a thread that reads results: 224 for those
  // warps, 56 for the others (together the 168 of each that the CTA starts with).
  // Spilled ones would go through the memory that feeds the products.
  if (warp < 4) {
    if (SUMS) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && elect_one()) {
      asm volatile("fence.proxy.async;" ::: "memory");   // (rows that kernels ahead wrote)
      copy_role<F32>(maps, a, plan, s, direct, rank);
    } else if (warp == 1 && rank == 0 && elect_one()) {
      mma_role<F32, SUMS>(a, plan, s, tmem);
    }
  } else {
    if (SUMS) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    result_role<F32, SUMS>(maps, a, plan, s, tmem, n, rank);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    uint32_t limit = kPolls;
    mbar_poll(s.done, 0, limit);
    __syncwarp();
    tc_fence_after();
  }
  __syncthreads();
  cluster_sync();
  if (warp == 2) pair_dealloc(tmem, 2 * kAccCols);
}

}  // namespace

// clusters: pairs of CTAs that the device holds at once.
cudaError_t setup_xent_mma(int dtype, int sms, int* clusters) {
  auto one = [&](auto kernel) {
    cudaError_t e = allow_max_smem(kernel);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms & ~1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg);
    return e == cudaSuccess && *clusters < 1 ? cudaErrorInvalidConfiguration : e;
  };
  if (dtype == CAT_F32) return one(xent_mma_kernel<true, true>);
  const cudaError_t e = one(xent_mma_kernel<false, false>);
  return e != cudaSuccess ? e : allow_max_smem(xent_mma_kernel<false, true>);
}

cudaError_t launch_xent_mma(const XentMaps& maps, const XentMma& a, int dtype, int clusters,
                            long long longest, cudaStream_t st) {
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, dim3(2 * clusters), dim3(kThreads), kSmem, st, maps, a);
  };
  if (dtype == CAT_F32) return go(xent_mma_kernel<true, true>);
  return longest > (long long)kLongChunk * kXtK ? go(xent_mma_kernel<false, true>)
                                                : go(xent_mma_kernel<false, false>);
}

}  // namespace cat
