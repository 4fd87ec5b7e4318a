// Forward softmax attention over packed sequences on the tensor cores
// (tcgen05), for bf16 rows that start on 16-byte boundaries, head width a
// multiple of 8 up to 128 (padded to 64 or 128 by the copies' zero fill).
//
// A CTA works on NT tiles of 128 query rows of one head (the MMA's M, one
// tensor-memory lane a row) and walks their keys in blocks of 128, from the
// diagonal (or the sequence's end) down to row 0, in one pass with a running
// maximum and sum.  CTAs are persistent: the next block of work is loaded
// while this one's last products run.  Roles, after NT warpgroups of rows:
//   - a warpgroup a tile, one thread a row: scores from tensor memory to
//     registers, mask, maximum, exponentials, and the probabilities back to
//     tensor memory as bf16 pairs;
//   - one warp finds the work and issues the tensor copies of Q, K and V (ring
//     of key blocks);
//   - a warp a tile issues the MMAs: S = Q·K^T into 128 columns, and O += P·V
//     with P as the tensor-memory operand A;
//   - one warp looks for infinities and NaN in V blocks that the mask cuts
//     (below).
// While one tile's warpgroup works on its scores the tensor core runs the
// other tile's products; with NT = 1 the two tiles are two CTAs on an SM.  At
// head width 64 P has columns of its own and the next block's scores are
// computed while P is still being made; at 128 the 512 columns are full and P
// takes the place of its scores.
//
// No unit is full: 16384 causal tokens of 16 heads over 4 (two such sequences
// and one of 4999) take 928 us, 1.24 PFLOP/s or 65 % of the measured bf16 rate; a
// block takes two tiles 2200 clocks, of which the row warps want 1520 (their
// exponentials, scaling, maxima, sums and packing, measured without any wait)
// and the MMAs and copies alone 1505.  The rest is waits of the roles for one
// another, not told apart yet (each tile has one buffer of scores, so its next
// ones are made only when the last have been read).  Four row warpgroups (two a
// tile) gained nothing.  Short documents (16 up to 1024 tokens, 12 heads) take 21 us
// against 7.5 for their bytes: each CTA has three blocks of work, and the
// first copies, the last products and the rows' stores of each are a chain.
//
// The maximum is followed lazily: while a block raises it by less than 2^8
// the old one stays (probabilities up to 2^8 and their fp32 sum lose nothing
// by it), so O in tensor memory is hardly ever rescaled.
//
// P is rounded to bf16 (half a step 2^-8 of each probability) as the
// MMA's operand; its row sum, the maximum, O and the scores are fp32.
//
// A masked pair has p = 0, but 0·inf and 0·NaN would reach the row through
// the MMA.  So in the one or two blocks of V that the mask cuts, values that
// are not finite are set to zero in shared memory, and, if a row of the
// sequence itself held one, added to the rows that see it at the end.
#include "../../include/cat.h"
#include "attn_tc.cuh"
#include "cat_internal.h"

namespace cat {

namespace {

constexpr int kNumBars = 40;               // room for every barrier
// Average length from which a CTA of head width 64 takes two tiles: they share
// the copies of K and V, but the work comes in larger pieces.  12 heads, causal,
// one tile against two (us): 16 documents of 57 .. 1024 tokens 25.2, 26.9;
// 8 x 1024 24.8, 24.9; 4 x 2048 35.0, 35.1; 4 x 4096 111.3, 103.6; 8192 102.3,
// 100.7; 16384 372.9, 347.3.  (At 128 a tile's tensor memory fills half the SM's
// and two tiles are one CTA.)
constexpr int kLongRows = 4096;
constexpr float kLazy = 8.f;               // log2 of the growth that is let pass

template <int DP, int NT>
struct FwdCfg {
  static constexpr int kThreads = 128 * (NT + 1);
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kStages = DP == 64 && NT == 2 ? 5 : 2;   // K and V of a key block each
  static constexpr size_t kSmem = 1024 + (size_t)(NT + 2 * kStages) * kTileBytes +
                                   kNumBars * 8 + 96;
  static constexpr bool kOwnP = DP == 64;  // P beside the scores, not in their place
  // Tensor-memory columns.
  static constexpr int kCols = 256 * NT;
  static constexpr int s(int t) { return kTile * t; }
  static constexpr int p(int t) { return kOwnP ? NT * kTile + 64 * t : kTile * t; }
  static constexpr int o(int t) { return kOwnP ? NT * (kTile + 64) + 64 * t : 256 + kTile * t; }
};

// What a block of work means for the forward.
struct FwdWork {
  int top[2];              // key blocks of tile t: top[t] - 1 .. 0 (0: the tile has no rows)
  int n;                   // blocks of the CTA: n - 1 .. 0
  int cut;                 // blocks from here on are cut by the mask for some row
  template <int NT>
  static __device__ __forceinline__ FwdWork of(const AttnBlock& b, int causal) {
    FwdWork w;
    const int nblk = (b.len + kTile - 1) / kTile;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int qb = b.row0 / kTile + t;
      w.top[t] = t >= NT || qb >= nblk ? 0 : causal ? qb + 1 : nblk;
    }
    w.n = max(w.top[0], w.top[1]);
    w.cut = causal ? b.row0 / kTile : (b.len % kTile ? nblk - 1 : nblk);
    return w;
  }
};

template <int DP, int NT>
__global__ void __launch_bounds__(FwdCfg<DP, NT>::kThreads, NT == 2 ? 1 : 2)
attn_tc_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const AttnArgs a) {
  using C = FwdCfg<DP, NT>;
  constexpr int kHelp = 4 * NT;              // first warp of the copy and MMA roles
  extern __shared__ unsigned char fa_raw[];
  const uint32_t raw = smem_addr(fa_raw);
  unsigned char* sm = fa_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* q_sm = sm;                                       // [NT][kTileBytes]
  unsigned char* kv_sm = sm + NT * C::kTileBytes;                 // [kStages][K, V][kTileBytes]
  uint64_t* bars = reinterpret_cast<uint64_t*>(kv_sm + 2 * C::kStages * C::kTileBytes);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  // Barriers by address.
  const uint32_t bar0 = smem_addr(bars);
  auto qfull = [&](int t) { return bar0 + 8 * t; };
  auto qempty = [&](int t) { return bar0 + 16 + 8 * t; };   // its last scores are done
  auto sfull = [&](int t) { return bar0 + 32 + 8 * t; };    // scores are in tensor memory
  auto sempty = [&](int t) { return bar0 + 48 + 8 * t; };   // ... and in registers
  auto pfull = [&](int t) { return bar0 + 64 + 8 * t; };    // probabilities in tensor memory
  auto odone = [&](int t) { return bar0 + 80 + 8 * t; };    // P·V is done
  auto done = [&](int t) { return bar0 + 96 + 8 * t; };     // every MMA is done
  auto full = [&](int st) { return bar0 + 152 + 8 * st; };
  auto empty = [&](int st) { return bar0 + 152 + 8 * (C::kStages + st); };
  // The V block of a stage has been looked through, where the mask cuts it.
  auto clean = [&](int st) { return bar0 + 152 + 8 * (2 * C::kStages + st); };
  const WorkRing ring = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 112,
                         smem_addr(tslot + 4)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    // sempty and pfull: a tile's warps; a slot's readers; empty: each tile's MMAs
    // and the look
    for (int i = 0; i < 19 + 3 * C::kStages; ++i)
      mbar_init(bars + i, i >= 6 && i < 10 ? 4
                          : i == 16 || i == 17 ? 4 * NT + NT + 1
                          : i >= 19 + C::kStages && i < 19 + 2 * C::kStages ? NT + 1
                          : 1);
    mbar_fence_init();
  }
  if (warp == kHelp + 1) tmem_alloc(tslot, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // The roles of the last warpgroup hand registers to those that hold a row of
  // scores: 2·208 + 88 = 3·168 and 208 + 48 = 2·128, the launch's own.
  uint32_t limit = kMaxPolls;                // 0 once a wait of this thread is lost
  if (warp >= kHelp) {
    if (NT == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kHelp) {
      int st = 0, used = 0, nq[2] = {0, 0};
      uint32_t round = 0;
      give_work(a, a.Hq, NT == 2 ? 8 : 7, true, ring, limit, [&](const AttnBlock& b, int h, WorkSlot*) {
        const FwdWork w = FwdWork::of<NT>(b, a.causal);
        const int g = h / (a.Hq / a.Hkv);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (w.top[t]) {
            if (nq[t] > 0) mbar_poll(qempty(t), (nq[t] - 1) & 1, limit);
            ++nq[t];
            if (limit == 0) return;
            if (lane == 0) {
              mbar_expect_tx(bars + t, C::kTileBytes);
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(q_sm + t * C::kTileBytes + x * (kTile * 128), &tmQ, 64 * x, h,
                            b.start + b.row0 + t * kTile, bars + t);
            }
          }
        for (int blk = w.n - 1; blk >= 0; --blk) {
          if (used >= C::kStages) mbar_poll(empty(st), round ^ 1u, limit);
          ++used;
          if (limit == 0) break;
          if (lane == 0) {
            uint64_t* bar = bars + 19 + st;
            unsigned char* k_sm = kv_sm + 2 * st * C::kTileBytes;
            const int row = b.start + blk * kTile;
            mbar_expect_tx(bar, 2 * C::kTileBytes);
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d(k_sm + x * (kTile * 128), &tmK, 64 * x, g, row, bar);
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d(k_sm + C::kTileBytes + x * (kTile * 128), &tmV, 64 * x, g, row, bar);
          }
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
        }
      });
    } else if (warp < kHelp + 1 + NT) {
      // MMAs of one tile.  The whole warp follows the waits (so that the loop
      // stays uniform), one lane of it issues.
      const int t = NT == 2 ? warp - kHelp - 1 : 0;
      constexpr uint32_t id_s = idesc_bf16_f32(kTile, kTile);
      constexpr uint32_t id_o = idesc_bf16_f32_bmn(kTile, DP);
      const uint64_t qd = sdesc_k128(q_sm + t * C::kTileBytes), kd = sdesc_k128(kv_sm);
      const uint64_t vd = sdesc_mn128(kv_sm + C::kTileBytes, kTile * 128);
      const uint32_t ts = tmem + C::s(t), tp = tmem + C::p(t), to = tmem + C::o(t);
      constexpr uint64_t kStep = 2 * C::kTileBytes >> 4;       // from stage to stage
      int st = 0;
      uint32_t round = 0;                      // parity of the ring's stage st
      uint32_t c = 0, nq = 0;                  // the tile's blocks and query tiles so far
      auto advance = [&]() {
        if (++st == C::kStages) {
          st = 0;
          round ^= 1u;
        }
      };
      auto scores = [&](bool last) {
        const uint64_t k0 = kd + st * kStep;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const int at = ((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
            tc_mma_bf16(ts, qd + at, k0 + at, id_s, k > 0);
          }
          tc_commit(sfull(t));
          if (last) tc_commit(qempty(t));
        }
        __syncwarp();
      };
      // A block that only the other tile sees.
      auto pass_block = [&]() {
        mbar_poll(full(st), round, limit);
        if (elect_one()) mbar_arrive(empty(st));
        __syncwarp();
        advance();
      };
      take_work(ring, limit, [&](const WorkSlot* slot) {
        const FwdWork w = FwdWork::of<NT>(slot->b, a.causal);
        const int top = w.top[t];
        for (int j = top; j < w.n; ++j) pass_block();
        if (top == 0) return;
        mbar_poll(qfull(t), nq++ & 1, limit);
        mbar_poll(full(st), round, limit);
        if (C::kOwnP && c > 0) mbar_poll(sempty(t), (c - 1) & 1, limit);
        tc_fence_after();
        scores(top == 1);
        for (int blk = top - 1; blk >= 0; --blk, ++c) {
          const uint64_t v0 = vd + st * kStep;
          const uint32_t done_v = empty(st);
          if (blk >= w.cut) mbar_poll(clean(st), round, limit);
          advance();
          if (C::kOwnP && blk > 0) {
            mbar_poll(full(st), round, limit);
            mbar_poll(sempty(t), c & 1, limit);
            tc_fence_after();
            scores(blk == 1);
          }
          mbar_poll(pfull(t), c & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            tc_mma_bf16_ts(to, tp, v0, id_o, blk < top - 1);
#pragma unroll
            for (int k = 1; k < kTile / 16; ++k)
              tc_mma_bf16_ts(to, tp + 8 * k, v0 + ((2048 * k) >> 4), id_o, 1);
            tc_commit(odone(t));
            tc_commit(done_v);
          }
          __syncwarp();
          if (!C::kOwnP && blk > 0) {
            // P took the place of the scores: the next ones follow its product.
            mbar_poll(full(st), round, limit);
            scores(blk == 1);
          }
        }
      });
      if (elect_one()) tc_commit(done(t));
      __syncwarp();
    } else if (warp == kHelp + 3) {
      int st = 0;
      uint32_t round = 0;
      take_work(ring, limit, [&](const WorkSlot* slot) {
        const FwdWork w = FwdWork::of<NT>(slot->b, a.causal);
        for (int blk = w.n - 1; blk >= 0; --blk) {
          mbar_poll(full(st), round, limit);
          if (blk >= w.cut) {
            unsigned char* v_sm = kv_sm + (2 * st + 1) * C::kTileBytes;
            if (odd_tile<DP>(v_sm)) {
              if (clean_tile<DP>(v_sm, slot->b.len - blk * kTile) && lane == 0)
                const_cast<WorkSlot*>(slot)->odd = 1;
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          // Given back here too: were the stage filled again without this warp, it
          // could come to a turn of the ring behind and stay there.
          if (lane == 0) {
            mbar_arrive(clean(st));
            mbar_arrive(empty(st));
          }
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
        }
      });
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = NT == 2 ? warp >> 2 : 0, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t ts = tmem + lanes + C::s(t), tp = tmem + lanes + C::p(t);
    const uint32_t to = tmem + lanes + C::o(t);
    const float sc = a.scale * kLog2e;
    uint32_t nb = 0;                           // the tile's blocks so far
    take_work(ring, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int h = slot->h, g = h / (a.Hq / a.Hkv);
    const FwdWork w = FwdWork::of<NT>(b, a.causal);
    const int row = b.row0 + t * kTile + 32 * quad + lane;     // within the sequence
    // (a row behind the sequence never makes its warp follow: the others' roundings
    // do not depend on what lies there)
    float m = row < b.len ? -INFINITY : INFINITY;
    float2 l2 = make_float2(0.f, 0.f), k2 = l2;      // row sum, in four parts
    for (int blk = w.top[t] - 1, it = 0; blk >= 0; --blk, ++it, ++nb) {
      mbar_poll(sfull(t), nb & 1, limit);
      tc_fence_after();
      uint32_t r[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tc_ld32(ts + c, r + c);
      tc_wait_ld();
      if (C::kOwnP) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty(t));
      }
      int kind[kTile / 32];
#pragma unroll
      for (int x = 0; x < kTile / 32; ++x) kind[x] = kEveryColumn;
      if (blk >= w.cut) {
        // The keys this row sees end before column hi of the block.
        const int hi = (a.causal ? min(row + 1, b.len) : b.len) - blk * kTile;
#pragma unroll
        for (int x = 0; x < kTile / 32; ++x) {
          kind[x] = chunk_kind(0, hi - 32 * x);
          if (kind[x] != kEveryColumn) {
            const uint32_t bits = chunk_bits(0, hi - 32 * x);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(bits >> c & 1u)) r[32 * x + c] = 0xff800000u;
          }
        }
      }
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = fmaxf(__uint_as_float(r[i]), __uint_as_float(r[4 + i]));
#pragma unroll
      for (int c = 8; c < kTile; c += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(r[c + i])), __uint_as_float(r[c + 4 + i]));
      const float top_s = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
      const bool grow = __any_sync(0xffffffffu, top_s > m + kLazy);
      float f = 1.f;
      if (grow) {
        const float nm = fmaxf(m, top_s);
        f = ex2(m - (nm == -INFINITY ? 0.f : nm));
        m = nm;
        l2.x *= f;
        l2.y *= f;
        k2.x *= f;
        k2.y *= f;
      }
      const float base = m == -INFINITY ? 0.f : m;
      const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(-base, -base);
#pragma unroll
      for (int c0 = 0; c0 < kTile; c0 += 32) {
        uint32_t p[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float2 x = fma2(make_float2(__uint_as_float(r[c0 + c]), __uint_as_float(r[c0 + c + 1])),
                          sc2, nb2);
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          if (c & 2)
            l2 = add2(l2, x);
          else
            k2 = add2(k2, x);
          p[c / 2] = bf16x2(x.x, x.y);
        }
        if (c0 == 0) {
          if (it > 0) {
            // The product of the block before has read P and written O.
            mbar_poll(odone(t), (nb - 1) & 1, limit);
            if (grow) {
              tc_fence_after();
#pragma unroll 1
              for (int d = 0; d < DP; d += 16) {
                float o[16];
                tc_ld16(to + d, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f;
                tc_st16(to + d, reinterpret_cast<uint32_t*>(o));
              }
            }
          }
          tc_fence_after();
        }
        tc_st16(tp + c0 / 2, p);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull(t));
    }
    if (w.top[t] > 0) {
      const float l = (l2.x + l2.y) + (k2.x + k2.y);
      mbar_poll(odone(t), (nb - 1) & 1, limit);
      // (rows of a CTA that lost a wait are not written)
      if (__all_sync(0xffffffffu, limit != 0)) {
        tc_fence_after();
        const float inv = 1.f / l;
        const long long tok = (long long)b.start + row;
        const bool live = row < b.len;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                             (tok * a.Hq + h) * (long long)a.dh;
        const bool wide = wide_rows(a.out, (long long)a.Hq * a.dh, a.dh);
        const bool odd = *reinterpret_cast<const volatile uint32_t*>(&slot->odd) != 0;
#pragma unroll 1
        for (int c = 0; c < a.dh; c += 16) {
          float o[16];
          tc_ld16(to + c, o);
          if (odd && live) {
            // What was taken out of the cut blocks of V, for the rows that
            // see it (an infinity or NaN times a positive probability).
            for (int j = w.cut * kTile; j < b.len && j < w.n * kTile; ++j) {
              if (a.causal && j > row) break;
              const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) +
                                       (b.start + (long long)j) * a.ldv + (long long)g * a.dh + c;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (c + i < a.dh) {
                  const float x = __bfloat162float(v[i]);
                  if (!isfinite(x)) o[i] += x;
                }
            }
          }
          if (live) store16(dst + c, o, inv, a.dh - c, wide);
        }
        if (live) a.lse[(long long)h * a.T + tok] = (m + log2f(l)) * kLn2;
        tc_fence_before();                     // O is read before the next block's products
      }
    }
    });
  }
  join_roles(a.status, limit, 0x711);
  if (warp == kHelp + 1) {
    // The columns are freed only after every MMA has completed.
    last_wait(done(0), a.status, 0x712);
    if (NT == 2) last_wait(done(1), a.status, 0x712);
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int DP, int NT>
cudaError_t fwd(const AttnArgs& a, cudaStream_t st) {
  using C = FwdCfg<DP, NT>;
  CUtensorMap q, k, v;
  if (!encode_map_heads_sw128(&q, a.q, a.dh, a.Hq, a.T, (unsigned long long)a.ldq * 2, kTile) ||
      !encode_map_heads_sw128(&k, a.k, a.dh, a.Hkv, a.T, (unsigned long long)a.ldk * 2, kTile) ||
      !encode_map_heads_sw128(&v, a.v, a.dh, a.Hkv, a.T, (unsigned long long)a.ldv * 2, kTile))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(attn_slots(a.T, a.S, NT == 2 ? 8 : 7) * a.Hq);
  attn_tc_fwd_kernel<DP, NT><<<grid, C::kThreads, C::kSmem, st>>>(q, k, v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t setup_attn_tc() {
  cudaError_t e = allow_max_smem(attn_tc_fwd_kernel<64, 1>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_fwd_kernel<64, 2>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_fwd_kernel<128, 2>);
  return e;
}

cudaError_t launch_attn_tc_forward(const AttnArgs& a, cudaStream_t st) {
  if (a.dh > 64) return fwd<128, 2>(a, st);
  return a.T / a.S < kLongRows ? fwd<64, 1>(a, st) : fwd<64, 2>(a, st);
}

}  // namespace cat
