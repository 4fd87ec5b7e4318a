// Backward softmax attention over packed sequences on the tensor cores
// (tcgen05), for bf16 rows that start on 16-byte boundaries, head width a
// multiple of 8 up to 128 (padded to 64 or 128 by the copies' zero fill).
//
// Three kernels.  attn_stats_kernel: delta_i = dO_i·o_i beside lse_i·log2 e,
// 128 rows of one head together, so that the next kernel fetches them with
// one bulk copy.  attn_tc_dkv_kernel: dK and dV of 128 keys over the query
// heads and blocks that see them,
//   S^T = K·Q^T, P^T = exp2(S^T·scale·log2 e - lse), dP^T = V·dO^T,
//   dS^T = P^T (dP^T - delta), dV += P^T·dO, dK += dS^T·Q.
// attn_tc_dq_kernel: dQ of 128 queries over the keys they see,
//   S = Q·K^T, P, dP = dO·V^T, dS, dQ += dS·K.
// It starts beside the last CTAs of the kernel ahead, where what the kernels
// ahead write is not visible yet: a CTA's first block makes lse and delta anew
// from the call's own inputs, the later ones wait for the kernels ahead and
// read them from the workspace (a backward of 16 documents 78.0 us, of 8192
// tokens 376; 78.6 and 386 with the wait before the first block too).
// Seven products instead of the five of one joint kernel, but dQ needs no
// atomics: results repeat bit for bit, and neither kernel's accumulators
// leave tensor memory.
//
// Roles of a CTA:
//   - one or two warpgroups, one thread a row, each with 64 columns of a
//     block: scores and dP from tensor memory, P and dS back to tensor memory
//     as bf16 pairs, in the columns of its own half;
//   - four warps more: tensor copies;  the MMAs S and dP;  the MMAs whose A
//     operand is P or dS (accumulators dV, dK or dQ);  values that are not
//     finite in blocks that the mask cuts.
// P takes the place of S, dS that of dP; dQ's S has two buffers, so that the
// next scores are computed while this block's probabilities are made.
//
// At head width 64 a CTA has one warpgroup of rows, works on blocks of 64 of
// the other side and takes half of the 512 columns, so that two CTAs share an
// SM and one's chain of waits runs beside the other's (12 heads, 16 documents
// up to 1024 tokens: all three kernels 86 us; 7.7 more with one CTA of two
// warpgroups; 8192 tokens: 373 and 25 more).  At 128 the accumulators fill the
// columns: two warpgroups, blocks of 128.
//
// Bound by the row warps' chain at 64: a block of 64 takes an SM 1150 clocks
// where the exponentials want 512 and the MMAs 640 (8192 tokens: 1.28 PFLOP/s
// counting nine products, 67 % of the measured bf16 rate), and by the MMAs, at
// the card's power limit, at 128 (16 heads over 4, 8192 + 4095 + 2049 + 1000 + ..
// tokens: 577 us for dK and dV, 498 for dQ, 1.5 PFLOP/s counting the nine products).
// Short documents: 47 us for dK and dV and 37 for dQ, with 2.3 us of each
// block of work between its last product and the next one's first.
//
// P is rounded to bf16 (half a step 2^-8 of each value) as an MMA operand, dS
// to two bf16 terms whose sum is within 2^-16: a row of dS sums to zero, and
// with one term the rounding of its parts made dQ and dK half as uncertain
// again as their own rounding to bf16 does (relative error 0.0026 against
// 0.0017 for a result rounded once).  Everything else is fp32.
//
// A masked pair has p = ds = 0, but 0·inf and 0·NaN would reach dV, dK and dQ
// through the MMA's other operand (dO, Q, K).  In blocks that the mask cuts
// such values are set to zero in shared memory once S and dP have been
// computed from them.  Where a pair is not masked, a value of q or k that is
// not finite has already made p and ds NaN; one of dO alone has not made p
// so, and is added to the dV of the keys its row sees at the end.
#include "../../include/cat.h"
#include "attn_tc.cuh"
#include "cat_internal.h"

namespace cat {

namespace {

constexpr int kHalf = 64;                  // columns of a block that a row's thread takes
constexpr int kNumBars = 40;               // room for every barrier

// NH: warpgroups of a CTA, and blocks of 64·NH on the other side.
template <int NH>
struct Shape {
  static constexpr int kW = kHalf * NH;                  // rows of a block
  static constexpr int kThreads = 128 * (NH + 1);
  static constexpr int kHelp = 4 * NH;                   // first warp of the other roles
  static constexpr int kCols = 256 * NH;                 // tensor-memory columns
  static constexpr int kStatBytes = 2 * kW * 4;          // lse and delta of a block
};

template <int DP, int NH>
struct DkvCfg : Shape<NH> {
  using S = Shape<NH>;
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kBlkBytes = S::kW * DP * 2;
  static constexpr int kStages = DP == 64 ? 4 : 2;       // Q, dO, lse and delta
  static constexpr size_t kSmem =
      1024 + 2 * kTileBytes + (size_t)kStages * (2 * kBlkBytes + S::kStatBytes) + kNumBars * 8 + 96;
  // Tensor-memory columns, after those of S.
  static constexpr int kDp = S::kW, kDv = kDp + S::kW, kDk = kDv + DP;
};

template <int DP, int NH>
struct DqCfg : Shape<NH> {
  using S = Shape<NH>;
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kBlkBytes = S::kW * DP * 2;
  static constexpr int kStages = DP == 64 ? 4 : 2;       // K, V
  static constexpr size_t kSmem = 1024 + 2 * kTileBytes + 2 * (2 * kTile * 4) +
                                  (size_t)kStages * 2 * kBlkBytes + kNumBars * 8 + 96;
  static constexpr int s(int b) { return S::kW * b; }
  static constexpr int kDp = 2 * S::kW, kDq = 3 * S::kW;
};

// D[128 x W] = A·B^T over DP columns: K-major tiles of 128 and W rows.
template <int DP, int W>
__device__ __forceinline__ void mma_kk(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16_f32(kTile, W);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k)
    tc_mma_bf16(d, a + (((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4),
                b + (((k / 4) * (W * 128) + (k % 4) * 32) >> 4), id, k > 0);
}
// D[128 x DP] (+)= A·B, A 128 x W in tensor memory (64 columns each as 32
// packed columns at the start of 64), B a tile of W rows.
template <int DP, int W>
__device__ __forceinline__ void mma_tn(uint32_t d, uint32_t a, uint64_t b, uint32_t add) {
  constexpr uint32_t id = idesc_bf16_f32_bmn(kTile, DP);
#pragma unroll
  for (int k = 0; k < W / 16; ++k)
    tc_mma_bf16_ts(d, a + (k / 4) * kHalf + (k % 4) * 8, b + ((2048 * k) >> 4), id,
                   k > 0 ? 1u : add);
}

// 64 fp32 values to 32 packed columns of this thread's lane.
__device__ __forceinline__ void store_half(uint32_t taddr, const float* v) {
#pragma unroll
  for (int c = 0; c < kHalf; c += 32) {
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = bf16x2(v[c + 2 * i], v[c + 2 * i + 1]);
    tc_st16(taddr + c / 2, p);
  }
  tc_wait_st();
}

// The same as two bf16 terms, the second in the next 32 columns.
__device__ __forceinline__ void store_half2(uint32_t taddr, const float* v) {
#pragma unroll
  for (int c = 0; c < kHalf; c += 32) {
    uint32_t p[16], q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = v[c + 2 * i], b = v[c + 2 * i + 1];
      p[i] = bf16x2(a, b);
      q[i] = bf16x2(a - __uint_as_float(p[i] << 16), b - __uint_as_float(p[i] & 0xffff0000u));
    }
    tc_st16(taddr + c / 2, p);
    tc_st16(taddr + kHalf / 2 + c / 2, q);
  }
  tc_wait_st();
}

// Columns outside lo .. hi - 1 of a half become zero, in chunks of 32.
__device__ __forceinline__ void mask_half(float* p, int lo, int hi) {
#pragma unroll
  for (int c0 = 0; c0 < kHalf; c0 += 32) {
    const int kind = chunk_kind(lo - c0, hi - c0);
    if (kind == kEveryColumn) continue;
    const uint32_t bits = chunk_bits(lo - c0, hi - c0);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!(bits >> c & 1u)) p[c0 + c] = 0.f;
  }
}

// f · accumulator columns c0 .. c1 - 1 of this thread's lane to a bf16 row.
__device__ __forceinline__ void store_row(uint32_t taddr, __nv_bfloat16* dst, int c0, int c1,
                                          float f, bool live, bool wide) {
#pragma unroll 1
  for (int c = c0; c < c1; c += 16) {
    float o[16];
    tc_ld16(taddr + c, o);
    if (live) store16(dst + c, o, f, c1 - c, wide);
  }
}

// d + the products of eight columns of dO and o.
__device__ __forceinline__ float add_products(float d, uint4 x, uint4 y) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), d);
    d = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), d);
  }
  return d;
}
// The sum over the eight lanes that share a row, in each of them.
__device__ __forceinline__ float sum_of_eight(float d) {
#pragma unroll
  for (int w = 4; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
  return d;
}

// delta of 32 rows of one head, of which the first `live` exist, in the warp's
// lanes: from `o` and `g` at the first row (rows ld elements apart), in the
// order of attn_stats_kernel.  All loads are under way at once: what is not
// there reads the last row or the first column instead.  (Not inlined: it would
// take registers from the loop behind it.)
template <int DP>
__device__ __noinline__ float warp_delta(const __nv_bfloat16* o, const __nv_bfloat16* g,
                                         long long ld, int live, int dh) {
  const int lane = threadIdx.x & 31;
  if (live <= 0) return 0.f;
  float part[8], del = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) part[i] = 0.f;
#pragma unroll
  for (int k = 0; k < DP / 64; ++k) {
    const int c = 64 * k + 8 * (lane & 7);
    const bool in = c < dh;
    uint4 x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long at = min(4 * i + (lane >> 3), live - 1) * ld + (in ? c : 0);
      x[i] = __ldg(reinterpret_cast<const uint4*>(o + at));
      y[i] = __ldg(reinterpret_cast<const uint4*>(g + at));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in) part[i] = add_products(part[i], x[i], y[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __shfl_sync(0xffffffffu, sum_of_eight(part[i]), 8 * (lane & 3));
    if (lane >> 2 == i) del = d;
  }
  return lane < live ? del : 0.f;
}

// One (slot of 128 rows, head): 8 lanes a row.
__global__ void __launch_bounds__(256)
attn_stats_kernel(const AttnArgs a, int slots) {
  pdl_trigger();
  if (blockIdx.x == 0) attn_check_sequences(a, threadIdx.x, 256);
  const int slot = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
  AttnBlock b;
  if (!attn_find_block(a, slot, 7, &b)) return;
  float* out = a.stats + ((long long)h * slots + slot) * (2 * kTile);
  const int sub = threadIdx.x & 7;
#pragma unroll
  for (int r0 = 0; r0 < kTile; r0 += 32) {
    const int r = r0 + (threadIdx.x >> 3), row = b.row0 + r;
    float d = 0.f, l = 0.f;
    if (row < b.len) {
      const long long tok = (long long)b.start + row;
      const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(a.o) + (tok * a.Hq + h) * a.dh;
      const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.dO) + (tok * a.Hq + h) * a.dh;
      for (int c = 8 * sub; c < a.dh; c += 64)
        d = add_products(d, __ldg(reinterpret_cast<const uint4*>(o + c)),
                         __ldg(reinterpret_cast<const uint4*>(g + c)));
      if (sub == 0) l = a.lse[(long long)h * a.T + tok] * kLog2e;
    }
    d = sum_of_eight(d);
    if (sub == 0) {
      out[r] = l;
      out[kTile + r] = d;
    }
  }
}

// What a tile of 128 keys means for dK and dV, in query blocks of W rows.
template <int W>
struct DkvWork {
  int nqb, qb0;            // query blocks qb0 .. nqb - 1 of every head see it
  int diag, last;          // cut by the mask: those below diag, and last (-1: none)
  static __device__ __forceinline__ DkvWork of(const AttnBlock& b, int causal) {
    DkvWork w;
    w.nqb = (b.len + W - 1) / W;
    w.qb0 = causal ? b.row0 / W : 0;
    w.diag = causal ? w.qb0 + kTile / W : -1;
    w.last = b.len % W ? w.nqb - 1 : -1;
    return w;
  }
  __device__ __forceinline__ bool is_cut(int qb) const { return qb < diag || qb == last; }
};

template <int DP, int NH>
__global__ void __launch_bounds__(Shape<NH>::kThreads, NH == 2 ? 1 : 2)
attn_tc_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                   const AttnArgs a, int slots) {
  using C = DkvCfg<DP, NH>;
  constexpr int kHelp = C::kHelp, W = C::kW;
  extern __shared__ unsigned char dkv_raw[];
  const uint32_t raw = smem_addr(dkv_raw);
  unsigned char* sm = dkv_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* kv_sm = sm;                                   // K, V
  unsigned char* ring = sm + 2 * C::kTileBytes;                // [kStages] Q, dO
  unsigned char* stat = ring + C::kStages * 2 * C::kBlkBytes;  // [kStages] lse, delta
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + C::kStages * C::kStatBytes);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t kvfull = bar0, dpfull = bar0 + 8, dsready = bar0 + 16, dkdone = bar0 + 24;
  const uint32_t done = bar0 + 40, sdone = bar0 + 32;           // all of either MMA warp's
  const uint32_t sfull = bar0 + 48, dvdone = bar0 + 80;
  auto pready = [&](int i) { return bar0 + 64 + 8 * i; };
  const uint32_t kvempty = bar0 + 104;
  auto full = [&](int st) { return bar0 + 152 + 8 * st; };
  auto empty = [&](int st) { return bar0 + 152 + 8 * (C::kStages + st); };
  // A stage's blocks have been looked through; S and dP have been made of them.
  auto clean = [&](int st) { return bar0 + 152 + 8 * (2 * C::kStages + st); };
  auto used_up = [&](int st) { return bar0 + 152 + 8 * (3 * C::kStages + st); };
  const WorkRing ring_w = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 112,
                           smem_addr(tslot + 4)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rep = a.Hq / a.Hkv;

  if (threadIdx.x == 0) {
    // dsready, pready; a slot's readers; empty: the products and the look
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i == 2 || i == 8 || i == 9 ? 4 * NH
                          : i == 16 || i == 17 ? 4 * NH + 3
                          : i >= 19 + C::kStages && i < 19 + 2 * C::kStages ? 2
                          : 1);
    mbar_fence_init();
  }
  if (warp == kHelp + 1) tmem_alloc(tslot, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  uint32_t limit = kMaxPolls;                // 0 once a wait of this thread is lost
  if (warp >= kHelp) {
    // (registers: 2·208 + 88 = 3·168 and 208 + 48 = 2·128, the launch's own)
    if (NH == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kHelp) {
      // The kernel ahead made lse and delta.  The next one may start from here
      // on: its first blocks read nothing that either of these two writes.
      pdl_wait();
      if (lane == 0) pdl_trigger();
      int st = 0, used = 0, items = 0;
      uint32_t round = 0;
      give_work(a, a.Hkv, 7, false, ring_w, limit, [&](const AttnBlock& b, int g, WorkSlot*) {
        const DkvWork<W> w = DkvWork<W>::of(b, a.causal);
        if (items > 0) mbar_poll(kvempty, (items - 1) & 1, limit);
        ++items;
        if (limit == 0) return;
        if (lane == 0) {
          mbar_expect_tx(bars, 2 * C::kTileBytes);
          for (int x = 0; x < C::kBoxes; ++x) {
            tma_load_3d(kv_sm + x * (kTile * 128), &tmK, 64 * x, g, b.start + b.row0, bars);
            tma_load_3d(kv_sm + C::kTileBytes + x * (kTile * 128), &tmV, 64 * x, g,
                        b.start + b.row0, bars);
          }
        }
        const int slot0 = (b.start >> 7) + b.seq;
        for (int h = g * rep; h < (g + 1) * rep; ++h)
          for (int qb = w.qb0; qb < w.nqb; ++qb) {
            if (used >= C::kStages) mbar_poll(empty(st), round ^ 1u, limit);
            ++used;
            if (limit == 0) return;
            if (lane == 0) {
              uint64_t* bar = bars + 19 + st;
              unsigned char* q_sm = ring + st * 2 * C::kBlkBytes;
              const int row = b.start + qb * W;
              mbar_expect_tx(bar, 2 * C::kBlkBytes + C::kStatBytes);
#pragma unroll
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(q_sm + x * (W * 128), &tmQ, 64 * x, h, row, bar);
#pragma unroll
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(q_sm + C::kBlkBytes + x * (W * 128), &tmG, 64 * x, h, row, bar);
              const float* src = a.stats +
                                 ((long long)h * slots + slot0 + qb * W / kTile) * (2 * kTile) +
                                 qb * W % kTile;
              bulk_g2s(stat + st * C::kStatBytes, src, W * 4, bar);
              bulk_g2s(stat + st * C::kStatBytes + W * 4, src + kTile, W * 4, bar);
            }
            if (++st == C::kStages) {
              st = 0;
              round ^= 1u;
            }
          }
      });
    } else if (warp == kHelp + 1) {
      const uint64_t kd = sdesc_k128(kv_sm), vd = sdesc_k128(kv_sm + C::kTileBytes);
      const uint64_t qd = sdesc_k128(ring), gd = sdesc_k128(ring + C::kBlkBytes);
      int st = 0, items = 0;
      uint32_t round = 0, c = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const DkvWork<W> w = DkvWork<W>::of(slot->b, a.causal);
        mbar_poll(kvfull, items++ & 1, limit);
        const int n = rep * (w.nqb - w.qb0);
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(2 * C::kBlkBytes >> 4);
          mbar_poll(full(st), round, limit);
          // S's columns are free once the dV product has read P from them.
          if (c >= 1) mbar_poll(dvdone, (c - 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_kk<DP, W>(tmem, kd, qd + at);
            tc_commit(sfull);
          }
          __syncwarp();
          // dP's columns are free once the dK product has read dS from them.
          if (c >= 1) mbar_poll(dkdone, (c - 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_kk<DP, W>(tmem + C::kDp, vd, gd + at);
            tc_commit(used_up(st));
            tc_commit(dpfull);
            if (j == n - 1) tc_commit(kvempty);
          }
          __syncwarp();
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
        }
      });
      if (elect_one()) tc_commit(sdone);
      __syncwarp();
    } else if (warp == kHelp + 2) {
      const uint64_t qd = sdesc_mn128(ring, W * 128);
      const uint64_t gd = sdesc_mn128(ring + C::kBlkBytes, W * 128);
      int st = 0;
      uint32_t round = 0, c = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const DkvWork<W> w = DkvWork<W>::of(slot->b, a.causal);
        const int n = rep * (w.nqb - w.qb0);
        int qb = w.qb0;
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(2 * C::kBlkBytes >> 4);
          if (w.is_cut(qb)) mbar_poll(clean(st), round, limit);
          // (the first of a block: both warpgroups have read the last one's dV, dK)
          mbar_poll(pready(c & 1), (c >> 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn<DP, W>(tmem + C::kDv, tmem, gd + at, j > 0);
            tc_commit(dvdone);
          }
          __syncwarp();
          mbar_poll(dsready, c & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn<DP, W>(tmem + C::kDk, tmem + C::kDp, qd + at, j > 0);
            mma_tn<DP, W>(tmem + C::kDk, tmem + C::kDp + kHalf / 2, qd + at, 1);
            tc_commit(dkdone);
            tc_commit(empty(st));
          }
          __syncwarp();
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
          if (++qb == w.nqb) qb = w.qb0;
        }
      });
      if (elect_one()) tc_commit(done);
      __syncwarp();
    } else {
      // Cut blocks are looked through as they land, ahead of their products;
      // what has to be taken out waits until S and dP have been made of it.
      int st = 0;
      uint32_t round = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const DkvWork<W> w = DkvWork<W>::of(slot->b, a.causal);
        const int n = rep * (w.nqb - w.qb0);
        int qb = w.qb0;
        for (int j = 0; j < n; ++j) {
          mbar_poll(full(st), round, limit);
          if (w.is_cut(qb)) {
            unsigned char* q_sm = ring + st * 2 * C::kBlkBytes;
            const bool q_odd = odd_tile<DP, W>(q_sm), g_odd = odd_tile<DP, W>(q_sm + C::kBlkBytes);
            if (q_odd || g_odd) {
              mbar_poll(used_up(st), round, limit);
              const int rows = slot->b.len - qb * W;
              clean_tile<DP, W>(q_sm, rows);
              if (clean_tile<DP, W>(q_sm + C::kBlkBytes, rows) && lane == 0)
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
          if (++qb == w.nqb) qb = w.qb0;
        }
      });
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int half = NH == 2 ? warp >> 2 : 0, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const float sc = a.scale * kLog2e;
    const float2 sc2 = make_float2(sc, sc);
    int st = 0;
    uint32_t round = 0, nb = 0;
    const uint32_t ts = tmem + lanes + half * kHalf;
    const uint32_t tdp = ts + C::kDp;
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int g = slot->h;
    const DkvWork<W> w = DkvWork<W>::of(b, a.causal);
    const int key = b.row0 + 32 * quad + lane;                 // within the sequence
    const int n = rep * (w.nqb - w.qb0);
    int qb = w.qb0;
    for (int j = 0; j < n; ++j, ++nb) {
      const float4* lse =
          reinterpret_cast<const float4*>(stat + st * C::kStatBytes) + half * 16;
      const float4* del = lse + W / 4;
      mbar_poll(sfull, nb & 1, limit);
      tc_fence_after();
      uint32_t r[kHalf];
      tc_ld32(ts, r);
      tc_ld32(ts + 32, r + 32);
      mbar_poll(full(st), round, limit);       // (lse and delta: long there)
      tc_wait_ld();
      float p[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; c += 4) {
        const float4 l = lse[c / 4];
        float2 x = fma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2,
                        make_float2(-l.x, -l.y));
        float2 y = fma2(make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), sc2,
                        make_float2(-l.z, -l.w));
        p[c] = ex2(x.x);
        p[c + 1] = ex2(x.y);
        p[c + 2] = ex2(y.x);
        p[c + 3] = ex2(y.y);
      }
      // Columns lo .. hi - 1 of the half are queries that see this key.
      const bool cut = w.is_cut(qb);
      const int q0 = qb * W + half * kHalf;
      const int lo = a.causal ? key - q0 : 0, hi = b.len - q0;
      if (cut) mask_half(p, lo, hi);
      store_half(ts, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready(nb & 1));
      mbar_poll(dpfull, nb & 1, limit);
      tc_fence_after();
      tc_ld32(tdp, r);
      tc_ld32(tdp + 32, r + 32);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < kHalf; c += 4) {
        const float4 d = del[c / 4];
        const float2 x = add2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])),
                              make_float2(-d.x, -d.y));
        const float2 y = add2(make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])),
                              make_float2(-d.z, -d.w));
        p[c] *= x.x;
        p[c + 1] *= x.y;
        p[c + 2] *= y.x;
        p[c + 3] *= y.y;
      }
      if (cut) mask_half(p, lo, hi);           // (0 times a delta or dP that is not finite)
      store_half2(tdp, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dsready);
      if (++st == C::kStages) {
        st = 0;
        round ^= 1u;
      }
      if (++qb == w.nqb) qb = w.qb0;
    }
    mbar_poll(dkdone, (nb - 1) & 1, limit);    // the block's last product
    // (rows of a CTA that lost a wait are not written)
    if (__all_sync(0xffffffffu, limit != 0)) {
      tc_fence_after();
      const bool live = key < b.len;
      const long long tok = (long long)b.start + key;
      if (half == 0) {
        __nv_bfloat16* dv =
            static_cast<__nv_bfloat16*>(a.dv) + tok * a.lddv + (long long)g * a.dh;
        store_row(tmem + lanes + C::kDv, dv, 0, a.dh, 1.f, live,
                  wide_rows(a.dv, a.lddv, a.dh));
        if (*reinterpret_cast<const volatile uint32_t*>(&slot->odd) != 0 && live) {
          // What was taken out of the cut blocks of dO, for the keys that its
          // rows see (an infinity or NaN times a positive probability).
          for (int h = g * rep; h < (g + 1) * rep; ++h)
            for (int i = a.causal ? key : (w.nqb - 1) * W; i < b.len; ++i) {
              if (!w.is_cut(i / W)) {          // on to the last block, if that is cut
                if (w.last < 0) break;
                i = w.last * W;
              }
              const __nv_bfloat16* go = static_cast<const __nv_bfloat16*>(a.dO) +
                                        (((long long)b.start + i) * a.Hq + h) * a.dh;
              for (int c = 0; c < a.dh; ++c) {
                const float x = __bfloat162float(go[c]);
                if (!isfinite(x)) dv[c] = __float2bfloat16_rn(__bfloat162float(dv[c]) + x);
              }
            }
        }
      }
      if (half == NH - 1) {
        __nv_bfloat16* dk =
            static_cast<__nv_bfloat16*>(a.dk) + tok * a.lddk + (long long)g * a.dh;
        store_row(tmem + lanes + C::kDk, dk, 0, a.dh, a.scale, live,
                  wide_rows(a.dk, a.lddk, a.dh));
      }
      tc_fence_before();                       // read before the next block's products
    }
    });
  }
  join_roles(a.status, limit, 0x721);
  if (warp == kHelp + 1) {
    // The columns are freed only after every MMA has completed.
    last_wait(done, a.status, 0x722);
    last_wait(sdone, a.status, 0x722);
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int DP, int NH>
__global__ void __launch_bounds__(Shape<NH>::kThreads, NH == 2 ? 1 : 2)
attn_tc_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                  const AttnArgs a, int slots) {
  using C = DqCfg<DP, NH>;
  constexpr int kHelp = C::kHelp, W = C::kW;
  extern __shared__ unsigned char dq_raw[];
  const uint32_t raw = smem_addr(dq_raw);
  unsigned char* sm = dq_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* q_sm = sm;                                    // Q, dO
  unsigned char* ring = sm + 2 * C::kTileBytes;                // [kStages] K, V
  float* stat = reinterpret_cast<float*>(ring + C::kStages * 2 * C::kBlkBytes);  // [2] lse, delta
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + 2 * 2 * kTile);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t dpfull = bar0 + 8, dsready = bar0 + 16, dqdone = bar0 + 24;
  const uint32_t qempty = bar0 + 32;
  const uint32_t done = bar0 + 40, sdone = bar0 + 64;           // all of either MMA warp's
  // Q, dO, lse and delta have landed (two barriers in turn: the warpgroups may
  // come to a block's after the next block's are there).
  constexpr int kQ1 = 17 + 2 * C::kStages;
  auto qfull = [&](int i) { return bar0 + 8 * (i & 1 ? kQ1 : 0); };
  auto sfull = [&](int i) { return bar0 + 48 + 8 * i; };
  auto full = [&](int st) { return bar0 + 136 + 8 * st; };
  auto empty = [&](int st) { return bar0 + 136 + 8 * (C::kStages + st); };
  // A stage's K has been looked through; S has been made of it.
  auto clean = [&](int st) { return bar0 + 8 * (kQ1 + 1) + 8 * st; };
  auto used_up = [&](int st) { return bar0 + 8 * (kQ1 + 1) + 8 * (C::kStages + st); };
  const WorkRing ring_w = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 96,
                           smem_addr(tslot + 4)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Key blocks n - 1 .. 0, of which the mask cuts some row of the first few.
  auto blocks = [&](const AttnBlock& b) {
    return ((a.causal ? min(b.len, b.row0 + kTile) : b.len) + W - 1) / W;
  };
  auto is_cut = [&](const AttnBlock& b, int blk) {
    return (blk + 1) * W > b.len || (a.causal && (blk + 1) * W > b.row0 + 1);
  };

  if (threadIdx.x == 0) {
    // dsready; a slot's readers; empty: the products and the look
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i == 2 ? 4 * NH
                          : i == 14 || i == 15 ? 4 * NH + 3
                          : i >= 17 + C::kStages && i < 17 + 2 * C::kStages ? 2
                          : 1);
    mbar_fence_init();
  }
  if (warp == kHelp + 1) tmem_alloc(tslot, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  uint32_t limit = kMaxPolls;                // 0 once a wait of this thread is lost
  if (warp >= kHelp) {
    // (registers: 2·208 + 88 = 3·168 and 208 + 48 = 2·128, the launch's own)
    if (NH == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kHelp) {
      int st = 0, used = 0, items = 0;
      uint32_t round = 0;
      give_work(a, a.Hq, 7, true, ring_w, limit, [&](const AttnBlock& b, int h, WorkSlot*) {
        const int g = h / (a.Hq / a.Hkv);
        if (items > 0) mbar_poll(qempty, (items - 1) & 1, limit);
        if (limit == 0) return;
        // From here on lse and delta come from the workspace: the kernels ahead,
        // which fill it, are waited for.
        if (items == 1) pdl_wait();
        if (lane == 0) {
          uint64_t* bar = bars + (items & 1 ? kQ1 : 0);
          mbar_expect_tx(bar, 2 * C::kTileBytes + (items > 0 ? 2 * kTile * 4 : 0));
          for (int x = 0; x < C::kBoxes; ++x) {
            tma_load_3d(q_sm + x * (kTile * 128), &tmQ, 64 * x, h, b.start + b.row0, bar);
            tma_load_3d(q_sm + C::kTileBytes + x * (kTile * 128), &tmG, 64 * x, h,
                        b.start + b.row0, bar);
          }
          // (its buffer's last reader has given back the slot of two blocks ago)
          const int slot = (b.start >> 7) + b.seq + b.row0 / kTile;
          if (items > 0)
            bulk_g2s(stat + (items & 1) * 2 * kTile,
                     a.stats + ((long long)h * slots + slot) * (2 * kTile), 2 * kTile * 4, bar);
        }
        ++items;
        for (int blk = blocks(b) - 1; blk >= 0; --blk) {
          if (used >= C::kStages) mbar_poll(empty(st), round ^ 1u, limit);
          ++used;
          if (limit == 0) break;
          if (lane == 0) {
            uint64_t* bar = bars + 17 + st;
            unsigned char* k_sm = ring + st * 2 * C::kBlkBytes;
            const int row = b.start + blk * W;
            mbar_expect_tx(bar, 2 * C::kBlkBytes);
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d(k_sm + x * (W * 128), &tmK, 64 * x, g, row, bar);
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d(k_sm + C::kBlkBytes + x * (W * 128), &tmV, 64 * x, g, row, bar);
          }
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
        }
      });
    } else if (warp == kHelp + 1) {
      const uint64_t qd = sdesc_k128(q_sm), gd = sdesc_k128(q_sm + C::kTileBytes);
      const uint64_t kd = sdesc_k128(ring), vd = sdesc_k128(ring + C::kBlkBytes);
      int st = 0, items = 0;
      uint32_t round = 0, c = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const int n = blocks(slot->b);
        mbar_poll(qfull(items), (items >> 1) & 1, limit);
        ++items;
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(2 * C::kBlkBytes >> 4);
          mbar_poll(full(st), round, limit);
          // (S's buffer was read before dS of two blocks ago was ready, which the
          // wait below for the product of that dS has shown.)
          if (elect_one()) {
            mma_kk<DP, W>(tmem + C::s(c & 1), qd, kd + at);
            tc_commit(used_up(st));
            tc_commit(sfull(c & 1));
          }
          __syncwarp();
          // dP's columns are free once the dQ product has read dS from them.
          if (c >= 1) mbar_poll(dqdone, (c - 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_kk<DP, W>(tmem + C::kDp, gd, vd + at);
            tc_commit(dpfull);
            if (j == n - 1) tc_commit(qempty);
          }
          __syncwarp();
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
        }
      });
      if (elect_one()) tc_commit(sdone);
      __syncwarp();
    } else if (warp == kHelp + 2) {
      const uint64_t kd = sdesc_mn128(ring, W * 128);
      int st = 0;
      uint32_t round = 0, c = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const int n = blocks(slot->b);
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(2 * C::kBlkBytes >> 4);
          if (is_cut(slot->b, n - 1 - j)) mbar_poll(clean(st), round, limit);
          // (the first of a block: both warpgroups have read the last one's dQ)
          mbar_poll(dsready, c & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn<DP, W>(tmem + C::kDq, tmem + C::kDp, kd + at, j > 0);
            mma_tn<DP, W>(tmem + C::kDq, tmem + C::kDp + kHalf / 2, kd + at, 1);
            tc_commit(dqdone);
            tc_commit(empty(st));
          }
          __syncwarp();
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
        }
      });
      if (elect_one()) tc_commit(done);
      __syncwarp();
    } else {
      int st = 0;
      uint32_t round = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        for (int blk = blocks(slot->b) - 1; blk >= 0; --blk) {
          mbar_poll(full(st), round, limit);
          unsigned char* k_sm = ring + st * 2 * C::kBlkBytes;
          if (is_cut(slot->b, blk) && odd_tile<DP, W>(k_sm)) {
            mbar_poll(used_up(st), round, limit);
            clean_tile<DP, W>(k_sm, 0);
            fence_proxy_async_smem();
            __syncwarp();
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
    const int half = NH == 2 ? warp >> 2 : 0, quad = warp & 3;
    const int lrow = 32 * quad + lane;                         // within the tile
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t tdp = tmem + lanes + C::kDp + half * kHalf;
    const float sc = a.scale * kLog2e;
    const float2 sc2 = make_float2(sc, sc);
    uint32_t nb = 0, items = 0;
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int h = slot->h, n = blocks(b);
    const int row = b.row0 + lrow;                             // within the sequence
    float lse, del;
    if (items == 0) {
      const int live = b.len - b.row0 - 32 * quad;
      const long long tok = (long long)b.start + b.row0 + 32 * quad;
      const long long ldo = (long long)a.Hq * a.dh, at = tok * ldo + (long long)h * a.dh;
      lse = lane < live ? a.lse[(long long)h * a.T + tok + lane] * kLog2e : 0.f;
      del = warp_delta<DP>(static_cast<const __nv_bfloat16*>(a.o) + at,
                           static_cast<const __nv_bfloat16*>(a.dO) + at, ldo, live, a.dh);
    } else {
      mbar_poll(qfull(items), (items >> 1) & 1, limit);
      lse = stat[(items & 1) * 2 * kTile + lrow];
      del = stat[(items & 1) * 2 * kTile + kTile + lrow];
    }
    ++items;
    const float2 nl2 = make_float2(-lse, -lse), nd2 = make_float2(-del, -del);
    for (int j = 0; j < n; ++j, ++nb) {
      const uint32_t ts = tmem + lanes + C::s(nb & 1) + half * kHalf;
      mbar_poll(sfull(nb & 1), (nb >> 1) & 1, limit);
      tc_fence_after();
      uint32_t r[kHalf];
      tc_ld32(ts, r);
      tc_ld32(ts + 32, r + 32);
      tc_wait_ld();
      float p[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; c += 2) {
        const float2 x =
            fma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, nl2);
        p[c] = ex2(x.x);
        p[c + 1] = ex2(x.y);
      }
      mbar_poll(dpfull, nb & 1, limit);
      tc_fence_after();
      tc_ld32(tdp, r);
      tc_ld32(tdp + 32, r + 32);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < kHalf; c += 2) {
        const float2 x =
            add2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), nd2);
        p[c] *= x.x;
        p[c + 1] *= x.y;
      }
      if (is_cut(b, n - 1 - j)) {
        // The keys this row sees end before this column of the half block.
        mask_half(p, 0, (a.causal ? min(row + 1, b.len) : b.len) - (n - 1 - j) * W - half * kHalf);
      }
      store_half2(tdp, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dsready);
    }
    mbar_poll(dqdone, (nb - 1) & 1, limit);    // the block's last product
    // (rows of a CTA that lost a wait are not written)
    if (__all_sync(0xffffffffu, limit != 0)) {
      tc_fence_after();
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dq) +
                           ((long long)b.start + row) * a.lddq + (long long)h * a.dh;
      const int c0 = half * (DP / NH);
      store_row(tmem + lanes + C::kDq, dst, c0, min(a.dh, c0 + DP / NH), a.scale, row < b.len,
                wide_rows(a.dq, a.lddq, a.dh));
      tc_fence_before();                       // read before the next block's products
    }
    });
  }
  // The kernel ahead (dK, dV) may still run: this one does not end before it.
  if (threadIdx.x == 0) pdl_wait();
  join_roles(a.status, limit, 0x731);
  if (warp == kHelp + 1) {
    // The columns are freed only after every MMA has completed.
    last_wait(done, a.status, 0x732);
    last_wait(sdone, a.status, 0x732);
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int DP, int NH>
cudaError_t bwd(const AttnArgs& a, cudaStream_t st) {
  constexpr int W = Shape<NH>::kW;
  // Tiles of 128 rows, and blocks of W on the other side.
  CUtensorMap q, k, v, g, qw, kw, vw, gw;
  const unsigned long long ldo = (unsigned long long)a.Hq * a.dh * 2;
  auto map = [&](CUtensorMap* m, const void* p, int heads, unsigned long long bytes, int rows) {
    return encode_map_heads_sw128(m, p, a.dh, heads, a.T, bytes, rows);
  };
  const unsigned long long lq = (unsigned long long)a.ldq * 2, lk = (unsigned long long)a.ldk * 2,
                           lv = (unsigned long long)a.ldv * 2;
  if (!map(&q, a.q, a.Hq, lq, kTile) || !map(&k, a.k, a.Hkv, lk, kTile) ||
      !map(&v, a.v, a.Hkv, lv, kTile) || !map(&g, a.dO, a.Hq, ldo, kTile) ||
      !map(&qw, a.q, a.Hq, lq, W) || !map(&kw, a.k, a.Hkv, lk, W) ||
      !map(&vw, a.v, a.Hkv, lv, W) || !map(&gw, a.dO, a.Hq, ldo, W))
    return cudaErrorInvalidValue;
  const int slots = (int)attn_slots(a.T, a.S, 7);
  attn_stats_kernel<<<(unsigned)(slots * a.Hq), 256, 0, st>>>(a, slots);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(attn_tc_dkv_kernel<DP, NH>, dim3((unsigned)(slots * a.Hkv)),
                       dim3(Shape<NH>::kThreads), DkvCfg<DP, NH>::kSmem, st, qw, k, v, gw, a,
                       slots);
  if (e != cudaSuccess) return e;
  return launch_dependent(attn_tc_dq_kernel<DP, NH>, dim3((unsigned)(slots * a.Hq)),
                          dim3(Shape<NH>::kThreads), DqCfg<DP, NH>::kSmem, st, q, kw, vw, g, a,
                          slots);
}

}  // namespace

size_t attn_tc_stats_count(int max_tokens, int max_seqs, int Hq) {
  return (size_t)attn_slots(max_tokens, max_seqs, 7) * Hq * 2 * kTile;
}

cudaError_t setup_attn_tc_bwd() {
  cudaError_t e = allow_max_smem(attn_tc_dkv_kernel<64, 1>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_dkv_kernel<128, 2>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_dq_kernel<64, 1>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_dq_kernel<128, 2>);
  return e;
}

cudaError_t launch_attn_tc_backward(const AttnArgs& a, cudaStream_t st) {
  if (a.dh > 64) return bwd<128, 2>(a, st);
  return bwd<64, 1>(a, st);
}

}  // namespace cat
