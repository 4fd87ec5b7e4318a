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
// Seven products instead of the five of one joint kernel, but dQ needs no
// atomics: results repeat bit for bit, and neither kernel's accumulators
// leave tensor memory.
//
// Roles of a CTA (384 threads, one CTA an SM):
//   - warps 0-7, two warpgroups, one thread a row, each with 64 of a block's
//     128 columns: scores and dP from tensor memory, P and dS back to tensor
//     memory as bf16 pairs, in the columns of its own half;
//   - warp 8: tensor copies;  warp 9: the MMAs S and dP;  warp 10: the MMAs
//     whose A operand is P or dS (accumulators dV, dK or dQ);
//   - warp 11: values that are not finite in blocks that the mask cuts.
// P takes the place of S, dS that of dP.  S has two buffers where 512
// columns allow it (always for dQ; for dK and dV at head width 64), so the
// next scores are computed while this block's probabilities are made.
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

constexpr int kBwdThreads = 384;
constexpr int kHalf = kTile / 2;           // columns of a block that a row's thread takes
constexpr int kStatBytes = 2 * kTile * 4;
constexpr int kNumBars = 32;               // room for every barrier

template <int DP>
struct DkvCfg {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kStages = DP == 64 ? 4 : 2;
  static constexpr int kStageBytes = 2 * kTileBytes + kStatBytes;    // Q, dO, lse and delta
  static constexpr size_t kSmem =
      1024 + 2 * kTileBytes + (size_t)kStages * kStageBytes + kNumBars * 8 + 96;
  static constexpr int kSBufs = DP == 64 ? 2 : 1;
  // Tensor-memory columns.
  static constexpr int s(int b) { return kTile * b; }
  static constexpr int kDp = kTile * kSBufs, kDv = kDp + kTile, kDk = kDv + DP;
};

template <int DP>
struct DqCfg {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kStages = DP == 64 ? 5 : 2;
  static constexpr int kStageBytes = 2 * kTileBytes;                  // K, V
  static constexpr size_t kSmem =
      1024 + 2 * kTileBytes + 2 * kStatBytes + (size_t)kStages * kStageBytes + kNumBars * 8 + 96;
  static constexpr int s(int b) { return kTile * b; }
  static constexpr int kDp = 2 * kTile, kDq = 3 * kTile;
};

// A product of two K-major tiles: D[128 x 128] = A·B^T over DP columns.
template <int DP>
__device__ __forceinline__ void mma_kk(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16_f32(kTile, kTile);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    const int at = ((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
    tc_mma_bf16(d, a + at, b + at, id, k > 0);
  }
}
// D[128 x DP] (+)= A·B, A 128 x 128 in tensor memory (each half of its 128
// columns as 32 packed columns at the start of 64), B a tile of 128 rows.
template <int DP>
__device__ __forceinline__ void mma_tn(uint32_t d, uint32_t a, uint64_t b, uint32_t add) {
  constexpr uint32_t id = idesc_bf16_f32_bmn(kTile, DP);
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
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

// One (slot of 128 rows, head): 8 lanes a row.
__global__ void __launch_bounds__(256)
attn_stats_kernel(const AttnArgs a, int slots) {
  if (blockIdx.x == 0) attn_check_sequences(a);
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
      for (int c = 8 * sub; c < a.dh; c += 64) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(o + c));
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(g + c));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), d);
          d = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), d);
        }
      }
      if (sub == 0) l = a.lse[(long long)h * a.T + tok] * kLog2e;
    }
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
    if (sub == 0) {
      out[r] = l;
      out[kTile + r] = d;
    }
  }
}

// What a block of 128 keys means for dK and dV.
struct DkvWork {
  int nqb, qb0;            // query blocks qb0 .. nqb - 1 of every head see it
  int diag, last;          // those that the mask cuts (-1: none)
  static __device__ __forceinline__ DkvWork of(const AttnBlock& b, int causal) {
    DkvWork w;
    w.nqb = (b.len + kTile - 1) / kTile;
    w.diag = causal ? b.row0 / kTile : -1;
    w.qb0 = causal ? w.diag : 0;
    w.last = b.len % kTile ? w.nqb - 1 : -1;
    return w;
  }
  __device__ __forceinline__ bool is_cut(int qb) const { return qb == diag || qb == last; }
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_tc_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                   const AttnArgs a, int slots) {
  using C = DkvCfg<DP>;
  extern __shared__ unsigned char dkv_raw[];
  const uint32_t raw = smem_addr(dkv_raw);
  unsigned char* sm = dkv_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* kv_sm = sm;                                   // K, V
  unsigned char* ring = sm + 2 * C::kTileBytes;                // [kStages] Q, dO
  unsigned char* stat = ring + C::kStages * 2 * C::kTileBytes; // [kStages] lse, delta
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + C::kStages * kStatBytes);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t kvfull = bar0, dpfull = bar0 + 8, dsready = bar0 + 16, dkdone = bar0 + 24;
  const uint32_t clean = bar0 + 32, done = bar0 + 40;
  auto sfull = [&](int i) { return bar0 + 48 + 8 * i; };
  auto pready = [&](int i) { return bar0 + 64 + 8 * i; };
  auto dvdone = [&](int i) { return bar0 + 80 + 8 * i; };
  const uint32_t cutgo = bar0 + 96, kvempty = bar0 + 104;
  auto full = [&](int st) { return bar0 + 152 + 8 * st; };
  auto empty = [&](int st) { return bar0 + 152 + 8 * (C::kStages + st); };
  const WorkRing ring_w = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 112,
                           smem_addr(tslot + 4)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rep = a.Hq / a.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i)       // dsready, pready: 8 warps; a slot's readers
      mbar_init(bars + i, i == 2 || i == 8 || i == 9 ? 8 : i == 16 || i == 17 ? 11 : 1);
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  uint32_t limit = kMaxPolls;                // 0 once a wait of this thread is lost
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      int st = 0, used = 0, items = 0;
      uint32_t round = 0;
      give_work(a, a.Hkv, 7, false, ring_w, limit, [&](const AttnBlock& b, int g) {
        const DkvWork w = DkvWork::of(b, a.causal);
        if (items > 0) mbar_poll(kvempty, (items - 1) & 1, limit);
        ++items;
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
              unsigned char* q_sm = ring + st * 2 * C::kTileBytes;
              const int row = b.start + qb * kTile;
              mbar_expect_tx(bar, 2 * C::kTileBytes + kStatBytes);
#pragma unroll
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(q_sm + x * (kTile * 128), &tmQ, 64 * x, h, row, bar);
#pragma unroll
              for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(q_sm + C::kTileBytes + x * (kTile * 128), &tmG, 64 * x, h, row, bar);
              bulk_g2s(stat + st * kStatBytes,
                       a.stats + ((long long)h * slots + slot0 + qb) * (2 * kTile), kStatBytes,
                       bar);
            }
            if (++st == C::kStages) {
              st = 0;
              round ^= 1u;
            }
          }
      });
    } else if (warp == 9) {
      const uint64_t kd = sdesc_k128(kv_sm), vd = sdesc_k128(kv_sm + C::kTileBytes);
      const uint64_t qd = sdesc_k128(ring), gd = sdesc_k128(ring + C::kTileBytes);
      int st = 0, sb = 0, items = 0;
      uint32_t round = 0, sround = 0, c = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const DkvWork w = DkvWork::of(slot->b, a.causal);
        mbar_poll(kvfull, items++ & 1, limit);
        const int n = rep * (w.nqb - w.qb0);
        int qb = w.qb0;
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(2 * C::kTileBytes >> 4);
          mbar_poll(full(st), round, limit);
          // S's buffer is free once the dV product has read P from it.
          if (c >= (uint32_t)C::kSBufs) mbar_poll(dvdone(sb), sround ^ 1u, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_kk<DP>(tmem + C::s(sb), kd, qd + at);
            tc_commit(sfull(sb));
          }
          __syncwarp();
          // dP's columns are free once the dK product has read dS from them.
          if (c >= 1) mbar_poll(dkdone, (c - 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_kk<DP>(tmem + C::kDp, vd, gd + at);
            tc_commit(dpfull);
            // A cut block has served as it came: it can be cleaned.
            if (w.is_cut(qb)) tc_commit(cutgo);
            if (j == n - 1) tc_commit(kvempty);
          }
          __syncwarp();
          if (++qb == w.nqb) qb = w.qb0;
          if (++st == C::kStages) {
            st = 0;
            round ^= 1u;
          }
          if (++sb == C::kSBufs) {
            sb = 0;
            sround ^= 1u;
          }
        }
      });
    } else if (warp == 10) {
      const uint64_t qd = sdesc_mn128(ring, kTile * 128);
      const uint64_t gd = sdesc_mn128(ring + C::kTileBytes, kTile * 128);
      int st = 0, sb = 0;
      uint32_t ncut = 0, c = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const DkvWork w = DkvWork::of(slot->b, a.causal);
        const int n = rep * (w.nqb - w.qb0);
        int qb = w.qb0;
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(2 * C::kTileBytes >> 4);
          if (w.is_cut(qb)) mbar_poll(clean, ncut++ & 1, limit);
          // (the first of a block: both warpgroups have read the last one's dV, dK)
          mbar_poll(pready(c & 1), (c >> 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn<DP>(tmem + C::kDv, tmem + C::s(sb), gd + at, j > 0);
            tc_commit(dvdone(sb));
          }
          __syncwarp();
          mbar_poll(dsready, c & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn<DP>(tmem + C::kDk, tmem + C::kDp, qd + at, j > 0);
            mma_tn<DP>(tmem + C::kDk, tmem + C::kDp + kHalf / 2, qd + at, 1);
            tc_commit(dkdone);
            tc_commit(empty(st));
          }
          __syncwarp();
          if (++st == C::kStages) st = 0;
          if (++sb == C::kSBufs) sb = 0;
          if (++qb == w.nqb) qb = w.qb0;
        }
      });
      if (elect_one()) tc_commit(done);
      __syncwarp();
    } else {
      // (the next cut block waits for the products of this one, so the phases
      // of cutgo and clean are taken one by one)
      int st = 0;
      uint32_t ncut = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const DkvWork w = DkvWork::of(slot->b, a.causal);
        const int n = rep * (w.nqb - w.qb0);
        int qb = w.qb0;
        for (int j = 0; j < n; ++j) {
          if (w.is_cut(qb)) {
            mbar_poll(cutgo, ncut++ & 1, limit);
            unsigned char* q_sm = ring + st * 2 * C::kTileBytes;
            const int rows = slot->b.len - qb * kTile;
            clean_tile<DP>(q_sm, rows);
            if (clean_tile<DP>(q_sm + C::kTileBytes, rows) && lane == 0)
              const_cast<WorkSlot*>(slot)->odd = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(clean);
          }
          if (++st == C::kStages) st = 0;
          if (++qb == w.nqb) qb = w.qb0;
        }
      });
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int half = warp >> 2, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const float sc = a.scale * kLog2e;
    const float2 sc2 = make_float2(sc, sc);
    int st = 0, sb = 0;
    uint32_t round = 0, sround = 0, nb = 0;
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int g = slot->h;
    const DkvWork w = DkvWork::of(b, a.causal);
    const int key = b.row0 + 32 * quad + lane;                 // within the sequence
    const int n = rep * (w.nqb - w.qb0);
    int qb = w.qb0;
    for (int j = 0; j < n; ++j, ++nb) {
      const uint32_t ts = tmem + lanes + C::s(sb) + half * kHalf;
      const uint32_t tdp = tmem + lanes + C::kDp + half * kHalf;
      const float4* lse = reinterpret_cast<const float4*>(stat + st * kStatBytes) + half * 16;
      const float4* del = lse + kTile / 4;
      mbar_poll(sfull(sb), sround, limit);
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
      const int q0 = qb * kTile + half * kHalf;
      const int lo = a.causal ? key - q0 : 0, hi = b.len - q0;
      if (cut) {
#pragma unroll
        for (int c = 0; c < kHalf; ++c)
          if (c < lo || c >= hi) p[c] = 0.f;
      }
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
      if (cut) {
        // (0 times a delta or dP that is not finite)
#pragma unroll
        for (int c = 0; c < kHalf; ++c)
          if (c < lo || c >= hi) p[c] = 0.f;
      }
      store_half2(tdp, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dsready);
      if (++st == C::kStages) {
        st = 0;
        round ^= 1u;
      }
      if (++sb == C::kSBufs) {
        sb = 0;
        sround ^= 1u;
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
            for (int i = a.causal ? key : (w.nqb - 1) * kTile; i < b.len; ++i) {
              if (!w.is_cut(i / kTile)) continue;
              const __nv_bfloat16* go = static_cast<const __nv_bfloat16*>(a.dO) +
                                        (((long long)b.start + i) * a.Hq + h) * a.dh;
              for (int c = 0; c < a.dh; ++c) {
                const float x = __bfloat162float(go[c]);
                if (!isfinite(x)) dv[c] = __float2bfloat16_rn(__bfloat162float(dv[c]) + x);
              }
            }
        }
      } else {
        __nv_bfloat16* dk =
            static_cast<__nv_bfloat16*>(a.dk) + tok * a.lddk + (long long)g * a.dh;
        store_row(tmem + lanes + C::kDk, dk, 0, a.dh, a.scale, live,
                  wide_rows(a.dk, a.lddk, a.dh));
      }
      tc_fence_before();                       // read before the next block's products
    }
    });
  }
  if (limit == 0) report(a.status, 0x721);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    // The columns are freed only after every MMA has completed (bounded).
    mbar_poll(done, 0, limit);
    if (limit == 0) report(a.status, 0x722);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_tc_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                  const AttnArgs a, int slots) {
  using C = DqCfg<DP>;
  extern __shared__ unsigned char dq_raw[];
  const uint32_t raw = smem_addr(dq_raw);
  unsigned char* sm = dq_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* q_sm = sm;                                    // Q, dO
  unsigned char* ring = sm + 2 * C::kTileBytes;                // [kStages] K, V
  float* stat = reinterpret_cast<float*>(ring + C::kStages * C::kStageBytes);  // [2] lse, delta
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + 2 * 2 * kTile);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t dpfull = bar0 + 8, dsready = bar0 + 16, dqdone = bar0 + 24;
  const uint32_t qempty = bar0 + 32, done = bar0 + 40;
  // Q, dO, lse and delta have landed (two barriers in turn: the warpgroups may
  // come to a block's after the next block's are there).
  constexpr int kQ1 = 17 + 2 * C::kStages;
  auto qfull = [&](int i) { return bar0 + 8 * (i & 1 ? kQ1 : 0); };
  auto sfull = [&](int i) { return bar0 + 48 + 8 * i; };
  auto cutgo = [&](int i) { return bar0 + 64 + 8 * i; };
  auto clean = [&](int i) { return bar0 + 80 + 8 * i; };
  auto full = [&](int st) { return bar0 + 136 + 8 * st; };
  auto empty = [&](int st) { return bar0 + 136 + 8 * (C::kStages + st); };
  const WorkRing ring_w = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 96,
                           smem_addr(tslot + 4)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Key blocks n - 1 .. 0; only the first of them can be cut by the mask.
  auto blocks = [&](const AttnBlock& b) {
    return a.causal ? b.row0 / kTile + 1 : (b.len + kTile - 1) / kTile;
  };
  auto is_cut = [&](const AttnBlock& b) { return a.causal || b.len % kTile != 0; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i)       // dsready: 8 warps; a slot's readers
      mbar_init(bars + i, i == 2 ? 8 : i == 14 || i == 15 ? 11 : 1);
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  uint32_t limit = kMaxPolls;                // 0 once a wait of this thread is lost
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      int st = 0, used = 0, items = 0;
      uint32_t round = 0;
      give_work(a, a.Hq, 7, true, ring_w, limit, [&](const AttnBlock& b, int h) {
        const int g = h / (a.Hq / a.Hkv);
        if (items > 0) mbar_poll(qempty, (items - 1) & 1, limit);
        if (lane == 0) {
          uint64_t* bar = bars + (items & 1 ? kQ1 : 0);
          mbar_expect_tx(bar, 2 * C::kTileBytes + kStatBytes);
          for (int x = 0; x < C::kBoxes; ++x) {
            tma_load_3d(q_sm + x * (kTile * 128), &tmQ, 64 * x, h, b.start + b.row0, bar);
            tma_load_3d(q_sm + C::kTileBytes + x * (kTile * 128), &tmG, 64 * x, h,
                        b.start + b.row0, bar);
          }
          // (its buffer's last reader has given back the slot of two blocks ago)
          const int slot = (b.start >> 7) + b.seq + b.row0 / kTile;
          bulk_g2s(stat + (items & 1) * 2 * kTile,
                   a.stats + ((long long)h * slots + slot) * (2 * kTile), kStatBytes, bar);
        }
        ++items;
        for (int blk = blocks(b) - 1; blk >= 0; --blk) {
          if (used >= C::kStages) mbar_poll(empty(st), round ^ 1u, limit);
          ++used;
          if (limit == 0) break;
          if (lane == 0) {
            uint64_t* bar = bars + 17 + st;
            unsigned char* k_sm = ring + st * C::kStageBytes;
            const int row = b.start + blk * kTile;
            mbar_expect_tx(bar, C::kStageBytes);
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
    } else if (warp == 9) {
      const uint64_t qd = sdesc_k128(q_sm), gd = sdesc_k128(q_sm + C::kTileBytes);
      const uint64_t kd = sdesc_k128(ring), vd = sdesc_k128(ring + C::kTileBytes);
      int st = 0, items = 0;
      uint32_t round = 0, c = 0, ncut = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const int n = blocks(slot->b);
        const bool cut = is_cut(slot->b);
        mbar_poll(qfull(items), (items >> 1) & 1, limit);
        ++items;
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(C::kStageBytes >> 4);
          mbar_poll(full(st), round, limit);
          // (S's buffer was read before dS of two blocks ago was ready, which the
          // wait below for the product of that dS has shown.)
          if (elect_one()) {
            mma_kk<DP>(tmem + C::s(c & 1), qd, kd + at);
            tc_commit(sfull(c & 1));
            // K of a cut block has served as it came: it can be cleaned.
            if (j == 0 && cut) tc_commit(cutgo(ncut & 1));
          }
          __syncwarp();
          if (j == 0 && cut) ++ncut;
          // dP's columns are free once the dQ product has read dS from them.
          if (c >= 1) mbar_poll(dqdone, (c - 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_kk<DP>(tmem + C::kDp, gd, vd + at);
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
    } else if (warp == 10) {
      const uint64_t kd = sdesc_mn128(ring, kTile * 128);
      int st = 0;
      uint32_t c = 0, ncut = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const int n = blocks(slot->b);
        if (is_cut(slot->b)) {
          mbar_poll(clean(ncut & 1), (ncut >> 1) & 1, limit);
          ++ncut;
        }
        for (int j = 0; j < n; ++j, ++c) {
          const uint64_t at = st * (uint64_t)(C::kStageBytes >> 4);
          // (the first of a block: both warpgroups have read the last one's dQ)
          mbar_poll(dsready, c & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn<DP>(tmem + C::kDq, tmem + C::kDp, kd + at, j > 0);
            mma_tn<DP>(tmem + C::kDq, tmem + C::kDp + kHalf / 2, kd + at, 1);
            tc_commit(dqdone);
            tc_commit(empty(st));
          }
          __syncwarp();
          if (++st == C::kStages) st = 0;
        }
      });
      if (elect_one()) tc_commit(done);
      __syncwarp();
    } else {
      // A cut block's scores may be there before the one before is cleaned, but
      // not those of the block after it: two barriers in turn.
      int first = 0;
      uint32_t ncut = 0;
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        if (is_cut(slot->b)) {
          mbar_poll(cutgo(ncut & 1), (ncut >> 1) & 1, limit);
          clean_tile<DP>(ring + first * C::kStageBytes, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(clean(ncut & 1));
          ++ncut;
        }
        first = (first + blocks(slot->b)) % C::kStages;
      });
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int half = warp >> 2, quad = warp & 3;
    const int lrow = 32 * quad + lane;                         // within the tile
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t tdp = tmem + lanes + C::kDp + half * kHalf;
    const float sc = a.scale * kLog2e;
    const float2 sc2 = make_float2(sc, sc);
    uint32_t nb = 0, items = 0;
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int h = slot->h, n = blocks(b);
    const bool cut0 = is_cut(b);
    const int row = b.row0 + lrow;                             // within the sequence
    mbar_poll(qfull(items), (items >> 1) & 1, limit);
    const float lse = stat[(items & 1) * 2 * kTile + lrow];
    const float del = stat[(items & 1) * 2 * kTile + kTile + lrow];
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
      if (j == 0 && cut0) {
        // The last key this row sees, within the half block.
        const int last = (a.causal ? min(row, b.len - 1) : b.len - 1) - (n - 1) * kTile -
                         half * kHalf;
#pragma unroll
        for (int c = 0; c < kHalf; ++c)
          if (c > last) p[c] = 0.f;
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
      const int c0 = half * (DP / 2);
      store_row(tmem + lanes + C::kDq, dst, c0, min(a.dh, c0 + DP / 2), a.scale, row < b.len,
                wide_rows(a.dq, a.lddq, a.dh));
      tc_fence_before();                       // read before the next block's products
    }
    });
  }
  if (limit == 0) report(a.status, 0x731);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    // The columns are freed only after every MMA has completed (bounded).
    mbar_poll(done, 0, limit);
    if (limit == 0) report(a.status, 0x732);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP>
cudaError_t bwd(const AttnArgs& a, cudaStream_t st) {
  CUtensorMap q, k, v, g;
  const unsigned long long ldo = (unsigned long long)a.Hq * a.dh * 2;
  if (!encode_map_heads_sw128(&q, a.q, a.dh, a.Hq, a.T, (unsigned long long)a.ldq * 2, kTile) ||
      !encode_map_heads_sw128(&k, a.k, a.dh, a.Hkv, a.T, (unsigned long long)a.ldk * 2, kTile) ||
      !encode_map_heads_sw128(&v, a.v, a.dh, a.Hkv, a.T, (unsigned long long)a.ldv * 2, kTile) ||
      !encode_map_heads_sw128(&g, a.dO, a.dh, a.Hq, a.T, ldo, kTile))
    return cudaErrorInvalidValue;
  const int slots = (int)attn_slots(a.T, a.S, 7);
  attn_stats_kernel<<<(unsigned)(slots * a.Hq), 256, 0, st>>>(a, slots);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attn_tc_dkv_kernel<DP><<<(unsigned)(slots * a.Hkv), kBwdThreads, DkvCfg<DP>::kSmem, st>>>(
      q, k, v, g, a, slots);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attn_tc_dq_kernel<DP><<<(unsigned)(slots * a.Hq), kBwdThreads, DqCfg<DP>::kSmem, st>>>(
      q, k, v, g, a, slots);
  return cudaGetLastError();
}

}  // namespace

size_t attn_tc_stats_count(int max_tokens, int max_seqs, int Hq) {
  return (size_t)attn_slots(max_tokens, max_seqs, 7) * Hq * 2 * kTile;
}

cudaError_t setup_attn_tc_bwd() {
  cudaError_t e = allow_max_smem(attn_tc_dkv_kernel<64>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_dkv_kernel<128>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_dq_kernel<64>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc_dq_kernel<128>);
  return e;
}

cudaError_t launch_attn_tc_backward(const AttnArgs& a, cudaStream_t st) {
  return a.dh <= 64 ? bwd<64>(a, st) : bwd<128>(a, st);
}

}  // namespace cat
