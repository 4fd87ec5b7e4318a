// Softmax attention over packed sequences on the tensor cores (tcgen05) for
// fp32 storage: the forward for head widths up to 128, the backward up to 64,
// any strides and alignment.
//
// Every operand is split into three bf16 terms, x = x0 + x1 + x2 with
// |x1| <= 2^-8 |x| and |x2| <= 2^-17 |x| (half steps of 8 bits, the second with a
// sign of its own), and no remainder short of underflow: 24 bits in three terms
// of 8.  A product A·B becomes the six products A_i·B_j with i + j <= 2,
// smallest first, into one fp32 accumulator; what is left out, A_1·B_2, A_2·B_1
// and A_2·B_2, is within 2·2^-25 = 2^-24 of |a||b|, half a rounding step of fp32.
// bf16 MMAs at a sixth of their rate are still four times what the FP32 pipe could
// do at best.
//
// The tensor core's fp32 accumulator drops what does not fit instead of
// rounding, always toward zero, so a long chain of MMAs drifts (4·10^-6 of the
// result after 240 of them).  An accumulator therefore holds one block's
// product, four full-size terms; the blocks are added in registers.
//
// A CTA takes 128 rows (the MMA's M, one tensor-memory lane each) and walks
// the other side in blocks of 64 rows.  Roles:
//   - warps 0-3, one thread a row: scores from tensor memory, softmax or its
//     gradient, and the results back as three planes of bf16 pairs (the A
//     operand of the next product);
//   - one warpgroup more (two in the forward at head width 64): load operands,
//     split them and write the planes to shared memory in the 128-byte swizzle
//     the MMA reads; rows outside the sequence and columns beyond the head
//     width become zeros;
//   - one warp issues the MMAs, one finds the work (two more only complete the
//     warpgroup).
//
// Bound by the chain of MMAs (six times 128·64·64 a product, 32 clocks each by
// their operations, about 51 as issued, whether the A operand comes from shared
// or tensor memory) and the row warps, with the splitting beside them.
// Measured, 12 heads of 64: 8192 causal tokens 501 us forward (632 with one
// splitting warpgroup, which took 1800 clocks a block for K and V), 1353 for dK
// and dV (two splitting warpgroups: 1 % faster here, but 10 % slower in short
// sequences for the registers that the second one takes), 882 for dQ; 16
// documents of 57 .. 1024 tokens 102, 243 and 153 us; 64 images of 196 tokens, 6
// heads, 59 us forward (223 us a pass on the FP32 pipe).
//
// Values that are not finite (or too large for bf16) do not split.  A CTA
// that met one, or whose masks could have hidden one, computes its rows again
// at its end by a plain loop over the pairs that count, straight from the
// definition: exact in what is NaN and what is not, and never taken by ordinary
// data (8192 causal tokens, 4 heads, with a NaN in the first key: 50 ms forward
// and 234 ms backward, instead of 0.20 and 0.83).
#include "../../include/cat.h"
#include "attn_tc.cuh"
#include "cat_internal.h"

namespace cat {

namespace {

constexpr int kThreads32 = 384;
constexpr int kB = 64;                     // rows of a block of the other side
constexpr int kNumBars = 32;               // room for every barrier
constexpr float kLazy = 8.f;               // log2 of the maximum's growth that is let pass

template <int DP>
struct Cfg32 {              // (the backward's shared memory holds DP = 64 only)
  static constexpr int kTilePlane = kTile * DP * 2;      // bytes of one plane of 128 rows
  static constexpr int kBlkPlane = kB * DP * 2;          // ... of 64 rows
  static constexpr int kStages = DP == 64 ? 2 : 1;
  // The forward's warpgroups that load and split, and the tiles that each has
  // under way or in work, as loaded (at 128 there is no room left).
  static constexpr int kGroups = DP == 64 ? 2 : 1, kAhead = DP == 64 ? 2 : 0;
  static constexpr int kPieceBytes = kB * DP * 4;
  static constexpr int kFwdThreads = 128 * (2 + kGroups);
  static constexpr size_t kFwdSmem = 1024 + 3 * (size_t)kTilePlane +
                                     kStages * 6 * (size_t)kBlkPlane +
                                     kGroups * kAhead * (size_t)kPieceBytes + kNumBars * 8 + 96;
};
constexpr size_t kBwdSmem32 = 1024 + 6 * (size_t)Cfg32<64>::kTilePlane +
                              Cfg32<64>::kStages * (6 * (size_t)Cfg32<64>::kBlkPlane + 2 * kB * 4) +
                              kNumBars * 8 + 96;

// Two values as three packed bf16 pairs.
__device__ __forceinline__ void split2(float a, float b, uint32_t* p0, uint32_t* p1, uint32_t* p2) {
  const uint32_t h = bf16x2(a, b);
  a -= __uint_as_float(h << 16);
  b -= __uint_as_float(h & 0xffff0000u);
  const uint32_t m = bf16x2(a, b);
  a -= __uint_as_float(m << 16);
  b -= __uint_as_float(m & 0xffff0000u);
  *p0 = h;
  *p1 = m;
  *p2 = bf16x2(a, b);
}

// A thread's share of 64 rows of a [.., dh] fp32 operand: pieces of 8 columns,
// zeros in rows from `rows` and columns from dh on.  By the 128 threads tid.
template <int DP>
struct Piece {
  float x[DP / 16][8];
  __device__ __forceinline__ void fetch(const float* src, long long ld, int rows, int dh, int vec,
                                        int tid) {
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int at = tid + 128 * i, r = at / (DP / 8), c = 8 * (at % (DP / 8));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
      if (r < rows) {
        const float* p = src + (long long)r * ld + c;
        if (vec) {
          if (c < dh) {
            const float4 y = __ldg(reinterpret_cast<const float4*>(p));
            x[i][0] = y.x; x[i][1] = y.y; x[i][2] = y.z; x[i][3] = y.w;
          }
          if (c + 4 < dh) {
            const float4 y = __ldg(reinterpret_cast<const float4*>(p + 4));
            x[i][4] = y.x; x[i][5] = y.y; x[i][6] = y.z; x[i][7] = y.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < dh) x[i][e] = __ldg(p + e);
        }
      }
    }
  }
  // The same by way of shared memory, where a thread writes and later reads
  // pieces of its own: copies that take no registers while they are under way.
  // (`base`: an address in the tensor, for copies of no bytes.)
  static __device__ __forceinline__ void fetch_ahead(uint32_t to, const float* src,
                                                     const float* base, long long ld, int rows,
                                                     int dh, int vec, int tid) {
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int at = tid + 128 * i, r = at / (DP / 8), c = 8 * (at % (DP / 8));
      const uint32_t q = to + 2 * i * 2048 + tid * 16;
      const float* p = src + (long long)r * ld + c;
      if (vec) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const bool in = r < rows && c + e < dh;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q + e * 512),
                       "l"(__cvta_generic_to_global(in ? p + e : base)), "r"(in ? 16 : 0)
                       : "memory");
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool in = r < rows && c + e < dh;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                           q + e / 4 * 2048 + e % 4 * 4),
                       "l"(__cvta_generic_to_global(in ? p + e : base)), "r"(in ? 4 : 0)
                       : "memory");
        }
      }
    }
  }
  __device__ __forceinline__ void take(const unsigned char* from, int tid) {
#pragma unroll
    for (int i = 0; i < 2 * (DP / 16); ++i)
      *reinterpret_cast<float4*>(&x[i / 2][4 * (i % 2)]) =
          *reinterpret_cast<const float4*>(from + i * 2048 + tid * 16);
  }
  // As rows row0 .. row0 + 63 of three bf16 planes of [DP/64][ROWS] 128-byte
  // rows, 128-byte swizzle.  Returns whether a value did not split.
  template <int ROWS>
  __device__ __forceinline__ bool put(unsigned char* dst, int row0, int tid) const {
    constexpr int kPlane = ROWS * DP * 2;
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int at = tid + 128 * i, r = row0 + at / (DP / 8), ch = at % (DP / 8);
      uint32_t w[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        split2(x[i][2 * e], x[i][2 * e + 1], &w[0][e], &w[1][e], &w[2][e]);
        odd |= odd2(w[0][e]);
      }
      unsigned char* q = dst + (ch / 8) * (ROWS * 128) + r * 128 + (((ch % 8) ^ (r & 7)) * 16);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint4*>(q + k * kPlane) =
            make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
    }
    return (odd & 0x80008000u) != 0;
  }
};
// A tile of 128 rows.
template <int DP>
__device__ __forceinline__ bool put_tile(unsigned char* dst, const float* src, long long ld,
                                         int rows, int dh, int vec, int tid) {
  Piece<DP> lo, hi;
  lo.fetch(src, ld, rows, dh, vec, tid);
  if (DP == 64) hi.fetch(src + 64 * ld, ld, rows - 64, dh, vec, tid);
  const bool bad = lo.template put<kTile>(dst, 0, tid);
  if (DP != 64) hi.fetch(src + 64 * ld, ld, rows - 64, dh, vec, tid);
  return hi.template put<kTile>(dst, 64, tid) || bad;
}

// The planes (i, j) with i + j <= 2, smallest products first.
__device__ constexpr int kPi[6] = {0, 2, 1, 0, 1, 0};
__device__ constexpr int kPj[6] = {2, 0, 1, 1, 0, 0};

// D[128 x 64] = A·B^T, both K-major planes in shared memory (128 and 64 rows).
template <int DP>
__device__ __forceinline__ void mma_kk3(uint32_t d, uint64_t a, uint64_t b) {
  using C = Cfg32<DP>;
  constexpr uint32_t id = idesc_bf16_f32(kTile, kB);
#pragma unroll
  for (int x = 0; x < 6; ++x)
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
      tc_mma_bf16(d, a + ((kPi[x] * C::kTilePlane + (k / 4) * (kTile * 128) + (k % 4) * 32) >> 4),
                  b + ((kPj[x] * C::kBlkPlane + (k / 4) * (kB * 128) + (k % 4) * 32) >> 4), id,
                  x > 0 || k > 0);
}
// D[128 x DP] = A·B: A three planes of 32 packed columns in tensor memory
// (128 x 64), B planes of 64 rows.
template <int DP>
__device__ __forceinline__ void mma_tn3(uint32_t d, uint32_t a, uint64_t b) {
  using C = Cfg32<DP>;
  constexpr uint32_t id = idesc_bf16_f32_bmn(kTile, DP);
#pragma unroll
  for (int x = 0; x < 6; ++x)
#pragma unroll
    for (int k = 0; k < kB / 16; ++k)
      tc_mma_bf16_ts(d, a + kPi[x] * (kB / 2) + 8 * k,
                     b + ((kPj[x] * C::kBlkPlane + 2048 * k) >> 4), id, x > 0 || k > 0);
}

// 64 fp32 values of this thread's lane to three planes of 32 packed columns.
__device__ __forceinline__ void store_planes(uint32_t taddr, const float* v) {
#pragma unroll
  for (int c = 0; c < kB; c += 32) {
    uint32_t p[3][16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      split2(v[c + 2 * i], v[c + 2 * i + 1], &p[0][i], &p[1][i], &p[2][i]);
#pragma unroll
    for (int k = 0; k < 3; ++k) tc_st16(taddr + k * (kB / 2) + c / 2, p[k]);
  }
  tc_wait_st();
}

// acc += DP accumulator columns of this thread's lane.
template <int DP>
__device__ __forceinline__ void add_columns(float* acc, uint32_t taddr) {
#pragma unroll
  for (int c = 0; c < DP; c += 16) {
    float o[16];
    tc_ld16(taddr + c, o);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[c + i] += o[i];
  }
}

// f · acc to an fp32 row.
template <int DP>
__device__ __forceinline__ void store_row32(const float* acc, float* dst, int dh, int vec,
                                            float f) {
#pragma unroll
  for (int c = 0; c < DP; c += 4) {
    if (vec) {
      if (c < dh)
        *reinterpret_cast<float4*>(dst + c) =
            make_float4(acc[c] * f, acc[c + 1] * f, acc[c + 2] * f, acc[c + 3] * f);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < dh) dst[c + e] = acc[c + e] * f;
    }
  }
}

// Rows by the definition (see the top of the file), one thread a row.  The
// thread's own operands stay with it, the other side's rows are the same for
// all lanes of a warp (one broadcast a load), and C columns of a result are
// made at a time.
template <int DP>
__device__ __forceinline__ void own_row(float* v, const float* x, int dh) {
#pragma unroll
  for (int c = 0; c < DP; ++c) v[c] = c < dh ? __ldg(x + c) : 0.f;
}
// Four columns from c on of a row, zeros from dh on.
__device__ __forceinline__ float4 four(const float* x, int c, int dh, int vec) {
  if (vec) return __ldg(reinterpret_cast<const float4*>(x + c));
  return make_float4(__ldg(x + c), c + 1 < dh ? __ldg(x + c + 1) : 0.f,
                     c + 2 < dh ? __ldg(x + c + 2) : 0.f, c + 3 < dh ? __ldg(x + c + 3) : 0.f);
}
template <int DP>
__device__ __forceinline__ float dot_row(const float* v, const float* x, int dh, int vec) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < DP; c += 4)
    if (c < dh) {
      const float4 y = four(x, c, dh, vec);
      s = fmaf(v[c], y.x, s);
      if (c + 1 < dh) s = fmaf(v[c + 1], y.y, s);
      if (c + 2 < dh) s = fmaf(v[c + 2], y.z, s);
      if (c + 3 < dh) s = fmaf(v[c + 3], y.w, s);
    }
  return s;
}
// acc += p · columns c0 .. c0 + C - 1 of a row.
template <int C>
__device__ __forceinline__ void add_row(float* acc, float p, const float* x, int c0, int dh,
                                        int vec) {
#pragma unroll
  for (int e = 0; e < C; e += 4)
    if (c0 + e < dh) {
      const float4 y = four(x, c0 + e, dh, vec);
      acc[e] = fmaf(p, y.x, acc[e]);
      acc[e + 1] = fmaf(p, y.y, acc[e + 1]);
      acc[e + 2] = fmaf(p, y.z, acc[e + 2]);
      acc[e + 3] = fmaf(p, y.w, acc[e + 3]);
    }
}
template <int C>
__device__ __forceinline__ void put_row(const float* acc, float f, float* dst, int c0, int dh) {
#pragma unroll
  for (int e = 0; e < C; ++e)
    if (c0 + e < dh) dst[c0 + e] = acc[e] * f;
}

// One row of the forward.
template <int DP>
__device__ __noinline__ void plain_fwd_row(const AttnArgs& a, const AttnBlock& b, int h, int g,
                                           int row) {
  constexpr int C = 64;
  const float sc = a.scale * kLog2e;
  const float* k = static_cast<const float*>(a.k) + b.start * a.ldk + (long long)g * a.dh;
  const float* v = static_cast<const float*>(a.v) + b.start * a.ldv + (long long)g * a.dh;
  float* o = static_cast<float*>(a.out) + ((b.start + (long long)row) * a.Hq + h) * a.dh;
  float q[DP];
  own_row<DP>(q, static_cast<const float*>(a.q) + (b.start + (long long)row) * a.ldq +
                     (long long)h * a.dh, a.dh);
  const int n = a.causal ? row + 1 : b.len;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) m = fmaxf(m, dot_row<DP>(q, k + j * a.ldk, a.dh, a.vec) * sc);
  const float base = m == -INFINITY ? 0.f : m;
  for (int c0 = 0; c0 < a.dh; c0 += C) {
    float acc[C];
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = 0.f;
    l = 0.f;
    for (int j = 0; j < n; ++j) {
      const float p = ex2(dot_row<DP>(q, k + j * a.ldk, a.dh, a.vec) * sc - base);
      l += p;
      add_row<C>(acc, p, v + j * a.ldv, c0, a.dh, a.vec);
    }
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (c0 + e < a.dh) o[c0 + e] = acc[e] / l;
  }
  a.lse[(long long)h * a.T + b.start + row] = (m + log2f(l)) * kLn2;
}

// Rows row (as query i or key j) of the backward.
template <int DP>
__device__ __noinline__ void plain_dq_row(const AttnArgs& a, const AttnBlock& b, int h, int g,
                                          int row) {
  constexpr int C = 32;
  const long long t = b.start + (long long)row, ldo = (long long)a.Hq * a.dh;
  const float* k = static_cast<const float*>(a.k) + b.start * a.ldk + (long long)g * a.dh;
  const float* v = static_cast<const float*>(a.v) + b.start * a.ldv + (long long)g * a.dh;
  float* dq = static_cast<float*>(a.dq) + t * a.lddq + (long long)h * a.dh;
  float q[DP], go[DP];
  own_row<DP>(q, static_cast<const float*>(a.q) + t * a.ldq + (long long)h * a.dh, a.dh);
  own_row<DP>(go, static_cast<const float*>(a.dO) + t * ldo + (long long)h * a.dh, a.dh);
  const float lse = a.lse[(long long)h * a.T + t], del = a.delta[(long long)h * a.T + t];
  const int n = a.causal ? row + 1 : b.len;
  for (int c0 = 0; c0 < a.dh; c0 += C) {
    float acc[C];
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = 0.f;
    for (int j = 0; j < n; ++j) {
      const float p =
          ex2((dot_row<DP>(q, k + j * a.ldk, a.dh, a.vec) * a.scale - lse) * kLog2e);
      const float ds = p * (dot_row<DP>(go, v + j * a.ldv, a.dh, a.vec) - del);
      add_row<C>(acc, ds, k + j * a.ldk, c0, a.dh, a.vec);
    }
    put_row<C>(acc, a.scale, dq, c0, a.dh);
  }
}
template <int DP>
__device__ __noinline__ void plain_dkv_row(const AttnArgs& a, const AttnBlock& b, int g, int row) {
  constexpr int C = 16;                    // (more take registers from the main loop)
  const long long t = b.start + (long long)row, ldo = (long long)a.Hq * a.dh;
  float* dk = static_cast<float*>(a.dk) + t * a.lddk + (long long)g * a.dh;
  float* dv = static_cast<float*>(a.dv) + t * a.lddv + (long long)g * a.dh;
  float k[DP], v[DP];
  own_row<DP>(k, static_cast<const float*>(a.k) + t * a.ldk + (long long)g * a.dh, a.dh);
  own_row<DP>(v, static_cast<const float*>(a.v) + t * a.ldv + (long long)g * a.dh, a.dh);
  const int rep = a.Hq / a.Hkv;
  for (int c0 = 0; c0 < a.dh; c0 += C) {
    float ak[C], av[C];
#pragma unroll
    for (int e = 0; e < C; ++e) ak[e] = av[e] = 0.f;
    for (int h = g * rep; h < (g + 1) * rep; ++h)
      // (from the tile's first row on, so that the warp's lanes stay together)
      for (int i = a.causal ? b.row0 : 0; i < b.len; ++i) {
        if (a.causal && i < row) continue;
        const long long ti = b.start + (long long)i;
        const float* q = static_cast<const float*>(a.q) + ti * a.ldq + (long long)h * a.dh;
        const float* go = static_cast<const float*>(a.dO) + ti * ldo + (long long)h * a.dh;
        const float p = ex2((dot_row<DP>(k, q, a.dh, a.vec) * a.scale -
                             a.lse[(long long)h * a.T + ti]) * kLog2e);
        const float ds =
            p * (dot_row<DP>(v, go, a.dh, a.vec) - a.delta[(long long)h * a.T + ti]);
        add_row<C>(ak, ds, q, c0, a.dh, a.vec);
        add_row<C>(av, p, go, c0, a.dh, a.vec);
      }
    put_row<C>(ak, a.scale, dk, c0, a.dh);
    put_row<C>(av, 1.f, dv, c0, a.dh);
  }
}

// Words that the roles of a CTA share.
enum Shared {
  kOddItems,               // the last item to be computed again (a.link leads to the one
                           // before), -1: none
  kLostWait,               // a role has lost a wait
};

// The wait for a whole block of work, however long its sequence: it ends with the
// roles it waits for, which either get there or lose a wait of their own.
__device__ __forceinline__ void wait_block(uint32_t bar, uint32_t parity, uint32_t polls,
                                           const volatile int* shared, uint32_t& limit) {
  if (limit == 0) return;
  do {
    limit = polls;
    mbar_poll(bar, parity, limit);
  } while (limit == 0 && shared[kLostWait] == 0);
}

// By one thread: puts a block that met a value that is not finite on the CTA's
// list of those to compute again.
__device__ __forceinline__ void note_odd(const AttnArgs& a, const WorkSlot* slot,
                                         volatile int* shared) {
  if (*reinterpret_cast<const volatile uint32_t*>(&slot->odd) == 0) return;
  a.link[slot->item] = shared[kOddItems];
  shared[kOddItems] = slot->item;
}
// By the four warps that keep the list, once they have done all their blocks:
// again(block, head) for each of the list.  No other role waits for them any
// more but at the CTA's end, so no wait has to last as long as these loops.
template <typename F>
__device__ __forceinline__ void redo_odd(const AttnArgs& a, int heads, bool rising, uint32_t limit,
                                         const volatile int* shared, F again) {
  asm volatile("bar.sync 1, 128;" ::: "memory");
  if (__any_sync(0xffffffffu, limit == 0)) return;
  for (int item = shared[kOddItems]; item >= 0;
       item = *reinterpret_cast<const volatile int*>(a.link + item)) {
    AttnBlock b;
    int h;
    if (find_work(a, heads, 7, rising, item, &b, &h)) again(b, h);
    __syncwarp();
  }
}

// This warp's writes to shared memory are visible to the MMA; one arrival.
__device__ __forceinline__ void planes_ready(uint32_t bar) {
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

template <int DP>
__global__ void __launch_bounds__(Cfg32<DP>::kFwdThreads, 1)
attn_tc32_fwd_kernel(const AttnArgs a) {
  using C = Cfg32<DP>;
  constexpr int kHelp = 4 + 4 * C::kGroups;                    // first warp of the other roles
  extern __shared__ unsigned char f32_raw[];
  const uint32_t raw = smem_addr(f32_raw);
  unsigned char* sm = f32_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* q_sm = sm;                                    // 3 planes of 128 rows
  unsigned char* k_sm = sm + 3 * C::kTilePlane;                // [kStages] 3 planes of 64
  unsigned char* v_sm = k_sm + C::kStages * 3 * C::kBlkPlane;
  unsigned char* raw_sm = v_sm + C::kStages * 3 * C::kBlkPlane;   // [kGroups][kAhead]
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(raw_sm + C::kGroups * C::kAhead * C::kPieceBytes);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t qready = bar0, pready = bar0 + 8, odone = bar0 + 16, done = bar0 + 24;
  auto sfull = [&](int i) { return bar0 + 32 + 8 * i; };
  auto kready = [&](int st) { return bar0 + 48 + 8 * st; };
  auto vready = [&](int st) { return bar0 + 64 + 8 * st; };
  auto kempty = [&](int st) { return bar0 + 80 + 8 * st; };
  auto vempty = [&](int st) { return bar0 + 96 + 8 * st; };
  const uint32_t qempty = bar0 + 112;
  const uint32_t splitdone = bar0 + 8 * (kNumBars - 6);
  const WorkRing ring_w = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 8 * (kNumBars - 5),
                           smem_addr(tslot + 4)};
  volatile int* shared = reinterpret_cast<volatile int*>(tslot + 1);   // see Shared
  // Tensor memory: scores (two buffers), probabilities, O.
  constexpr int kP = 128, kO = 256;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Key blocks n - 1 .. 0.
  auto blocks = [&](const AttnBlock& b) {
    return ((a.causal ? min(b.len, b.row0 + kTile) : b.len) + kB - 1) / kB;
  };

  if (threadIdx.x == 0) {
    shared[kOddItems] = -1;
    shared[kLostWait] = 0;
    // pready, kready and vready: four warps; qready and splitdone: the splitting
    // warps; a slot's readers
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i == 0 || i == kNumBars - 6 ? 4 * C::kGroups
                          : i == 1 || (i >= 6 && i < 10) ? 4
                          : i == kNumBars - 3 || i == kNumBars - 2 ? 5 + 4 * C::kGroups
                          : 1);
    mbar_fence_init();
  }
  if (warp == kHelp) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  uint32_t limit = a.polls;                  // 0 once a wait of this thread is lost

  // Registers of the warpgroups: 208 + 2·112 + 80 = 4·128 and 240 + 168 + 96 =
  // 3·168, the launch's own.
  if (warp >= kHelp) {
    if (DP == 64)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == kHelp) {
      const uint64_t qd = sdesc_k128(q_sm), kd = sdesc_k128(k_sm);
      const uint64_t vd = sdesc_mn128(v_sm, kB * 128);
      constexpr uint64_t kStep = 3 * C::kBlkPlane >> 4;
      uint32_t c = 0, items = 0;               // blocks and query tiles so far
      auto scores = [&](uint32_t x, bool last) {
        const int st = x % C::kStages;
        mbar_poll(kready(st), (x / C::kStages) & 1, limit);
        if (elect_one()) {
          mma_kk3<DP>(tmem + kB * (x & 1), qd, kd + st * kStep);
          tc_commit(sfull(x & 1));
          tc_commit(kempty(st));
          if (last) tc_commit(qempty);
        }
        __syncwarp();
      };
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const int n = blocks(slot->b);
        mbar_poll(qready, items++ & 1, limit);
        scores(c, n == 1);
        for (int j = 0; j < n; ++j, ++c) {
          // (the buffer of the next block was read before P of the one before was ready)
          if (j + 1 < n) scores(c + 1, j + 2 == n);
          const int st = c % C::kStages;
          mbar_poll(vready(st), (c / C::kStages) & 1, limit);
          mbar_poll(pready, c & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn3<DP>(tmem + kO, tmem + kP, vd + st * kStep);
            tc_commit(odone);
            tc_commit(vempty(st));
          }
          __syncwarp();
        }
      });
      if (elect_one()) tc_commit(done);
      __syncwarp();
    } else if (warp == kHelp + 1) {
      // Finds the work, the next block when this one's operands are all but split.
      uint32_t items = 0;
      give_work(a, a.Hq, 7, true, ring_w, limit, [&](const AttnBlock&, int, WorkSlot*) {
        wait_block(splitdone, items++ & 1, a.polls, shared, limit);
      });
    }
  } else if (warp >= 4) {
    if (DP == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    const int group = (warp - 4) >> 2, tid = threadIdx.x - 128 * (1 + group);
    uint32_t c = 0, items = 0;
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
      const AttnBlock b = slot->b;
      const int h = slot->h;
      const int g = h / (a.Hq / a.Hkv), n = blocks(b);
      const float* q = static_cast<const float*>(a.q) + (b.start + (long long)b.row0) * a.ldq +
                       (long long)h * a.dh;
      const float* k = static_cast<const float*>(a.k) + b.start * a.ldk + (long long)g * a.dh;
      const float* v = static_cast<const float*>(a.v) + b.start * a.ldv + (long long)g * a.dh;
      bool bad = false;
      // K's or V's block j to its stage, split.
      auto put = [&](const Piece<DP>& x, bool ik, int j) {
        const uint32_t at = c + j, st = at % C::kStages;
        if (at >= C::kStages)
          mbar_poll(ik ? kempty(st) : vempty(st), ((at / C::kStages) - 1) & 1, limit);
        bad |= x.template put<kB>((ik ? k_sm : v_sm) + st * 3 * C::kBlkPlane, 0, tid);
        if (bad) const_cast<WorkSlot*>(slot)->odd = 1;
        planes_ready(ik ? kready(st) : vready(st));
      };
      if constexpr (DP == 64) {
        // One warpgroup takes Q's first half and K, the other Q's second half and
        // V; the next tile is under way while one is split and written.
        const bool ik = group == 0;
        const float* src = ik ? k : v;
        const long long ld = ik ? a.ldk : a.ldv;
        unsigned char* mine = raw_sm + group * C::kAhead * C::kPieceBytes;
        auto fetch = [&](int u) {
          const uint32_t to = smem_addr(mine) + u % C::kAhead * C::kPieceBytes;
          if (u == 0) {
            Piece<DP>::fetch_ahead(to, q + 64 * group * a.ldq, q, a.ldq,
                                   b.len - b.row0 - 64 * group, a.dh, a.vec, tid);
          } else if (u <= n) {
            const long long r0 = (long long)(n - u) * kB;
            Piece<DP>::fetch_ahead(to, src + r0 * ld, src, ld, b.len - (int)r0, a.dh, a.vec, tid);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        fetch(0);
        if (items > 0) mbar_poll(qempty, (items - 1) & 1, limit);
        for (int u = 0; u <= n; ++u) {
          // The next block of work is looked for beside the last two tiles.
          if (u == max(n - 1, 0) && lane == 0) mbar_arrive(splitdone);
          fetch(u + 1);                      // (its place was read a tile ago)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          Piece<DP> x;
          x.take(mine + u % C::kAhead * C::kPieceBytes, tid);
          if (u > 0) {
            put(x, ik, u - 1);
          } else {
            bad = x.template put<kTile>(q_sm, 64 * group, tid);
            planes_ready(qready);
          }
        }
      } else {
        // K0 K1 V0 K2 V1 .. (the registers hold one tile).
        auto load = [&](bool ik, int j) {
          const long long r0 = (long long)(n - 1 - j) * kB, ld = ik ? a.ldk : a.ldv;
          Piece<DP> x;
          x.fetch((ik ? k : v) + r0 * ld, ld, b.len - (int)r0, a.dh, a.vec, tid);
          put(x, ik, j);
        };
        if (items > 0) mbar_poll(qempty, (items - 1) & 1, limit);
        bad = put_tile<DP>(q_sm, q, a.ldq, min(kTile, b.len - b.row0), a.dh, a.vec, tid);
        planes_ready(qready);
        load(true, 0);
        for (int j = 0; j < n; ++j) {
          if (j + 1 < n) load(true, j + 1);
          load(false, j);
        }
      }
      ++items;
      c += n;
      if (DP != 64 && lane == 0) mbar_arrive(splitdone);
    });
  } else {
    if (DP == 64)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t to = tmem + lanes + kO;
    const float sc = a.scale * kLog2e;
    uint32_t nb = 0;                           // blocks so far
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int h = slot->h, n = blocks(b);
    const int row = b.row0 + 32 * warp + lane;                 // within the sequence
    float m = -INFINITY;
    float2 l2 = make_float2(0.f, 0.f), k2 = l2;
    float o[DP];
#pragma unroll
    for (int c = 0; c < DP; ++c) o[c] = 0.f;
    for (int j = 0; j < n; ++j, ++nb) {
      // The product of the block before: beside this block's scores at head
      // width 128 (registers), beside its probabilities at 64.
      if (DP == 128 && j > 0) {
        mbar_poll(odone, (nb - 1) & 1, limit);
        tc_fence_after();
        add_columns<DP>(o, to);
      }
      mbar_poll(sfull(nb & 1), (nb >> 1) & 1, limit);
      tc_fence_after();
      uint32_t r[kB];
      tc_ld32(tmem + lanes + kB * (nb & 1), r);
      tc_ld32(tmem + lanes + kB * (nb & 1) + 32, r + 32);
      tc_wait_ld();
      // The last key this row sees, within the block.
      const int k0 = (n - 1 - j) * kB;
      const int last = (a.causal ? min(row, b.len - 1) : b.len - 1) - k0;
      if (k0 + kB > b.len || (a.causal && k0 + kB > b.row0)) {
#pragma unroll
        for (int c = 0; c < kB; ++c)
          if (c > last) r[c] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = fmaxf(__uint_as_float(r[i]), __uint_as_float(r[4 + i]));
#pragma unroll
      for (int c = 8; c < kB; c += 8)
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
      float p[kB];
#pragma unroll
      for (int c = 0; c < kB; c += 2) {
        float2 x = fma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, nb2);
        x.x = ex2(x.x);
        x.y = ex2(x.y);
        if (c & 2)
          l2 = add2(l2, x);
        else
          k2 = add2(k2, x);
        p[c] = x.x;
        p[c + 1] = x.y;
      }
      if (DP == 64 && j > 0) {
        mbar_poll(odone, (nb - 1) & 1, limit);
        tc_fence_after();
        add_columns<DP>(o, to);
      }
      if (grow) {
#pragma unroll
        for (int c = 0; c < DP; ++c) o[c] *= f;
      }
      store_planes(tmem + lanes + kP, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready);
    }
    mbar_poll(odone, (nb - 1) & 1, limit);
    // (rows of a CTA that lost a wait are not written)
    if (__all_sync(0xffffffffu, limit != 0)) {
      tc_fence_after();
      const bool live = row < b.len;
      const float l = (l2.x + l2.y) + (k2.x + k2.y);
      const long long tok = (long long)b.start + row;
      add_columns<DP>(o, to);
      if (live)
        store_row32<DP>(o, static_cast<float*>(a.out) + (tok * a.Hq + h) * a.dh, a.dh, a.vec,
                        1.f / l);
      if (live) a.lse[(long long)h * a.T + tok] = (m + log2f(l)) * kLn2;
      if (threadIdx.x == 0) note_odd(a, slot, shared);
      tc_fence_before();                       // read before the next block's products
    }
    });
    redo_odd(a, a.Hq, true, limit, shared, [&](const AttnBlock& b, int h) {
      const int row = b.row0 + 32 * warp + lane;
      if (row < b.len) plain_fwd_row<DP>(a, b, h, h / (a.Hq / a.Hkv), row);
    });
  }
  if (limit == 0) shared[kLostWait] = 1;
  join_roles(a.status, limit, 0x741);
  if (warp == kHelp) {
    // The columns are freed only after every MMA has completed.
    last_wait(done, a.status, 0x742);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dK and dV of 128 keys: S^T = K·Q^T, dP^T = V·dO^T, dV += P^T·dO, dK += dS^T·Q.
template <int DP>
__global__ void __launch_bounds__(kThreads32, 1)
attn_tc32_dkv_kernel(const AttnArgs a) {
  using C = Cfg32<DP>;
  extern __shared__ unsigned char f32_raw[];
  const uint32_t raw = smem_addr(f32_raw);
  unsigned char* sm = f32_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* k_sm = sm;                                    // 3 planes of 128 rows
  unsigned char* v_sm = sm + 3 * C::kTilePlane;
  unsigned char* ring = sm + 6 * C::kTilePlane;                // [kStages] Q, dO: 3 planes of 64
  float* stat = reinterpret_cast<float*>(ring + C::kStages * 6 * C::kBlkPlane);  // lse, delta
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + C::kStages * 2 * kB);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t kvready = bar0, pready = bar0 + 8, dsready = bar0 + 16, done = bar0 + 24;
  const uint32_t sfull = bar0 + 32, dpfull = bar0 + 40, dvdone = bar0 + 48, dkdone = bar0 + 56;
  auto ready = [&](int st) { return bar0 + 64 + 8 * st; };
  auto empty = [&](int st) { return bar0 + 80 + 8 * st; };
  const uint32_t dvread = bar0 + 96, dkread = bar0 + 104;      // added to the registers
  const uint32_t kvempty = bar0 + 112;
  const uint32_t splitdone = bar0 + 8 * (kNumBars - 6);
  const WorkRing ring_w = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 8 * (kNumBars - 5),
                           smem_addr(tslot + 4)};
  volatile int* shared = reinterpret_cast<volatile int*>(tslot + 1);   // see Shared
  // Tensor memory: scores, probabilities, dP, dS, dV, dK.
  constexpr int kP = 64, kDp = 160, kDs = 224, kDv = 320, kDk = 384;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rep = a.Hq / a.Hkv;
  // Query blocks qb0 .. nqb - 1 of every head.
  auto first_block = [&](const AttnBlock& b) { return a.causal ? b.row0 / kB : 0; };
  auto blocks = [&](const AttnBlock& b) { return (b.len + kB - 1) / kB; };

  if (threadIdx.x == 0) {
    shared[kOddItems] = -1;
    shared[kLostWait] = 0;
    // those that four warps arrive on, splitdone among them; a slot's readers
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i < 3 || i == 8 || i == 9 || i == 12 || i == 13 || i == kNumBars - 6 ? 4
                          : i == kNumBars - 3 || i == kNumBars - 2 ? 9
                          : 1);
    mbar_fence_init();
  }
  if (warp == 8) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  uint32_t limit = a.polls;                  // 0 once a wait of this thread is lost

  // Registers of the three warpgroups: 168 + 232 + 104 = 3·168, the launch's own.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8) {
      const uint64_t kd = sdesc_k128(k_sm), vd = sdesc_k128(v_sm);
      const uint64_t qk = sdesc_k128(ring), gk = sdesc_k128(ring + 3 * C::kBlkPlane);
      const uint64_t qn = sdesc_mn128(ring, kB * 128);
      const uint64_t gn = sdesc_mn128(ring + 3 * C::kBlkPlane, kB * 128);
      constexpr uint64_t kStep = 6 * C::kBlkPlane >> 4;
      uint32_t c = 0, items = 0;               // blocks and key tiles so far
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const int n = rep * (blocks(slot->b) - first_block(slot->b));
        mbar_poll(kvready, items++ & 1, limit);
        mbar_poll(ready(c % C::kStages), (c / C::kStages) & 1, limit);
        tc_fence_after();
        if (elect_one()) {
          const uint64_t at = c % C::kStages * kStep;
          mma_kk3<DP>(tmem, kd, qk + at);
          tc_commit(sfull);
          mma_kk3<DP>(tmem + kDp, vd, gk + at);
          tc_commit(dpfull);
          if (n == 1) tc_commit(kvempty);
        }
        __syncwarp();
        for (int j = 0; j < n; ++j, ++c) {
          const int st = c % C::kStages, nx = (c + 1) % C::kStages;
          mbar_poll(pready, c & 1, limit);     // P is there, the scores are read
          if (j + 1 < n) mbar_poll(ready(nx), ((c + 1) / C::kStages) & 1, limit);
          if (c > 0) mbar_poll(dvread, (c - 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            if (j + 1 < n) {
              mma_kk3<DP>(tmem, kd, qk + nx * kStep);
              tc_commit(sfull);
            }
            mma_tn3<DP>(tmem + kDv, tmem + kP, gn + st * kStep);
            tc_commit(dvdone);
          }
          __syncwarp();
          mbar_poll(dsready, c & 1, limit);    // dS is there, dP is read
          if (c > 0) mbar_poll(dkread, (c - 1) & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            if (j + 1 < n) {
              mma_kk3<DP>(tmem + kDp, vd, gk + nx * kStep);
              tc_commit(dpfull);
              if (j + 2 == n) tc_commit(kvempty);
            }
            mma_tn3<DP>(tmem + kDk, tmem + kDs, qn + st * kStep);
            tc_commit(dkdone);
            tc_commit(empty(st));
          }
          __syncwarp();
        }
      });
      if (elect_one()) tc_commit(done);
      __syncwarp();
    } else if (warp == 9) {
      // Finds the work, the next block once this one's operands are split.
      uint32_t items = 0;
      give_work(a, a.Hkv, 7, false, ring_w, limit, [&](const AttnBlock&, int, WorkSlot*) {
        wait_block(splitdone, items++ & 1, a.polls, shared, limit);
      });
    }
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int tid = threadIdx.x - 128;
    const long long ldo = (long long)a.Hq * a.dh;
    // This warpgroup also adds the blocks' dV and dK, one thread a key.
    const uint32_t lanes = (uint32_t)(32 * (warp - 4)) << 16;
    uint32_t c = 0, items = 0;
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
      const AttnBlock b = slot->b;
      const int g = slot->h;
      const long long t0 = b.start + (long long)b.row0;
      const int keys = min(kTile, b.len - b.row0), qb0 = first_block(b), nqb = blocks(b);
      const int n = rep * (nqb - qb0);
      float dv[DP], dk[DP];
#pragma unroll
      for (int x = 0; x < DP; ++x) dv[x] = dk[x] = 0.f;
      auto add_block = [&](uint32_t x) {
        mbar_poll(dvdone, x & 1, limit);
        tc_fence_after();
        add_columns<DP>(dv, tmem + lanes + kDv);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dvread);
        mbar_poll(dkdone, x & 1, limit);
        tc_fence_after();
        add_columns<DP>(dk, tmem + lanes + kDk);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dkread);
      };
      int qb = qb0, h = g * rep;
      Piece<DP> xq, xg;
      auto fetch = [&]() {
        const long long r = b.start + (long long)qb * kB;
        const int have = b.len - qb * kB;
        xq.fetch(static_cast<const float*>(a.q) + r * a.ldq + (long long)h * a.dh, a.ldq, have,
                 a.dh, a.vec, tid);
        xg.fetch(static_cast<const float*>(a.dO) + r * ldo + (long long)h * a.dh, ldo, have, a.dh,
                 a.vec, tid);
      };
      if (items > 0) mbar_poll(kvempty, (items - 1) & 1, limit);
      ++items;
      bool bad = put_tile<DP>(k_sm, static_cast<const float*>(a.k) + t0 * a.ldk +
                                        (long long)g * a.dh, a.ldk, keys, a.dh, a.vec, tid);
      bad |= put_tile<DP>(v_sm, static_cast<const float*>(a.v) + t0 * a.ldv + (long long)g * a.dh,
                          a.ldv, keys, a.dh, a.vec, tid);
      fetch();
      planes_ready(kvready);
      for (int j = 0; j < n; ++j, ++c) {
        const uint32_t st = c % C::kStages;
        if (c >= C::kStages) mbar_poll(empty(st), ((c / C::kStages) - 1) & 1, limit);
        const long long r = b.start + (long long)qb * kB;
        const int have = b.len - qb * kB;
        unsigned char* q_sm = ring + st * 6 * C::kBlkPlane;
        bad |= xq.template put<kB>(q_sm, 0, tid);
        bad |= xg.template put<kB>(q_sm + 3 * C::kBlkPlane, 0, tid);
        if (tid < kB) {
          const long long i = (long long)h * a.T + r + tid;
          const float l = tid < have ? a.lse[i] * kLog2e : 0.f;
          const float d = tid < have ? a.delta[i] : 0.f;
          stat[st * 2 * kB + tid] = l;
          stat[st * 2 * kB + kB + tid] = d;
          bad |= !isfinite(l) || !isfinite(d);
        }
        if (bad) const_cast<WorkSlot*>(slot)->odd = 1;
        planes_ready(ready(st));
        if (++qb == nqb) {
          qb = qb0;
          ++h;
        }
        // The next block's rows are on their way while this one's sums come in.
        if (j + 1 < n) fetch();
        if (j > 0) add_block(c - 1);
      }
      if (lane == 0) mbar_arrive(splitdone);
      add_block(c - 1);
      // (rows of a CTA that lost a wait are not written)
      const int key = b.row0 + 32 * (warp - 4) + lane;
      if (limit != 0 && key < b.len) {
        const long long tok = (long long)b.start + key;
        store_row32<DP>(dv, static_cast<float*>(a.dv) + tok * a.lddv + (long long)g * a.dh, a.dh,
                        a.vec, 1.f);
        store_row32<DP>(dk, static_cast<float*>(a.dk) + tok * a.lddk + (long long)g * a.dh, a.dh,
                        a.vec, a.scale);
      }
      if (limit != 0 && tid == 0) note_odd(a, slot, shared);
      __syncwarp();
    });
    redo_odd(a, a.Hkv, false, limit, shared, [&](const AttnBlock& b, int g) {
      const int key = b.row0 + 32 * (warp - 4) + lane;
      if (key < b.len) plain_dkv_row<DP>(a, b, g, key);
    });
  } else {
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const float sc = a.scale * kLog2e;
    const float2 sc2 = make_float2(sc, sc);
    uint32_t nb = 0;                           // blocks so far
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int key = b.row0 + 32 * warp + lane;                 // within the sequence
    const int qb0 = first_block(b), nqb = blocks(b), n = rep * (nqb - qb0);
    int qb = qb0;
    for (int j = 0; j < n; ++j, ++nb) {
      const int st = nb % C::kStages;
      const float4* lse = reinterpret_cast<const float4*>(stat + st * 2 * kB);
      const float4* del = lse + kB / 4;
      mbar_poll(sfull, nb & 1, limit);
      tc_fence_after();
      uint32_t r[kB];
      tc_ld32(tmem + lanes, r);
      tc_ld32(tmem + lanes + 32, r + 32);
      mbar_poll(ready(st), (nb / C::kStages) & 1, limit);      // (lse and delta: long there)
      tc_wait_ld();
      float p[kB];
#pragma unroll
      for (int c = 0; c < kB; c += 4) {
        const float4 l = lse[c / 4];
        const float2 x = fma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2,
                              make_float2(-l.x, -l.y));
        const float2 y = fma2(make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])),
                              sc2, make_float2(-l.z, -l.w));
        p[c] = ex2(x.x);
        p[c + 1] = ex2(x.y);
        p[c + 2] = ex2(y.x);
        p[c + 3] = ex2(y.y);
      }
      // Columns lo .. hi - 1 are queries that see this key.
      const int q0 = qb * kB, lo = a.causal ? key - q0 : 0, hi = b.len - q0;
      const bool cut = q0 + kB > b.len || (a.causal && q0 < b.row0 + kTile);
      if (cut) {
#pragma unroll
        for (int c = 0; c < kB; ++c)
          if (c < lo || c >= hi) p[c] = 0.f;
      }
      if (nb > 0) mbar_poll(dvdone, (nb - 1) & 1, limit);      // P of before has been used
      tc_fence_after();
      store_planes(tmem + lanes + kP, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready);
      mbar_poll(dpfull, nb & 1, limit);
      tc_fence_after();
      tc_ld32(tmem + lanes + kDp, r);
      tc_ld32(tmem + lanes + kDp + 32, r + 32);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < kB; c += 4) {
        const float4 d = del[c / 4];
        p[c] *= __uint_as_float(r[c]) - d.x;
        p[c + 1] *= __uint_as_float(r[c + 1]) - d.y;
        p[c + 2] *= __uint_as_float(r[c + 2]) - d.z;
        p[c + 3] *= __uint_as_float(r[c + 3]) - d.w;
      }
      if (nb > 0) mbar_poll(dkdone, (nb - 1) & 1, limit);      // dS of before has been used
      tc_fence_after();
      store_planes(tmem + lanes + kDs, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dsready);
      if (++qb == nqb) qb = qb0;
    }
    });
  }
  if (limit == 0) shared[kLostWait] = 1;
  join_roles(a.status, limit, 0x751);
  if (warp == 8) {
    // The columns are freed only after every MMA has completed.
    last_wait(done, a.status, 0x752);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dQ of 128 queries: S = Q·K^T, dP = dO·V^T, dQ += dS·K.
template <int DP>
__global__ void __launch_bounds__(kThreads32, 1)
attn_tc32_dq_kernel(const AttnArgs a) {
  using C = Cfg32<DP>;
  extern __shared__ unsigned char f32_raw[];
  const uint32_t raw = smem_addr(f32_raw);
  unsigned char* sm = f32_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* q_sm = sm;                                    // 3 planes of 128 rows
  unsigned char* g_sm = sm + 3 * C::kTilePlane;
  unsigned char* ring = sm + 6 * C::kTilePlane;                // [kStages] K, V: 3 planes of 64
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + C::kStages * 6 * C::kBlkPlane);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t qready = bar0, dsready = bar0 + 8, dqdone = bar0 + 16, done = bar0 + 24;
  auto sfull = [&](int i) { return bar0 + 32 + 8 * i; };       // S and dP of a block
  auto ready = [&](int st) { return bar0 + 48 + 8 * st; };
  auto empty = [&](int st) { return bar0 + 64 + 8 * st; };
  const uint32_t qempty = bar0 + 80;
  const uint32_t splitdone = bar0 + 8 * (kNumBars - 6);
  const WorkRing ring_w = {reinterpret_cast<WorkSlot*>(tslot + 8), bar0 + 8 * (kNumBars - 5),
                           smem_addr(tslot + 4)};
  volatile int* shared = reinterpret_cast<volatile int*>(tslot + 1);   // see Shared
  // Tensor memory: scores and dP (two buffers each), dS, dQ.
  constexpr int kDp = 128, kDs = 256, kDq = 384;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto blocks = [&](const AttnBlock& b) {
    return ((a.causal ? min(b.len, b.row0 + kTile) : b.len) + kB - 1) / kB;
  };

  if (threadIdx.x == 0) {
    shared[kOddItems] = -1;
    shared[kLostWait] = 0;
    // qready, dsready, ready, splitdone: a warp each; a slot's readers
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i < 2 || i == 6 || i == 7 || i == kNumBars - 6 ? 4
                          : i == kNumBars - 3 || i == kNumBars - 2 ? 9
                          : 1);
    mbar_fence_init();
  }
  if (warp == 8) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  uint32_t limit = a.polls;                  // 0 once a wait of this thread is lost

  // Registers of the three warpgroups: 216 + 168 + 120 = 3·168, the launch's own.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == 8) {
      const uint64_t qd = sdesc_k128(q_sm), gd = sdesc_k128(g_sm);
      const uint64_t kk = sdesc_k128(ring), vk = sdesc_k128(ring + 3 * C::kBlkPlane);
      const uint64_t kn = sdesc_mn128(ring, kB * 128);
      constexpr uint64_t kStep = 6 * C::kBlkPlane >> 4;
      uint32_t c = 0, items = 0;               // blocks and query tiles so far
      auto front = [&](uint32_t x, bool last) {
        const int st = x % C::kStages;
        mbar_poll(ready(st), (x / C::kStages) & 1, limit);
        if (elect_one()) {
          mma_kk3<DP>(tmem + kB * (x & 1), qd, kk + st * kStep);
          mma_kk3<DP>(tmem + kDp + kB * (x & 1), gd, vk + st * kStep);
          tc_commit(sfull(x & 1));
          if (last) tc_commit(qempty);
        }
        __syncwarp();
      };
      take_work(ring_w, limit, [&](const WorkSlot* slot) {
        const int n = blocks(slot->b);
        mbar_poll(qready, items++ & 1, limit);
        front(c, n == 1);
        for (int j = 0; j < n; ++j, ++c) {
          // (the buffers of the next block were read before dS of the one before was ready)
          if (j + 1 < n) front(c + 1, j + 2 == n);
          const int st = c % C::kStages;
          mbar_poll(dsready, c & 1, limit);
          tc_fence_after();
          if (elect_one()) {
            mma_tn3<DP>(tmem + kDq, tmem + kDs, kn + st * kStep);
            tc_commit(dqdone);
            tc_commit(empty(st));
          }
          __syncwarp();
        }
      });
      if (elect_one()) tc_commit(done);
      __syncwarp();
    } else if (warp == 9) {
      // Finds the work, the next block once this one's operands are split.
      uint32_t items = 0;
      give_work(a, a.Hq, 7, true, ring_w, limit, [&](const AttnBlock&, int, WorkSlot*) {
        wait_block(splitdone, items++ & 1, a.polls, shared, limit);
      });
    }
  } else if (warp >= 4) {
    const int tid = threadIdx.x - 128;
    const long long ldo = (long long)a.Hq * a.dh;
    uint32_t c = 0, items = 0;
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
      const AttnBlock b = slot->b;
      const int h = slot->h;
      const int g = h / (a.Hq / a.Hkv), n = blocks(b), rows = min(kTile, b.len - b.row0);
      const long long t0 = b.start + (long long)b.row0;
      const float* k = static_cast<const float*>(a.k) + b.start * a.ldk + (long long)g * a.dh;
      const float* v = static_cast<const float*>(a.v) + b.start * a.ldv + (long long)g * a.dh;
      Piece<DP> xk, xv;
      auto fetch = [&](int j) {
        const long long r0 = (long long)(n - 1 - j) * kB;
        const int have = b.len - (int)r0;
        xk.fetch(k + r0 * a.ldk, a.ldk, have, a.dh, a.vec, tid);
        xv.fetch(v + r0 * a.ldv, a.ldv, have, a.dh, a.vec, tid);
      };
      if (items > 0) mbar_poll(qempty, (items - 1) & 1, limit);
      ++items;
      bool bad = put_tile<DP>(q_sm, static_cast<const float*>(a.q) + t0 * a.ldq +
                                        (long long)h * a.dh, a.ldq, rows, a.dh, a.vec, tid);
      bad |= put_tile<DP>(g_sm, static_cast<const float*>(a.dO) + t0 * ldo + (long long)h * a.dh,
                          ldo, rows, a.dh, a.vec, tid);
      fetch(0);
      planes_ready(qready);
      for (int j = 0; j < n; ++j, ++c) {
        const uint32_t st = c % C::kStages;
        // (the next block of work is looked for beside the last two blocks)
        if (j == max(n - 2, 0) && lane == 0) mbar_arrive(splitdone);
        if (c >= C::kStages) mbar_poll(empty(st), ((c / C::kStages) - 1) & 1, limit);
        unsigned char* k_to = ring + st * 6 * C::kBlkPlane;
        bad |= xk.template put<kB>(k_to, 0, tid);
        bad |= xv.template put<kB>(k_to + 3 * C::kBlkPlane, 0, tid);
        if (bad) const_cast<WorkSlot*>(slot)->odd = 1;
        planes_ready(ready(st));
        if (j + 1 < n) fetch(j + 1);
      }
    });
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const float sc = a.scale * kLog2e;
    uint32_t nb = 0;                           // blocks so far
    take_work(ring_w, limit, [&](const WorkSlot* slot) {
    const AttnBlock b = slot->b;
    const int h = slot->h, n = blocks(b);
    const int row = b.row0 + 32 * warp + lane;                 // within the sequence
    const bool live = row < b.len;
    const long long at = (long long)h * a.T + b.start + row;
    const float lse = live ? a.lse[at] * kLog2e : 0.f, del = live ? a.delta[at] : 0.f;
    const float2 sc2 = make_float2(sc, sc), nl2 = make_float2(-lse, -lse);
    float dq[DP];
#pragma unroll
    for (int c = 0; c < DP; ++c) dq[c] = 0.f;
    for (int j = 0; j < n; ++j, ++nb) {
      const uint32_t ts = tmem + lanes + kB * (nb & 1);
      mbar_poll(sfull(nb & 1), (nb >> 1) & 1, limit);
      tc_fence_after();
      uint32_t r[kB];
      tc_ld32(ts, r);
      tc_ld32(ts + 32, r + 32);
      tc_wait_ld();
      float p[kB];
#pragma unroll
      for (int c = 0; c < kB; c += 2) {
        const float2 x =
            fma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, nl2);
        p[c] = ex2(x.x);
        p[c + 1] = ex2(x.y);
      }
#pragma unroll
      for (int c0 = 0; c0 < kB; c0 += 32) {
        tc_ld32(ts + kDp + c0, r);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) p[c0 + c] *= __uint_as_float(r[c]) - del;
      }
      const int k0 = (n - 1 - j) * kB;
      const int last = (a.causal ? min(row, b.len - 1) : b.len - 1) - k0;
      if (k0 + kB > b.len || (a.causal && k0 + kB > b.row0)) {
#pragma unroll
        for (int c = 0; c < kB; ++c)
          if (c > last) p[c] = 0.f;
      }
      if (j > 0) {
        mbar_poll(dqdone, (nb - 1) & 1, limit);                // dS of before has been used
        tc_fence_after();
        add_columns<DP>(dq, tmem + lanes + kDq);
      }
      store_planes(tmem + lanes + kDs, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dsready);
    }
    mbar_poll(dqdone, (nb - 1) & 1, limit);
    // (rows of a CTA that lost a wait are not written)
    if (__all_sync(0xffffffffu, limit != 0)) {
      tc_fence_after();
      add_columns<DP>(dq, tmem + lanes + kDq);
      if (live)
        store_row32<DP>(dq, static_cast<float*>(a.dq) + ((long long)b.start + row) * a.lddq +
                                (long long)h * a.dh, a.dh, a.vec, a.scale);
      if (threadIdx.x == 0) note_odd(a, slot, shared);
      tc_fence_before();                       // read before the next block's products
    }
    });
    redo_odd(a, a.Hq, true, limit, shared, [&](const AttnBlock& b, int h) {
      const int row = b.row0 + 32 * warp + lane;
      if (row < b.len) plain_dq_row<DP>(a, b, h, h / (a.Hq / a.Hkv), row);
    });
  }
  if (limit == 0) shared[kLostWait] = 1;
  join_roles(a.status, limit, 0x761);
  if (warp == 8) {
    // The columns are freed only after every MMA has completed.
    last_wait(done, a.status, 0x762);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP>
cudaError_t fwd(const AttnArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)(attn_slots(a.T, a.S, 7) * a.Hq);
  attn_tc32_fwd_kernel<DP><<<grid, Cfg32<DP>::kFwdThreads, Cfg32<DP>::kFwdSmem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t setup_attn_tc32() {
  cudaError_t e = allow_max_smem(attn_tc32_fwd_kernel<64>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc32_fwd_kernel<128>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc32_dkv_kernel<64>);
  if (e == cudaSuccess) e = allow_max_smem(attn_tc32_dq_kernel<64>);
  return e;
}

cudaError_t launch_attn_tc32_forward(const AttnArgs& a, cudaStream_t st) {
  return a.dh <= 64 ? fwd<64>(a, st) : fwd<128>(a, st);
}

cudaError_t launch_attn_tc32_backward(const AttnArgs& a, cudaStream_t st) {
  const long long slots = attn_slots(a.T, a.S, 7);
  attn_tc32_dkv_kernel<64><<<(unsigned)(slots * a.Hkv), kThreads32, kBwdSmem32, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attn_tc32_dq_kernel<64><<<(unsigned)(slots * a.Hq), kThreads32, kBwdSmem32, st>>>(a);
  return cudaGetLastError();
}

}  // namespace cat
