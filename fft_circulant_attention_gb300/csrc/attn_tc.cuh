// What the tensor-core attention kernels share: packed fp32 arithmetic, the
// exponential, bf16 packing and the care for values that are not finite.
#pragma once
#include <cuda_bf16.h>

#include "attn.cuh"
#include "tc.cuh"

namespace cat {

constexpr int kTile = 128;                 // rows of a query tile, keys of a block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// a·b + c on two fp32 values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// A mask cuts a block of scores along a row's columns lo .. hi - 1.  Chunks of
// 32 columns are told apart by whole warps, so that only those that the edge
// runs through are masked value by value (a compare and a select on the pipe
// of half rate, which for 64 columns took longer than their exponentials) and
// those behind it are not computed at all.
enum Chunk { kNoColumn = 0, kSomeColumns = 1, kEveryColumn = 2 };
__device__ __forceinline__ int chunk_kind(int lo, int hi) {
  if (__all_sync(0xffffffffu, lo <= 0 && hi >= 32)) return kEveryColumn;
  return __all_sync(0xffffffffu, lo >= 32 || hi <= 0 || hi <= lo) ? kNoColumn : kSomeColumns;
}
// The chunk's columns as bits.
__device__ __forceinline__ uint32_t chunk_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  return hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
}

// A bf16 half whose exponent is all ones (an infinity or NaN) sets the high
// bit of its half: adding one to the exponent carries there.
__device__ __forceinline__ uint32_t odd2(uint32_t w) {
  return (w & 0x7f807f80u) + 0x00800080u;
}
__device__ __forceinline__ uint32_t drop_odd(uint32_t w) {
  const uint32_t o = odd2(w);
  return w & ~((o & 0x8000u ? 0xffffu : 0u) | (o & 0x80000000u ? 0xffff0000u : 0u));
}

// Whether a [ROWS][DP] tile in shared memory holds a value that is not finite,
// by one warp (9 operations per 8 values: about 0.3 us a tile of 128 x 64).
template <int DP, int ROWS = kTile>
__device__ __forceinline__ bool odd_tile(const unsigned char* tile) {
  constexpr int kVec = ROWS * DP * 2 / 16;
  const uint4* v = reinterpret_cast<const uint4*>(tile);
  uint32_t any = 0;
#pragma unroll 16
  for (int i = threadIdx.x & 31; i < kVec; i += 32) {
    const uint4 x = v[i];
    any |= odd2(x.x) | odd2(x.y) | odd2(x.z) | odd2(x.w);
  }
  return __any_sync(0xffffffffu, (any & 0x80008000u) != 0);
}

// Values of the tile that are not finite become zero.  True if one of them lay
// in a row below `rows`.
template <int DP, int ROWS = kTile>
__device__ __forceinline__ bool clean_tile(unsigned char* tile, int rows) {
  constexpr int kVec = ROWS * DP * 2 / 16;
  uint4* v = reinterpret_cast<uint4*>(tile);
  bool found = false;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < kVec; i += 32) {
    const uint4 x = v[i];
    if (((odd2(x.x) | odd2(x.y) | odd2(x.z) | odd2(x.w)) & 0x80008000u) != 0) {
      // 8 pieces a row, ROWS rows a box of 64 columns.
      if ((i / 8) % ROWS < rows) found = true;
      v[i] = make_uint4(drop_odd(x.x), drop_odd(x.y), drop_odd(x.z), drop_odd(x.w));
    }
  }
  return __any_sync(0xffffffffu, found);
}

// f · 16 fp32 values as bf16 to a row, its first `cols` (a multiple of 8).
// wide: 32-byte aligned rows, one store of a whole sector (the lanes of a warp
// write 32 different rows, so the number of stores is what counts).
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float* o, float f, int cols,
                                        bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = bf16x2(o[2 * i] * f, o[2 * i + 1] * f);
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                     __cvta_generic_to_global(dst)),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                 "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    if (cols > 8) *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Whether store16 may take whole sectors: head rows of 16·k elements that
// start on 32-byte boundaries.
__device__ __forceinline__ bool wide_rows(const void* base, long long ld, int dh) {
  return ((uintptr_t)base & 31) == 0 && ld % 16 == 0 && dh % 16 == 0;
}

// Work of a persistent CTA.  The grid has one CTA for every slot and head; a
// CTA that runs takes over CTAs that have not started yet (cluster launch
// control: the hardware's own queue, no counter in memory that calls or
// graphs could share), so that the copies and first products of its next
// block run beside the last ones of this block, and the set-up of a CTA is
// paid once an SM.  The copy warp finds the blocks and hands them to the other
// roles through two slots in shared memory.
struct WorkSlot {
  AttnBlock b;
  int h, valid;
  uint32_t odd;            // values that are not finite have been met (bf16: in a cut
                           // block's own rows)
  int item;                // the block's number (find_work)
};

// Barriers at `bars`: [0, 1] slot filled, [2, 3] slot released, [4] the queue's
// answer, which lands in `answer` (16 bytes).
struct WorkRing {
  WorkSlot* slots;
  uint32_t bars, answer;
  __device__ __forceinline__ uint32_t filled(int s) const { return bars + 8 * s; }
  __device__ __forceinline__ uint32_t released(int s) const { return bars + 16 + 8 * s; }
  __device__ __forceinline__ uint32_t answered() const { return bars + 32; }
};

// Block and head of work item `item`, in blocks of 2^shift rows by `heads` heads, by
// one whole warp; false where there is none.  rising: under a causal mask the
// work of a block grows with its row.  The largest blocks come first where
// there are few sequences; where there are many, blocks are small beside the
// work of an SM, and they are taken as they lie.
__device__ __forceinline__ bool find_work(const AttnArgs& a, int heads, int shift, bool rising,
                                          int item, AttnBlock* b, int* h) {
  *h = item % heads;
  int slot = item / heads;
  if (a.S <= kSortedSeqs) return attn_find_by_size(a, slot, shift, rising, b);
  if (rising) slot = (int)(gridDim.x / heads) - 1 - slot;
  return attn_find_block(a, slot, shift, b);
}

// The copy warp's loop: load(block, head, slot) for each of the CTA's blocks.
template <typename F>
__device__ __forceinline__ void give_work(const AttnArgs& a, int heads, int shift, bool rising,
                                          const WorkRing& ring, uint32_t& limit, F load) {
  const int lane = threadIdx.x & 31;
  int item = blockIdx.x, count = 0;
  auto publish = [&](const AttnBlock& b, int h, int valid) {
    const int s = count & 1;
    if (count >= 2) mbar_poll(ring.released(s), ((count >> 1) - 1) & 1, limit);
    if (lane == 0) {
      ring.slots[s].b = b;
      ring.slots[s].h = h;
      ring.slots[s].valid = valid;
      ring.slots[s].odd = 0;
      ring.slots[s].item = item;
      mbar_arrive(ring.filled(s));
    }
    __syncwarp();
    ++count;
  };
  for (uint32_t par = 0;; par ^= 1u) {
    AttnBlock b;
    int h;
    if (find_work(a, heads, shift, rising, item, &b, &h)) {
      publish(b, h, 1);
      load(b, h, ring.slots + ((count - 1) & 1));
      __syncwarp();
    }
    if (item == 0) attn_check_sequences(a, lane, 32);
    if (__any_sync(0xffffffffu, limit == 0)) break;
    // Asked only now, with this block's copies issued: a block taken over early
    // would wait here while another SM ran dry.
    if (lane == 0) {
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], 16;" ::"r"(ring.answered())
                   : "memory");
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
          "[%0], [%1];" ::"r"(ring.answer),
          "r"(ring.answered())
          : "memory");
    }
    mbar_poll(ring.answered(), par, limit);
    uint32_t more, next;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(more), "=r"(next)
        : "r"(ring.answer)
        : "memory");
    fence_proxy_async_smem();                // the answer is read before the next one lands
    __syncwarp();
    if (!more || __any_sync(0xffffffffu, limit == 0)) break;
    item = (int)next;
  }
  publish(AttnBlock{0, 0, 0, 0}, 0, 0);
}

// Where the roles of a CTA meet at the end.  A lost wait is reported, and then
// the CTA stays on for 2 ms: copies and the queue's answer that it no longer
// waited for take microseconds, and land in shared memory that is still its own.
__device__ __forceinline__ void join_roles(unsigned int* status, uint32_t limit,
                                           unsigned int code) {
  if (limit == 0) report(status, code);
  tc_fence_before();
  if (__syncthreads_or(limit == 0))
    for (int i = 0; i < 4; ++i) __nanosleep(500000);
}
// A wait of its own limit, whatever has been lost before: for MMAs that must
// have completed before their columns are freed.
__device__ __forceinline__ void last_wait(uint32_t bar, unsigned int* status, unsigned int code) {
  uint32_t limit = kMaxPolls;
  mbar_poll(bar, 0, limit);
  if (limit == 0) report(status, code);
}

// Another role's loop: work(slot) for each of the CTA's blocks.  One arrival
// a warp gives the slot back.
template <typename F>
__device__ __forceinline__ void take_work(const WorkRing& ring, uint32_t& limit, F work) {
  for (int i = 0;; ++i) {
    const int s = i & 1;
    mbar_poll(ring.filled(s), (i >> 1) & 1, limit);
    if (__any_sync(0xffffffffu, limit == 0)) break;
    const WorkSlot* w = ring.slots + s;
    if (!w->valid) break;
    work(w);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(ring.released(s));
  }
}

}  // namespace cat
