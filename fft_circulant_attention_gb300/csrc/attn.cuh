// Softmax attention over packed sequences (plans of cat_plan_create_attn):
// what its kernels share.
//
// T token rows hold S sequences one after another, sequence s in rows
// cu[s] .. cu[s+1] - 1 (cu on the device, S + 1 entries).  A kernel works on
// blocks of 2^shift rows of one sequence.  Blocks are numbered without a
// prefix sum: sequence s owns the slots from (cu[s] >> shift) + s on, which
// never meet those of sequence s + 1, since a sequence of L rows has at most
// (cu[s+1] >> shift) - (cu[s] >> shift) + 1 blocks.  So (T >> shift) + S
// slots cover every block, their number needs no look at cu on the host, and
// a slot's sequence is a search in cu.
#pragma once
#include <cuda_runtime.h>

#include "elem.cuh"
#include "fft_device.cuh"

namespace cat {

// Arguments of every attention kernel.  Strides are in elements between
// token rows; heads are dense inside a row.
struct AttnArgs {
  const void* q; const void* k; const void* v; const void* o; const void* dO;
  void* out;               // forward's O
  void* dq; void* dk; void* dv;
  float* lse;              // [Hq][T], natural logarithm
  float* delta;            // [Hq][T] Σ_c dO·O (backward workspace)
  float* stats;            // [Hq][slots of 128 rows][2][128] lse·log2 e, then delta
                           // (backward workspace of the tensor-core kernels)
  const int* cu;
  long long ldq, ldk, ldv, lddq, lddk, lddv;
  int T, S, Hq, Hkv, dh, causal;
  float scale;
  int vec;                 // every row start is aligned for 4-element accesses
  int tc;                  // bf16, every row and head starts on a 16-byte boundary
  unsigned int* status;
  int* link;               // [slots of 128 rows · Hq] blocks to compute again (fp32
                           // workspace)
  unsigned int polls;      // of a wait of the fp32 kernels until it is lost (3.8 us each)
};
constexpr unsigned int kWaitPolls = 1u << 22;

struct AttnBlock {
  int seq;                 // the sequence
  int start, len;          // its first row and its length
  int row0;                // the block's first row within the sequence
};

// Looks over the whole of cu (the search below may pass over a fault), `step`
// threads from thread `first` on: entries that do not ascend within 0 .. T are
// reported.
__device__ __forceinline__ void attn_check_sequences(const AttnArgs& a, int first, int step) {
  for (int i = first; i < a.S; i += step) {
    const int c0 = __ldg(a.cu + i), c1 = __ldg(a.cu + i + 1);
    if (c0 < 0 || c1 < c0 || c1 > a.T) report(a.status, 0x701);
  }
}

// The block of `slot`, by one whole warp; false for a slot without one.  A
// sequence that is not ascending within 0 .. T is skipped, so that no access
// leaves the tensors.
__device__ __forceinline__ bool attn_find_block(const AttnArgs& a, int slot, int shift,
                                                AttnBlock* b) {
  const int lane = threadIdx.x & 31;
  // The last s with (cu[s] >> shift) + s <= slot, 32 candidates at a time.
  int lo = 0, n = a.S;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool in = at < n && (__ldg(a.cu + lo + at) >> shift) + lo + at <= slot;
    const int k = max(__popc(__ballot_sync(0xffffffffu, in)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int c0 = __ldg(a.cu + lo), c1 = __ldg(a.cu + lo + 1);
  if (c0 < 0 || c1 < c0 || c1 > a.T) return false;
  const int blk = slot - ((c0 >> shift) + lo);
  b->seq = lo;
  b->start = c0;
  b->len = c1 - c0;
  b->row0 = blk << shift;
  return blk >= 0 && blk <= ((c1 - c0) >> shift) && b->row0 < b->len;
}

// The block of rank `r`, the largest amount of work first, by one whole warp;
// for up to kSortedSeqs sequences.  A causal sequence of m blocks has one
// block of each size 1 .. m (rising: the last row's block is the largest,
// else the first one's), one that is not causal m blocks of size m.  So the
// number of blocks above a size k is a sum over the sequences, and size and
// sequence of rank r are found from such sums, without a sorted list in
// memory that another call's kernel could be reading.
//
// Against blocks as they lie (12 heads of 64, bf16 forward and backward, us):
// 16 documents of 57 .. 1024 tokens 25.0 for 27.8, 84.0 for 92.1; 8 x 1024 24.8
// for 27.2, 79.2 for 89.2; 128 documents of 20 .. 200 tokens 30.9 for 31.0, 92.9
// for 92.9, where the last block is small whatever the order: so this search,
// whose cost grows with the sequences, ends there.
constexpr int kSortedSeqs = 128;
__device__ __forceinline__ bool attn_find_by_size(const AttnArgs& a, int r, int shift, bool rising,
                                                  AttnBlock* b) {
  const int lane = threadIdx.x & 31;
  int m[kSortedSeqs / 32];
#pragma unroll
  for (int i = 0; i < kSortedSeqs / 32; ++i) {
    const int s = 32 * i + lane;
    m[i] = 0;
    if (s < a.S) {
      const int c0 = __ldg(a.cu + s), c1 = __ldg(a.cu + s + 1);
      if (c0 >= 0 && c1 >= c0 && c1 <= a.T) m[i] = (c1 - c0 + (1 << shift) - 1) >> shift;
    }
  }
  auto above = [&](int k) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSortedSeqs / 32; ++i)
      n += a.causal ? max(m[i] - k, 0) : m[i] > k ? m[i] : 0;
    return __reduce_add_sync(0xffffffffu, n);
  };
  if (r >= above(0)) return false;
  int lo = 0, size = 0;                      // above(lo) > r >= above(size)
#pragma unroll
  for (int i = 0; i < kSortedSeqs / 32; ++i) size = max(size, m[i]);
  size = __reduce_max_sync(0xffffffffu, size);
  while (size - lo > 1) {
    const int mid = (lo + size) >> 1;
    if (above(mid) > r)
      lo = mid;
    else
      size = mid;
  }
  r -= above(size);
  int blk = 0, seq = -1;
  if (!a.causal) {
    blk = r % size;
    r /= size;
  }
  // The r-th of the sequences that have blocks of this size.
#pragma unroll
  for (int i = 0; i < kSortedSeqs / 32; ++i) {
    const bool in = a.causal ? m[i] >= size : m[i] == size;
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    const unsigned at = __ballot_sync(
        0xffffffffu, in && __popc(mask & ((1u << lane) - 1u)) == r);
    if (at) seq = 32 * i + __ffs(at) - 1;
    r -= __popc(mask);
  }
  if (seq < 0) return false;
  b->seq = seq;
  b->start = __ldg(a.cu + seq);
  b->len = __ldg(a.cu + seq + 1) - b->start;
  if (a.causal) blk = rising ? size - 1 : ((b->len + (1 << shift) - 1) >> shift) - size;
  b->row0 = blk << shift;
  return true;
}

__host__ __device__ inline long long attn_slots(int T, int S, int shift) {
  return (long long)(T >> shift) + S;
}

}  // namespace cat
