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
};

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

__host__ __device__ inline long long attn_slots(int T, int S, int shift) {
  return (long long)(T >> shift) + S;
}

}  // namespace cat
