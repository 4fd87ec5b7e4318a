// Token ids: 32- or 64-bit integers on the device.
#pragma once
#include <cuda_runtime.h>

namespace cat {

struct Ids {
  const void* p;
  int wide;                // 64 bits each
};

// An id as 32 bits that compare as unsigned: itself where it is 0 .. 2^31 - 1, the
// largest of those where it is larger, 2^31 or more where it is negative.
__device__ __forceinline__ unsigned id_key(int v) { return (unsigned)v; }
__device__ __forceinline__ unsigned id_key(long long v) {
  const int hi = (int)(v >> 32);
  return hi == 0 ? min((unsigned)v, 0x7fffffffu) : hi < 0 ? 0xffffffffu : 0x7fffffffu;
}
// -1 where the token has none (a negative id), -2 where the id is outside the
// vocabulary.
__device__ __forceinline__ int id_of(unsigned key, int vocab) {
  return key < (unsigned)vocab ? (int)key : key >> 31 ? -1 : -2;
}
__device__ __forceinline__ int id_at(const Ids& ids, long long i, int vocab) {
  return id_of(ids.wide ? id_key(__ldg(static_cast<const long long*>(ids.p) + i))
                        : id_key(__ldg(static_cast<const int*>(ids.p) + i)),
               vocab);
}

// The keys of U ids at i, i + step, .. (none from n on), all loads on their way at
// once.
template <int U>
__device__ __forceinline__ void keys_at(const Ids& ids, long long i, int step, long long n,
                                        unsigned (&key)[U]) {
  if (ids.wide) {
    long long v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = i + u * step < n ? __ldg(static_cast<const long long*>(ids.p) + i + u * step) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) key[u] = id_key(v[u]);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
      key[u] = i + u * step < n
                   ? id_key(__ldg(static_cast<const int*>(ids.p) + i + u * step)) : 0xffffffffu;
  }
}

}  // namespace cat
