// Token ids: 32- or 64-bit integers on the device.
#pragma once
#include <cuda_runtime.h>

namespace cat {

struct Ids {
  const void* p;
  int wide;                // 64 bits each
};

// Id i of a call: -1 where the token has none (a negative id), -2 where the id
// is outside the vocabulary.
__device__ __forceinline__ int id_at(const Ids& ids, long long i, int vocab) {
  if (ids.wide) {
    const long long v = __ldg(static_cast<const long long*>(ids.p) + i);
    return v < 0 ? -1 : v >= vocab ? -2 : (int)v;
  }
  const int v = __ldg(static_cast<const int*>(ids.p) + i);
  return v < 0 ? -1 : v >= vocab ? -2 : v;
}

// U ids at i, i + step, .. (-1 from n on), all loads on their way at once.
template <int U>
__device__ __forceinline__ void ids_at(const Ids& ids, long long i, int step, long long n,
                                       int vocab, int (&id)[U]) {
  if (ids.wide) {
    long long v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = i + u * step < n ? __ldg(static_cast<const long long*>(ids.p) + i + u * step) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = v[u] < 0 ? -1 : v[u] >= vocab ? -2 : (int)v[u];
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
      id[u] = i + u * step < n ? __ldg(static_cast<const int*>(ids.p) + i + u * step) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = id[u] < 0 ? -1 : id[u] >= vocab ? -2 : id[u];
  }
}

}  // namespace cat
