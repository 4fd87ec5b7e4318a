// What the C entry points of the operator plans share: operands' ranges and
// their overlaps, a plan's creation and its workspace.
#pragma once
#include <new>

#include "../../include/cat.h"
#include "cat_internal.h"

namespace cat {

inline int status_of(cudaError_t e) { return e == cudaSuccess ? CAT_OK : CAT_ERR_CUDA; }

inline size_t elem_size(int dtype) { return dtype == CAT_BF16 ? 2 : 4; }

// One operand: `rows` rows of `width` bytes, `stride` bytes apart.
struct Span2 {
  const void* p;
  size_t rows, width, stride;
};

inline Span2 flat(const void* p, size_t bytes) { return Span2{p, 1, bytes, bytes}; }

// Whether two operands share a byte.  Rows of the same stride may interleave
// (the columns of one projection's output): they meet only if their columns
// do.  Different strides count as meeting wherever the ranges do.
inline bool overlap(const Span2& a, const Span2& b) {
  if (!a.p || !b.p || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  const size_t nx = (a.rows - 1) * a.stride + a.width, ny = (b.rows - 1) * b.stride + b.width;
  if (x >= y + ny || y >= x + nx) return false;
  if (a.stride != b.stride || a.rows == 1) return true;
  const size_t s = a.stride;
  const size_t d = y >= x ? (y - x) % s : (s - (x - y) % s) % s;   // b's column offset from a's
  return d < a.width || d + b.width > s;
}

// No output meets an input or another output.
inline bool aliased(const Span2* in, int nin, const Span2* out, int nout) {
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i)
      if (overlap(out[o], in[i])) return true;
    for (int q = o + 1; q < nout; ++q)
      if (overlap(out[o], out[q])) return true;
  }
  return false;
}

inline cat_plan_s* new_plan(int op, int dtype, void* stream, int* st) {
  cat_plan_s* p = new (std::nothrow) cat_plan_s();
  if (!p) {
    *st = CAT_ERR_ALLOC;
    return nullptr;
  }
  p->op = op;
  p->dtype = dtype;
  p->stream = (cudaStream_t)stream;
  *st = CAT_OK;
  if (cudaGetDevice(&p->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->sms, cudaDevAttrMultiProcessorCount, p->device) != cudaSuccess) {
    cudaGetLastError();
    delete p;
    *st = CAT_ERR_CUDA;
    return nullptr;
  }
  return p;
}

template <typename T>
bool alloc(cat_plan_s* p, T** ptr, size_t count) {
  const size_t bytes = count ? count * sizeof(T) : 16;
  if (cudaMalloc((void**)ptr, bytes) != cudaSuccess) {
    cudaGetLastError();
    *ptr = nullptr;
    return false;
  }
  p->workspace_bytes += bytes;
  return true;
}

// Releases a half-built plan and passes its error on.
inline int fail(cat_plan_s* p, int st) {
  cudaGetLastError();
  cat_plan_destroy(p);
  return st;
}

// The status word, cleared.
inline bool alloc_status(cat_plan_s* p) {
  return alloc(p, &p->status, 1) && cat::settled([&](cudaStream_t s) {
           return cudaMemsetAsync(p->status, 0, sizeof(unsigned int), s);
         }) == cudaSuccess;
}

}  // namespace cat
