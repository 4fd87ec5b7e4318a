// Host-side tensor-map encoding through the driver entry point (the runtime
// library exposes it without linking the driver library directly).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "bulk.cuh"
#include "tc.cuh"
#include "xent_mma.cuh"

namespace cat {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_once;

void find_encode() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}
}  // namespace

bool encode_map_4d(CUtensorMap* map, const void* base, CUtensorMapDataType type,
                   const unsigned long long dims[4], const unsigned long long strides[3],
                   const unsigned int box[4]) {
  std::call_once(g_once, find_encode);
  if (!g_encode) return false;
  cuuint64_t gd[4] = {dims[0], dims[1], dims[2], dims[3]};
  cuuint64_t gs[3] = {strides[0], strides[1], strides[2]};
  cuuint32_t bx[4] = {box[0], box[1], box[2], box[3]};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = g_encode(map, type, 4, const_cast<void*>(base), gd, gs, bx, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_map_2d_sw128(CUtensorMap* map, const void* base, unsigned long long cols,
                         unsigned long long rows, unsigned long long row_bytes,
                         unsigned int box_cols, unsigned int box_rows) {
  std::call_once(g_once, find_encode);
  if (!g_encode) return false;
  cuuint64_t gd[2] = {cols, rows};
  cuuint64_t gs[1] = {row_bytes};
  cuuint32_t bx[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gd, gs,
                        bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_map_heads_sw128(CUtensorMap* map, const void* base, unsigned long long width,
                            unsigned long long heads, unsigned long long rows,
                            unsigned long long row_bytes, unsigned int box_rows) {
  std::call_once(g_once, find_encode);
  if (!g_encode) return false;
  cuuint64_t gd[3] = {width, heads, rows};
  cuuint64_t gs[2] = {width * 2, row_bytes};
  cuuint32_t bx[3] = {64, 1, box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gd, gs,
                        bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_map_planes_sw128(CUtensorMap* map, const void* base, bool f32, unsigned long long width,
                             unsigned long long planes, unsigned long long rows,
                             unsigned long long row_bytes, unsigned int box_rows) {
  std::call_once(g_once, find_encode);
  if (!g_encode) return false;
  const unsigned int es1 = f32 ? 4 : 2;
  cuuint64_t gd[3] = {width, planes, rows};
  cuuint64_t gs[2] = {planes > 1 ? width * es1 : row_bytes, row_bytes};
  cuuint32_t bx[3] = {128 / es1, 1, box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = g_encode(
      map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
      const_cast<void*>(base), gd, gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_map_blocks_sw128(CUtensorMap* map, const void* base, unsigned long long width,
                             unsigned long long planes, unsigned long long rows,
                             unsigned long long row_bytes) {
  std::call_once(g_once, find_encode);
  if (!g_encode) return false;
  cuuint64_t gd[4] = {64, rows, width / 64, planes};
  cuuint64_t gs[3] = {row_bytes, 128, planes > 1 ? width * 2 : row_bytes};
  cuuint32_t bx[4] = {64, 64, 2, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), gd, gs,
                        bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace cat
