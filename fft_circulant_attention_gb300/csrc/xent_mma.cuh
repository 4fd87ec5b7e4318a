// Products of the cross entropy on the tensor cores (xent_mma.cu).
#pragma once
#include <cuda.h>

#include "cat_internal.h"

namespace cat {

constexpr int kXtM = 256;                // rows of a tile (a pair of CTAs)
constexpr int kXtN = 256;                // its columns
constexpr int kXtK = 64;                 // K of a stage: 128 bytes of bf16

// Operands and results as tensors of bf16 terms (one, or three of fp32 values),
// [row][term][column], in boxes of 64 columns by 128 rows; "r": by rows, as
// (64 columns, row, block of 64 columns, term) in boxes of 64 by 64 rows by two
// blocks (where the user's rows are not whole blocks: as the others, 64 rows a
// box).  Results by 32 rows.
struct XentMaps {
  CUtensorMap x, xr;                     // X itself (bf16 rows on 16-byte boundaries)
  CUtensorMap xp, xpr;                   // the list's rows of X
  CUtensorMap w, wr;                     // W
  CUtensorMap d, dr;                     // d of two pieces, one after the other
  CUtensorMap acc;                       // dX in fp32: slices of rows of the list
  CUtensorMap dw;                        // dW
};

// Slices of a piece's K that DX is cut into where it has few tiles, each with rows
// of its own: as many as give each pair of CTAs a tile, at least eight K stages a
// slice.
__host__ __device__ inline int xent_slices(int pairs, int mt, int nt, int piece, int acc_tiles) {
  if (mt < 1) return 1;
  int s = pairs / (mt * nt);
  if (s > acc_tiles / mt) s = acc_tiles / mt;
  if (s > piece / (8 * kXtK)) s = piece / (8 * kXtK);
  return s < 1 ? 1 : s;
}

// One launch: the forward's runs, or up to three kinds of a backward's work.
struct XentMma {
  int V, D;
  int rows;                              // rows of X and of one piece of d (allocated)
  int piece;                             // columns of a piece of d
  int lse;                               // 1: the forward, `run` tiles of the vocabulary a part
  int run;
  int dw_piece, dx_piece, d_piece;       // pieces to work on, -1: none
  int pairs;                             // pairs of CTAs that the device holds
  int acc_tiles;                         // row tiles that dX's slices have room for
  int two_w;                             // wr takes two boxes
  int first, dw_tma;                     // dx_piece is the first; dW's rows fit a tensor map
  int ld;                                // part's rows
  const int* count;                      // [0] rows of the list, [1] 1: it is X itself
  const int* tgt;
  const int* rows_of;                    // the list's tokens
  const void* x; const void* w;          // X and W as they are
  const float2* stat;
  const float* factor;                   // of dW (d is without it), or null: 1
  float* hit;
  float2* part;
  void* d;
  void* dw;
  unsigned int* status;
};

// longest: of the sums over K that a tile takes.
cudaError_t launch_xent_mma(const XentMaps& maps, const XentMma& a, int dtype, int clusters,
                            long long longest, cudaStream_t st);
// Host: [rows][planes][width] of bf16 (or fp32) with rows row_bytes apart, boxes
// of 128 bytes by box_rows rows, 128-byte swizzle.
bool encode_map_planes_sw128(CUtensorMap* map, const void* base, bool f32, unsigned long long width,
                             unsigned long long planes, unsigned long long rows,
                             unsigned long long row_bytes, unsigned int box_rows);

// The same rows as (64 columns, row, block of 64 columns, plane), width a multiple
// of 64, boxes of 64 rows by two blocks.
bool encode_map_blocks_sw128(CUtensorMap* map, const void* base, unsigned long long width,
                             unsigned long long planes, unsigned long long rows,
                             unsigned long long row_bytes);

}  // namespace cat
