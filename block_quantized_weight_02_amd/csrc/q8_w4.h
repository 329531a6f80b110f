// q8_w4.h -- the products over 4-bit weights: the packed layout, and what the
// host side (q8_w4_api.cpp) and the kernels (q8_w4.hip, q8_w4_tile.h,
// q8_w4_gemm.hip) share.
//
// A weight is K x N values u of 4 bits with one 16-bit scale s, and where it has
// them one zero point z of a byte, per group of 32, 64 or 128 rows of a column:
// w = s (u - z), z = 8 where there are none.
//
// Packed values: tiles of 64 columns (N padded to T tiles), blocks of 32 rows,
// tile t's block b one KiB at (t * NB + b) * 1024.  Lane l = 16 q + i of a wave
// finds at 16 l its operand of a 16x16x32 matrix product for each of the four
// column groups g, one dword each: rows 8q .. 8q+7 of column 16 g + i.  So a block
// is one 16-byte load a lane, with nothing to move between lanes.  In a dword, row
// 2p is nibble p and row 2p + 1 nibble p + 4: one shift and one and-or bring a row
// pair into the two halves of a bf16 pair.
//
// Packed scales: a tile's groups in turn.  Groups of 128 rows: 64 scales a group,
// column 16 g + i at 4 i + g (a lane's four columns are 8 bytes).  Groups of 32 and
// 64 rows: two groups together, lane i's 8 bytes of the first, then of the second
// (16 bytes a lane).  The zero points follow all tiles' scales, in the same order.
// Pad columns and a missing second group hold zeros.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "q8_internal.h"

namespace q8 {

constexpr int kW4Chunk = 1024;   // one tile x one block of values

// Groups of a column as they are laid out (pairs of them below 128 rows).
__host__ __device__ inline int64_t w4_groups(int64_t K, int group) {
  const int64_t n = (K + group - 1) / group;
  return group == 128 ? n : (n + 1) / 2 * 2;
}
// Place of column c's scale of group j within a tile's scales (and zero points).
__host__ __device__ inline int64_t w4_scale_pos(int64_t j, int c, int group) {
  const int i = c & 15, g = c >> 4;
  return group == 128 ? j * 64 + i * 4 + g : (j >> 1) * 128 + i * 8 + (j & 1) * 4 + g;
}

// A weight as the kernels take it.
struct W4 {
  const char *values;
  const char *scales;
  const char *zeros;   // null: 8
};

struct W4Args {
  const void *x;         // bf16 m x K, or the quantized activation buffer
  W4 w, w_u;             // w_u: the gated pair's second weight
  float *y;              // m x Npad
  float *partial;        // the splits' carries (split_k > 1)
  unsigned *counters;    // one a tile, zero between calls (split_k > 1)
  int m, K, NB, Npad, T;
  int group;             // rows a group
  int scale_bf16;        // the scales are bf16, not fp16
  int split_k;
  unsigned act_scale_off, act_view_off;
  Epi ep;
};

hipError_t launch_w4_repack(const uint8_t *u, const uint16_t *s, const uint8_t *z, int64_t K,
                            int64_t N, int group, char *values, char *scales, char *zeros,
                            hipStream_t stream);
hipError_t launch_w4_unpack(const char *values, const char *scales, const char *zeros, int64_t K,
                            int64_t N, int group, uint8_t *u, uint16_t *s, uint8_t *z,
                            hipStream_t stream);

// The tile kernel: rows 4, 16, 32 or 64 (Q8_0: 8 and 24 too) a workgroup (more in chunks), its waves (8
// or 16) splitting K, each over `tiles` column tiles (the pair: both weights' tile).
struct W4Plan {
  int rows, waves, tiles;
};
hipError_t launch_w4_tile_bf16(const W4Plan &p, bool pair, const W4Args &a, hipStream_t stream);
hipError_t launch_w4_tile_q8(const W4Plan &p, bool pair, const W4Args &a, hipStream_t stream);

// The GEMM: blocks of 128 rows.
hipError_t launch_w4_gemm(int act, bool pair, const W4Args &a, hipStream_t stream);

}  // namespace q8
