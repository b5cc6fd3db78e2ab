// Where the codes and scales of a microscaled 4-bit matrix stand, as plain functions of its sizes: the kernels
// and host programs alike compute with these.
#pragma once

#include "../../include/dit.h"

#ifdef __CUDACC__
#define DIT_HOST_DEVICE __host__ __device__
#else
#define DIT_HOST_DEVICE
#endif

namespace dit {

// Code bytes of a row: two codes per byte (even column in the low half), rows padded with zero codes
// to whole 32 columns, so every row starts on 16 bytes (the TMA's rule for strides).
DIT_HOST_DEVICE constexpr long long fp4_code_row_bytes(int cols) { return (cols + 31LL) / 32 * 16; }
// Groups of four blocks along a row (the last one padded).
DIT_HOST_DEVICE constexpr int fp4_groups(int fmt, int cols) {
  const int block = fmt == DIT_FP4_NV ? 16 : 32;
  return (cols + 4 * block - 1) / (4 * block);
}
// Scale bytes stand in tiles of 128 rows x 4 blocks, 512 bytes each, the tiles of a 128-row band one
// after another: inside a tile row r is at 16 (r % 32) + 4 (r / 32), its four blocks consecutive. This
// is the order tcgen05.cp (32 x 128 bit) spreads over tensor memory for the block-scaled MMA.
DIT_HOST_DEVICE constexpr long long fp4_scale_row(int fmt, int row, int cols) {
  return (long long)(row >> 7) * fp4_groups(fmt, cols) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}
// (64 bits: from 2^24 blocks on, a band's tiles of one row reach past 2 GB.)
DIT_HOST_DEVICE constexpr long long fp4_scale_block(int block) { return (block >> 2) * 512LL + (block & 3); }

}  // namespace dit
