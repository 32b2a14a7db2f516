// The order in which the NVFP4 products take block scales (internal header).
//
// tcgen05.mma with one scale per 16 values reads, for a step of 64 columns, four
// E4M3 bytes per row from TMEM: row r of 128 in lane r % 32, 32-bit column r / 32,
// the four blocks of the step in the four bytes. tcgen05.cp brings 32 x 16 bytes of
// shared memory there as they lie, so the scales are kept in memory as tiles of 128
// rows x 4 blocks of 512 bytes: byte (r, j) of a tile at 16 (r % 32) + 4 (r / 32) + j.
// The tiles of 128 rows follow one another by their four blocks, and a stage of
// several steps is one contiguous piece.
//
// Rows of group g of a batch (tokens offsets[g] .. offsets[g+1]) start on a tile of
// their own: tile offsets[g] / 128 + g, which needs no sum over the earlier groups
// and leaves room for them, since floor((a + n) / 128) + 1 >= floor(a / 128) +
// ceil(n / 128). A batch of n rows in G groups takes n / 128 + G tiles of rows.
#pragma once

#include <stdint.h>

namespace lh {

constexpr int kTileRows = 128;
constexpr int kTileBytes = 512;

__host__ __device__ __forceinline__ int64_t scale_steps(int64_t c_in) { return (c_in + 63) / 64; }
__host__ __device__ __forceinline__ int64_t group_tile(int64_t first_row, int64_t g) { return first_row / kTileRows + g; }

}  // namespace lh
