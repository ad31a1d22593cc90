// zero_mx4.cuh -- the format of a microscaled 4-bit matrix (OCP Microscaling
// Formats v1.0, MXFP4): e2m1 values, one e8m0 scale for 32 consecutive
// elements of a row.
//
// data    row r starts at r * ld bytes (ld a multiple of 16): two elements a
//         byte, the even one in the low half; rows are padded with zeros to
//         whole blocks of 32
// scales  ZERO_MX4_ROWS: byte [r][b], ceil(cols / 32) a row, so that a
//         contiguous range of a flat parameter vector has a contiguous range
//         of scales and a part can be gathered like any other bytes.
//         ZERO_MX4_TILES: what the tensor cores read -- tiles of 128 rows by 4
//         blocks, 512 bytes each, byte (r % 32) * 16 + (r / 32) * 4 + b inside
//         one, the tiles of 128 rows following one another along the blocks.
//         Rows are padded to 128 and blocks to 8 (one step of the product)
//         with scale bytes of 0.
#pragma once

#include <stdint.h>

#include "zero.h"

namespace zdp {

__host__ __device__ __forceinline__ int64_t mx4_blocks(int64_t cols) { return (cols + 31) / 32; }
__host__ __device__ __forceinline__ int64_t mx4_tiles(int64_t cols) { return (cols + 255) / 256 * 2; }
__host__ __device__ __forceinline__ int64_t mx4_scale_bytes(int64_t rows, int64_t cols, int layout) {
    return layout == ZERO_MX4_ROWS ? rows * mx4_blocks(cols) : (rows + 127) / 128 * mx4_tiles(cols) * 512;
}
// Byte of the scale of (row, block) in the tiled layout.
__host__ __device__ __forceinline__ int64_t mx4_tiled_at(int64_t r, int64_t b, int64_t tiles) {
    return ((r >> 7) * tiles + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

int check_mx4(const zero_mx4* m, const char* call, const char* what);

}  // namespace zdp
