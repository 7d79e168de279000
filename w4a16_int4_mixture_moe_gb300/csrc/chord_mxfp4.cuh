// Microscaled 4-bit matrices (CHORD_LAYOUT_MXFP4): where a code and a scale of
// row r, column k live in the packed bytes, and the values they stand for.
//
// An element is an E2M1 code (sign, two exponent bits, one mantissa bit:
// 0, .5, 1, 1.5, 2, 3, 4, 6) and every 32 consecutive columns of a row share
// an E8M0 scale 2^(b - 127), b = 255 standing for NaN (the MXFP4 format of the
// OCP Microscaling specification v1.0).  After a 256-byte header the matrix is
// a grid of tiles of 128 rows x 256 columns, 17408 bytes each, the tiles of one
// row band contiguous along K.  Inside a tile:
//   * bytes [0, 16384): row r at 128 r, its 32-column group j (16 bytes, the
//     lower column in the lower nibble) at 16 (j ^ (r mod 8)): the 128-byte
//     swizzle that the tensor cores read from shared memory, so a tile goes
//     there with one bulk copy and no rearrangement;
//   * bytes [16384, 17408): two 512-byte scale blocks, one per 128 columns, the
//     scale of row r and group j at 512 (j / 4) + 16 (r mod 32) + 4 (r / 32) +
//     j mod 4: the order in which the tensor cores take the scales of 128 rows
//     (row r mod 32 a tensor-memory lane, r / 32 a column, four groups a word).
// Rows past N and columns past K of the last tiles hold zeros with scale 1.
#pragma once

#include <stdint.h>

#include "chord_common.cuh"

namespace chord {

constexpr int kMxTileRows = 128;
constexpr int kMxTileCols = 256;
constexpr int kMxCodeBytes = kMxTileRows * kMxTileCols / 2;   // 16384
constexpr int kMxScaleBlock = 512;                            // 128 rows x 4 groups
constexpr int kMxTileBytes = kMxCodeBytes + 2 * kMxScaleBlock;

__host__ __device__ __forceinline__ int64_t mx_row_tiles(int64_t N) { return (N + kMxTileRows - 1) / kMxTileRows; }
__host__ __device__ __forceinline__ int64_t mx_col_tiles(int64_t K) { return (K + kMxTileCols - 1) / kMxTileCols; }

// Byte offset inside a tile of the 16 codes bytes of (row r, group j), r < 128, j < 8.
__host__ __device__ __forceinline__ uint32_t mx_code_offset(uint32_t r, uint32_t j) {
    return r * 128u + ((j ^ (r & 7u)) << 4);
}
__host__ __device__ __forceinline__ uint32_t mx_scale_offset(uint32_t r, uint32_t j) {
    return (uint32_t)kMxCodeBytes + (j >> 2) * (uint32_t)kMxScaleBlock + (r & 31u) * 16u + (r >> 5) * 4u + (j & 3u);
}

// Header of a matrix of G groups of N x K (same words as the INT4 blobs, the
// 64-bit group stride counting whole tiles).
__host__ __device__ __forceinline__ unsigned long long mx_group_bytes(int64_t N, int64_t K) {
    return (unsigned long long)mx_row_tiles(N) * (unsigned long long)mx_col_tiles(K) * (unsigned)kMxTileBytes;
}

__device__ __forceinline__ bool mx_header_ok(const uint8_t* blob, int64_t G, int64_t N, int K) {
    const uint32_t* h = reinterpret_cast<const uint32_t*>(blob);
    const unsigned long long* h64 = reinterpret_cast<const unsigned long long*>(blob + 32);
    return h[0] == kMagic && h[1] == 1u && h[2] == (uint32_t)CHORD_LAYOUT_MXFP4 && h[3] == (uint32_t)kGroup &&
           h[4] == (uint32_t)G && h[5] == (uint32_t)N && h[6] == (uint32_t)K && h64[0] == mx_group_bytes(N, K) &&
           h64[1] == (unsigned long long)kHeaderBytes;
}

// Header check by one warp, a word per lane (one memory latency).
__device__ __forceinline__ bool mx_header_ok_warp(const uint8_t* blob, int64_t G, int64_t N, int K) {
    const int i = threadIdx.x & 31;
    const unsigned long long bytes = mx_group_bytes(N, K);
    const uint32_t v = i < 12 ? reinterpret_cast<const uint32_t*>(blob)[i] : 0u;
    const uint32_t want[4] = {kMagic, 1u, (uint32_t)CHORD_LAYOUT_MXFP4, (uint32_t)kGroup};
    uint32_t w = i < 4 ? want[i & 3] : 0u;
    if (i == 4) w = (uint32_t)G;
    if (i == 5) w = (uint32_t)N;
    if (i == 6) w = (uint32_t)K;
    if (i == 8) w = (uint32_t)bytes;
    if (i == 9) w = (uint32_t)(bytes >> 32);
    if (i == 10) w = (uint32_t)kHeaderBytes;
    return __all_sync(0xffffffffu, v == w);
}

// Scale 2^(b - 127) as FP32; b = 255 is NaN, b = 0 the subnormal 2^-127.
__device__ __forceinline__ float mx_scale_f32(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FC00000u : (b == 0u ? 0x00400000u : b << 23));
}

}  // namespace chord
