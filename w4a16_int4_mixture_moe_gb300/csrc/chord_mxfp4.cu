// Microscaled 4-bit quantisation (MXFP4) of weight matrices and of routed
// activation rows, and the values a quantised matrix stands for.
//
// For 32 columns v of a row with largest magnitude a:
//   e    = floor(log2 a) - 2, clamped to [-127, 127]   (a = 0: e = -127)
//   code = the E2M1 number nearest to v * 2^-e (ties to the even code), at most 6
// stored as (codes, b = e + 127).  2 is the largest exponent of E2M1, so the
// block's largest element lands in [4, 8) and at most a third of that range
// saturates at 6 (the OCP Microscaling specification's conversion).  v * 2^-e is exact in
// FP32 (a power of two), so the only rounding is the code's.  A block that
// holds an infinity or NaN gets the NaN scale: it stays visible downstream.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chord_internal.h"
#include "chord_mxfp4.cuh"

namespace chord {
namespace {

__device__ __forceinline__ float load_elem(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Nearest E2M1 code of y (finite): ties to even, |y| above 5 to 6.
__device__ __forceinline__ uint32_t e2m1_code(float y) {
    const float a = fabsf(y);
    const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
    return c | (__float_as_uint(y) >> 31 << 3);
}

// Where the rows of a packed matrix come from: row i of group g is row
// g * N + i of src (weights), or the activation row of the pair in
// sorted_ids[g * N + i] (routed rows; no pair: row not written).
struct RowSource {
    const void* src;
    int f32;
    int64_t row_stride, mat_stride;
    const int32_t* sorted_ids;   // null: plain matrices
    const int32_t* ntp;
    int64_t id_limit;
    int divisor;
};

__global__ void mx_header_kernel(uint8_t* packed, int64_t G, int64_t N, int K) {
    const unsigned long long stride = mx_group_bytes(N, K);
    const int i = threadIdx.x;
    if (i >= kHeaderBytes / 4) return;
    uint32_t v = 0;
    switch (i) {
        case 0: v = kMagic; break;
        case 1: v = 1u; break;
        case 2: v = CHORD_LAYOUT_MXFP4; break;
        case 3: v = kGroup; break;
        case 4: v = (uint32_t)G; break;
        case 5: v = (uint32_t)N; break;
        case 6: v = (uint32_t)K; break;
        case 8: v = (uint32_t)stride; break;
        case 9: v = (uint32_t)(stride >> 32); break;
        case 10: v = kHeaderBytes; break;
        default: v = 0u;
    }
    reinterpret_cast<uint32_t*>(packed)[i] = v;
}

// One thread per (row, 32-column group) of the padded tiles.
__global__ void mx_quantize_kernel(RowSource s, int64_t G, int64_t N, int K, uint8_t* __restrict__ packed, int* err) {
    const int64_t rt = mx_row_tiles(N), kb = mx_col_tiles(K);
    int64_t groups = G;
    if (s.ntp) {
        const int64_t ntp = *s.ntp;
        if (ntp < 0 || ntp > G * N || ntp % N) {
            if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, CHORD_DEV_BAD_PADDED);
            return;
        }
        groups = ntp / N;
    }
    const int64_t total = groups * rt * kb * (kMxTileRows * 8);
    uint8_t* data = packed + kHeaderBytes;
    for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < total; q += (int64_t)gridDim.x * blockDim.x) {
        const uint32_t j = (uint32_t)(q & 7), r = (uint32_t)(q >> 3) & 127u;
        const int64_t tile = q >> 10;
        const int64_t kt = tile % kb, band = tile / kb;
        const int64_t g = band / rt, row = (band % rt) * kMxTileRows + r;
        const int64_t k0 = kt * kMxTileCols + j * 32;
        int64_t base = -1;
        if (row < N && k0 < K) {
            if (!s.sorted_ids) {
                base = g * s.mat_stride + row * s.row_stride + k0;
            } else {
                const int32_t id = s.sorted_ids[g * N + row];
                if (id >= 0 && id < s.id_limit) base = (int64_t)(id / s.divisor) * s.row_stride + k0;
            }
        }
        float v[32];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v[i] = base >= 0 ? load_elem(s.src, base + i, s.f32 != 0) : 0.0f;
            top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        }
        const uint32_t ex = top >> 23;   // biased exponent; 0 for zero and subnormals
        uint32_t b = ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
        if (base < 0) b = 127u;
        const float up = __uint_as_float((254u - min(b, 253u)) << 23);   // 2^(127 - b)
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i >> 3] |= (b == 255u ? 0u : e2m1_code(v[i] * up)) << (4 * (i & 7));
        uint8_t* t = data + tile * kMxTileBytes;
        *reinterpret_cast<uint4*>(t + mx_code_offset(r, j)) = make_uint4(w[0], w[1], w[2], w[3]);
        t[mx_scale_offset(r, j)] = (uint8_t)b;
    }
}

__global__ void mx_dequantize_kernel(const uint8_t* __restrict__ packed, int64_t G, int64_t N, int K, int f32,
                                     void* __restrict__ out, int* err) {
    if (!mx_header_ok(packed, G, N, K)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, CHORD_DEV_BAD_HEADER);
        return;
    }
    const int64_t rt = mx_row_tiles(N), kb = mx_col_tiles(K);
    const int kg = K / kGroup;
    const int64_t total = G * N * kg;
    const uint8_t* data = packed + kHeaderBytes;
    for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < total; q += (int64_t)gridDim.x * blockDim.x) {
        const int64_t grow = q / kg;
        const int jg = (int)(q % kg);
        const int64_t g = grow / N, row = grow % N;
        const uint8_t* t = data + ((g * rt + row / kMxTileRows) * kb + jg / 8) * kMxTileBytes;
        const uint32_t r = (uint32_t)(row % kMxTileRows), j = (uint32_t)(jg % 8);
        const uint4 c = *reinterpret_cast<const uint4*>(t + mx_code_offset(r, j));
        const float sc = mx_scale_f32(t[mx_scale_offset(r, j)]);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float v = e2m1_f32((w[i >> 3] >> (4 * (i & 7))) & 15u) * sc;
            const int64_t o = grow * K + jg * 32 + i;
            if (f32)
                static_cast<float*>(out)[o] = v;
            else
                static_cast<__nv_bfloat16*>(out)[o] = __float2bfloat16_rn(v);
        }
    }
}

unsigned grid_for(int64_t items, int threads) {
    const int64_t b = (items + threads - 1) / threads, cap = (int64_t)device_info().sm_count * 16;
    return (unsigned)(b < 1 ? 1 : (b > cap ? cap : b));
}

cudaError_t launch_quantize(const RowSource& s, int64_t G, int64_t N, int K, uint8_t* packed, int* err,
                            cudaStream_t st) {
    mx_header_kernel<<<1, 64, 0, st>>>(packed, G, N, K);
    const int64_t items = G * mx_row_tiles(N) * mx_col_tiles(K) * kMxTileRows * 8;
    if (items > 0) mx_quantize_kernel<<<grid_for(items, 256), 256, 0, st>>>(s, G, N, K, packed, err);
    return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known_dtype(int d) { return d == CHORD_DTYPE_BF16 || d == CHORD_DTYPE_F32; }

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

size_t chord_mxfp4_bytes(int64_t G, int64_t N, int K) {
    if (G < 0 || N < 0 || K <= 0 || K % kGroup || G > INT32_MAX || N > INT32_MAX) return 0;
    return (size_t)kHeaderBytes + (size_t)G * (size_t)mx_group_bytes(N, K);
}

size_t chord_mxfp4_rows_bytes(int64_t capacity, int block_m, int K) {
    if (capacity < 0 || block_m <= 0 || capacity % block_m) return 0;
    return chord_mxfp4_bytes(capacity / block_m, block_m, K);
}

chord_status chord_mxfp4_quantize(const void* src, int src_dtype, int64_t row_stride, int64_t mat_stride, int64_t G,
                                  int64_t N, int K, void* packed, size_t packed_bytes, void* stream) {
    if (G < 0 || N < 0 || K <= 0 || !known_dtype(src_dtype)) return CHORD_ERR_INVALID_ARG;
    if (chord_mxfp4_bytes(G, N, K) == 0) return CHORD_ERR_UNSUPPORTED;
    if (packed_bytes != chord_mxfp4_bytes(G, N, K)) return CHORD_ERR_LAYOUT_MISMATCH;
    if ((N > 1 && row_stride < K) || (G > 1 && mat_stride < 0)) return CHORD_ERR_INVALID_ARG;
    if (!packed || !aligned16(packed)) return CHORD_ERR_INVALID_ARG;
    if (G * N > 0 && (!src || !aligned_to(src, src_dtype == CHORD_DTYPE_F32 ? 4 : 2))) return CHORD_ERR_INVALID_ARG;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    RowSource s{src, src_dtype == CHORD_DTYPE_F32, row_stride, mat_stride, nullptr, nullptr, 0, 1};
    return launch_quantize(s, G, N, K, static_cast<uint8_t*>(packed), di.err, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? CHORD_OK
               : CHORD_ERR_CUDA;
}

chord_status chord_mxfp4_quantize_rows(const void* A, int a_dtype, int64_t a_rows, int64_t row_stride,
                                       int a_row_divisor, int K, const int32_t* sorted_ids,
                                       const int32_t* num_tokens_padded, int64_t capacity, int block_m,
                                       int64_t num_pairs, void* packed, size_t packed_bytes, void* stream) {
    if (a_rows < 0 || a_row_divisor <= 0 || K <= 0 || capacity < 0 || block_m <= 0 || num_pairs < 0 ||
        !known_dtype(a_dtype))
        return CHORD_ERR_INVALID_ARG;
    if (K % kGroup || num_pairs >= INT32_MAX || capacity >= INT32_MAX) return CHORD_ERR_UNSUPPORTED;
    if (capacity % block_m) return CHORD_ERR_INVALID_ARG;
    if (packed_bytes != chord_mxfp4_rows_bytes(capacity, block_m, K)) return CHORD_ERR_LAYOUT_MISMATCH;
    if (a_rows > 1 && row_stride < K) return CHORD_ERR_INVALID_ARG;
    if (!packed || !aligned16(packed) || !num_tokens_padded || (capacity > 0 && !sorted_ids))
        return CHORD_ERR_INVALID_ARG;
    if (a_rows > 0 && (!A || !aligned_to(A, a_dtype == CHORD_DTYPE_F32 ? 4 : 2))) return CHORD_ERR_INVALID_ARG;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    const int64_t limit = a_rows * (int64_t)a_row_divisor;
    RowSource s{A,         a_dtype == CHORD_DTYPE_F32, row_stride, 0, sorted_ids, num_tokens_padded,
                limit < num_pairs ? limit : num_pairs, a_row_divisor};
    return launch_quantize(s, capacity / block_m, block_m, K, static_cast<uint8_t*>(packed), di.err,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? CHORD_OK
               : CHORD_ERR_CUDA;
}

chord_status chord_mxfp4_dequantize(const void* packed, size_t packed_bytes, int64_t G, int64_t N, int K, void* out,
                                    int out_dtype, void* stream) {
    if (G < 0 || N < 0 || K <= 0 || !known_dtype(out_dtype)) return CHORD_ERR_INVALID_ARG;
    if (chord_mxfp4_bytes(G, N, K) == 0) return CHORD_ERR_UNSUPPORTED;
    if (packed_bytes != chord_mxfp4_bytes(G, N, K)) return CHORD_ERR_LAYOUT_MISMATCH;
    if (!packed || !aligned16(packed) || (G * N > 0 && (!out || !aligned16(out)))) return CHORD_ERR_INVALID_ARG;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    const int64_t items = G * N * (K / kGroup);
    if (items == 0) return CHORD_OK;
    mx_dequantize_kernel<<<grid_for(items, 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t*>(packed), G, N, K, out_dtype == CHORD_DTYPE_F32, out, di.err);
    return cudaGetLastError() == cudaSuccess ? CHORD_OK : CHORD_ERR_CUDA;
}

}  // extern "C"
