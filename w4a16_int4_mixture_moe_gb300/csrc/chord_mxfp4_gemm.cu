// Microscaled 4-bit product: both operands in CHORD_LAYOUT_MXFP4,
//   C[p, n] = sum_k a[row(p), k] * w[e, n, k]     (FP32 sums),
// dense (one weight matrix, row p of C is row p of a) or grouped by expert
// through the routing arrays of chord_moe_align.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "chord_internal.h"
#include "chord_mxfp4.cuh"

namespace chord {
namespace {

struct MxGemmArgs {
    const uint8_t* a;        // groups of a_rows rows (grouped: one group per align block)
    const uint8_t* w;        // E groups of N rows
    int64_t a_groups, a_rows;
    int E, N, K;
    const int32_t* sorted_ids;   // null: dense
    const int32_t* expert_ids;
    const int32_t* ntp;
    int64_t num_pairs;
    void* C;
    int out_f32;
    int* err;
};

__device__ __forceinline__ float group_dot(uint4 x, uint4 w) {
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {w.x, w.y, w.z, w.w};
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        s = fmaf(e2m1_f32((a[i >> 3] >> (4 * (i & 7))) & 15u), e2m1_f32((b[i >> 3] >> (4 * (i & 7))) & 15u), s);
    return s;
}

// One thread per output element.
__global__ void mx_gemm_kernel(MxGemmArgs g) {
    if (!mx_header_ok(g.a, g.a_groups, g.a_rows, g.K) || !mx_header_ok(g.w, g.E, g.N, g.K)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_error(g.err, CHORD_DEV_BAD_HEADER);
        return;
    }
    const int n = blockIdx.x * blockDim.x + threadIdx.x;
    int64_t rows = g.a_groups * g.a_rows;
    if (g.ntp) {
        const int64_t ntp = *g.ntp;
        if (ntp < 0 || ntp > rows || ntp % g.a_rows) {
            if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_error(g.err, CHORD_DEV_BAD_PADDED);
            return;
        }
        rows = ntp;
    }
    if (n >= g.N) return;
    const int64_t kb = mx_col_tiles(g.K), art = mx_row_tiles(g.a_rows), wrt = mx_row_tiles(g.N);
    for (int64_t i = blockIdx.y; i < rows; i += gridDim.y) {
        int64_t grp = 0, ar = i, p = i;
        int e = 0;
        if (g.sorted_ids) {
            grp = i / g.a_rows;
            ar = i % g.a_rows;
            p = g.sorted_ids[i];
            e = g.expert_ids[grp];
            if (e < 0 || e >= g.E) {
                if (n == 0) set_error(g.err, CHORD_DEV_BAD_EXPERT);
                continue;
            }
            if (p < 0 || p >= g.num_pairs) {
                if (p != g.num_pairs && n == 0) set_error(g.err, CHORD_DEV_BAD_ROW);
                continue;
            }
        }
        const uint8_t* at = g.a + kHeaderBytes + (grp * art + ar / kMxTileRows) * kb * kMxTileBytes;
        const uint8_t* wt = g.w + kHeaderBytes + ((int64_t)e * wrt + n / kMxTileRows) * kb * kMxTileBytes;
        const uint32_t r = (uint32_t)(ar % kMxTileRows), q = (uint32_t)(n % kMxTileRows);
        float sum = 0.0f;
        for (int k = 0; k < g.K / kGroup; ++k) {
            const uint8_t* a = at + (k >> 3) * (int64_t)kMxTileBytes;
            const uint8_t* w = wt + (k >> 3) * (int64_t)kMxTileBytes;
            const uint32_t j = k & 7;
            const float d = group_dot(*reinterpret_cast<const uint4*>(a + mx_code_offset(r, j)),
                                      *reinterpret_cast<const uint4*>(w + mx_code_offset(q, j)));
            sum += d * mx_scale_f32(a[mx_scale_offset(r, j)]) * mx_scale_f32(w[mx_scale_offset(q, j)]);
        }
        if (g.out_f32)
            static_cast<float*>(g.C)[p * g.N + n] = sum;
        else
            static_cast<__nv_bfloat16*>(g.C)[p * g.N + n] = __float2bfloat16_rn(sum);
    }
}

cudaError_t launch_mx_gemm(const MxGemmArgs& g, cudaStream_t st) {
    const int64_t rows = g.a_groups * g.a_rows;
    const dim3 grid((unsigned)((g.N + 127) / 128), (unsigned)(rows < 65535 ? rows : 65535));
    mx_gemm_kernel<<<grid, 128, 0, st>>>(g);
    return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMxMaxBlockM = 224;

// After a call in validate mode: wait for it and turn the error word into a status.
chord_status mx_finish(const chord_opts* o, cudaStream_t st) {
    if (cudaGetLastError() != cudaSuccess) return CHORD_ERR_CUDA;
    if (!o || !o->validate) return CHORD_OK;
    int32_t code = 0;
    const chord_status s = chord_get_device_error(st, &code);
    if (s != CHORD_OK) return s;
    if (code == CHORD_DEV_TIMEOUT) return CHORD_ERR_TIMEOUT;
    return code ? CHORD_ERR_DEVICE_VALIDATION : CHORD_OK;
}

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

int chord_mxfp4_select_block_m(int T, int topk, int E_local, int E_global) {
    const int eg = E_global > 0 ? E_global : (E_local > 0 ? E_local : 1);
    const double tok_e = (double)T * (double)(topk > 0 ? topk : 1) / (double)eg;
    // rows that an expert rarely exceeds (mean + 3 sd of a Poisson count), in
    // as few equal blocks as the kernel's largest allows
    const double need = tok_e + 3.0 * sqrt(tok_e) + 1.0;
    const double blocks = ceil(need / kMxMaxBlockM);
    const int bm = (int)ceil(need / blocks / 32.0) * 32;
    return bm > kMxMaxBlockM ? kMxMaxBlockM : bm;
}

chord_status chord_mxfp4_moe_gemm(const void* Aq, size_t aq_bytes, const void* packed, size_t packed_bytes, int E,
                                  int N, int K, const int32_t* sorted_ids, const int32_t* expert_ids,
                                  const int32_t* num_tokens_padded, int64_t capacity, int block_m, int64_t num_pairs,
                                  void* C, int c_dtype, const chord_opts* opts, void* stream) {
    if (E <= 0 || N <= 0 || K <= 0 || block_m <= 0 || capacity < 0 || num_pairs < 0) return CHORD_ERR_INVALID_ARG;
    if (K % kGroup || block_m % 32 || block_m > kMxMaxBlockM || num_pairs >= INT32_MAX || capacity >= INT32_MAX)
        return CHORD_ERR_UNSUPPORTED;
    if (capacity % block_m || (c_dtype != CHORD_DTYPE_BF16 && c_dtype != CHORD_DTYPE_F32)) return CHORD_ERR_INVALID_ARG;
    if (packed_bytes != chord_mxfp4_bytes(E, N, K) || aq_bytes != chord_mxfp4_rows_bytes(capacity, block_m, K))
        return CHORD_ERR_LAYOUT_MISMATCH;
    if (!packed || !aligned16(packed) || !Aq || !aligned16(Aq) || !num_tokens_padded ||
        (capacity > 0 && (!sorted_ids || !expert_ids)) || (num_pairs > 0 && (!C || !aligned16(C))))
        return CHORD_ERR_INVALID_ARG;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    if (capacity == 0 || num_pairs == 0) return CHORD_OK;
    MxGemmArgs g{static_cast<const uint8_t*>(Aq), static_cast<const uint8_t*>(packed), capacity / block_m, block_m, E,
                 N, K, sorted_ids, expert_ids, num_tokens_padded, num_pairs, C, c_dtype == CHORD_DTYPE_F32, di.err};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_mx_gemm(g, st) != cudaSuccess) return CHORD_ERR_CUDA;
    return mx_finish(opts, st);
}

chord_status chord_mxfp4_gemm(const void* Aq, size_t aq_bytes, int64_t M, const void* packed, size_t packed_bytes,
                              int N, int K, void* C, int c_dtype, const chord_opts* opts, void* stream) {
    if (M < 0 || N <= 0 || K <= 0 || (c_dtype != CHORD_DTYPE_BF16 && c_dtype != CHORD_DTYPE_F32))
        return CHORD_ERR_INVALID_ARG;
    if (K % kGroup || M >= INT32_MAX) return CHORD_ERR_UNSUPPORTED;
    if (packed_bytes != chord_mxfp4_bytes(1, N, K) || aq_bytes != chord_mxfp4_bytes(1, M, K))
        return CHORD_ERR_LAYOUT_MISMATCH;
    if (!packed || !aligned16(packed) || !Aq || !aligned16(Aq) || (M > 0 && (!C || !aligned16(C))))
        return CHORD_ERR_INVALID_ARG;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    if (M == 0) return CHORD_OK;
    MxGemmArgs g{static_cast<const uint8_t*>(Aq), static_cast<const uint8_t*>(packed), 1, M, 1, N, K, nullptr,
                 nullptr, nullptr, M, C, c_dtype == CHORD_DTYPE_F32, di.err};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_mx_gemm(g, st) != cudaSuccess) return CHORD_ERR_CUDA;
    return mx_finish(opts, st);
}

}  // extern "C"
