// Low-rank adapters of many requests beside a projection that they share:
//   y[p] = base[p] + scale[a] * B[a, e] (A[a, e] x[p / div])
// in two steps, v = A x (FP32, in the workspace) and y = base + scale * B v.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chord_common.cuh"
#include "chord_internal.h"

namespace chord {
namespace {

struct AdapterArgs {
    const __nv_bfloat16* x;
    int64_t x_stride;
    int div;
    const int32_t* adapter_ids;   // [T]
    const int32_t* topk_ids;      // [T, topk], null: one projection
    int64_t P;
    int topk, S, E;
    const __nv_bfloat16* A;       // [S, E, parts * rank, K]
    const __nv_bfloat16* B;       // [S, E, N, rank]
    const float* scale;           // [S], null: 1
    int rank, parts, N, K;
    const void* base;
    void* y;
    int f32;
    int64_t base_stride, y_stride;
    float* v;                     // [P, parts * rank]
    int* err;
};

// Slot of pair p: adapter * E + expert; -1: no adapter, the row is base's; -2: the pair's expert is on another GPU.
__device__ __forceinline__ int64_t slot_of(const AdapterArgs& g, int64_t p, bool report) {
    int64_t e = 0;
    if (g.topk_ids) {
        e = g.topk_ids[p];
        if (e < 0 || e >= g.E) return -2;
    }
    int k;
    const int a = g.adapter_ids[divmod_idx(p, g.topk, k)];
    if (a < 0 || a >= g.S) {
        if (a != -1 && report) set_error(g.err, CHORD_DEV_BAD_ADAPTER);
        return -1;
    }
    return (int64_t)a * g.E + e;
}

__global__ void __launch_bounds__(256) adapter_down_kernel(const AdapterArgs g) {
    const int lane = threadIdx.x & 31, R = g.rank * g.parts;
    const int64_t n = g.P * R;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * 8) {
        int j, q;
        const int64_t p = divmod_idx(i, R, j), s = slot_of(g, p, lane == 0);
        if (s < 0) continue;
        const __nv_bfloat16* w = g.A + (s * R + j) * g.K;
        const __nv_bfloat16* x = g.x + divmod_idx(p, g.div, q) * g.x_stride;
        float sum = 0.0f;
        for (int k = lane; k < g.K; k += 32) sum = fmaf(__bfloat162float(x[k]), __bfloat162float(w[k]), sum);
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) g.v[i] = sum;
    }
}

__global__ void __launch_bounds__(256) adapter_up_kernel(const AdapterArgs g) {
    const int64_t n = g.P * g.N;
    const int R = g.rank * g.parts;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        int c;
        const int64_t p = divmod_idx(i, g.N, c), s = slot_of(g, p, false);
        const int64_t from = p * g.base_stride + c, to = p * g.y_stride + c;
        if (s == -2 || (s == -1 && g.base == g.y)) continue;
        float sum = 0.0f;
        if (s >= 0) {
            const __nv_bfloat16* b = g.B + (s * g.N + c) * g.rank;
            const float* v = g.v + p * R + c / (g.N / g.parts) * g.rank;
            for (int k = 0; k < g.rank; ++k) sum = fmaf(v[k], __bfloat162float(b[k]), sum);
            if (g.scale) sum *= g.scale[s / g.E];
        }
        if (g.f32) {
            const float o = static_cast<const float*>(g.base)[from];
            static_cast<float*>(g.y)[to] = s >= 0 ? o + sum : o;
        } else {
            const __nv_bfloat16 o = static_cast<const __nv_bfloat16*>(g.base)[from];
            static_cast<__nv_bfloat16*>(g.y)[to] = s >= 0 ? __float2bfloat16_rn(__bfloat162float(o) + sum) : o;
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The bytes from a to a + na and from b to b + nb have one in common.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

size_t chord_adapter_workspace_bytes(int64_t T, int topk, int adapters, int E, int rank, int parts) {
    if (T < 0 || topk <= 0 || adapters <= 0 || E <= 0 || rank <= 0 || parts <= 0 || rank > 128 || parts > 4) return 0;
    if (T > INT32_MAX / topk || adapters > 65536 / E) return 0;
    return ((size_t)T * topk * rank * parts * 4 + 255) / 256 * 256 + 256;
}

chord_status chord_adapter_add(const void* x, int64_t x_rows, int64_t x_stride, int a_row_divisor, const int32_t* adapter_ids,
                               const int32_t* topk_ids, int T, int topk, int adapters, int E, const void* A, const void* B,
                               const float* scale, int rank, int parts, int N, int K, const void* base, int64_t base_stride,
                               void* y, int64_t y_stride, int y_dtype, void* workspace, size_t workspace_bytes,
                               const chord_opts* opts, void* stream) {
    if (T < 0 || topk <= 0 || adapters <= 0 || E <= 0 || rank <= 0 || parts <= 0 || N <= 0 || K <= 0 || a_row_divisor <= 0 ||
        x_rows < 0 || (y_dtype != CHORD_DTYPE_BF16 && y_dtype != CHORD_DTYPE_F32))
        return CHORD_ERR_INVALID_ARG;
    const int64_t P = (int64_t)T * topk;
    const int per = y_dtype == CHORD_DTYPE_F32 ? 4 : 8;
    if (P >= INT32_MAX || adapters > 65536 / E || rank % 8 || rank > 128 || parts > 4 || N % (8 * parts) || K % 8)
        return CHORD_ERR_UNSUPPORTED;
    if (!topk_ids && E != 1) return CHORD_ERR_INVALID_ARG;
    if (P == 0) return CHORD_OK;
    if ((P - 1) / a_row_divisor >= x_rows) return CHORD_ERR_INVALID_ARG;
    // the stride of a single row is not used
    if (P <= a_row_divisor) x_stride = K;
    if (P == 1) base_stride = y_stride = N;
    if (x_stride < K || base_stride < N || y_stride < N) return CHORD_ERR_INVALID_ARG;
    if (x_stride % 8 || base_stride % per || y_stride % per) return CHORD_ERR_UNSUPPORTED;
    if (!x || !aligned16(x) || !adapter_ids || !A || !aligned16(A) || !B || !aligned16(B) || !base || !aligned16(base) || !y ||
        !aligned16(y) || !workspace || !aligned16(workspace))
        return CHORD_ERR_INVALID_ARG;
    const int64_t esize = 16 / per;
    const int64_t y_bytes = ((P - 1) * y_stride + N) * esize, base_bytes = ((P - 1) * base_stride + N) * esize;
    const int64_t x_bytes = ((P - 1) / a_row_divisor * x_stride + K) * 2;
    if (overlap(y, y_bytes, x, x_bytes) || (base == y ? base_stride != y_stride : overlap(y, y_bytes, base, base_bytes)))
        return CHORD_ERR_INVALID_ARG;
    if (workspace_bytes < chord_adapter_workspace_bytes(T, topk, adapters, E, rank, parts)) return CHORD_ERR_BUFFER_TOO_SMALL;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    AdapterArgs g{static_cast<const __nv_bfloat16*>(x), x_stride, a_row_divisor, adapter_ids, topk_ids, P, topk, adapters, E,
                  static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B), scale, rank, parts, N, K, base, y,
                  y_dtype == CHORD_DTYPE_F32, base_stride, y_stride, static_cast<float*>(workspace), di.err};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t down = ceil_div64(P * rank * parts, 8), up = ceil_div64(P * N, 256);
    adapter_down_kernel<<<(unsigned)(down < 65536 ? down : 65536), 256, 0, st>>>(g);
    adapter_up_kernel<<<(unsigned)(up < 65536 ? up : 65536), 256, 0, st>>>(g);
    if (cudaGetLastError() != cudaSuccess) return CHORD_ERR_CUDA;
    if (!opts || !opts->validate) return CHORD_OK;
    int32_t code = 0;
    const chord_status s = chord_get_device_error(stream, &code);
    if (s != CHORD_OK) return s;
    if (code == CHORD_DEV_TIMEOUT) return CHORD_ERR_TIMEOUT;
    return code ? CHORD_ERR_DEVICE_VALIDATION : CHORD_OK;
}

}  // extern "C"
