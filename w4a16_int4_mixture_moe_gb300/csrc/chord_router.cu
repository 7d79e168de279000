// Router logits: bf16 activations times the router's weights, FP32 sums and result.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chord_common.cuh"
#include "chord_internal.h"
#include "chord_rows.cuh"

namespace chord {
namespace {

struct LogitArgs {
    const __nv_bfloat16* x;
    int64_t stride;
    int T;
    const __nv_bfloat16* W;   // [parts, E, H]
    int parts, E, H;
    float* out;
};

constexpr int kFewTokens = 16;

// A warp per logit.
__global__ void __launch_bounds__(256) logits_kernel(const LogitArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)a.T * a.E;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * 8) {
        int e;
        const int64_t t = divmod_idx(i, a.E, e);
        float sum = 0.0f;
        for (int p = a.parts - 1; p >= 0; --p) {
            const __nv_bfloat16* w = a.W + ((int64_t)p * a.E + e) * a.H;
            const __nv_bfloat16* x = a.x + t * a.stride;
            for (int k = lane; k < a.H; k += 32) sum = fmaf(__bfloat162float(x[k]), __bfloat162float(w[k]), sum);
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) a.out[i] = sum;
    }
}

// Eight significant bits a part, cut off towards zero: the three parts add up to the number
// exactly (down to 2^-110, where the last part's bits end), and none overflows.  An infinity
// or NaN is the first part alone.
__global__ void __launch_bounds__(256) split_kernel(const float* __restrict__ w, int64_t n, __nv_bfloat16* __restrict__ parts) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float v = w[i];
        const bool finite = fabsf(v) <= 3.4028235e38f;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const __nv_bfloat16 h = finite ? __float2bfloat16_rz(v) : __float2bfloat16_rn(p ? 0.0f : v);
            parts[p * n + i] = h;
            v = finite ? v - __bfloat162float(h) : 0.0f;
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

chord_status chord_router_split_weights(const float* W, int64_t n, void* parts, void* stream) {
    if (n < 0 || (n > 0 && (!W || !parts || (reinterpret_cast<uintptr_t>(W) & 3) || (reinterpret_cast<uintptr_t>(parts) & 1))))
        return CHORD_ERR_INVALID_ARG;
    if (n > INT64_MAX / 8) return CHORD_ERR_UNSUPPORTED;
    if (n == 0) return CHORD_OK;
    const int64_t blocks = ceil_div64(n, 256);
    split_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        W, n, static_cast<__nv_bfloat16*>(parts));
    return cudaGetLastError() == cudaSuccess ? CHORD_OK : CHORD_ERR_CUDA;
}

chord_status chord_router_logits(const void* x, int64_t x_stride, int T, const void* W, int parts, int E, int H, float* logits,
                                 const chord_opts* opts, void* stream) {
    if (T < 0 || E <= 0 || H <= 0 || x_stride < (T > 1 ? H : 0)) return CHORD_ERR_INVALID_ARG;
    if ((parts != 1 && parts != 3) || E > 1024 || H % 8 || (T > 1 && x_stride % 8)) return CHORD_ERR_UNSUPPORTED;
    if (!W || !aligned16(W)) return CHORD_ERR_INVALID_ARG;
    if (T > 0 && (!x || !aligned16(x) || !logits || (reinterpret_cast<uintptr_t>(logits) & 3))) return CHORD_ERR_INVALID_ARG;
    if (T == 0) return CHORD_OK;
    LogitArgs a{static_cast<const __nv_bfloat16*>(x), x_stride, T, static_cast<const __nv_bfloat16*>(W), parts, E, H, logits};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T <= kFewTokens) {
        const int64_t blocks = ceil_div64((int64_t)T * E, 8);
        logits_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(a);
        return cudaGetLastError() == cudaSuccess ? CHORD_OK : CHORD_ERR_CUDA;
    }
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    RowsArgs r{};
    r.x = x, r.x_rows = T, r.x_stride = T > 1 ? x_stride : H;
    r.W = W, r.w_rows = (int64_t)parts * E, r.K = H, r.parts = parts, r.part_rows = E;
    r.nb = T >= 64 ? 64 : (T + 15) / 16 * 16;
    const int64_t tiles = ceil_div64(T, r.nb);
    const int m_tiles = (E + 127) / 128;
    // three tiles of 128 experts share the tokens' copy; fewer where that leaves SMs idle even with K cut in eight
    r.groups = tiles * ((m_tiles + 2) / 3) * 8 < di.sm_count ? m_tiles : (m_tiles + 2) / 3;
    r.R = ((E + r.groups - 1) / r.groups + 7) / 8 * 8;
    r.items = tiles * r.groups;
    r.E = E, r.out = logits, r.err = di.err;
    r.splits = rows_splits(r.R, r.nb, (H + 63) / 64 * parts, r.items, di.sm_count);
    if (launch_rows(r, pdl_enabled(), st) != cudaSuccess || cudaGetLastError() != cudaSuccess) return CHORD_ERR_CUDA;
    if (!opts || !opts->validate) return CHORD_OK;
    int32_t code = 0;
    const chord_status s = chord_get_device_error(stream, &code);
    if (s != CHORD_OK) return s;
    if (code == CHORD_DEV_TIMEOUT) return CHORD_ERR_TIMEOUT;
    return code ? CHORD_ERR_DEVICE_VALIDATION : CHORD_OK;
}

}  // extern "C"
