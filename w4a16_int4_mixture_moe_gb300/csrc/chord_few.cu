// One mixture-of-experts layer for a few tokens (at most CHORD_FEW_MAX_TOKENS),
// expert weights in 4 bits:
//   h[t, e]   = topk_w[t, e] * SiLU(W13[e][:I] x_t) * (W13[e][I:] x_t)
//   out[t]    = bf16( sum over the token's local experts of W2[e] h[t, e] )
// in two launches: gate_up with the activation and the routing weight, then
// the down projection with the sum over the experts.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chord_internal.h"
#include "chord_mxfp4.cuh"

namespace chord {
namespace {

struct FewArgs {
    const uint16_t* x;
    const int32_t* ids;
    const float* wts;
    int T, topk, E, H, I;
    int mx;              // weights: 0 INT4 blobs, 1 MXFP4
    const uint8_t* w13;
    const uint8_t* w2;
    float* h;            // [T * topk, I]
    uint16_t* out;
    int* err;
    int validate;        // report ids outside [-1, E)
};

__device__ __forceinline__ float bf(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// 32 consecutive columns (group j) of row `row` of expert e.
__device__ __forceinline__ void weights32(const uint8_t* blob, int mx, int e, int row, int N, int K, int j, float* v) {
    if (mx) {
        const uint8_t* t = blob + kHeaderBytes +
                           (((int64_t)e * mx_row_tiles(N) + row / 128) * mx_col_tiles(K) + j / 8) * kMxTileBytes;
        const uint4 c = *reinterpret_cast<const uint4*>(t + mx_code_offset(row % 128, j % 8));
        const float s = mx_scale_f32(t[mx_scale_offset(row % 128, j % 8)]);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        for (int i = 0; i < 32; ++i) v[i] = e2m1_f32((w[i >> 3] >> (4 * (i & 7))) & 15u) * s;
        return;
    }
    const uint8_t* t = blob + kHeaderBytes +
                       (uint64_t)e * ((uint64_t)N * (uint64_t)K * 9ull / 16ull) + ((int64_t)(row / 128) * (K / 64) + j / 2) * 4608;
    const int r = row % 128, hf = j & 1;
    const uint4 c = *reinterpret_cast<const uint4*>(t + hf * 2048 + r * 16);
    const uint32_t s = *reinterpret_cast<const uint16_t*>(t + 4096 + r * 4 + 2 * hf);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t d[16];
    for (int i = 0; i < 4; ++i) dequant_row8(w[i], s | (s << 16), d + 4 * i);
    for (int i = 0; i < 16; ++i) {
        v[2 * i] = __uint_as_float(d[i] << 16);
        v[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
    }
}

// Gate and up rows of column c in the packed w13; false: not a w13 of this shape.
__device__ __forceinline__ bool gate_up_rows(const FewArgs& a, int c, int& rg, int& ru) {
    rg = c;
    ru = a.I + c;
    if (a.mx) return mx_header_ok(a.w13, a.E, 2 * a.I, a.H);
    if (header_ok_layout(a.w13, a.E, 2 * a.I, a.H, CHORD_LAYOUT_TCGEN05)) return true;
    rg = 16 * (c / 8) + c % 8;
    ru = rg + 8;
    return header_ok_layout(a.w13, a.E, 2 * a.I, a.H, CHORD_LAYOUT_GATE_UP_INTERLEAVED);
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp per (pair, column of I).
__global__ void few_gate_up_kernel(FewArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t q = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (q >= (int64_t)a.T * a.topk * a.I) return;
    const int p = (int)(q / a.I), c = (int)(q % a.I);
    const int e = a.ids[p];
    if (a.validate && lane == 0 && c == 0 && (e < -1 || e >= a.E)) set_error(a.err, CHORD_DEV_BAD_EXPERT);
    if (e < 0 || e >= a.E) return;
    int rg, ru;
    if (!gate_up_rows(a, c, rg, ru)) {
        set_error(a.err, CHORD_DEV_BAD_HEADER);
        return;
    }
    const uint16_t* x = a.x + (int64_t)(p / a.topk) * a.H;
    float g = 0.0f, u = 0.0f;
    for (int j = lane; j < a.H / kGroup; j += 32) {
        float vg[32], vu[32];
        weights32(a.w13, a.mx, e, rg, 2 * a.I, a.H, j, vg);
        weights32(a.w13, a.mx, e, ru, 2 * a.I, a.H, j, vu);
        for (int i = 0; i < 32; ++i) {
            const float xv = bf(x[j * 32 + i]);
            g = fmaf(xv, vg[i], g);
            u = fmaf(xv, vu[i], u);
        }
    }
    g = warp_sum(g);
    u = warp_sum(u);
    if (lane == 0) a.h[(int64_t)p * a.I + c] = a.wts[p] * silu_times(g, u);
}

// One warp per (token, column of H).
__global__ void few_down_kernel(FewArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t q = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (q >= (int64_t)a.T * a.H) return;
    const int t = (int)(q / a.H), n = (int)(q % a.H);
    const bool ok = a.mx ? mx_header_ok(a.w2, a.E, a.H, a.I) : header_ok_layout(a.w2, a.E, a.H, a.I, CHORD_LAYOUT_TCGEN05);
    if (!ok) {
        set_error(a.err, CHORD_DEV_BAD_HEADER);
        return;
    }
    float s = 0.0f;
    for (int k = 0; k < a.topk; ++k) {
        const int p = t * a.topk + k, e = a.ids[p];
        if (e < 0 || e >= a.E) continue;
        for (int j = lane; j < a.I / kGroup; j += 32) {
            float v[32];
            weights32(a.w2, a.mx, e, n, a.H, a.I, j, v);
            for (int i = 0; i < 32; ++i) s = fmaf(a.h[(int64_t)p * a.I + j * 32 + i], v[i], s);
        }
    }
    s = warp_sum(s);
    if (lane == 0) a.out[(int64_t)t * a.H + n] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
}

cudaError_t launch_few(const FewArgs& a, cudaStream_t st) {
    const int64_t w1 = (int64_t)a.T * a.topk * a.I, w2 = (int64_t)a.T * a.H;
    few_gate_up_kernel<<<(unsigned)((w1 + 7) / 8), 256, 0, st>>>(a);
    few_down_kernel<<<(unsigned)((w2 + 7) / 8), 256, 0, st>>>(a);
    return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

size_t chord_moe_few_workspace_bytes(int T, int topk, int E, int H, int I) {
    if (T < 0 || topk <= 0 || E <= 0 || H <= 0 || I <= 0) return 0;
    return ((size_t)T * (size_t)topk * (size_t)I * 4 + 255) / 256 * 256;
}

chord_status chord_moe_layer_few(const void* x, const int32_t* topk_ids, const float* topk_w, int T, int topk, int E,
                                 int H, int I, int weights, const void* packed_w13, size_t w13_bytes,
                                 const void* packed_w2, size_t w2_bytes, void* workspace, size_t workspace_bytes,
                                 void* out, const chord_opts* opts, void* stream) {
    if (T < 0 || topk <= 0 || E <= 0 || H <= 0 || I <= 0) return CHORD_ERR_INVALID_ARG;
    if (weights != CHORD_WEIGHTS_INT4 && weights != CHORD_WEIGHTS_MXFP4) return CHORD_ERR_INVALID_ARG;
    if (T > CHORD_FEW_MAX_TOKENS || topk > 32 || E > 1024 || H > (1 << 20) || I > (1 << 20)) return CHORD_ERR_UNSUPPORTED;
    const bool mx = weights == CHORD_WEIGHTS_MXFP4;
    if (mx ? (H % 32 || I % 32) : (H % 128 || I % 64)) return CHORD_ERR_UNSUPPORTED;
    const size_t n13 = mx ? chord_mxfp4_bytes(E, 2 * I, H) : chord_packed_weight_bytes(E, 2 * I, H, CHORD_LAYOUT_TCGEN05);
    const size_t n2 = mx ? chord_mxfp4_bytes(E, H, I) : chord_packed_weight_bytes(E, H, I, CHORD_LAYOUT_TCGEN05);
    if (w13_bytes != n13 || w2_bytes != n2) return CHORD_ERR_LAYOUT_MISMATCH;
    if (workspace_bytes < chord_moe_few_workspace_bytes(T, topk, E, H, I)) return CHORD_ERR_BUFFER_TOO_SMALL;
    if (!packed_w13 || !aligned16(packed_w13) || !packed_w2 || !aligned16(packed_w2)) return CHORD_ERR_INVALID_ARG;
    if (T == 0) return CHORD_OK;
    if (!workspace || !aligned16(workspace) || !x || !aligned16(x) || !topk_ids || !topk_w || !out || !aligned16(out))
        return CHORD_ERR_INVALID_ARG;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    FewArgs a{static_cast<const uint16_t*>(x), topk_ids, topk_w, T, topk, E, H, I, mx ? 1 : 0,
              static_cast<const uint8_t*>(packed_w13), static_cast<const uint8_t*>(packed_w2),
              static_cast<float*>(workspace), static_cast<uint16_t*>(out), di.err,
              opts && opts->validate ? 1 : 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_few(a, st) != cudaSuccess) return CHORD_ERR_CUDA;
    if (!opts || !opts->validate) return CHORD_OK;
    int32_t code = 0;
    const chord_status s = chord_get_device_error(st, &code);
    if (s != CHORD_OK) return s;
    if (code == CHORD_DEV_TIMEOUT) return CHORD_ERR_TIMEOUT;
    return code ? CHORD_ERR_DEVICE_VALIDATION : CHORD_OK;
}

}  // extern "C"
