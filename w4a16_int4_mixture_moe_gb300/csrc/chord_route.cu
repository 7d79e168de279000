// Choice of experts from router logits: scores, groups, top-k, weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "chord_common.cuh"
#include "chord_internal.h"

namespace chord {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouteWarps = 4;

struct RouteArgs {
    const void* logits;
    int f32;
    int64_t stride;
    int T, E, topk;
    const float* bias;
    int score, groups, topk_groups, best, renorm;
    float scale;
    int first, local;
    int32_t* ids;
    float* w;
};

// A logit as the scores use it: +inf counts as the largest number, so that the softmax has a limit.
__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t t, int e) {
    const int64_t i = t * a.stride + e;
    const float l = a.f32 ? static_cast<const float*>(a.logits)[i]
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[i]);
    return l > FLT_MAX ? FLT_MAX : l;
}

__device__ __forceinline__ float warp_max(float v) {
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// The weights of one token's choice: lane k < topk holds choice k (expert e, its logit l; e < 0: none).
//   softmax: exp(l - m) / sum over all, renormalised exp(l - c) / sum over the chosen
//   sigmoid: 1 / (1 + exp(-l))
// Renormalised, both numerators are scaled by exp(-c) with c the largest chosen logit (sigmoid: at
// most 0), which the quotient does not change and which keeps far negative logits from all
// becoming 0.
__device__ __forceinline__ void write_choice(const RouteArgs& a, int64_t t, int lane, int e, float l, float m, float total) {
    const bool have = lane < a.topk && e >= 0;
    float s = 0.0f;
    if (a.renorm) {
        float c = warp_max(have ? l : -FLT_MAX);
        if (a.score == CHORD_SCORE_SIGMOID) {
            c = fminf(c, 0.0f);
            s = l > 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l - c) / (1.0f + expf(l));
        } else {
            s = expf(l - c);
        }
        if (!have) s = 0.0f;
        const float sum = warp_sum(s);
        s = have ? s / sum : 0.0f;
    } else if (have) {
        s = a.score == CHORD_SCORE_SIGMOID ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / total;
    }
    if (lane < a.topk) {
        const int id = have && e >= a.first && e - a.first < a.local ? e - a.first : -1;
        a.ids[t * a.topk + lane] = id;
        a.w[t * a.topk + lane] = s * a.scale;
    }
}

__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a) {
    extern __shared__ double route_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    double* z = route_smem + (size_t)warp * (a.E + 32);
    double* gz = z + a.E;
    const double ninf = -INFINITY;
    float mx = -INFINITY;
    for (int e = lane; e < a.E; e += 32) mx = fmaxf(mx, logit_at(a, t, e));
    mx = warp_max(mx);
    double total = 0;
    if (a.score == CHORD_SCORE_SOFTMAX) {
        for (int e = lane; e < a.E; e += 32) {
            const float l = logit_at(a, t, e);
            if (l > -INFINITY) total += exp((double)l - (double)mx);
        }
        total = warp_sum(total);
    }
    const bool by_logit = !a.bias && (a.groups == 1 || a.best == 1);
    for (int e = lane; e < a.E; e += 32) {
        const float l = logit_at(a, t, e), b = a.bias ? a.bias[e] : 0.0f;
        double v = ninf;
        if (l > -INFINITY && b > -INFINITY) {
            if (by_logit)
                v = l;
            else if (a.score == CHORD_SCORE_SOFTMAX)
                v = exp((double)l - (double)mx) / total + (double)b;
            else
                v = 1.0 / (1.0 + exp(-(double)l)) + (double)b;
        }
        z[e] = v;
    }
    __syncwarp();
    if (a.groups > 1) {
        const int size = a.E / a.groups;
        if (lane < a.groups) {
            double b1 = ninf, b2 = ninf;
            for (int i = 0; i < size; ++i) {
                const double v = z[lane * size + i];
                if (v > b1) {
                    b2 = b1;
                    b1 = v;
                } else if (v > b2) {
                    b2 = v;
                }
            }
            gz[lane] = a.best == 2 && b2 > ninf ? b1 + b2 : b1;
        }
        __syncwarp();
        bool keep = false;
        if (lane < a.groups) {
            int rank = 0;
            for (int g = 0; g < a.groups; ++g) rank += gz[g] > gz[lane] || (gz[g] == gz[lane] && g < lane);
            keep = rank < a.topk_groups;
        }
        const unsigned kept = __ballot_sync(kAll, keep);
        for (int e = lane; e < a.E; e += 32)
            if (!(kept >> (e / size) & 1u)) z[e] = ninf;
        __syncwarp();
    }
    if (!a.bias && !by_logit)
        for (int e = lane; e < a.E; e += 32)
            if (z[e] > ninf) z[e] = logit_at(a, t, e);
    int mine = -1;
    for (int k = 0; k < a.topk; ++k) {
        double best = ninf;
        int at = INT32_MAX;
        for (int e = lane; e < a.E; e += 32)
            if (z[e] > best) {
                best = z[e];
                at = e;
            }
        for (int o = 16; o; o >>= 1) {
            const double ob = __shfl_xor_sync(kAll, best, o);
            const int oa = __shfl_xor_sync(kAll, at, o);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
        if (!(best > ninf)) break;
        if (at % 32 == lane) z[at] = ninf;
        if (lane == k) mine = at;
        __syncwarp();
    }
    write_choice(a, t, lane, mine, mine >= 0 ? logit_at(a, t, mine) : 0.0f, mx, (float)total);
}

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

chord_status chord_moe_route(const void* logits, int logits_dtype, int64_t row_stride, int T, int E, const float* bias,
                             int topk, const chord_route* how, int32_t* topk_ids, float* topk_w, void* stream) {
    if (!how || T < 0 || E <= 0 || topk <= 0 || (logits_dtype != CHORD_DTYPE_BF16 && logits_dtype != CHORD_DTYPE_F32))
        return CHORD_ERR_INVALID_ARG;
    if ((how->score != CHORD_SCORE_SOFTMAX && how->score != CHORD_SCORE_SIGMOID) || how->groups < 1 || how->topk_groups < 1 ||
        how->topk_groups > how->groups || E % how->groups || how->group_best < 1 || how->group_best > 2 || how->first < 0 ||
        how->E_local < 1 || how->E_local > E - how->first || row_stride < (T > 1 ? E : 0))
        return CHORD_ERR_INVALID_ARG;
    if (E > 1024 || topk > 32 || how->groups > 32 || (int64_t)T * topk >= INT32_MAX) return CHORD_ERR_UNSUPPORTED;
    if (topk > (int64_t)how->topk_groups * (E / how->groups)) return CHORD_ERR_INVALID_ARG;
    const uintptr_t align = logits_dtype == CHORD_DTYPE_F32 ? 3 : 1;
    if (T > 0 && (!logits || !topk_ids || !topk_w || (reinterpret_cast<uintptr_t>(logits) & align))) return CHORD_ERR_INVALID_ARG;
    if (T == 0) return CHORD_OK;
    RouteArgs a{logits, logits_dtype == CHORD_DTYPE_F32, row_stride, T, E, topk, bias, how->score, how->groups,
                how->topk_groups, how->group_best, how->renormalize != 0, how->scale, how->first, how->E_local, topk_ids, topk_w};
    const size_t smem = (size_t)kRouteWarps * (E + 32) * 8;
    if (ensure_smem_limit(reinterpret_cast<const void*>(route_kernel), kRouteWarps * (1024 + 32) * 8) != cudaSuccess)
        return CHORD_ERR_CUDA;
    route_kernel<<<(unsigned)ceil_div64(T, kRouteWarps), kRouteWarps * 32, smem, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? CHORD_OK : CHORD_ERR_CUDA;
}

}  // extern "C"
