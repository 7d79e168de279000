// Choice of experts from router logits: scores, groups, top-k, weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

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
//   sigmoid: 1 / (1 + exp(-l)), in terms of q = exp(-|l|): 1 / (1 + q) or q / (1 + q)
// Renormalised, the numerators are scaled by exp(-c) with c the largest chosen logit (sigmoid: only
// if that is negative), which the quotient does not change and which keeps far negative logits
// from all becoming 0.
__device__ __forceinline__ void write_choice(const RouteArgs& a, int64_t t, int lane, int e, float l, float m, float total) {
    const bool have = e >= 0;   // no lane from topk on has one
    const bool sigmoid = a.score == CHORD_SCORE_SIGMOID;
    const bool far = a.renorm && !__any_sync(kAll, have && sigmoid && l >= 0.0f);   // warp-uniform
    float c = sigmoid ? 0.0f : m;
    if (far) c = warp_max(have ? l : -FLT_MAX);
    const float q = expf(sigmoid ? -fabsf(l) : l - c);
    float s = q;
    if (sigmoid) {
        if (far) s = expf(l - c);
        s = (l > 0.0f ? 1.0f : s) / (1.0f + q);
    }
    if (!have) s = 0.0f;
    const float sum = a.renorm ? warp_sum(s) : sigmoid ? 1.0f : total;
    if (lane < a.topk) {
        const int id = have && e >= a.first && e - a.first < a.local ? e - a.first : -1;
        a.ids[t * a.topk + lane] = id;
        a.w[t * a.topk + lane] = (have ? s / sum : 0.0f) * a.scale;
    }
}

// The softmax's sum in binary64.
__device__ __noinline__ double total_in_64_bits(const RouteArgs& a, int64_t t, int lane, float mx) {
    double total = 0;
    for (int e = lane; e < a.E; e += 32) {
        const float l = logit_at(a, t, e);
        if (l > -INFINITY) total += exp((double)l - (double)mx);
    }
    return warp_sum(total);
}

// A value in binary64 (-inf: not available); total: the softmax's sum.
__device__ __forceinline__ double value_in_64_bits(const RouteArgs& a, float l, float b, float mx, double total) {
    if (!(l > -INFINITY && b > -INFINITY)) return -INFINITY;
    return (a.score == CHORD_SCORE_SOFTMAX ? exp((double)l - (double)mx) / total : 1.0 / (1.0 + exp(-(double)l))) + (double)b;
}

// The choice with a bias by the definition, every value in binary64, one expert after the other: lane k gets
// the k-th (-1: none).  z: E + 32 doubles of the warp's own.  (Without a bias the logits order the experts, and
// nothing is in doubt.)
__device__ __noinline__ int choose_in_64_bits(const RouteArgs& a, int64_t t, int lane, float mx, double* z) {
    double* gz = z + a.E;
    const double ninf = -INFINITY;
    const double total = a.score == CHORD_SCORE_SOFTMAX ? total_in_64_bits(a, t, lane, mx) : 0.0;
    for (int e = lane; e < a.E; e += 32) z[e] = value_in_64_bits(a, logit_at(a, t, e), a.bias[e], mx, total);
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
    return mine;
}

// A number's place among unsigned integers, in the order of the numbers (-inf is not 0: 0 is below all).
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and +0 are the same number
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float number_of(uint32_t key) {
    return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// e^x and 1 / x in one approximate instruction each (relative error below 2^-22 and 2^-23; e^x next to
// that |x| 2^-24 from its argument).
__device__ __forceinline__ float fast_exp(float x) {
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One token per warp; lane l holds experts l, l + 32, ...  Bound by instructions: 16384 tokens of 384 experts, sigmoid, a
// bias, top-8, 18.4 us in a graph (1.4 TB/s of logits, 2.7 of 4 instructions a cycle issued).  Eight CTAs to an SM
// (64 registers; 8 bytes a thread spilled at 8 values a lane, 44 to 64 at 12 and 16): 8192 tokens of 512 experts top-16 15.8 us,
// without the bound, at 88 registers, 17.5.
//   1. Values in FP32, each off by a known slack.
//   2. The topk-th largest of the 32 lanes' largest values bounds the topk-th largest value from
//      below: what is not below it (by twice the slack) are the candidates, about ten for a
//      top-8 of 384.  One per lane, each counts those before it.
//   3. Where two candidates' values are too close for FP32 to tell (some of a thousand tokens of a
//      sigmoid router of 384 experts), the candidates' are computed in binary64; where two groups' are, those
//      of the groups in question.
//   4. More than 32 candidates: choose_one_by_one.  Where that is still in doubt, or biases are +inf, the whole
//      token is done by choose_in_64_bits.
// A value in FP32 is off by at most slack + kRounding |value|.  A sigmoid of the fast functions is off by s (1 - s)
// (2^-22 + |l| 2^-24) + 2^-23, below 3e-7, of the accurate ones by s (1 - s) 2^-22 + s 2^-23, below 1.8e-7.  A softmax's score e / total, of E <= 1024
// experts: the sum by 37 half ulps for its additions, 2 ulps for the function and 7 half ulps for the exponents' rounding
// (their mean weighted by the scores is below ln E), each exponential by 2 ulps and 0.37 half ulps; all below 4e-6 / total.
constexpr float kSlackFast = 1e-6f, kSlackAccurate = 2.5e-7f, kSlackSoftmax = 4e-6f, kRounding = 1.2e-7f;

// Shared memory of a warp, in doubles: the list (16), its candidates (16), their inputs or values in
// binary64 (32); or the list and all values (E / 2); or the groups' rows; or all values in binary64 and the groups' (E + 32).
__host__ __device__ inline int own_doubles(int E) { return (E > 32 ? E + 33 : 65) & ~1; }

// The groups that take part, where FP32 does not decide: lane g has group g's value in FP32, those above `above` are
// in, those below `below` out, the ones between are ordered by their values in binary64, the lower index first of equal
// ones.  z: E doubles of the warp's own; lpg lanes (a power of two) share a group.
__device__ __noinline__ unsigned groups_in_64_bits(const RouteArgs& a, int64_t t, int lane, float value, float above, float below, float mx, int lpg,
                                                   double* z) {
    const int size = a.E / a.groups;
    const bool in = lane < a.groups && value > above, open = lane < a.groups && !in && value > -INFINITY && !(value < below);
    const unsigned sure = __ballot_sync(kAll, in), asked = __ballot_sync(kAll, open);
    const double total = a.score == CHORD_SCORE_SOFTMAX ? total_in_64_bits(a, t, lane, mx) : 0.0;
    for (int e = lane; e < a.E; e += 32)
        if (asked >> (e / size) & 1u) z[e] = value_in_64_bits(a, logit_at(a, t, e), a.bias ? a.bias[e] : 0.0f, mx, total);
    __syncwarp();
    double b1 = -INFINITY, b2 = -INFINITY;
    const int g = lane / lpg;
    if (g < a.groups && asked >> g & 1u)
        for (int i = lane % lpg; i < size; i += lpg) {
            const double v = z[g * size + i];
            b2 = fmax(b2, fmin(b1, v));
            b1 = fmax(b1, v);
        }
    for (int o = 1; o < lpg; o <<= 1) {
        const double o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
        b2 = fmax(fmax(b2, o2), fmin(b1, o1));
        b1 = fmax(b1, o1);
    }
    double mine = __shfl_sync(kAll, a.best == 2 && b2 > -INFINITY ? b1 + b2 : b1, (lane * lpg) & 31);
    int rank = __popc(sure);
    for (int k = 0; k < a.groups; ++k) {
        const double v = __shfl_sync(kAll, mine, k);
        rank += (asked >> k & 1u) && (v > mine || (v == mine && k < lane));
    }
    __syncwarp();
    return sure | __ballot_sync(kAll, open && rank < a.topk_groups);
}

// The places of the n <= 32 candidates, a lane each, by their values in binary64.
__device__ __noinline__ int rank_in_64_bits(const RouteArgs& a, int64_t t, int lane, float mx, int n, double* own) {
    const int* list = reinterpret_cast<const int*>(own);
    double* values = own + 16 + 16;
    const double total = a.score == CHORD_SCORE_SOFTMAX ? total_in_64_bits(a, t, lane, mx) : 0.0;
    const int e = list[min(lane, n - 1)];
    const double d = value_in_64_bits(a, logit_at(a, t, e), a.bias[e], mx, total);   // without a bias nothing is in doubt
    if (lane < n) values[lane] = d;
    __syncwarp();
    int rank = 0;
    for (int k = 0; k < n; ++k) rank += values[k] > d || (values[k] == d && list[k] < e);
    return rank;
}

// More candidates than lanes (many equal logits, a top-k that comes near to 32): the largest of all values z, one after
// the other, until one is certainly below the topk-th; where FP32 does not tell the order of those before it, that is
// found in binary64.  -2 in every lane: still in doubt after 32.  z lies behind the list in the warp's own memory.
__device__ __noinline__ int choose_one_by_one(const RouteArgs& a, int64_t t, int lane, float mx, bool exact_order, float slack, double* own) {
    int* list = reinterpret_cast<int*>(own);
    float* z = reinterpret_cast<float*>(own + 16);
    bool sure = true;
    float before = INFINITY, bound = -INFINITY;
    int n = 0;
    for (;; ++n) {
        float best = -INFINITY;
        int at = lane;
        for (int e = lane; e < a.E; e += 32)
            if (z[e] > best) {
                best = z[e];
                at = e;
            }
        const uint32_t mine_key = key_of(best), key = __reduce_max_sync(kAll, mine_key);
        const float v = number_of(key);
        if (!(v > -INFINITY)) break;
        if (n >= a.topk && (exact_order || bound - v > 2.0f * slack + kRounding * (fabsf(v) + fabsf(bound)))) break;
        if (n == 32) return -2;
        if (!exact_order && n > 0 && !(before - v > 2.0f * slack + kRounding * (fabsf(v) + fabsf(before)))) sure = false;
        before = v;
        if (n < a.topk) bound = v;
        const int e = (int)__reduce_min_sync(kAll, mine_key == key ? (unsigned)at : 0xffffffffu);
        if (lane == 0) list[n] = e;
        if (e == at) z[e] = -INFINITY;   // this lane's own
    }
    __syncwarp();
    if (!sure) {
        const int e = list[min(lane, n - 1)], rank = rank_in_64_bits(a, t, lane, mx, n, own);
        __syncwarp();
        if (lane < n && rank < a.topk) list[rank] = e;
        __syncwarp();
    }
    return lane < min(n, a.topk) ? list[lane] : -1;
}

template <int VPL, bool F32>
__global__ void __launch_bounds__(kRouteWarps * 32, VPL > 16 ? 4 : 8) route_kernel(const RouteArgs a) {
    using In = typename std::conditional<F32, float, __nv_bfloat16>::type;
    extern __shared__ double route_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    double* own = route_smem + (size_t)warp * own_doubles(a.E);
    const bool by_logit = !a.bias && (a.groups == 1 || a.best == 1);
    const bool softmax = a.score == CHORD_SCORE_SOFTMAX;
    const In* row = static_cast<const In*>(a.logits) + t * a.stride + lane;
    // a logit as the scores use it: +inf counts as the largest number
    auto logit = [&](int i) { return fminf((float)row[32 * i], FLT_MAX); };
    float z[VPL], bias[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool in = lane + 32 * i < a.E;
        z[i] = in ? (float)row[32 * i] : -INFINITY;
        bias[i] = in && a.bias ? a.bias[lane + 32 * i] : 0.0f;
    }
    float mx = 0.0f, total = 1.0f;
    if (softmax) {
        mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) mx = fmaxf(mx, z[i]);   // leaves out NaN
        mx = fminf(warp_max(mx), FLT_MAX);
        if (!(by_logit && a.renorm)) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) total += z[i] > -INFINITY ? expf(fminf(z[i], FLT_MAX) - mx) : 0.0f;
            total = warp_sum(total);
        }
    }
    const float slack = softmax ? kSlackSoftmax / total : a.groups > 1 ? kSlackAccurate : kSlackFast;
    auto off_by = [&](float v) { return slack + kRounding * fabsf(v); };
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) z[i] = z[i] > -INFINITY ? fminf(z[i], FLT_MAX) : -INFINITY;
    } else if (softmax) {
        const float inv = 1.0f / total;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool open = z[i] > -INFINITY && bias[i] > -INFINITY;
            z[i] = open ? expf(fminf(z[i], FLT_MAX) - mx) * inv + bias[i] : -INFINITY;
        }
    } else if (a.groups > 1) {
        // accurate here already: few pairs of groups are then too close
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool open = z[i] > -INFINITY && bias[i] > -INFINITY;
            z[i] = open ? 1.0f / (1.0f + expf(-z[i])) + bias[i] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool open = z[i] > -INFINITY && bias[i] > -INFINITY;
            z[i] = open ? fast_rcp(1.0f + fast_exp(-z[i])) + bias[i] : -INFINITY;
        }
    }
    bool fine = true;
    if (a.groups > 1) {
        float* rows = reinterpret_cast<float*>(own);
        const int size = a.E / a.groups;
        const uint32_t inv = (1u << 20) / (uint32_t)size + 1u;   // e * inv >> 20 = e / size for e < 1024
        int lpg = 32;                                            // lanes that share a group
        while (lpg * a.groups > 32) lpg >>= 1;
        // groups lie lpg words further apart, so that lanes read different banks
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) rows[e + lpg * (int)((uint32_t)e * inv >> 20)] = z[i];
        }
        __syncwarp();
        const int g = lane / lpg;
        float b1 = -INFINITY, b2 = -INFINITY;
        if (g < a.groups) {
            const float* mine = rows + g * (size + lpg);
#pragma unroll 4
            for (int i = lane % lpg; i < size; i += lpg) {
                const float v = mine[i];
                b2 = fmaxf(b2, fminf(b1, v));
                b1 = fmaxf(b1, v);
            }
        }
        for (int o = 1; o < lpg; o <<= 1) {
            const float o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
            b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
            b1 = fmaxf(b1, o1);
        }
        const bool pair = a.best == 2 && b2 > -INFINITY;
        // A sum below FP32's range is still a number, not a group without experts; which of such sums is larger is
        // found in binary64 below, since size_of is infinite then.
        float gv = __shfl_sync(kAll, pair ? fmaxf(b1 + b2, -FLT_MAX) : b1, (lane * lpg) & 31);
        const float size_of = warp_max(b1 > -INFINITY ? (pair ? fabsf(b1) + fabsf(b2) : fabsf(b1)) : 0.0f);
        if (lane >= a.groups) gv = -INFINITY;
        int rank = 0;
        for (int k = 0; k < a.groups; ++k) {
            const float v = __shfl_sync(kAll, gv, k);
            rank += v > gv || (v == gv && k < lane);
        }
        if (lane >= a.groups) rank = 32;
        unsigned kept = __ballot_sync(kAll, rank < a.topk_groups);
        if (!by_logit && a.topk_groups < a.groups) {
            // the last group that is kept and the first that is not: two values each, each off by the slack
            const unsigned last = __ballot_sync(kAll, rank == a.topk_groups - 1), next = __ballot_sync(kAll, rank == a.topk_groups);
            const float v = __shfl_sync(kAll, gv, __ffs(last) - 1), w = __shfl_sync(kAll, gv, __ffs(next) - 1);
            const float apart = 4.0f * slack + 4.0f * kRounding * size_of;   // of two groups, two values each and their sum
            __syncwarp();
            if (w > -INFINITY && !(v < INFINITY && v - w > apart)) kept = groups_in_64_bits(a, t, lane, gv, v + apart, w - apart, mx, lpg, own);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool in = kept >> ((uint32_t)(lane + 32 * i) * inv >> 20 & 31u) & 1u;
            z[i] = in ? z[i] : -INFINITY;
            if (!a.bias && !by_logit && z[i] > -INFINITY) z[i] = logit(i);
        }
    }
    // from here on the logit orders the experts wherever there is no bias
    const bool exact_order = !a.bias;
    float top = z[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = fmaxf(top, z[i]);
    uint32_t key = key_of(top), bound = 0;
    for (int k = 0; k < a.topk;) {
        bound = __reduce_max_sync(kAll, key);
        if (bound == 0) break;   // fewer than topk lanes
        k += __popc(__ballot_sync(kAll, key == bound));
        if (key == bound) key = 0;
    }
    // bound back to a number; 0: fewer than topk lanes hold anything
    float least = bound == 0 ? -INFINITY : number_of(bound);
    if (!exact_order) {
        if (!(least < INFINITY)) fine = false;   // biases of +inf: least becomes NaN, the list empty
        least -= 2.0f * off_by(least);
    }
    least = fmaxf(least, -FLT_MAX);   // -inf is never chosen (the lowest number is)
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) mask |= z[i] >= least ? 1u << i : 0u;
    const int n = (int)__reduce_add_sync(kAll, (unsigned)__popc(mask));
    int mine = -1;
    if (fine && n > 32) {
        float* rows = reinterpret_cast<float*>(own + 16);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane + 32 * i < a.E) rows[lane + 32 * i] = z[i];
        mine = choose_one_by_one(a, t, lane, mx, exact_order, slack, own);
        fine = mine != -2;
    } else if (fine) {
        int* list = reinterpret_cast<int*>(own);
        float* cand = reinterpret_cast<float*>(own + 16);
        int at = 0;
        for (unsigned left; (left = __ballot_sync(kAll, mask != 0)) != 0;) {
            if (mask) {
                list[at + __popc(left & ((1u << lane) - 1u))] = lane + 32 * (__ffs(mask) - 1);
                mask &= mask - 1;
            }
            at += __popc(left);
        }
        __syncwarp();
        int e = INT32_MAX;
        float l = 0.0f, b = 0.0f, v = -INFINITY;
        if (lane < n) {
            e = list[lane];
            l = fminf((float)row[e - lane], FLT_MAX);
            v = l;
            if (a.bias) {
                b = a.bias[e];
                v = (softmax ? expf(l - mx) / total : 1.0f / (1.0f + expf(-l))) + b;   // accurate: fewer are too close then
            }
            cand[lane] = v;
        }
        __syncwarp();
        // Those before this one, and those that FP32 cannot tell from it (without a bias: that are equal), itself among them.
        int rank = 0, close = 0;
        const float tol = exact_order ? 0.0f : 2.0f * ((softmax ? slack : kSlackAccurate) + kRounding * fabsf(v));
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float c = cand[k];
            rank += c > v;
            close += !(fabsf(c - v) > tol);
        }
        if (__any_sync(kAll, lane < n && rank < a.topk && close > 1)) {
            // Equal inputs are equal values in any precision: the lower index is first.
            float2* inputs = reinterpret_cast<float2*>(own + 16 + 16);
            if (lane < n) inputs[lane] = make_float2(l, b);
            __syncwarp();
            int before = 0;
            for (int k = 0; k < n; ++k) {
                const float2 c = inputs[k];
                const bool same = c.x == l && c.y == b;
                close -= same;
                before += same && list[k] < e;
            }
            __syncwarp();
            rank += before;
            if (__any_sync(kAll, lane < n && rank < a.topk && close > 0)) {
                // the candidates are certain, their order is not
                rank = rank_in_64_bits(a, t, lane, mx, n, own);
            }
        }
        __syncwarp();
        if (lane < n && rank < a.topk) list[rank] = e;
        __syncwarp();
        mine = lane < min(n, a.topk) ? list[lane] : -1;
    }
    __syncwarp();
    if (!fine) mine = choose_in_64_bits(a, t, lane, mx, own);
    write_choice(a, t, lane, mine, mine >= 0 ? fminf((float)row[mine - lane], FLT_MAX) : 0.0f, mx, total);
}

template <bool F32>
auto route_kernel_for(int E) {
    return E <= 64    ? route_kernel<2, F32>
           : E <= 128 ? route_kernel<4, F32>
           : E <= 256 ? route_kernel<8, F32>
           : E <= 384 ? route_kernel<12, F32>
           : E <= 512 ? route_kernel<16, F32>
                      : route_kernel<32, F32>;
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
    const size_t smem = (size_t)kRouteWarps * own_doubles(E) * 8;   // at most 36 KB
    void (*kern)(RouteArgs) = logits_dtype == CHORD_DTYPE_F32 ? route_kernel_for<true>(E) : route_kernel_for<false>(E);
    kern<<<(unsigned)ceil_div64(T, kRouteWarps), kRouteWarps * 32, smem, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? CHORD_OK : CHORD_ERR_CUDA;
}

}  // extern "C"
