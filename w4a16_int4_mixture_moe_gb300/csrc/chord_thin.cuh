// Thin products on the warp-level tensor cores: up to 64 rows of x times up to 64 rows of weights over a long
// K, for the router's logits and the first half of an adapter.  There is little to compute and every
// byte is used once or a few times, so nothing is staged: a lane loads 16 bytes of its rows
// straight into the fragments of m16n8k16 instructions.  Lane (g, c) takes columns 8c .. 8c + 7 of a
// 32-column step; the instruction's k order is whatever puts them into its slots, the same for
// both operands.  The warps of a CTA take every eighth step, so a CTA reads 512 neighbouring bytes of a row, and
// add their sums up through shared memory.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "chord_common.cuh"

namespace chord {
namespace thin {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStep = 32;     // columns
// The instructions' additions chop: chains end after 24 steps (48 instructions) and are added up in FP32.
constexpr int kChain = 24;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What one warp multiplies: MT tiles of 16 rows of x, NT tiles of eight weight rows.  Rows that are not
// there are any others: their sums are not looked at.
template <int MT, int NT>
struct Warp {
    static constexpr int kRows = MT * 16, kCols = NT * 8;
    // Steps in registers, all but one of them on their way: as many as a few rows need to cover the latency.
    static constexpr int kDepth = MT * NT <= 2 ? 4 : MT * NT <= 4 ? 3 : 2;
    const uint4* x[2 * MT];    // this lane's rows and piece of a step: row start + c
    const uint4* w[NT];
    float acc[MT][NT][4];

    struct Step {
        uint4 a[2 * MT], b[NT];
    };

    template <bool TAIL>
    __device__ __forceinline__ void load(Step& s, int at, bool in) const {
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j) s.a[j] = !TAIL || in ? x[j][at] : zero;
#pragma unroll
        for (int j = 0; j < NT; ++j) s.b[j] = !TAIL || in ? w[j][at] : zero;
    }
    __device__ __forceinline__ void multiply(const Step& s) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mma(acc[m][t], s.a[2 * m].x, s.a[2 * m + 1].x, s.a[2 * m].y, s.a[2 * m + 1].y, s.b[t].x, s.b[t].y);
                mma(acc[m][t], s.a[2 * m].z, s.a[2 * m + 1].z, s.a[2 * m].w, s.a[2 * m + 1].w, s.b[t].z, s.b[t].w);
            }
    }
    __device__ __forceinline__ void move(int pieces) {
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j) x[j] += pieces;
#pragma unroll
        for (int j = 0; j < NT; ++j) w[j] += pieces;
    }
    // Steps first, first + 8, ... below last of K = 8 * pieces columns: the sums go to (or, with `more`, are
    // added to) mine, the warp's [kRows][kCols] floats in shared memory.  Moves x and w.
    __device__ __forceinline__ void run(int first, int last, int pieces, float* mine, bool more) {
        constexpr int kNext = kWarps * 4;   // pieces from a step of this warp to its next
        const int lane = threadIdx.x & 31;
        float* to0 = mine + (lane >> 2) * kCols + 2 * (lane & 3);
        const int full = min(last, pieces / 4);                                        // whole steps end here
        int left = first < full ? (full - first + kWarps - 1) / kWarps : 0;            // whole steps of this warp
        const int after = first + left * kWarps;                                       // and its step behind them
        move(first * 4);
        do {
            int n = min(left, kChain);
            left -= n;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < 4; ++u) acc[m][t][u] = 0.0f;
            Step s[kDepth];
#pragma unroll
            for (int d = 0; d < kDepth - 1; ++d)
                if (d < n) load<false>(s[d], d * kNext, true);
            while (n > 0) {
#pragma unroll
                for (int d = 0; d < kDepth; ++d) {
                    if (n > kDepth - 1) load<false>(s[(d + kDepth - 1) % kDepth], (d + kDepth - 1) * kNext, true);
                    if (n > 0) {
                        multiply(s[d]);
                        if (d + 1 == kDepth) move(kDepth * kNext);
                        else if (n == 1) move((d + 1) * kNext);
                    }
                    --n;
                }
            }
            if (left == 0 && after < last) {   // the last columns, not a whole step
                load<true>(s[0], 0, after * 4 + (lane & 3) < pieces);
                multiply(s[0]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2* to = reinterpret_cast<float2*>(to0 + (m * 16 + h * 8) * kCols + t * 8);
                        float2 o = make_float2(acc[m][t][2 * h], acc[m][t][2 * h + 1]);
                        if (more) o.x += to->x, o.y += to->y;
                        *to = o;
                    }
            more = true;
        } while (left > 0);
    }
};

// Sum i of all warps' (red: [kWarps][n]), in warp order.
__device__ __forceinline__ float joined(const float* red, int n, int i) {
    float v = red[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += red[w * n + i];
    return v;
}

}  // namespace thin
}  // namespace chord
