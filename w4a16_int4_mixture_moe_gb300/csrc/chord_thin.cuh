// Thin products on the warp-level tensor cores: some rows of x times some rows of weights over a long K, for the
// router's logits and the first half of an adapter.
// Up to 16 rows (Warp): there is little to compute and every byte is used once or a few times, so nothing is staged: a
// lane loads 16 bytes of its rows straight into the fragments of m16n8k16 instructions.  Lane (g, c) takes columns
// 8c .. 8c + 7 of a 32-column step; the instruction's k order is whatever puts them into its slots, the same for
// both operands.  The warps of a CTA take every eighth step, so a CTA reads 512 neighbouring bytes of a row, and
// add their sums up through shared memory.  Bound by latency: one row of 7168 columns times 384 rows 3.9 us in a graph,
// 1.4 TB/s of weights.
// Up to 64 rows (Staged): below.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "chord_common.cuh"
#include "chord_tcgen05.cuh"

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

// Four 8 x 8 matrices of 16-bit numbers, lane l gives the address of row l mod 8 of matrix l / 8.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// What one warp multiplies: 16 rows of x, NT tiles of eight weight rows.  Rows that are not
// there are any others: their sums are not looked at.
template <int NT>
struct Warp {
    static constexpr int kRows = 16, kCols = NT * 8;
    // Steps in registers, all but one of them on their way: as many as a few rows need to cover the latency.
    static constexpr int kDepth = NT <= 2 ? 4 : NT <= 4 ? 3 : 2;
    const uint4* x[2];    // this lane's rows and piece of a step: row start + c
    const uint4* w[NT];
    float acc[NT][4];

    struct Step {
        uint4 a[2], b[NT];
    };

    template <bool TAIL>
    __device__ __forceinline__ void load(Step& s, int at, bool in) const {
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 2; ++j) s.a[j] = !TAIL || in ? x[j][at] : zero;
#pragma unroll
        for (int j = 0; j < NT; ++j) s.b[j] = !TAIL || in ? w[j][at] : zero;
    }
    __device__ __forceinline__ void multiply(const Step& s) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mma(acc[t], s.a[0].x, s.a[1].x, s.a[0].y, s.a[1].y, s.b[t].x, s.b[t].y);
            mma(acc[t], s.a[0].z, s.a[1].z, s.a[0].w, s.a[1].w, s.b[t].z, s.b[t].w);
        }
    }
    __device__ __forceinline__ void move(int pieces) {
#pragma unroll
        for (int j = 0; j < 2; ++j) x[j] += pieces;
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
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[t][u] = 0.0f;
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
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2* to = reinterpret_cast<float2*>(to0 + h * 8 * kCols + t * 8);
                    float2 o = make_float2(acc[t][2 * h], acc[t][2 * h + 1]);
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

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Sum i of kCount over the CTAs of a cluster (splits, a power of two), put(i, sum) for each by one of them: every CTA
// pushes each one the share of its sums that that one adds up, in rank order.  `mine(i)` is this CTA's sum, `shares` kCount
// floats that no earlier call's reads are left on.
template <int kCount, typename Mine, typename Put>
__device__ __forceinline__ void join_slices(int splits, float* shares, Mine mine, Put put) {
    static_assert((kCount & (kCount - 1)) == 0, "shares are powers of two");
    if (splits == 1) {
        for (int i = threadIdx.x; i < kCount; i += kThreads) put(i, mine(i));
        return;
    }
    const int rank = (int)tc5::cluster_rank(), share = kCount / splits, bits = __ffs(share) - 1;   // a power of two, as splits is
    tc5::cluster_sync();                                                                           // every CTA of the cluster runs
    for (int i = threadIdx.x; i < kCount; i += kThreads)
        st_cluster(tc5::at_cta(smem_u32(shares + rank * share + (i & (share - 1))), (uint32_t)(i >> bits)), mine(i));
    tc5::cluster_sync();
    for (int i = threadIdx.x; i < share; i += kThreads) {
        float v = shares[i];
        for (int s = 1; s < splits; ++s) v += shares[s * share + i];
        put(rank * share + i, v);
    }
}

// ---- the same for many rows, staged in shared memory ----------------------------------------
// 64 rows of x times NT x 8 weight rows: every thread copies 16-byte pieces of a stage of 128 columns, two tiles of 64,
// with cp.async, kStages - 1 stages are on their way.  A warp takes 32 rows, 32 weight rows (or all) and a share of a
// stage's columns, a half or a quarter, so that a fragment read from shared memory serves two or four instructions; the
// shares' sums are joined at the end.  A tile's rows are 128 bytes, piece p of row r at p xor (r mod 8).  (Stages of 64
// columns meet twice as often: 48 tokens of 384 experts in FP32 14.6 us for 13.9.  Warps of 16 rows and 64 weight rows read a
// quarter more fragments: the same 11.0 for 10.6, 256 tokens 13.1 for 12.4.)
template <int NT>
struct Staged {
    static constexpr int kRows = 64, kCols = NT * 8, kTileCols = 128, kHalf = (kRows + kCols) * 128;
    static constexpr int kStageBytes = 2 * kHalf, kStages = NT == 4 ? 4 : 3;
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes;          // the ring
    static constexpr int kTiles = NT < 4 ? NT : 4, kShares = NT == 8 ? 2 : 4, kSteps = 8 / kShares;   // of a warp: weight tiles; a stage's k steps
    static constexpr size_t kSums = (size_t)kShares * kRows * kCols * 4;    // over it, afterwards: [kShares][kRows][kCols]
    static constexpr size_t kBytes = kSmem > kSums ? kSmem : kSums;
    static constexpr int kChainStages = 16 / kSteps;                        // chains of sixteen instructions

    // This thread's rows of x (t / 8 and t / 8 + 32) and weight rows, at piece t mod 8; null: not copied,
    // whatever is multiplied in its place is not looked at.
    const __nv_bfloat16* x[2];
    const __nv_bfloat16* w[2];
    float acc[2][kTiles][4], sum[2][kTiles][4];

    __device__ __forceinline__ void copy(uint32_t st, int col, int64_t w_offset, int K) const {
        const int t = threadIdx.x, row = t >> 3, piece = t & 7;
        const uint32_t at = st + (uint32_t)row * 128u + (uint32_t)(((piece ^ row) & 7) << 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int k = col + half * 64;
            const bool in = k + piece * 8 < K;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t to = at + (uint32_t)(half * kHalf + h * 4096);
                if (x[h]) fill(to, in ? x[h] + k : x[h], in);
                if (h * 32 < kCols && w[h]) fill(to + kRows * 128u, in ? w[h] + w_offset + k : w[h], in);
            }
        }
    }
    // 16 bytes, or zeros behind the last column.
    __device__ __forceinline__ static void fill(uint32_t dst, const __nv_bfloat16* src, bool in) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
    }
    // This warp's first row, weight row and k step of a stage.
    __device__ __forceinline__ static int first_row() { return (threadIdx.x >> 5 & 1) * 32; }
    __device__ __forceinline__ static int first_col() { return NT == 8 ? (threadIdx.x >> 6 & 1) * 32 : 0; }
    __device__ __forceinline__ static int share() { return NT == 8 ? threadIdx.x >> 7 : threadIdx.x >> 6; }
    __device__ __forceinline__ void multiply(uint32_t st) {
        const int lane = threadIdx.x & 31, ar = first_row() + (lane & 15), br = first_col() + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int step = share() * kSteps + s, kk = step & 3;
            const uint32_t from = st + (uint32_t)((step >> 2) * kHalf);
            uint32_t a[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
                ldsm4(a[m], from + (uint32_t)(ar + m * 16) * 128u + (uint32_t)(((kk * 2 + (lane >> 4)) ^ (ar & 7)) << 4));
#pragma unroll
            for (int t = 0; t < kTiles; t += 2) {
                uint32_t b[4];
                // with one tile of weights the second half of the lanes reads its rows again
                const int r = t * 8 + (NT > 1 ? br : (lane & 7));
                ldsm4(b, from + kRows * 128u + (uint32_t)r * 128u + (uint32_t)(((kk * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma(acc[m][t], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
                    if (t + 1 < kTiles) mma(acc[m][t + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
                }
            }
        }
    }
    __device__ __forceinline__ void end_chain() {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    sum[m][t][u] += acc[m][t][u];
                    acc[m][t][u] = 0.0f;
                }
    }
    // Sum i of the tile, of its shares in order; sums: what run left.
    __device__ __forceinline__ static float joined(const float* sums, int i) {
        float v = sums[i];
#pragma unroll
        for (int z = 1; z < kShares; ++z) v += sums[z * kRows * kCols + i];
        return v;
    }
    // Stages s0 .. s1 - 1 of `parts` weight matrices one behind the other, part_stride elements apart, the last
    // one first.  Every thread of the CTA; the sums are in smem ([kShares][kRows][kCols] floats) when it returns.
    __device__ __forceinline__ void run(uint8_t* smem, int s0, int s1, int K, int parts, int64_t part_stride) {
        const uint32_t base = smem_u32(smem);
        const int per = (K + kTileCols - 1) / kTileCols;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[m][t][u] = sum[m][t][u] = 0.0f;
        int next = s0, part = s0 / per, k = s0 - part * per, slot_in = 0, slot_out = 0, chain = 0;
        auto issue = [&]() {
            if (next < s1) {
                copy(base + (uint32_t)(slot_in * kStageBytes), k * kTileCols, (int64_t)(parts - 1 - part) * part_stride, K);
                if (++k == per) k = 0, ++part;
                ++next;
            }
            cp_async_commit();
            if (++slot_in == kStages) slot_in = 0;
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue();
        for (int s = s0; s < s1; ++s) {
            cp_async_wait<kStages - 2>();
            __syncthreads();   // the stage is there for all, and the one before has been read by all
            issue();
            multiply(base + (uint32_t)(slot_out * kStageBytes));
            if (++slot_out == kStages) slot_out = 0;
            if (++chain == kChainStages) {
                chain = 0;
                end_chain();
            }
        }
        end_chain();
        cp_async_wait<0>();
        __syncthreads();
        const int lane = threadIdx.x & 31;
        float* to = reinterpret_cast<float*>(smem) + (share() * kRows + first_row() + (lane >> 2)) * kCols + first_col() + 2 * (lane & 3);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2*>(to + (m * 16 + h * 8) * kCols + t * 8) = make_float2(sum[m][t][2 * h], sum[m][t][2 * h + 1]);
        __syncthreads();
    }
};

}  // namespace thin
}  // namespace chord
