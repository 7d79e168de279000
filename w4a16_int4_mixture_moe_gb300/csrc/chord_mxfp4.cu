// Microscaled 4-bit quantisation (MXFP4) of weight matrices and of routed
// activation rows, and the values a quantised matrix stands for.
//
// For 32 columns v of a row with largest magnitude a:
//   e    = floor(log2 a) - 2, clamped to [-127, 127]   (a = 0: e = -127)
//   code = the E2M1 number nearest to v * 2^-e (ties to the even code), at most 6
// stored as (codes, b = e + 127).  2 is the largest exponent of E2M1, so the
// block's largest element lands in [4, 8); what is above 6 saturates, off by less than
// 2 units, a quarter of it (the OCP Microscaling specification's conversion).  v * 2^-e is exact in
// FP32 (a power of two), so the only rounding is the code's.  A block that
// holds an infinity or NaN gets the NaN scale: it stays visible downstream.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chord_internal.h"
#include "chord_mxfp4.cuh"

namespace chord {
namespace {

// E2M1 codes of eight columns, column i in bits 4i (the hardware conversion:
// round to nearest, ties to even, magnitudes above 5 to 6).
__device__ __forceinline__ uint32_t e2m1_codes8(const float (&y)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return w;
}

// The values of eight codes as four half pairs (exact).
__device__ __forceinline__ void e2m1_halves8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Eight consecutive elements as loaded: bf16 pairs or FP32.  VEC: 16-byte loads
// (the address is aligned).
template <bool F32>
struct Raw {
    uint32_t w[F32 ? 8 : 4];
};

template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* src, int64_t at, Raw<F32>& v) {
    if constexpr (VEC) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) + at * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) {
            const uint4 a = __ldg(p + i);
            v.w[4 * i] = a.x, v.w[4 * i + 1] = a.y, v.w[4 * i + 2] = a.z, v.w[4 * i + 3] = a.w;
        }
    } else if constexpr (F32) {
        const uint32_t* p = static_cast<const uint32_t*>(src) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i) v.w[i] = __ldg(p + i);
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(src) + at;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
    }
}

// Codes of a lane's eight columns and the biased scale b of their group (the lane's quad).
// The largest magnitude is found on the bit patterns, whose order is the values' order with
// infinities and NaN on top.  A block with one of those: b = 255, and whatever codes come out.
template <bool F32>
__device__ __forceinline__ uint32_t quantize8(const Raw<F32>& v, uint32_t& b) {
    uint32_t ex;   // biased exponent of the largest magnitude; 0 for zero and subnormals
    float y[8];
    if constexpr (F32) {
        uint32_t top = v.w[0] & 0x7fffffffu;
#pragma unroll
        for (int i = 1; i < 8; ++i) top = max(top, v.w[i] & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        ex = top >> 23;
    } else {
        uint32_t top = v.w[0] & 0x7fff7fffu;
#pragma unroll
        for (int i = 1; i < 4; ++i) top = __vmaxu2(top, v.w[i] & 0x7fff7fffu);
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        ex = max(top >> 16, top & 0xffffu) >> 7;
    }
    const uint32_t e = max(ex, 2u) - 2u;
    const uint32_t up = 254u - e;   // exponent field of 2^(127 - e)
    b = ex == 255u ? 255u : e;
    if constexpr (F32) {
        const float f = __uint_as_float(up << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(v.w[i]) * f;
    } else {
        // exact: a power of two; what falls below bf16's range has code 0
        const __nv_bfloat162 f = u32_as_bf2(up * 0x00800080u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = bf2_as_u32(__hmul2(u32_as_bf2(v.w[i]), f));
            y[2 * i] = __uint_as_float(p << 16);
            y[2 * i + 1] = __uint_as_float(p & 0xffff0000u);
        }
    }
    return e2m1_codes8(y);
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
    int64_t id_limit;            // ids below this have a row
    int32_t sentinel;            // the id of positions without a pair
    int divisor;
};

__device__ __forceinline__ void mx_write_header(uint8_t* packed, int i, int64_t G, int64_t N, int K) {
    const unsigned long long stride = mx_group_bytes(N, K);
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

// One warp takes rows r, r + 32, r + 64, r + 96 of a band of tiles (four
// independent loads; their scales are 16 contiguous bytes of each scale block)
// over a run of `run` tiles along K, the next tile's loads in flight while one is
// converted.  A lane holds eight columns of each row: a group of 32 columns is
// four lanes, its largest magnitude two shuffles, a row's codes one 128-byte store.
// ROUTED: the rows of a routing array's positions (those without a pair are skipped).
// Bound by HBM: 8 x 4096 x 7168 bf16 weights (470 MB read, 125 MB written) in 102 us,
// 5.8 TB/s; next to it the conversion (logical pipe 66 % busy).  Four rows and whole runs
// keep enough loads in flight: one row a warp and a tile at a time took 401 us.
template <bool F32, bool VEC, bool ROUTED>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const RowSource s, int64_t G, int64_t N, int K, int run,
                                                          uint8_t* __restrict__ packed, int* err) {
    pdl_trigger();   // a product that follows sets itself up meanwhile
    if (blockIdx.x == 0 && threadIdx.x < kHeaderBytes / 4) mx_write_header(packed, threadIdx.x, G, N, K);
    const int64_t rt = mx_row_tiles(N);
    const int kb = (int)mx_col_tiles(K);
    const int runs = (kb + run - 1) / run;
    int64_t groups = G;
    if (ROUTED) {
        const int64_t ntp = *s.ntp;
        if (ntp < 0 || ntp > G * N || ntp % N) {
            if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, CHORD_DEV_BAD_PADDED);
            return;
        }
        groups = ntp / N;
    }
    const int lane = threadIdx.x & 31;
    const uint32_t j = lane >> 2;
    const int64_t tasks = groups * rt * runs * 32;
    uint8_t* data = packed + kHeaderBytes;
    for (int64_t q = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; q < tasks;
         q += ((int64_t)gridDim.x * blockDim.x) >> 5) {
        const uint32_t r0 = (uint32_t)(q & 31);
        int part, bt;
        const int64_t band = divmod_idx(q >> 5, runs, part);
        const int64_t g = divmod_idx(band, (int)rt, bt);
        const int kt0 = part * run, kt1 = min(kt0 + run, kb);
        int64_t at[4];   // first element of the row
        uint32_t live = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = (int64_t)bt * kMxTileRows + r0 + 32 * i;
            at[i] = 0;
            if (row < N) {
                if (!ROUTED) {
                    at[i] = g * s.mat_stride + row * s.row_stride;
                    live |= 1u << i;
                } else {
                    const int32_t id = __ldg(s.sorted_ids + g * N + row);
                    if (id >= 0 && id < s.id_limit) {
                        at[i] = (int64_t)((uint32_t)id / (uint32_t)s.divisor) * s.row_stride;
                        live |= 1u << i;
                    } else if (id != s.sentinel && part == 0 && lane == 0) {
                        set_error(err, CHORD_DEV_BAD_ROW);
                    }
                }
            }
        }
        if (ROUTED && !live) continue;
        Raw<F32> cur[4] = {}, nxt[4] = {};
        auto fetch = [&](Raw<F32>(&v)[4], int kt) {
            const int k0 = kt * kMxTileCols + lane * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)   // a row's last columns past K stay zero: in the last tile only
                if (live >> i & 1u) {
                    if (k0 < K)
                        load8<F32, VEC>(s.src, at[i] + k0, v[i]);
                    else
                        v[i] = Raw<F32>{};
                }
        };
        fetch(cur, kt0);
        uint8_t* t = data + (band * kb + kt0) * kMxTileBytes;
        for (int kt = kt0; kt < kt1; ++kt, t += kMxTileBytes) {
            if (kt + 1 < kt1) fetch(nxt, kt + 1);
            const bool in_k = kt * kMxTileCols + lane * 8 < K;
            uint32_t col = 0x7F7F7F7Fu;   // this group's scales of the four rows; padding: 1
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!ROUTED || (live >> i & 1u)) {
                    uint32_t b;
                    const uint32_t codes = quantize8<F32>(cur[i], b);
                    if (in_k && (live >> i & 1u)) col = (col & ~(255u << (8 * i))) | b << (8 * i);
                    *reinterpret_cast<uint32_t*>(t + mx_code_offset(r0 + 32 * i, j) + 4 * (lane & 3)) = codes;
                    cur[i] = nxt[i];
                }
            }
            // transpose the 4 groups x 4 rows of each half-warp: lane i of its first quad gets row
            // i's word
            const uint32_t pick = 0x0040u | (lane & 3) * 0x0011u;   // byte i of either operand
            const int half = lane & 16;
            const uint32_t c0 = __shfl_sync(0xffffffffu, col, half), c1 = __shfl_sync(0xffffffffu, col, half + 4);
            const uint32_t c2 = __shfl_sync(0xffffffffu, col, half + 8), c3 = __shfl_sync(0xffffffffu, col, half + 12);
            const uint32_t w = __byte_perm(__byte_perm(c0, c1, pick), __byte_perm(c2, c3, pick), 0x5410u);
            if ((lane & 12) == 0) *reinterpret_cast<uint32_t*>(t + mx_scale_offset(r0 + 32 * (lane & 3), j)) = w;
        }
    }
}

// Where each pair's row goes, for rows that several pairs share: index[p] = the position of
// pair p in sorted_ids.  Entries of pairs without a position are not written; a reader
// checks sorted_ids[index[p]] == p.
__global__ void __launch_bounds__(256) mx_index_kernel(const RowSource s, int64_t G, int64_t N, int K,
                                                       uint8_t* __restrict__ packed, int32_t* __restrict__ index, int* err) {
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x < kHeaderBytes / 4) mx_write_header(packed, threadIdx.x, G, N, K);
    const int64_t ntp = *s.ntp;
    if (ntp < 0 || ntp > G * N || ntp % N) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, CHORD_DEV_BAD_PADDED);
        return;
    }
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < ntp; i += (int64_t)gridDim.x * blockDim.x) {
        const int32_t id = __ldg(s.sorted_ids + i);
        if (id >= 0 && id < s.id_limit)
            index[id] = (int32_t)i;
        else if (id != s.sentinel)
            set_error(err, CHORD_DEV_BAD_ROW);
    }
}

// Activation rows shared by `divisor` pairs (a token's experts): a row is loaded and
// quantised once and stored at each of its pairs' positions.  One warp, kRows rows,
// `run` tiles along K; lane k keeps where pair k of a row goes.  (A warp per position
// quantised every row `divisor` times: 1024 rows of 7168 for eight experts each took 45 us,
// this 23.)  Bound by the eight scattered stores of a row's codes, 31 MB in 128-byte pieces.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) mx_quantize_shared_kernel(const RowSource s, int64_t a_rows, int64_t G, int64_t N, int K,
                                                                 int run, uint8_t* __restrict__ packed,
                                                                 const int32_t* index) {
    pdl_trigger();
    constexpr int kRows = 2;
    const int64_t ntp = *s.ntp;   // older than the index kernel, as the rows and sorted_ids are
    bool waited = false;
    if (ntp < 0 || ntp > G * N || ntp % N) {   // reported by the index kernel
        pdl_wait();
        return;
    }
    const int kb = (int)mx_col_tiles(K), rt = (int)mx_row_tiles(N), runs = (kb + run - 1) / run;
    const int lane = threadIdx.x & 31;
    const uint32_t j = lane >> 2;
    const int64_t groups = (a_rows + kRows - 1) / kRows, tasks = groups * runs;
    uint8_t* data = packed + kHeaderBytes;
    for (int64_t q = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; q < tasks;
         q += ((int64_t)gridDim.x * blockDim.x) >> 5) {
        int part;
        const int64_t row0 = divmod_idx(q, runs, part) * kRows;
        const int kt0 = part * run, kt1 = min(kt0 + run, kb);
        Raw<F32> cur[kRows] = {}, nxt[kRows];
        auto fetch = [&](Raw<F32>(&v)[kRows], int kt) {
            const int k0 = kt * kMxTileCols + lane * 8;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                v[i] = Raw<F32>{};
                if (row0 + i < a_rows && k0 < K) load8<F32, VEC>(s.src, (row0 + i) * s.row_stride + k0, v[i]);
            }
        };
        // pairs 32 at a time (a row is read again for each such group; 32 experts a token is
        // far above common use)
        for (int first = 0; first < s.divisor; first += 32) {
            fetch(cur, kt0);
            if (!waited) pdl_wait();   // the index
            waited = true;
            uint64_t to[kRows];   // the pair's row in its block's first tile, row mod 8 in the low bits
            uint32_t on[kRows];   // pairs of this group that have a position
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t p = (row0 + i) * s.divisor + first + lane;
                int64_t pos = -1;
                if (row0 + i < a_rows && first + lane < s.divisor && p < s.id_limit) {
                    pos = __ldcg(index + p);   // not as a read-only value: that might be fetched ahead of the wait
                    if (pos < 0 || pos >= ntp || __ldg(s.sorted_ids + pos) != (int32_t)p) pos = -1;
                }
                on[i] = __ballot_sync(0xffffffffu, pos >= 0);
                int r = 0;
                const int64_t blk = pos >= 0 ? divmod_idx(pos, (int)N, r) : 0;
                to[i] = (uint64_t)((blk * rt + (r >> 7)) * kb) * kMxTileBytes << 7 | (uint32_t)(r & 127);
            }
            for (int kt = kt0; kt < kt1; ++kt) {
                if (kt + 1 < kt1) fetch(nxt, kt + 1);
                const bool in_k = kt * kMxTileCols + lane * 8 < K;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    if (!on[i]) continue;
                    uint32_t b;
                    const uint32_t codes = quantize8<F32>(cur[i], b);
                    uint32_t w = (in_k ? b : 127u) << (8 * (j & 3));
                    w |= __shfl_xor_sync(0xffffffffu, w, 4);
                    w |= __shfl_xor_sync(0xffffffffu, w, 8);
                    uint8_t* tile = data + (int64_t)kt * kMxTileBytes;
                    for (uint32_t m = on[i]; m; m &= m - 1) {
                        const uint64_t d = __shfl_sync(0xffffffffu, to[i], __ffs(m) - 1);
                        const uint32_t r = (uint32_t)d & 127u;
                        *reinterpret_cast<uint32_t*>(tile + (d >> 7) + mx_code_offset(r, j) + 4 * (lane & 3)) = codes;
                    }
                    // scale words: lane 2 k + h stores half h of pair k, sixteen pairs at a time
                    const uint32_t wh = __shfl_sync(0xffffffffu, w, (lane & 1) * 16);
#pragma unroll
                    for (int k0 = 0; k0 < 32; k0 += 16) {
                        const uint64_t d = __shfl_sync(0xffffffffu, to[i], k0 + (lane >> 1));
                        if (on[i] >> (k0 + (lane >> 1)) & 1u)
                            *reinterpret_cast<uint32_t*>(tile + (d >> 7) + mx_scale_offset((uint32_t)d & 127u, 4 * (lane & 1))) = wh;
                        if (first + 16 >= s.divisor) break;
                    }
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) cur[i] = nxt[i];
            }
        }
    }
    if (!waited) pdl_wait();
}

// The same split; a lane writes the values of its eight columns of each row.  Bound by the
// writes to HBM: 8 x 4096 x 7168 values to bf16 (125 MB read, 470 MB written) in 100 us,
// 5.9 TB/s (streaming stores: the same).
template <bool F32>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* __restrict__ packed, int64_t G, int64_t N,
                                                            int K, int run, void* __restrict__ out, int* err) {
    if (!mx_header_ok(packed, G, N, K)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, CHORD_DEV_BAD_HEADER);
        return;
    }
    const int64_t rt = mx_row_tiles(N);
    const int kb = (int)mx_col_tiles(K);
    const int runs = (kb + run - 1) / run;
    const int lane = threadIdx.x & 31;
    const uint32_t j = lane >> 2;
    const int64_t tasks = G * rt * runs * 32;
    const uint8_t* data = packed + kHeaderBytes;
    for (int64_t q = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; q < tasks;
         q += ((int64_t)gridDim.x * blockDim.x) >> 5) {
        const uint32_t r0 = (uint32_t)(q & 31);
        int part, bt;
        const int64_t band = divmod_idx(q >> 5, runs, part);
        const int64_t g = divmod_idx(band, (int)rt, bt);
        const int kt0 = part * run, kt1 = min(kt0 + run, kb);
        const uint8_t* t = data + (band * kb + kt0) * kMxTileBytes;
        uint32_t w[4], wn[4] = {};
        uint4 sc, scn = {};
        auto fetch = [&](uint32_t(&c)[4], uint4& s4, const uint8_t* tile) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] = __ldg(reinterpret_cast<const uint32_t*>(tile + mx_code_offset(r0 + 32 * i, j) + 4 * (lane & 3)));
            s4 = __ldg(reinterpret_cast<const uint4*>(tile + mx_scale_offset(r0, j & 4u)));
        };
        fetch(w, sc, t);
        const int64_t row0 = (int64_t)bt * kMxTileRows + r0;
        int64_t o = (g * N + row0) * K + kt0 * kMxTileCols + lane * 8;   // K % 32 == 0: 16-byte aligned
        for (int kt = kt0; kt < kt1; ++kt, t += kMxTileBytes, o += kMxTileCols) {
            if (kt + 1 < kt1) fetch(wn, scn, t + kMxTileBytes);
            const uint32_t scw[4] = {sc.x, sc.y, sc.z, sc.w};
            if (kt * kMxTileCols + lane * 8 < K) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (row0 + 32 * i >= N) continue;
                    const float f = mx_scale_f32((scw[i] >> (8 * (j & 3))) & 255u);
                    uint32_t h[4];
                    e2m1_halves8(w[i], h);
                    float v[8];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[c]));
                        v[2 * c] = p.x * f;
                        v[2 * c + 1] = p.y * f;
                    }
                    const int64_t oi = o + (int64_t)(32 * i) * K;
                    if constexpr (F32) {
                        float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + oi);
                        d[0] = make_float4(v[0], v[1], v[2], v[3]);
                        d[1] = make_float4(v[4], v[5], v[6], v[7]);
                    } else {
                        uint4 d;
                        d.x = bf2_as_u32(__floats2bfloat162_rn(v[0], v[1]));
                        d.y = bf2_as_u32(__floats2bfloat162_rn(v[2], v[3]));
                        d.z = bf2_as_u32(__floats2bfloat162_rn(v[4], v[5]));
                        d.w = bf2_as_u32(__floats2bfloat162_rn(v[6], v[7]));
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + oi) = d;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = wn[i];
            sc = scn;
        }
    }
}

// Tiles along K per warp task: up to 4 (loads of the next tile overlap the
// conversion), fewer while that leaves fewer tasks than the GPU holds warps.
int run_for(int64_t bands, int kb) {
    const int64_t warps = (int64_t)device_info().sm_count * 32;
    int run = 4;
    while (run > 1 && bands * 32 * ((kb + run - 1) / run) < warps) run >>= 1;
    return run;
}

// CTAs of 8 warps for `tasks` warp tasks: at most 8 per SM (the kernels stride).
unsigned grid_for(int64_t tasks) {
    const int64_t b = (tasks + 7) / 8, cap = (int64_t)device_info().sm_count * 8;
    return (unsigned)(b < 1 ? 1 : (b > cap ? cap : b));
}

cudaError_t launch_quantize(const RowSource& s, int64_t G, int64_t N, int K, uint8_t* packed, int* err,
                            cudaStream_t st) {
    const int esz = s.f32 ? 4 : 2;
    // 16-byte loads where every row starts on a 16-byte boundary
    const bool vec = (reinterpret_cast<uintptr_t>(s.src) | (s.sorted_ids || N > 1 ? (uintptr_t)(s.row_stride * esz) : 0) |
                      (G > 1 ? (uintptr_t)(s.mat_stride * esz) : 0)) % 16 == 0;
    const int kb = (int)mx_col_tiles(K);
    const int64_t bands = G * mx_row_tiles(N);
    const int run = run_for(bands, kb);
    const unsigned grid = grid_for(bands * ((kb + run - 1) / run) * 32);
    auto kern = s.sorted_ids ? (s.f32 ? (vec ? mx_quantize_kernel<true, true, true> : mx_quantize_kernel<true, false, true>)
                                      : (vec ? mx_quantize_kernel<false, true, true> : mx_quantize_kernel<false, false, true>))
                             : (s.f32 ? (vec ? mx_quantize_kernel<true, true, false> : mx_quantize_kernel<true, false, false>)
                                      : (vec ? mx_quantize_kernel<false, true, false> : mx_quantize_kernel<false, false, false>));
    kern<<<grid, 256, 0, st>>>(s, G, N, K, run, packed, err);
    return cudaGetLastError();
}

// Routed rows: shared ones through the index (it has an entry per position, so room for every
// pair id unless the caller routes a few pairs of many), others position by position.
cudaError_t launch_quantize_rows(const RowSource& s, int64_t a_rows, int64_t G, int64_t N, int K, uint8_t* packed,
                                 int32_t* index, int* err, cudaStream_t st) {
    if (s.divisor == 1 || a_rows == 0 || s.id_limit > G * N) return launch_quantize(s, G, N, K, packed, err, st);
    const int esz = s.f32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(s.src) | (a_rows > 1 ? (uintptr_t)(s.row_stride * esz) : 0)) % 16 == 0;
    const int kb = (int)mx_col_tiles(K);
    const int run = run_for((a_rows + 63) / 64, kb);
    const int64_t ids = (G * N + 255) / 256, cap = (int64_t)device_info().sm_count * 8;
    // a plain launch: the next kernel reads rows and counts before its wait (see pdl_wait)
    mx_index_kernel<<<(unsigned)(ids < 1 ? 1 : (ids > cap ? cap : ids)), 256, 0, st>>>(s, G, N, K, packed, index, err);
    auto kern = s.f32 ? (vec ? mx_quantize_shared_kernel<true, true> : mx_quantize_shared_kernel<true, false>)
                      : (vec ? mx_quantize_shared_kernel<false, true> : mx_quantize_shared_kernel<false, false>);
    return launch_pdl(pdl_enabled(), kern, dim3(grid_for((a_rows + 1) / 2 * ((kb + run - 1) / run))), dim3(256), 0, st, s, a_rows,
                      G, N, K, run, packed, (const int32_t*)index);
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
    const unsigned long long group = mx_group_bytes(N, K);   // below 2^62
    // what 64 bits of byte offset cannot hold is no size: a wrapped one would pass for a small buffer
    if (group && (unsigned long long)G > ((1ull << 62) - kHeaderBytes) / group) return 0;
    return (size_t)kHeaderBytes + (size_t)G * (size_t)group;
}

size_t chord_mxfp4_rows_bytes(int64_t capacity, int block_m, int K) {
    if (capacity < 0 || block_m <= 0 || capacity % block_m) return 0;
    const size_t n = chord_mxfp4_bytes(capacity / block_m, block_m, K);
    return n ? n + ((size_t)capacity * 4 + 255) / 256 * 256 : 0;   // and each pair's position
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
    RowSource s{src, src_dtype == CHORD_DTYPE_F32, row_stride, mat_stride, nullptr, nullptr, 0, 0, 1};
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
    const size_t need = chord_mxfp4_rows_bytes(capacity, block_m, K);
    if (need == 0 || packed_bytes != need) return CHORD_ERR_LAYOUT_MISMATCH;
    if (a_rows > 1 && row_stride < K) return CHORD_ERR_INVALID_ARG;
    if (!packed || !aligned16(packed) || !num_tokens_padded || (capacity > 0 && !sorted_ids))
        return CHORD_ERR_INVALID_ARG;
    if (a_rows > 0 && (!A || !aligned_to(A, a_dtype == CHORD_DTYPE_F32 ? 4 : 2))) return CHORD_ERR_INVALID_ARG;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    const int64_t limit = a_rows * (int64_t)a_row_divisor;
    RowSource s{A,         a_dtype == CHORD_DTYPE_F32, row_stride, 0, sorted_ids, num_tokens_padded,
                limit < num_pairs ? limit : num_pairs, (int32_t)num_pairs, a_row_divisor};
    uint8_t* out = static_cast<uint8_t*>(packed);
    int32_t* index = reinterpret_cast<int32_t*>(out + chord_mxfp4_bytes(capacity / block_m, block_m, K));
    return launch_quantize_rows(s, a_rows, capacity / block_m, block_m, K, out, index, di.err,
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
    const int kb = (int)mx_col_tiles(K);
    const int64_t bands = G * mx_row_tiles(N);
    if (bands == 0) return CHORD_OK;
    const int run = run_for(bands, kb);
    auto kern = out_dtype == CHORD_DTYPE_F32 ? mx_dequantize_kernel<true> : mx_dequantize_kernel<false>;
    kern<<<grid_for(bands * ((kb + run - 1) / run) * 32), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t*>(packed), G, N, K, run, out, di.err);
    return cudaGetLastError() == cudaSuccess ? CHORD_OK : CHORD_ERR_CUDA;
}

}  // extern "C"
