// One mixture-of-experts layer for a few tokens (at most CHORD_FEW_MAX_TOKENS),
// expert weights in 4 bits:
//   h[t, e]   = topk_w[t, e] * SiLU(W13[e][:I] x_t) * (W13[e][I:] x_t)
//   out[t]    = bf16( sum over the token's local experts of W2[e] h[t, e] )
// in two launches: gate_up with the activation and the routing weight, then
// the down projection with the sum over the experts.
//
// The weights' bytes bound the layer, so both kernels stream every used
// expert's weights once, each lane into its own shared-memory slots (16-byte
// cp.async, a ring of units per warp, no barrier in the loop), and multiply on the
// warp-level tensor cores: a tile is 16 weight rows x 128 columns, the MMA's A
// side, with tokens on the B side.  Lane (g, c) of a warp holds rows g and g + 8 and
// the 32-column group c of the tile: one 16-byte load and one scale per row.  The
// MMA's k order inside a tile is whatever puts a lane's own 32 columns into its
// slots, the same for A and B.
//   gate_up: an item is 16 gate rows and their 16 up rows of one expert (two
//     tiles of 8 + 8), B column j its j-th token, the K range split over the warps of
//     a group and joined in shared memory in warp order; a lane then holds a gate
//     sum and its up sum, and h is written as two bf16 numbers (value and
//     remainder, 16 significant bits together).
//   down: a CTA owns rows of the output for all experts, B column t token t of the
//     call (zero where it does not use the expert); its warps split the (expert, K
//     unit) pairs and join their sums in warp order, so neither atomics nor a
//     combine pass are needed.  The kernel is launched early (programmatic
//     dependent launch) and fills its rings while gate_up still runs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chord_internal.h"
#include "chord_mxfp4.cuh"

namespace chord {
namespace {

constexpr int kUpWarps = 8;
constexpr int kUpThreads = kUpWarps * 32;
constexpr int kTileBytes = 1280;     // a tile's slots: 32 lanes x (2 x 16 bytes of codes + 2 x 4 bytes of scales)
constexpr int kUpDepth = 3;          // units (two tiles) in flight per warp, gate_up
constexpr int kDownDepth = 2;        // units (RT tiles) in flight per warp, down
constexpr size_t kSmemMax = 226 * 1024;    // dynamic; the kernels hold a few static bytes too
constexpr size_t kSmemHalf = 112 * 1024;   // two CTAs per SM

struct FewArgs {
    const uint16_t* x;
    const int32_t* ids;
    const float* wts;
    int T, topk, E, H, I;
    const uint8_t* w13;
    const uint8_t* w2;
    uint16_t* h;         // [2][T * topk, I]: bf16 values, then bf16 remainders; one row per (expert, token) in use
    uint16_t* out;
    int* err;
    int validate;        // report ids outside [-1, E)
    int used_cap;        // min(E, T * topk)
    int warps_item;      // gate_up: warps that share an item's K range
    int units_warp;      // gate_up: K units of one warp, at most
    int x_cap;           // gate_up: tokens of an expert whose activations fit in shared memory
};

// ---- which experts are used, by which tokens --------------------------------
struct Route {
    int used;
    const uint16_t* expert;    // ascending
    const uint32_t* tokens;    // bit t: token t uses it
    const uint16_t* first;     // its first row of h
};

__host__ __device__ __forceinline__ size_t route_bytes(int E, int P, int used_cap) {
    return (size_t)E * 4 + (size_t)P * 8 + (size_t)used_cap * 8 + 128 + 16;
}

// Builds the route in shared memory (all threads) and leaves the ids and
// weights there too.
template <int WARPS>
__device__ Route build_route(const FewArgs& a, uint8_t* sm, int32_t*& s_ids, float*& s_w, bool report) {
    const int P = a.T * a.topk, tid = threadIdx.x;
    uint32_t* mask = reinterpret_cast<uint32_t*>(sm);
    s_ids = reinterpret_cast<int32_t*>(mask + a.E);
    s_w = reinterpret_cast<float*>(s_ids + P);
    uint32_t* tokens = reinterpret_cast<uint32_t*>(s_w + P);
    uint16_t* expert = reinterpret_cast<uint16_t*>(tokens + a.used_cap);
    uint16_t* first = expert + a.used_cap;
    uint32_t* sums = reinterpret_cast<uint32_t*>((reinterpret_cast<uintptr_t>(first + a.used_cap) + 15) & ~(uintptr_t)15);
    constexpr int kThreads = WARPS * 32, kPer = 1024 / kThreads;   // experts per thread in the scan (E <= 1024)
    for (int e = tid; e < a.E; e += kThreads) mask[e] = 0;
    __syncthreads();
    for (int p = tid; p < P; p += kThreads) {
        const int32_t e = a.ids[p];
        s_ids[p] = e;
        s_w[p] = a.wts[p];
        if (e >= 0 && e < a.E)
            atomicOr(&mask[e], 1u << (p / a.topk));
        else if (report && e != -1)
            set_error(a.err, CHORD_DEV_BAD_EXPERT);
    }
    __syncthreads();
    // exclusive scan over the experts of (used, rows of h), packed as
    // used << 16 | rows (both at most 1024)
    uint32_t m[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        m[i] = e < a.E ? mask[e] : 0u;
        mine += m[i] ? (1u << 16) + __popc(m[i]) : 0u;
    }
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if ((tid & 31) >= o) inc += v;
    }
    if ((tid & 31) == 31) sums[tid >> 5] = inc;
    __syncthreads();
    uint32_t at = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < (tid >> 5)) at += sums[w];
        total += sums[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (!m[i]) continue;
        const uint32_t u = at >> 16;
        expert[u] = (uint16_t)(tid * kPer + i);
        tokens[u] = m[i];
        first[u] = (uint16_t)at;
        at += (1u << 16) + __popc(m[i]);
    }
    __syncthreads();
    return Route{(int)(total >> 16), expert, tokens, first};
}

// ---- weights: addresses and dequantisation ------------------------------------
// Offsets from an expert's first byte of a lane's codes (group c of K unit 0)
// and scale word of weight row `row`; the next row of the same 8-row phase (row + 8) is
// kRow8 and kScale8 further on, K unit u at unit_offset(u).
template <bool MX>
struct Lay {
    static constexpr uint32_t kRow8 = MX ? 1024 : 128, kScale8 = MX ? 128 : 32;
    static __device__ __forceinline__ uint64_t expert_bytes(int N, int K) {
        return MX ? mx_group_bytes(N, K) : (uint64_t)N * (uint64_t)K * 9ull / 16ull;
    }
    static __device__ __forceinline__ uint32_t code(int row, int K, int c) {
        const uint32_t r = row & 127;
        if constexpr (MX)
            return (uint32_t)(row >> 7) * (uint32_t)mx_col_tiles(K) * kMxTileBytes + r * 128 + ((c ^ (r & 7)) << 4);
        else
            return (uint32_t)(row >> 7) * (uint32_t)(K / 64) * 4608u + (c >> 1) * 4608 + (c & 1) * 2048 + r * 16;
    }
    static __device__ __forceinline__ uint32_t scale(int row, int K, int c) {
        const uint32_t r = row & 127;
        if constexpr (MX)
            return (uint32_t)(row >> 7) * (uint32_t)mx_col_tiles(K) * kMxTileBytes + mx_scale_offset(r, 0);
        else
            return (uint32_t)(row >> 7) * (uint32_t)(K / 64) * 4608u + (c >> 1) * 4608 + 4096 + r * 4;
    }
    // MXFP4: two units share a 256-column tile; the swizzled code slot of the second
    // one is 64 bytes up or down (g: the lane's row mod 8)
    static __device__ __forceinline__ int64_t code_unit(int u, int g) {
        if constexpr (MX) return (int64_t)(u >> 1) * kMxTileBytes + (u & 1 ? (g & 4 ? -64 : 64) : 0);
        return (int64_t)u * 9216;
    }
    static __device__ __forceinline__ int64_t scale_unit(int u) {
        if constexpr (MX) return (int64_t)(u >> 1) * kMxTileBytes + (u & 1) * kMxScaleBlock;
        return (int64_t)u * 9216;
    }
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A tile's rows g and g + 8 to this lane's slots: codes at 0 and 512, the two
// scale words together at 1024.  Columns past K (off): zeros.
__device__ __forceinline__ void fetch_tile(uint32_t slot, int lane, const uint8_t* c0, const uint8_t* c1, const uint8_t* s0,
                                           const uint8_t* s1, bool on) {
    const uint32_t d = slot + lane * 16, ds = slot + 1024 + lane * 8;
    if (on) {
        cp_async16(d, c0);
        cp_async16(d + 512, c1);
        cp_async4(ds, s0);
        cp_async4(ds + 4, s1);
    } else {
        const uint4 z = make_uint4(0, 0, 0, 0);
        sts128(d, z);
        sts128(d + 512, z);
        asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(ds), "r"(0) : "memory");
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// The scale of a lane's group, ready for the dequantisation in use.
//   INT4, every scale in the one-FMA range: (s * 2^129, -8 s); else (s, s).
//   MXFP4: a code's three magnitude bits at bits 6..8 of a half-word are the bf16
//   number value * 2^-126 (subnormal 0.5 included), so one multiply by
//   2^(b - 1) gives the weight exactly; it fits bf16 for b <= 128, and larger scales
//   (wide) take two multiplies, 2^126 and 2^(b - 127).
struct Scale {
    uint32_t m, n;
};

template <bool MX, bool FAST>
__device__ __forceinline__ Scale make_scale(uint32_t word, int c) {
    Scale s;
    if constexpr (MX) {
        const uint32_t b = (word >> (8 * c)) & 255u;
        const uint32_t m = b <= 128u ? (b + 126u) << 7 : (b == 255u ? 0x7FC0u : (b << 7));
        s.m = m | m << 16;
        s.n = b > 128u ? 1u : 0u;
    } else {
        const uint32_t sp = prmt(word, c & 1 ? 0x3232u : 0x1010u);
        s.m = sp;
        s.n = 0;
        if constexpr (FAST) fma_scale_pair(sp, s.m, s.n);
    }
    return s;
}

// Eight codes to four bf16 pairs; wide: MXFP4 scales above 2 are present.
template <bool MX, bool FAST>
__device__ __forceinline__ void dequant8(uint32_t w, const Scale& s, bool wide, uint32_t (&o)[4]) {
    if constexpr (MX) {
        uint32_t v[4];
        v[0] = ((w << 6) & 0x01C001C0u) | ((w << 12) & 0x80008000u);   // columns 0, 4
        v[1] = ((w << 2) & 0x01C001C0u) | ((w << 8) & 0x80008000u);    // 1, 5
        v[2] = ((w >> 2) & 0x01C001C0u) | ((w << 4) & 0x80008000u);    // 2, 6
        v[3] = ((w >> 6) & 0x01C001C0u) | (w & 0x80008000u);           // 3, 7
        if (wide) {
            const __nv_bfloat162 big = u32_as_bf2(0x7E807E80u);        // 2^126
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s.n) v[i] = bf2_as_u32(__hmul2(u32_as_bf2(v[i]), big));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = bf2_as_u32(__hmul2(u32_as_bf2(v[i]), u32_as_bf2(s.m)));
    } else if constexpr (FAST) {
        dequant_row8_fma(w, s.m, s.n, o);
    } else {
        dequant_row8(w, s.m, o);
    }
}

// Activations in the order in which dequant8 leaves the columns: INT4 natural,
// MXFP4 (0, 4), (1, 5), (2, 6), (3, 7).
template <bool MX>
__device__ __forceinline__ uint4 b_order(uint4 v) {
    if constexpr (!MX) return v;
    uint4 r;
    asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(r.x) : "r"(v.x), "r"(v.z));
    asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(r.y) : "r"(v.x), "r"(v.z));
    asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(r.z) : "r"(v.y), "r"(v.w));
    asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(r.w) : "r"(v.y), "r"(v.w));
    return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Headers of both blobs; inter: w13 in the gate/up-interleaved layout; fast:
// the one-FMA dequantisation fits the blob asked for.
template <bool MX>
__device__ __forceinline__ int check_headers(const FewArgs& a, bool down) {
    bool inter = false, ok;
    if constexpr (MX) {
        ok = mx_header_ok(a.w13, a.E, 2 * a.I, a.H) && mx_header_ok(a.w2, a.E, a.H, a.I);
    } else {
        inter = header_ok_layout(a.w13, a.E, 2 * a.I, a.H, CHORD_LAYOUT_GATE_UP_INTERLEAVED);
        ok = (inter || header_ok_layout(a.w13, a.E, 2 * a.I, a.H, CHORD_LAYOUT_TCGEN05)) &&
             header_ok_layout(a.w2, a.E, a.H, a.I, CHORD_LAYOUT_TCGEN05);
    }
    const bool fast = !MX && ok && header_scales_in_fma_range(down ? a.w2 : a.w13);
    return (ok ? 1 : 0) | (inter ? 2 : 0) | (fast ? 4 : 0);
}

// Position of the n-th set bit of m (n below their number; mostly 0 or 1 here).
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
    for (; n > 0; --n) m &= m - 1;
    return __ffs(m) - 1;
}

// ---- gate_up ----------------------------------------------------------------
struct UpSmem {
    uint32_t ring;      // this warp's slots
    uint32_t x;         // this warp's activations
    uint32_t zero;      // 256 bytes of zeros: what lanes without a token read
    float4* red;        // [2][kUpWarps][2][32]
};

// One item's K range of one warp.  SPILL: the expert has more tokens than x_cap,
// the others' activations are read from global memory.
template <bool MX, int NT, bool FAST, bool SPILL, typename Fetch>
__device__ __forceinline__ void up_units(const FewArgs& a, const UpSmem& sm, int ua, int ub, int nts, int& slot,
                                         const uint32_t (&xa)[NT], const uint32_t (&step)[NT], const int (&far)[NT],
                                         float (&acc)[2][NT][4], Fetch&& fetch) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    for (int u = ua; u < ub; ++u) {
        cp_async_wait<kUpDepth - 2>();
        const uint32_t st = sm.ring + slot * 2 * kTileBytes + lane * 16;
        if (++slot == kUpDepth) slot = 0;
        uint4 q[2][2];
        Scale s[2][2];
        bool wide = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            q[i][0] = lds128(st + i * kTileBytes);
            q[i][1] = lds128(st + i * kTileBytes + 512);
            const uint2 w = lds64(st + i * kTileBytes + 1024 - lane * 8);
            s[i][0] = make_scale<MX, FAST>(w.x, c);
            s[i][1] = make_scale<MX, FAST>(w.y, c);
            if constexpr (MX) wide |= (s[i][0].n | s[i][1].n) != 0;
        }
        if constexpr (MX) wide = __any_sync(0xffffffffu, wide);
        fetch();   // into the slots that the unit before this one left
        const uint32_t at = (uint32_t)(u - ua) * 256u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t x[2][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                dequant8<MX, FAST>(word(q[i][0], j), s[i][0], wide, x[i][0]);
                dequant8<MX, FAST>(word(q[i][1], j), s[i][1], wide, x[i][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (NT > 1 && nt >= nts) continue;
                uint4 b = lds128(xa[nt] + (at & step[nt]) + j * 64);
                if constexpr (SPILL) {
                    if (far[nt] >= 0 && (u * 4 + c) * 32 < a.H)
                        b = b_order<MX>(__ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)far[nt] * a.H + u * 128 + c * 32 + j * 8)));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma16816(acc[i][nt], x[i][0][0], x[i][1][0], x[i][0][1], x[i][1][1], b.x, b.y);
                    mma16816(acc[i][nt], x[i][0][2], x[i][1][2], x[i][0][3], x[i][1][3], b.z, b.w);
                }
            }
        }
    }
}

template <bool MX, int NT, bool FAST>
__device__ __forceinline__ void gate_up_loop(const FewArgs& a, const Route& rt, const int32_t* s_ids, const float* s_w,
                                             const UpSmem& sm, bool inter) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int W = a.warps_item, ngrp = kUpWarps / W, grp = warp / W, rank = warp % W;
    const int U = (a.H + 127) / 128, kgroups = a.H / 32;
    const int ua = rank * U / W, ub = (rank + 1) * U / W, nu = ub - ua;
    const int per_e = a.I / 16;
    const int n_items = rt.used * per_e;
    const int i0 = (int)((int64_t)blockIdx.x * n_items / gridDim.x), i1 = (int)((int64_t)(blockIdx.x + 1) * n_items / gridDim.x);
    const int first = i0 + grp;
    const int mine = first < i1 ? (i1 - first + ngrp - 1) / ngrp : 0;
    const int steps = mine * nu;
    const uint64_t expert_bytes = Lay<MX>::expert_bytes(2 * a.I, a.H);
    // interleaved: rows of tile i at 16 i of the item's 32 (8 gate, 8 up); else gate and up rows 8 i apart
    const uint32_t d_code = (inter ? 2 : 1) * Lay<MX>::kRow8, d_scale = (inter ? 2 : 1) * Lay<MX>::kScale8;

    // producer: the next unit to fetch
    const uint8_t *gc = nullptr, *gs = nullptr, *uc = nullptr, *us = nullptr;
    int p_item = first, p_u = ub, p_slot = 0, fetched = 0;
    auto fetch = [&]() {
        if (fetched < steps) {
            if (p_u == ub) {
                if (fetched) p_item += ngrp;
                p_u = ua;
                const int ue = p_item / per_e, it = p_item - ue * per_e;
                const uint8_t* base = a.w13 + kHeaderBytes + (uint64_t)rt.expert[ue] * expert_bytes;
                const int gr = inter ? 32 * it + g : 16 * it + g, ur = inter ? gr + 8 : a.I + gr;
                gc = base + Lay<MX>::code(gr, a.H, c);
                gs = base + Lay<MX>::scale(gr, a.H, c);
                uc = base + Lay<MX>::code(ur, a.H, c);
                us = base + Lay<MX>::scale(ur, a.H, c);
            }
            const int64_t co = Lay<MX>::code_unit(p_u, g), so = Lay<MX>::scale_unit(p_u);
            const bool on = p_u * 4 + c < kgroups;
            const uint32_t slot = sm.ring + p_slot * 2 * kTileBytes;
            fetch_tile(slot, lane, gc + co, uc + co, gs + so, us + so, on);
            fetch_tile(slot + kTileBytes, lane, gc + co + d_code, uc + co + d_code, gs + so + d_scale, us + so + d_scale, on);
            ++p_u;
            ++fetched;
            if (++p_slot == kUpDepth) p_slot = 0;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kUpDepth - 1; ++i) fetch();

    const uint32_t x_stride = (uint32_t)a.units_warp * 256u + 64u;   // one token's activations of this warp's K range
    int cur = -1, slot = 0, join = 0, ntok = 0;
    uint32_t tokens = 0;
    // B column 8 nt + g: address and step (all ones, or 0 for the zeros) of its
    // activations in shared memory; far: the token whose activations are in global memory
    uint32_t xa[NT], step[NT];
    int far[NT];
    for (int n = 0; n < mine; ++n) {
        const int item = first + n * ngrp, ue = item / per_e;
        if (ue != cur) {
            cur = ue;
            tokens = rt.tokens[ue];
            ntok = __popc(tokens);
            __syncwarp();
            int at = 0;
            for (uint32_t m = tokens; m && at < a.x_cap; m &= m - 1, ++at) {
                const int t = __ffs(m) - 1;
                for (int q = lane; q < nu * 16; q += 32) {
                    // piece q: 8 columns; kept as (unit, piece of the group, group) so that a
                    // quad's four loads of one piece are contiguous
                    const int k = (ua * 16 + q) * 8;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (k < a.H) v = b_order<MX>(__ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H + k)));
                    sts128(sm.x + (uint32_t)at * x_stride + (uint32_t)((q >> 4) * 256 + (q & 3) * 64 + ((q >> 2) & 3) * 16), v);
                }
            }
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int col = 8 * nt + g;
                const bool near = col < ntok && col < a.x_cap;
                xa[nt] = (near ? sm.x + (uint32_t)col * x_stride : sm.zero) + c * 16;
                step[nt] = near ? 0xffffffffu : 0u;
                far[nt] = -1;
                if (col < ntok && !near) far[nt] = nth_bit(tokens, col);
            }
        }
        float acc[2][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i >> 2][nt][i & 3] = 0.0f;
        const int nts = (ntok + 7) / 8;
        if (ntok > a.x_cap)
            up_units<MX, NT, FAST, true>(a, sm, ua, ub, nts, slot, xa, step, far, acc, fetch);
        else
            up_units<MX, NT, FAST, false>(a, sm, ua, ub, nts, slot, xa, step, far, acc, fetch);
        // join the K ranges of the group's warps in warp order, eight tokens at a time (the
        // buffers alternate, so one barrier each is enough; the warps take turns joining)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt >= nts) continue;
            float4* red = sm.red + (size_t)(join & 1) * kUpWarps * 64;
            red[warp * 64 + lane] = make_float4(acc[0][nt][0], acc[0][nt][1], acc[0][nt][2], acc[0][nt][3]);
            red[warp * 64 + 32 + lane] = make_float4(acc[1][nt][0], acc[1][nt][1], acc[1][nt][2], acc[1][nt][3]);
            if (W > 1)
                group_sync(1 + grp, W * 32);
            else
                __syncwarp();
            if (rank == join++ % W) {
                const int e = rt.expert[ue];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float4 s = red[grp * W * 64 + i * 32 + lane];
                    for (int w = 1; w < W; ++w) {
                        const float4 v = red[(grp * W + w) * 64 + i * 32 + lane];
                        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                    }
                    const int col = (item - ue * per_e) * 16 + i * 8 + g;
                    const int pos = MX ? (col & ~7) | ((col & 3) << 1) | ((col >> 2) & 1) : col;
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        const int jt = 8 * nt + 2 * c + h2;
                        if (jt >= ntok) continue;
                        const int t = nth_bit(tokens, jt);
                        float wt = 0.0f;
                        for (int k = 0; k < a.topk; ++k)
                            if (s_ids[t * a.topk + k] == e) wt += s_w[t * a.topk + k];
                        const float h = wt * silu_times(h2 ? s.y : s.x, h2 ? s.w : s.z);
                        // bf16 value and remainder; no remainder for infinities and NaN
                        const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                        const float rest = h - __bfloat162float(hi);
                        const int64_t to = (int64_t)(rt.first[ue] + jt) * a.I + pos;
                        a.h[to] = __bfloat16_as_ushort(hi);
                        a.h[to + (int64_t)a.T * a.topk * a.I] =
                            __bfloat16_as_ushort(__float2bfloat16_rn(isfinite(rest) ? rest : 0.0f));
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
}

template <bool MX, int NT>
__global__ void __launch_bounds__(kUpThreads, 2) few_gate_up_kernel(const FewArgs a) {
    pdl_trigger();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int flags;
    __shared__ __align__(16) uint8_t zeros[256];
    if (threadIdx.x < 64) reinterpret_cast<uint32_t*>(zeros)[threadIdx.x] = 0u;
    if (threadIdx.x == 0) {
        flags = check_headers<MX>(a, false);
        if (!(flags & 1) && blockIdx.x == 0) set_error(a.err, CHORD_DEV_BAD_HEADER);
    }
    const int warp = threadIdx.x >> 5;
    UpSmem sm;
    sm.ring = smem_u32(smem) + warp * kUpDepth * 2 * kTileBytes;
    uint8_t* red = smem + kUpWarps * kUpDepth * 2 * kTileBytes;
    sm.red = reinterpret_cast<float4*>(red);
    uint8_t* xs = red + 2 * kUpWarps * 64 * sizeof(float4);
    const uint32_t x_warp = (uint32_t)a.x_cap * ((uint32_t)a.units_warp * 256u + 64u);
    sm.x = smem_u32(xs) + warp * x_warp;
    sm.zero = smem_u32(zeros);
    int32_t* s_ids;
    float* s_w;
    const Route rt = build_route<kUpWarps>(a, xs + kUpWarps * x_warp, s_ids, s_w, a.validate && blockIdx.x == 0);
    if (!(flags & 1)) return;
    if (MX || (flags & 4))
        gate_up_loop<MX, NT, true>(a, rt, s_ids, s_w, sm, (flags & 2) != 0);
    else
        gate_up_loop<MX, NT, false>(a, rt, s_ids, s_w, sm, (flags & 2) != 0);
}

// ---- down -------------------------------------------------------------------
// Warps per CTA: 16, or 8 where the sums of more than 16 tokens need the registers.
template <int NT>
constexpr int kDownWarps = NT > 2 ? 8 : 16;

template <bool MX, int NT, int RT, bool FAST>
__device__ __forceinline__ void down_loop(const FewArgs& a, const Route& rt, uint32_t ring, int tile0, int rank, int ranks,
                                          float (&acc)[RT][NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int KU = (a.I + 127) / 128, kgroups = a.I / 32, tiles = a.H / 16;
    const int total = rt.used * KU;
    const uint64_t expert_bytes = Lay<MX>::expert_bytes(a.H, a.I);
    uint32_t co[RT], so[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = min(tile0 + i, tiles - 1) * 16 + g;   // a tile past H repeats the last one and is not written
        co[i] = Lay<MX>::code(row, a.I, c);
        so[i] = Lay<MX>::scale(row, a.I, c);
    }
    int pv = rank, p_slot = 0;
    auto fetch = [&]() {
        if (pv < total) {
            const int ue = pv / KU, ku = pv - ue * KU;
            const uint8_t* base = a.w2 + kHeaderBytes + (uint64_t)rt.expert[ue] * expert_bytes;
            const uint8_t *cb = base + Lay<MX>::code_unit(ku, g), *sb = base + Lay<MX>::scale_unit(ku);
            const bool on = ku * 4 + c < kgroups;
#pragma unroll
            for (int i = 0; i < RT; ++i)
                fetch_tile(ring + (p_slot * RT + i) * kTileBytes, lane, cb + co[i], cb + co[i] + Lay<MX>::kRow8, sb + so[i],
                           sb + so[i] + Lay<MX>::kScale8, on);
            pv += ranks;
            if (++p_slot == kDownDepth) p_slot = 0;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDownDepth - 1; ++i) fetch();
    pdl_wait();   // h of the gate_up kernel is complete from here on
    const int64_t lo_plane = (int64_t)a.T * a.topk * a.I;
    int slot = 0;
    for (int v = rank; v < total; v += ranks) {
        const int ue = v / KU, ku = v - ue * KU;
        const uint32_t tokens = rt.tokens[ue];
        const uint16_t* hp[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int t = 8 * nt + g;
            const bool on = (tokens >> t & 1u) && ku * 4 + c < kgroups;
            hp[nt] = on ? a.h + (int64_t)(rt.first[ue] + __popc(tokens & ((1u << t) - 1u))) * a.I + ku * 128 + c * 32 : nullptr;
        }
        fetch();
        cp_async_wait<kDownDepth - 1>();
        const uint32_t st = ring + slot * RT * kTileBytes + lane * 16;
        if (++slot == kDownDepth) slot = 0;
        uint4 q[RT][2];
        Scale s[RT][2];
        bool wide = false;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            q[i][0] = lds128(st + i * kTileBytes);
            q[i][1] = lds128(st + i * kTileBytes + 512);
            const uint2 w = lds64(st + i * kTileBytes + 1024 - lane * 8);
            s[i][0] = make_scale<MX, FAST>(w.x, c);
            s[i][1] = make_scale<MX, FAST>(w.y, c);
            if constexpr (MX) wide |= (s[i][0].n | s[i][1].n) != 0;
        }
        if constexpr (MX) wide = __any_sync(0xffffffffu, wide);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 bh[NT], bl[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                bh[nt] = bl[nt] = make_uint4(0, 0, 0, 0);
                if (hp[nt]) {
                    bh[nt] = *reinterpret_cast<const uint4*>(hp[nt] + j * 8);
                    bl[nt] = *reinterpret_cast<const uint4*>(hp[nt] + lo_plane + j * 8);
                }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                uint32_t x0[4], x1[4];
                dequant8<MX, FAST>(word(q[i][0], j), s[i][0], wide, x0);
                dequant8<MX, FAST>(word(q[i][1], j), s[i][1], wide, x1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (NT > 1 && !(tokens >> (8 * nt) & 0xffu)) continue;
                    mma16816(acc[i][nt], x0[0], x1[0], x0[1], x1[1], bh[nt].x, bh[nt].y);
                    mma16816(acc[i][nt], x0[2], x1[2], x0[3], x1[3], bh[nt].z, bh[nt].w);
                    mma16816(acc[i][nt], x0[0], x1[0], x0[1], x1[1], bl[nt].x, bl[nt].y);
                    mma16816(acc[i][nt], x0[2], x1[2], x0[3], x1[3], bl[nt].z, bl[nt].w);
                }
            }
        }
    }
    cp_async_wait<0>();
}

__device__ __forceinline__ void few_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t cta) {
    uint32_t ra;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(cta));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(ra)
                 : "memory");
    return v;
}

// gridDim.x = row groups x cluster size; the CTAs of a cluster split the
// (expert, K unit) pairs of one row group and CTA 0 joins their sums in order.
template <bool MX, int NT, int RT>
__global__ void __launch_bounds__(kDownWarps<NT> * 32, 1) few_down_kernel(const FewArgs a, int cluster) {
    constexpr int kWarps = kDownWarps<NT>, kThreads = kWarps * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int flags;
    if (threadIdx.x == 0) flags = check_headers<MX>(a, true);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = cluster > 1 ? (int)(blockIdx.x % cluster) : 0;
    const int tile0 = (int)(blockIdx.x / cluster) * RT, tiles = a.H / 16;
    constexpr int kRing = kDownDepth * RT * kTileBytes;
    int32_t* s_ids;
    float* s_w;
    const Route rt = build_route<kWarps>(a, smem + kWarps * kRing, s_ids, s_w, false);
    if (!(flags & 1)) return;   // the same in every CTA; the gate_up kernel reported it
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT * NT * 4; ++i) acc[i / (NT * 4)][i / 4 % NT][i % 4] = 0.0f;
    const uint32_t ring = smem_u32(smem) + warp * kRing;
    if (MX || (flags & 4))
        down_loop<MX, NT, RT, true>(a, rt, ring, tile0, cta * kWarps + warp, cluster * kWarps, acc);
    else
        down_loop<MX, NT, RT, false>(a, rt, ring, tile0, cta * kWarps + warp, cluster * kWarps, acc);
    // join the warps' sums in warp order (the rings' space is free now)
    __syncthreads();
    float4* red = reinterpret_cast<float4*>(smem);
    constexpr int kPer = RT * NT * 32;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            red[warp * kPer + (i * NT + nt) * 32 + lane] =
                make_float4(acc[i][nt][0], acc[i][nt][1], acc[i][nt][2], acc[i][nt][3]);
    __syncthreads();
    if (cluster > 1) {
        for (int q = threadIdx.x; q < kPer; q += kThreads) {
            float4 s = red[q];
            for (int w = 1; w < kWarps; ++w) {
                const float4 v = red[w * kPer + q];
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            red[q] = s;   // only this thread reads slot q of any warp
        }
        few_cluster_sync();
    }
    if (cta == 0) {
        for (int q = threadIdx.x; q < kPer; q += kThreads) {
            float4 s = red[q];
            if (cluster > 1) {
                for (int r = 1; r < cluster; ++r) {
                    const float4 v = ld_cluster(smem_u32(red + q), r);
                    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                }
            } else {
                for (int w = 1; w < kWarps; ++w) {
                    const float4 v = red[w * kPer + q];
                    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                }
            }
            const int l = q & 31, nt = (q >> 5) % NT, tile = tile0 + (q >> 5) / NT;
            if (tile >= tiles) continue;
            const int row = tile * 16 + (l >> 2), t = 8 * nt + 2 * (l & 3);
            // + 0.0f: a sum of nothing, or of zeros of either sign, is +0
            if (t < a.T) {
                a.out[(int64_t)t * a.H + row] = __bfloat16_as_ushort(__float2bfloat16_rn(s.x + 0.0f));
                a.out[(int64_t)t * a.H + row + 8] = __bfloat16_as_ushort(__float2bfloat16_rn(s.z + 0.0f));
            }
            if (t + 1 < a.T) {
                a.out[(int64_t)(t + 1) * a.H + row] = __bfloat16_as_ushort(__float2bfloat16_rn(s.y + 0.0f));
                a.out[(int64_t)(t + 1) * a.H + row + 8] = __bfloat16_as_ushort(__float2bfloat16_rn(s.w + 0.0f));
            }
        }
    }
    if (cluster > 1) few_cluster_sync();   // CTA 0 has read the others' sums
}

template <bool MX, int NT>
cudaError_t launch_up(FewArgs a, cudaStream_t st) {
    auto kern = few_gate_up_kernel<MX, NT>;
    const int U = (a.H + 127) / 128;
    a.warps_item = U >= 8 ? 8 : (U >= 4 ? 4 : (U >= 2 ? 2 : 1));
    a.units_warp = (U + a.warps_item - 1) / a.warps_item;
    // two CTAs per SM; the activations of as many of an expert's tokens as then fit
    const size_t fixed = (size_t)kUpWarps * kUpDepth * 2 * kTileBytes + 2 * kUpWarps * 64 * sizeof(float4) +
                         route_bytes(a.E, a.T * a.topk, a.used_cap);
    const size_t tok = (size_t)kUpWarps * (a.units_warp * 256 + 64);
    const int cap = (int)((kSmemHalf - fixed) / tok);
    a.x_cap = cap < a.T ? cap : a.T;
    const size_t smem = fixed + tok * a.x_cap;
    int per_sm = 1;
    cudaError_t e = kernel_ctas_per_sm(reinterpret_cast<const void*>(kern), kUpThreads, smem, kSmemMax, &per_sm);
    if (e != cudaSuccess) return e;
    if (per_sm > 2) per_sm = 2;
    const int64_t items = (int64_t)a.used_cap * (a.I / 16), groups = kUpWarps / a.warps_item;
    const int64_t want = (items + groups - 1) / groups, cap_ctas = (int64_t)device_info().sm_count * per_sm;
    kern<<<(unsigned)(want < cap_ctas ? want : cap_ctas), kUpThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <bool MX, int NT, int RT>
cudaError_t launch_down(const FewArgs& a, int cluster, cudaStream_t st) {
    auto kern = few_down_kernel<MX, NT, RT>;
    constexpr int kWarps = kDownWarps<NT>;
    constexpr size_t ring = (size_t)kWarps * kDownDepth * RT * kTileBytes, sums = (size_t)kWarps * RT * NT * 512;
    const size_t smem = (ring > sums ? ring : sums) + route_bytes(a.E, a.T * a.topk, a.used_cap);
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.H / 16 + RT - 1) / RT * cluster));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, a, cluster);
}

template <bool MX, int NT>
cudaError_t launch_few_nt(const FewArgs& a, cudaStream_t st) {
    cudaError_t e = launch_up<MX, NT>(a, st);
    if (e != cudaSuccess) return e;
    // Row tiles per CTA: enough that one wave of CTAs covers H.  Few tiles: clusters
    // that split the (expert, K unit) pairs, while every warp still gets one.
    const int tiles = a.H / 16, sms = device_info().sm_count;
    const int rt = tiles > 2 * sms ? 3 : (tiles > sms ? 2 : 1);
    int cluster = 1;
    const int64_t pairs = (int64_t)a.used_cap * ((a.I + 127) / 128);
    while (cluster < 8 && rt == 1 && tiles * cluster * 2 <= sms && cluster * 2 * kDownWarps<NT> <= pairs) cluster *= 2;
    return rt == 3 ? launch_down<MX, NT, 3>(a, cluster, st)
                   : (rt == 2 ? launch_down<MX, NT, 2>(a, cluster, st) : launch_down<MX, NT, 1>(a, cluster, st));
}

cudaError_t launch_few(const FewArgs& a, bool mx, cudaStream_t st) {
    if (a.T <= 8) return mx ? launch_few_nt<true, 1>(a, st) : launch_few_nt<false, 1>(a, st);
    if (a.T <= 16) return mx ? launch_few_nt<true, 2>(a, st) : launch_few_nt<false, 2>(a, st);
    return mx ? launch_few_nt<true, 4>(a, st) : launch_few_nt<false, 4>(a, st);
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
    if (T > CHORD_FEW_MAX_TOKENS || topk > 32 || E > 1024 || (int64_t)H * I > (1LL << 31))
        return CHORD_ERR_UNSUPPORTED;   // an expert's bytes are addressed with 32 bits
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
    FewArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.ids = topk_ids;
    a.wts = topk_w;
    a.T = T;
    a.topk = topk;
    a.E = E;
    a.H = H;
    a.I = I;
    a.w13 = static_cast<const uint8_t*>(packed_w13);
    a.w2 = static_cast<const uint8_t*>(packed_w2);
    a.h = static_cast<uint16_t*>(workspace);
    a.out = static_cast<uint16_t*>(out);
    a.err = di.err;
    a.validate = opts && opts->validate ? 1 : 0;
    a.used_cap = T * topk < E ? T * topk : E;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_few(a, mx, st) != cudaSuccess) return CHORD_ERR_CUDA;
    if (!opts || !opts->validate) return CHORD_OK;
    int32_t code = 0;
    const chord_status s = chord_get_device_error(st, &code);
    if (s != CHORD_OK) return s;
    if (code == CHORD_DEV_TIMEOUT) return CHORD_ERR_TIMEOUT;
    return code ? CHORD_ERR_DEVICE_VALIDATION : CHORD_OK;
}

}  // extern "C"
