// Microscaled 4-bit product: both operands in CHORD_LAYOUT_MXFP4,
//   C[p, n] = sum_k a[row(p), k] * w[e, n, k]     (FP32 sums),
// dense (one weight matrix, row p of C is row p of a) or grouped by expert
// through the routing arrays of chord_moe_align.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "chord_internal.h"
#include "chord_mxfp4.cuh"
#include "chord_tcgen05.cuh"

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

// One work item is (row block, 128 rows of N).  The weight rows are the MMA's M
// side and the block's rows its N side, so a block of 11 rows costs an N = 16
// instruction.  Roles, each a warp that keeps its addresses warp-uniform and lets one
// elected lane issue (a lane on its own issued at half the rate):
//   * two producers copy K stages of 256 columns into shared-memory rings with
//     cp.async.bulk: one the weight tiles (17408 contiguous bytes, from HBM), one the codes
//     of the block's rows with their scales (from L2);
//   * a scale warp copies the stages' scales to tensor memory;
//   * an issuing warp issues the stages' four K = 64 instructions into one of two FP32
//     accumulators and commits the stages back to the producers.  It paces the
//     kernel, so it takes two stages a turn and learns what an item is from the
//     producer, beside the stage (one stage a turn: dense 4096 x 4096 x 7168 84 us with its
//     quantisation, two: 76);
//   * eight warps read the finished accumulator and write C while the next item
//     is computed into the other one.
// Every wait is bounded; the grid is persistent (static round robin).
// Blocks of 96 rows or more run in pairs of CTAs on neighbouring tiles of N, whose
// instructions are one of 256 weight rows: each CTA copies its own weights and half of the
// block's rows, which the tensor cores of both read, so a stage is 31 KB a CTA instead of
// 44 and the rings are half as deep again (of measured 208-row blocks, 48 experts: 4096 x 7168
// 152 us against 174 with single CTAs, 7168 x 2048 104 against 113; dense 4096 x 4096 x
// 7168 59 against 76).  The first CTA issues for both.  What the second one has copied reaches it
// through the copies themselves: they are counted on the first CTA's barrier, which only
// copies through a tensor map can (cta_group::2), so a stage is full there when both CTAs' bytes
// have landed.  (A barrier of the second CTA's own and an arrival on the first's would have to
// release at cluster scope: 229 us for 152, 141 for 104, 78 for 59.)  A block's rows go in boxes of 32 and
// then 8 rows (8 alone: 166, 107 and 80 us).  Small blocks leave the rows' share small (64 rows: 135 us single, 137 paired;
// 112 and 128 rows: equal).
// What bounds it: the weights' bytes (4096 x 7168 for 8192 rows: 749 MB, and 67 MB of C, in
// 152 us = 5.4 TB/s; reading these weights alone takes 130 us), and in the dense product,
// whose tiles come from L2, those copies again: 650 MB in 59 us, 51 us with no matrix
// instruction issued; the instructions alone take 40.
constexpr int kEpiWarps = 8;
constexpr int kWeightWarp = kEpiWarps, kRowWarp = kEpiWarps + 1, kScaleWarp = kEpiWarps + 2, kMmaWarp = kEpiWarps + 3;
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr uint32_t kStop = 0xffffffffu;   // stage info: no more items
constexpr int kMaxStages = 12;
constexpr int kDone = 16;                // barriers of finished stages, above any ring's depth
constexpr int kPairRows = 96;            // blocks from here on run in pairs of CTAs
constexpr int kTileLines = kMxTileBytes / 128;   // 128-byte rows of a tile
constexpr int kBoxRows = 32, kScaleRows = 8;   // a pair's copies of rows: half of a block is a multiple of 8, a tile's scales are 8
constexpr int kStgBytes = 2048;          // one epilogue warp's buffer: 16 rows x 32 columns x FP32
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCols = 24;      // tensor-memory columns of a stage's scales: 2 x (4 + 8)
constexpr int kTurns = 16;               // scale barriers, one per turn in flight (a turn is one or two stages)
constexpr long long kLandCycles = 4000000;   // about 2 ms
constexpr size_t kSmemBudget = 227 * 1024;
constexpr int kMxMaxBlockM = 208;        // two accumulators and four stages' scales fill the tensor memory

struct MxPlan {
    int tok;        // rows of a block (dense: a multiple of 64)
    int w_stages;   // ring of weight tiles
    int r_stages;   // ring of rows
    int r_bytes;    // one stage of rows: codes (a pair's CTA: of half of them), then 1 KB of scales per 128 rows
    int slots;      // stages whose scales tensor memory holds
};

// Pairs of CTAs: both matrices as rows of 128 bytes (136 a tile: its code rows, then 8 of scales).
struct MxMaps {
    CUtensorMap w;      // boxes of a tile
    CUtensorMap a, a8;  // boxes of 32 and of 8 rows
};

struct Item {
    int64_t b;      // row block
    int nt;         // 128-row tile of N
    int e;          // expert
    int rows;       // rows of the block that hold pairs (a prefix), rounded up to 16; 0: nothing to do
    int off;        // first row inside its 128-row tile (dense blocks of 64 or 192: 0 or 64)
    bool write;     // false: a pair's repeat of an odd last tile
};

// The routing of one item's block as loaded: issued an item ahead, so that no role
// waits for it between two items.
struct Routing {
    int32_t e, ids[7];   // lane l: rows l, l + 32, ... of the block
};

struct Walk {
    int64_t n_items, step;
    int nper, ntiles;
    uint32_t rank;
};

__device__ __forceinline__ Routing load_routing(const MxGemmArgs& g, const MxPlan& pl, const Walk& w, int64_t i, int lane) {
    Routing r{};
    if (!g.sorted_ids || i >= w.n_items) return r;
    int q;
    const int64_t b = divmod_idx(i, w.nper, q);
    r.e = g.expert_ids[b];
#pragma unroll
    for (int k = 0; k < 7; ++k) {
        const int row = lane + 32 * k;
        r.ids[k] = row < pl.tok ? g.sorted_ids[b * pl.tok + row] : (int32_t)g.num_pairs;
    }
    return r;
}

// Facts of item i, computed identically by every warp from the same arrays.
template <bool PAIR>
__device__ __forceinline__ Item item_at(const MxGemmArgs& g, const MxPlan& pl, const Walk& w, int64_t i, const Routing& rt,
                                        int lane, bool report) {
    Item it;
    it.b = divmod_idx(i, w.nper, it.nt);
    it.write = true;
    if (PAIR) {
        it.nt = 2 * it.nt + (int)w.rank;
        it.write = it.nt < w.ntiles;
        if (!it.write) --it.nt;
    }
    it.e = 0;
    it.off = 0;
    if (!g.sorted_ids) {
        const int64_t r0 = it.b * pl.tok;
        const int64_t n = min((int64_t)pl.tok, g.a_rows - r0);
        it.rows = (int)((n + 15) / 16 * 16);
        it.off = (int)(r0 % kMxTileRows);
        return it;
    }
    it.e = rt.e;
    it.rows = 0;
    if (it.e < 0 || it.e >= g.E) {
        if (report && lane == 0) set_error(g.err, CHORD_DEV_BAD_EXPERT);
        return it;
    }
    int last = 0;
#pragma unroll
    for (int k = 0; k < 7; ++k) {
        const bool ok = rt.ids[k] >= 0 && rt.ids[k] < g.num_pairs;
        if (report && !ok && rt.ids[k] != g.num_pairs) set_error(g.err, CHORD_DEV_BAD_ROW);
        if (ok) last = lane + 32 * k + 1;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    it.rows = (last + 15) / 16 * 16;
    return it;
}

// Accumulator columns of one epilogue warp (its 32 lanes are rows of N; warp group wg
// takes every other slice of 32 block rows) to C, through the warp's buffer so that C is
// written in 16-byte pieces: 32 (bf16) or twice 16 (FP32) block rows of 32 columns.  Lane l
// of rt.ids[k] holds the pair of block row 32 k + l, so nothing is loaded here.
template <bool F32>
__device__ __forceinline__ void drain(const MxGemmArgs& g, const MxPlan& pl, const Item& it, const Routing& rt, uint32_t acc,
                                      int wg, int quarter, int lane, uint8_t* stg) {
    constexpr int kEsz = F32 ? 4 : 2, kPer = 16 / kEsz, kPieces = 32 / kPer;   // pieces of a block row's 32 columns
    constexpr int kHalf = F32 ? 16 : 32;                                       // block rows per pass
    const int n0 = it.nt * kMxTileRows + quarter * 32;
    if (n0 >= g.N) return;
    const bool wide = (int64_t)g.N * kEsz % 16 == 0;
    const uint32_t sbase = smem_u32(stg);
#pragma unroll
    for (int k = 0; k < 7; ++k) {
        if ((k & 1) != wg || 32 * k >= it.rows) continue;
        int32_t mine;   // C row of block row 32 k + lane, -1: none
        if (g.sorted_ids) {
            mine = rt.ids[k] >= 0 && rt.ids[k] < g.num_pairs ? rt.ids[k] : -1;
        } else {
            const int64_t r = it.b * pl.tok + 32 * k + lane;
            mine = 32 * k + lane < pl.tok && r < g.a_rows ? (int32_t)r : -1;
        }
        uint32_t v[2][16];
        const uint32_t at = acc + ((uint32_t)(quarter * 32) << 16) + 32 * k;
        tc5::ld16(at, v[0]);
        if (32 * k + 16 < it.rows) tc5::ld16(at + 16, v[1]);
        tc5::wait_ld();
        if (!wide) {
#pragma unroll
            for (int u = 0; u < 32; ++u) {
                const int32_t p = __shfl_sync(0xffffffffu, mine, u);
                if (p < 0 || 32 * k + u >= it.rows || n0 + lane >= g.N) continue;
                const int64_t o = (int64_t)p * g.N + n0 + lane;
                if (F32)
                    static_cast<float*>(g.C)[o] = __uint_as_float(v[u >> 4][u & 15]);
                else
                    static_cast<__nv_bfloat16*>(g.C)[o] = __float2bfloat16_rn(__uint_as_float(v[u >> 4][u & 15]));
            }
            continue;
        }
#pragma unroll
        for (int h = 0; h < 32 / kHalf; ++h) {
            if (32 * k + h * kHalf >= it.rows) continue;
#pragma unroll
            for (int u = 0; u < kHalf; ++u) {
                const uint32_t x = v[(h * kHalf + u) >> 4][u & 15];
                const uint32_t to = sbase + (uint32_t)((u * 32 + lane) * kEsz);
                if (F32)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(x) : "memory");
                else
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(to),
                                 "h"(__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(x))))
                                 : "memory");
            }
            __syncwarp();
            uint4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[q].x), "=r"(w[q].y), "=r"(w[q].z), "=r"(w[q].w)
                             : "r"(sbase + (uint32_t)((q * 32 + lane) * 16))
                             : "memory");
            const int c = n0 + (lane % kPieces) * kPer;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int u = h * kHalf + (q * 32 + lane) / kPieces;
                const int32_t p = __shfl_sync(0xffffffffu, mine, u);
                // N is a multiple of kPer here, so a piece lies wholly inside or outside
                if (p >= 0 && 32 * k + u < it.rows && c < g.N)
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.C) + ((int64_t)p * g.N + c) * kEsz) = w[q];
            }
            __syncwarp();
        }
    }
}

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(const MxGemmArgs g, const MxPlan pl, const __grid_constant__ MxMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* ring_r = smem + pl.w_stages * kMxTileBytes;
    uint8_t* stg = ring_r + pl.r_stages * pl.r_bytes;
    uint64_t* full_w = reinterpret_cast<uint64_t*>(stg + kEpiWarps * kStgBytes);
    uint64_t* full_r = full_w + kMaxStages;
    uint64_t* done = full_r + kMaxStages;      // stage g's instructions: barrier g mod kDone
    uint64_t* turn_full = done + kDone;
    uint64_t* acc_full = turn_full + kTurns;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);   // [0] row blocks, [1] abort, [2] skip
    // what each stage's item is, written by the producer before the stage is full:
    // rows | offset << 16, or kStop
    volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(tmem_slot + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? tc5::cluster_rank() : 0u;
    if (warp == kMmaWarp) tc5::alloc<PAIR>(tmem_slot, kTmemCols);
    pdl_wait();   // before the first access to global memory
    if (warp == 0) {
        const bool oka = mx_header_ok_warp(g.a, g.a_groups, g.a_rows, g.K), okw = mx_header_ok_warp(g.w, g.E, g.N, g.K);
        if (lane == 0) {
            bool ok = oka && okw;
            if (!ok) set_error(g.err, CHORD_DEV_BAD_HEADER);
            int64_t blocks = (g.a_rows + pl.tok - 1) / pl.tok;
            if (g.sorted_ids) {
                const int64_t ntp = *g.ntp;
                if (ntp < 0 || ntp > g.a_groups * g.a_rows || ntp % pl.tok) {
                    if (ok) set_error(g.err, CHORD_DEV_BAD_PADDED);
                    ok = false;
                }
                blocks = ok ? ntp / pl.tok : 0;
            }
            flags[0] = (int)blocks;
            flags[1] = 0;
            flags[2] = ok ? 0 : 1;
            for (int s = 0; s < kMaxStages; ++s) {
                mbar_init(&full_w[s], 1);
                mbar_init(&full_r[s], 1);
            }
            for (int s = 0; s < kDone; ++s) mbar_init(&done[s], 1);
            for (int s = 0; s < kTurns; ++s) mbar_init(&turn_full[s], 1);
            for (int s = 0; s < 2; ++s) {
                mbar_init(&acc_full[s], 1);
                mbar_init(&acc_empty[s], PAIR ? 2 * kEpiWarps : kEpiWarps);
            }
            fence_barrier_init();
        }
    }
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    // a pair's barriers are initialised before the other CTA's arrivals and commits reach them
    if (PAIR) tc5::cluster_sync();
    const uint32_t tmem = *tmem_slot;
    const int ntiles = (g.N + kMxTileRows - 1) / kMxTileRows;
    const int kstages = (g.K + kMxTileCols - 1) / kMxTileCols;
    // a pair's item is (row block, two tiles of N); an odd last tile leaves the second CTA a
    // repeat of the first's that it does not write
    const int nper = PAIR ? (ntiles + 1) / 2 : ntiles;
    const int64_t n_items = flags[2] ? 0 : (int64_t)flags[0] * nper;
    const int64_t first = PAIR ? blockIdx.x >> 1 : blockIdx.x;
    const Walk wk{n_items, PAIR ? gridDim.x >> 1 : gridDim.x, nper, ntiles, rank};
    Routing nxt = load_routing(g, pl, wk, first, lane);
    const int64_t art = mx_row_tiles(g.a_rows);

    // Position in a ring: stage number, slot, its address and the parity of its current
    // fill; barriers as shared-memory addresses.
    struct Pos {
        uint32_t g, slot, st, parity;
    };
    const uint32_t base_w = smem_u32(smem), base_r = smem_u32(ring_r), r_codes = (uint32_t)pl.tok * (PAIR ? 64u : 128u);
    const uint32_t full_w_a = smem_u32(full_w), full_r_a = smem_u32(full_r), done_a = smem_u32(done), turn_a = smem_u32(turn_full);
    const uint32_t slots = (uint32_t)pl.slots;
    const uint32_t w_stages = (uint32_t)pl.w_stages, r_stages = (uint32_t)pl.r_stages, r_bytes = (uint32_t)pl.r_bytes;
    auto next_w = [&](const Pos& p) {
        return p.slot + 1 == w_stages ? Pos{p.g + 1, 0, base_w, p.parity ^ 1u}
                                      : Pos{p.g + 1, p.slot + 1, p.st + kMxTileBytes, p.parity};
    };
    auto next_r = [&](const Pos& p) {
        return p.slot + 1 == r_stages ? Pos{p.g + 1, 0, base_r, p.parity ^ 1u}
                                      : Pos{p.g + 1, p.slot + 1, p.st + r_bytes, p.parity};
    };
    auto wait_full = [&](uint32_t bars, const Pos& p) {
        return tc5::wait<false, PAIR>(bars + p.slot * 8, p.parity, &flags[1], g.err);
    };
    // the instructions of a stage are done
    auto wait_done = [&](uint32_t stage) {
        return tc5::wait<false, PAIR>(done_a + (stage % kDone) * 8, (stage / kDone) & 1u, &flags[1], g.err);
    };
    // the slot of stage p.g is free: the instructions of the stage a ring before are done
    auto wait_free = [&](const Pos& p, uint32_t depth) { return p.g < depth || wait_done(p.g - depth); };
    // a stage's copies are counted on one barrier: a pair's, both CTAs' bytes, on the first CTA's
    auto counted_on = [&](uint32_t bar) { return PAIR ? tc5::at_cta(bar, 0) : bar; };
    bool ok = true;

    if (warp == kWeightWarp) {
        Pos p{0, 0, base_w, 0};
        for (int64_t i = first; i < n_items && ok; i += wk.step) {
            const Item it = item_at<PAIR>(g, pl, wk, i, nxt, lane, false);
            nxt = load_routing(g, pl, wk, i + wk.step, lane);
            if (it.rows == 0) continue;
            const int64_t tile = ((int64_t)it.e * ntiles + it.nt) * kstages;
            const uint8_t* src = g.w + kHeaderBytes + tile * kMxTileBytes;
            for (int ks = 0; ks < kstages; ++ks, src += kMxTileBytes) {
                ok = wait_free(p, w_stages);
                if (!ok) break;
                if (tc5::elect()) {
                    const uint32_t bar = full_w_a + p.slot * 8;
                    if (!rank) tc5::arrive_expect_tx(bar, PAIR ? 2u * kMxTileBytes : kMxTileBytes);
                    if constexpr (PAIR)
                        tc5::box_g2s_pair(p.st, &maps.w, (int)(tile + ks) * kTileLines, counted_on(bar));
                    else
                        tc5::bulk_g2s(p.st, src, kMxTileBytes, bar);
                }
                __syncwarp();
                p = next_w(p);
            }
        }
        // leave only after every copy issued here has landed
        if (PAIR && p.g > 0) wait_done(p.g - 1);
        for (uint32_t k = 0; k < w_stages && p.g > 0 && !PAIR; ++k) {
            p = p.slot == 0 ? Pos{p.g - 1, w_stages - 1, 0, p.parity ^ 1u} : Pos{p.g - 1, p.slot - 1, 0, p.parity};
            if (!wait_full(full_w_a, p)) break;
        }
    } else if (warp == kRowWarp) {
        Pos p{0, 0, base_r, 0};
        for (int64_t i = first; i < n_items && ok; i += wk.step) {
            const Item it = item_at<PAIR>(g, pl, wk, i, nxt, lane, false);
            nxt = load_routing(g, pl, wk, i + wk.step, lane);
            if (it.rows == 0) continue;
            // tiles of the block's rows: its own (grouped), or those of the matrix it starts in (dense)
            const int64_t t0 = g.sorted_ids ? it.b * art : it.b * pl.tok / kMxTileRows;
            const int64_t tstride = (int64_t)kstages * kMxTileBytes;
            const uint8_t* src = g.a + kHeaderBytes + t0 * tstride;
            const int rows = it.rows, r0 = min(rows, kMxTileRows - it.off);   // r0 of them in the first tile
            // a pair's CTA copies rows [h0, h1), and the scales of all
            const int h0 = PAIR ? (int)rank * (rows / 2) : 0, h1 = PAIR ? h0 + rows / 2 : rows;
            const int a0 = min(h0, r0), a1 = min(h1, r0), b0 = max(h0, r0), b1 = max(h1, r0);   // in the first, second tile
            const uint32_t scales = rows > r0 ? 2048u : 1024u;
            const uint32_t bytes = (uint32_t)rows * 128u + (PAIR ? 2u * scales : scales);
            const uint32_t inf = (uint32_t)rows | (uint32_t)it.off << 16;
            for (int ks = 0; ks < kstages; ++ks, src += kMxTileBytes) {
                ok = wait_free(p, r_stages);
                if (!ok) break;
                if (tc5::elect()) {
                    const uint32_t bar = full_r_a + p.slot * 8, ss = p.st + r_codes;
                    if (!rank) {
                        info[p.slot] = inf;
                        tc5::arrive_expect_tx(bar, bytes);
                    }
                    if constexpr (PAIR) {
                        const uint32_t to = counted_on(bar);
                        const int line = (int)(t0 * kstages + ks) * kTileLines, line2 = line + kstages * kTileLines;
                        uint32_t st = p.st;
                        auto copy = [&](int at, int n) {
                            for (; n >= kBoxRows; n -= kBoxRows, at += kBoxRows, st += kBoxRows * 128)
                                tc5::box_g2s_pair(st, &maps.a, at, to);
                            for (; n > 0; n -= kScaleRows, at += kScaleRows, st += kScaleRows * 128)
                                tc5::box_g2s_pair(st, &maps.a8, at, to);
                        };
                        copy(line + it.off + a0, a1 - a0);
                        copy(line2 + b0 - r0, b1 - b0);
                        tc5::box_g2s_pair(ss, &maps.a8, line + kMxTileRows, to);
                        if (rows > r0) tc5::box_g2s_pair(ss + 1024, &maps.a8, line2 + kMxTileRows, to);
                    } else {
                        tc5::bulk_g2s(p.st, src + it.off * 128, (uint32_t)a1 * 128u, bar);
                        if (b1 > b0) tc5::bulk_g2s(p.st + a1 * 128, src + tstride, (uint32_t)(b1 - b0) * 128u, bar);
                        tc5::bulk_g2s(ss, src + kMxCodeBytes, 1024u, bar);
                        if (rows > r0) tc5::bulk_g2s(ss + 1024, src + tstride + kMxCodeBytes, 1024u, bar);
                    }
                }
                __syncwarp();
                p = next_r(p);
            }
        }
        if (!rank && ok && wait_free(p, r_stages)) {
            if (tc5::elect()) {
                info[p.slot] = kStop;
                tc5::arrive(full_r_a + p.slot * 8);
            }
            __syncwarp();
            p = next_r(p);
        }
        if (PAIR && rank && p.g > 0) wait_done(p.g - 1);
        for (uint32_t k = 0; k < r_stages && p.g > 0 && !rank; ++k) {
            p = p.slot == 0 ? Pos{p.g - 1, r_stages - 1, 0, p.parity ^ 1u} : Pos{p.g - 1, p.slot - 1, 0, p.parity};
            if (!wait_full(full_r_a, p)) break;
        }
    } else if (rank && (warp == kScaleWarp || warp == kMmaWarp)) {
        // the first CTA of the pair issues
    } else if (warp == kScaleWarp) {
        // Scales of a stage's two 128-column halves to the columns of its rows' slot: 4 columns
        // per 128 rows (and four groups), weights first.  They are free when the slot is.
        const uint32_t sf_base = tmem + 2u * (uint32_t)pl.tok;
        Pos w{0, 0, base_w, 0}, r{0, 0, base_r, 0};
        uint32_t turn = 0;
        while (ok) {
            ok = wait_full(full_r_a, r);
            if (!ok) break;
            const uint32_t inf = __shfl_sync(0xffffffffu, info[r.slot], 0);
            if (inf == kStop) break;
            const bool two = (inf >> 16) + (inf & 0xffffu) > (uint32_t)kMxTileRows;
            for (int ks = 0; ks < kstages; ks += 2, ++turn) {
                const Pos w2 = next_w(w), r2 = next_r(r);
                const bool second = ks + 1 < kstages;
                ok = wait_full(full_r_a, r) && wait_full(full_w_a, w) &&
                     (!second || (wait_full(full_r_a, r2) && wait_full(full_w_a, w2)));
                if (!ok) break;
                ok = wait_free(second ? r2 : r, slots);
                if (!ok) break;
                if (tc5::elect()) {
                    auto copy = [&](const Pos& wp, const Pos& rp) {
                        const uint32_t sf = sf_base + rp.g % slots * kScaleCols;
                        const uint64_t dsa = tc5::desc_scales(wp.st + kMxCodeBytes), dsb = tc5::desc_scales(rp.st + r_codes);
#pragma unroll
                        for (uint32_t h = 0; h < 2; ++h) {
                            tc5::cp_scales<PAIR>(sf + 4u * h, dsa + h * (kMxScaleBlock >> 4));
                            tc5::cp_scales<PAIR>(sf + 8u + 8u * h, dsb + h * (kMxScaleBlock >> 4));
                            if (two) tc5::cp_scales<PAIR>(sf + 12u + 8u * h, dsb + (1024u >> 4) + h * (kMxScaleBlock >> 4));
                        }
                    };
                    copy(w, r);
                    if (second) copy(w2, r2);
                    tc5::commit<PAIR, false>(turn_a + (turn % kTurns) * 8);
                }
                __syncwarp();
                w = second ? next_w(w2) : w2;
                r = second ? next_r(r2) : r2;
            }
        }
        // the last instructions are done: before tensor memory is released
        if (w.g > 0) wait_done(w.g - 1);
        __syncwarp();
    } else if (warp == kMmaWarp) {
        const uint32_t sf_base = tmem + 2u * (uint32_t)pl.tok;
        Pos w{0, 0, base_w, 0}, r{0, 0, base_r, 0};
        uint32_t nitem = 0, turn = 0;
        while (ok) {
            ok = wait_full(full_r_a, r);
            if (!ok) break;
            const uint32_t inf = __shfl_sync(0xffffffffu, info[r.slot], 0);
            if (inf == kStop) break;
            const uint32_t rows = inf & 0xffffu, off = inf >> 21, buf = nitem & 1u;   // off: in 32 rows
            ok = tc5::wait<false, PAIR>(smem_u32(&acc_empty[buf]), ((nitem >> 1) & 1u) ^ 1u, &flags[1], g.err);
            if (!ok) break;
            const uint32_t acc = tmem + buf * (uint32_t)pl.tok;
            const uint32_t id0 = tc5::idesc_mxf4<PAIR>((int)rows, 0), id2 = tc5::idesc_mxf4<PAIR>((int)rows, 2);
            for (int ks = 0; ks < kstages; ks += 2, ++turn) {
                const Pos w2 = next_w(w), r2 = next_r(r);
                const bool second = ks + 1 < kstages;
                // the scale warp has waited for both stages' copies before it committed this turn
                ok = tc5::wait(turn_a + (turn % kTurns) * 8, (turn / kTurns) & 1u, &flags[1], g.err);
                if (!ok) break;
                tc5::fence_after();
                if (tc5::elect()) {
                    auto mma = [&](const Pos& wp, const Pos& rp, int k) {
                        const uint32_t sf = sf_base + rp.g % slots * kScaleCols;
                        const uint64_t da = tc5::desc_sw128(wp.st), db = tc5::desc_sw128(rp.st);
                        const int nk = min(4, (g.K - k * kMxTileCols + 63) / 64);
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk)
                            if ((int)kk < nk)
                                tc5::mma_mxf4<PAIR>(acc, da + 2u * kk, db + 2u * kk, kk & 1 ? id2 : id0, sf + 4u * (kk >> 1),
                                              sf + 8u + 8u * (kk >> 1) + off, k > 0 || kk > 0 ? 1u : 0u);
                        tc5::commit<PAIR, true>(done_a + (wp.g % kDone) * 8);
                    };
                    mma(w, r, ks);
                    if (second) mma(w2, r2, ks + 1);
                    if (ks + 2 >= kstages) tc5::commit<PAIR, true>(smem_u32(&acc_full[buf]));
                }
                __syncwarp();
                w = second ? next_w(w2) : w2;
                r = second ? next_r(r2) : r2;
            }
            ++nitem;
        }
    } else {
        const int wg = warp >> 2, quarter = warp & 3;
        int64_t nitem = 0;
        for (int64_t i = first; i < n_items; i += wk.step) {
            const Routing cur = nxt;
            const Item it = item_at<PAIR>(g, pl, wk, i, cur, lane, warp == 0);
            nxt = load_routing(g, pl, wk, i + wk.step, lane);
            if (it.rows == 0) continue;
            const int buf = (int)(nitem & 1);
            if (!tc5::wait<true, PAIR>(&acc_full[buf], (uint32_t)((nitem >> 1) & 1), &flags[1], g.err)) break;
            tc5::fence_after();
            if (it.write) {
                const uint32_t acc = tmem + (uint32_t)(buf * pl.tok);
                if (g.out_f32)
                    drain<true>(g, pl, it, cur, acc, wg, quarter, lane, stg + warp * kStgBytes);
                else
                    drain<false>(g, pl, it, cur, acc, wg, quarter, lane, stg + warp * kStgBytes);
            }
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR)
                    tc5::arrive_relaxed_at(smem_u32(&acc_empty[buf]), 0);
                else
                    mbar_arrive(&acc_empty[buf]);
            }
            ++nitem;
        }
    }
    tc5::fence_before();
    __syncthreads();
    // A role that gave up has made the others' last waits return at once: what is still in flight
    // (copies into this CTA's shared memory, instructions on its tensor memory) gets its time here,
    // some hundred times what it takes, before either is handed to the next CTA.
    if (flags[1])
        for (const long long t0 = clock64(); clock64() - t0 < kLandCycles;) __nanosleep(1000);
    if (PAIR) tc5::cluster_sync();   // the pair's instructions, and arrivals on the other CTA's barriers, are done
    tc5::fence_after();
    if (warp == kMmaWarp) tc5::dealloc<PAIR>(tmem, kTmemCols);
}

// The tiles of a packed matrix as rows of 128 bytes, copied `box` at a time.
bool tile_map(CUtensorMap* map, const uint8_t* packed, int64_t tiles, int box) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess;
        return reinterpret_cast<Encode>(ok && r == cudaDriverEntryPointSuccess ? f : nullptr);
    }();
    const cuuint64_t dims[2] = {128, (cuuint64_t)(tiles * kTileLines)}, strides[1] = {128};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, ones[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(packed) + kHeaderBytes, dims, strides,
                            boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_mx_gemm(const MxGemmArgs& g, cudaStream_t st) {
    MxPlan pl;
    // Dense blocks: 192 rows (two accumulators and the scales fill the tensor
    // memory), fewer when the matrix is shorter.
    pl.tok = g.sorted_ids ? (int)g.a_rows : (g.a_rows > 128 ? 192 : (g.a_rows > 64 ? 128 : 64));
    // 128-row tiles a block may touch (dense blocks of 192 start at row 0 or 64 of one)
    const int tiles = (pl.tok + kMxTileRows - 1) / kMxTileRows;
    const int64_t ntiles = (g.N + kMxTileRows - 1) / kMxTileRows;
    // tiles of either matrix; their 128-byte rows are a pair's 32-bit tensor-map coordinates
    const int64_t w_tiles = (int64_t)g.E * ntiles * mx_col_tiles(g.K), a_tiles = g.a_groups * mx_row_tiles(g.a_rows) * mx_col_tiles(g.K);
    const bool pair = pl.tok >= kPairRows && ntiles > 1 && (w_tiles > a_tiles ? w_tiles : a_tiles) <= INT32_MAX / kTileLines;
    pl.r_bytes = pl.tok * (pair ? 64 : 128) + 1024 * tiles;
    const size_t fixed = 1024 + kEpiWarps * kStgBytes + (2 * kMaxStages + kDone + kTurns + 4) * 8 + 64 + 4 * kMaxStages;
    const size_t room = kSmemBudget - fixed;
    pl.slots = (int)((kTmemCols - 2 * pl.tok) / kScaleCols);
    if (pl.slots > kMaxStages) pl.slots = kMaxStages;
    pl.r_stages = (int)(room / (kMxTileBytes + pl.r_bytes));
    if (pl.r_stages > kMaxStages) pl.r_stages = kMaxStages;
    pl.w_stages = (int)((room - (size_t)pl.r_stages * pl.r_bytes) / kMxTileBytes);
    if (pl.w_stages > kMaxStages) pl.w_stages = kMaxStages;
    if (pl.r_stages < 2 || pl.w_stages < 2 || pl.slots < 2) return cudaErrorInvalidConfiguration;
    // one CTA per SM: it takes the whole tensor memory, and more than half of the shared memory
    const size_t smem = fixed + (size_t)pl.w_stages * kMxTileBytes + (size_t)pl.r_stages * pl.r_bytes;
    MxMaps maps{};
    if (pair && !(tile_map(&maps.w, g.w, w_tiles, kTileLines) && tile_map(&maps.a, g.a, a_tiles, kBoxRows) &&
                  tile_map(&maps.a8, g.a, a_tiles, kScaleRows)))
        return cudaErrorInvalidValue;
    void (*kern)(MxGemmArgs, MxPlan, MxMaps) = pair ? mx_gemm_kernel<true> : mx_gemm_kernel<false>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kSmemBudget);
    if (e != cudaSuccess) return e;
    const int64_t blocks = g.sorted_ids ? g.a_groups : (g.a_rows + pl.tok - 1) / pl.tok;
    const int64_t sms = device_info().sm_count;
    const int64_t items = pair ? blocks * ((ntiles + 1) / 2) : blocks * ntiles, ctas = pair ? sms / 2 : sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items < ctas ? items : ctas) * (pair ? 2 : 1)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pair) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
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
    return cudaLaunchKernelEx(&cfg, kern, g, pl, maps);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
    const double tok_e = (double)(T > 0 ? T : 0) * (double)(topk > 0 ? topk : 1) / (double)eg;
    // rows that an expert rarely exceeds (mean + 3 sd of a Poisson count), in
    // as few equal blocks as the kernel's largest allows
    const double need = tok_e + 3.0 * sqrt(tok_e) + 1.0;
    // a second block streams the expert's weights again: the few experts above mean + 2 sd may take one
    const double blocks = ceil((tok_e + 2.0 * sqrt(tok_e) + 1.0) / kMxMaxBlockM);
    const int bm = (int)ceil(need / blocks / 16.0) * 16;
    return bm > kMxMaxBlockM ? kMxMaxBlockM : bm;
}

chord_status chord_mxfp4_moe_gemm(const void* Aq, size_t aq_bytes, const void* packed, size_t packed_bytes, int E,
                                  int N, int K, const int32_t* sorted_ids, const int32_t* expert_ids,
                                  const int32_t* num_tokens_padded, int64_t capacity, int block_m, int64_t num_pairs,
                                  void* C, int c_dtype, const chord_opts* opts, void* stream) {
    if (E <= 0 || N <= 0 || K <= 0 || block_m <= 0 || capacity < 0 || num_pairs < 0) return CHORD_ERR_INVALID_ARG;
    if (K % kGroup || block_m % 16 || block_m > kMxMaxBlockM || num_pairs >= INT32_MAX || capacity >= INT32_MAX)
        return CHORD_ERR_UNSUPPORTED;
    if (capacity % block_m || (c_dtype != CHORD_DTYPE_BF16 && c_dtype != CHORD_DTYPE_F32)) return CHORD_ERR_INVALID_ARG;
    const size_t need_w = chord_mxfp4_bytes(E, N, K), need_a = chord_mxfp4_rows_bytes(capacity, block_m, K);
    if (need_w == 0 || packed_bytes != need_w || need_a == 0 || aq_bytes != need_a) return CHORD_ERR_LAYOUT_MISMATCH;
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
