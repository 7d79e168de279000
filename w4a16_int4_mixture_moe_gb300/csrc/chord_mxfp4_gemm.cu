// Microscaled 4-bit product: both operands in CHORD_LAYOUT_MXFP4,
//   C[p, n] = sum_k a[row(p), k] * w[e, n, k]     (FP32 sums),
// dense (one weight matrix, row p of C is row p of a) or grouped by expert
// through the routing arrays of chord_moe_align.
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
// instruction.  Roles:
//   * a producer lane copies K stages of 256 columns into a shared-memory ring
//     with cp.async.bulk: the weight tile (17408 contiguous bytes) and the codes
//     of the block's rows with their scales;
//   * an issuing warp copies the stage's scales to tensor memory, issues its four
//     K = 64 instructions into one of two FP32 accumulators and commits the stage
//     back to the producer.  This warp paces the kernel (a stage's instructions
//     take 400 to 500 cycles, and its loop took as long again), so it takes two stages a
//     turn and learns what an item is from the producer, beside the stage;
//   * eight warps read the finished accumulator and write C while the next item
//     is computed into the other one.
// Every wait is bounded; the grid is persistent (static round robin).
// Blocks of many rows run in clusters of two CTAs on neighbouring tiles of N: each
// copies its own weights and half of the block's rows, the rows going to both CTAs
// (multicast), since at fp4 rates the rows re-read from L2 for every 128 rows of N
// are what an SM waits for.  A stage is then free once both CTAs have used it.
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr uint32_t kStop = 0xffffffffu;   // stage info: no more items
constexpr int kMaxStages = 12;
constexpr int kPairRows = 96;            // blocks from here on run in pairs of CTAs
constexpr int kStgBytes = 2048;          // one epilogue warp's buffer: 16 rows x 32 columns x FP32
constexpr uint32_t kTmemCols = 512;
constexpr size_t kSmemBudget = 227 * 1024;

struct MxPlan {
    int tok;        // rows of a block (dense: a multiple of 64)
    int stages;     // shared-memory ring
    int sf_slots;   // tensor-memory scale ring
    int stage_bytes;
    int pair;       // clusters of two CTAs
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
__device__ __forceinline__ Item item_at(const MxGemmArgs& g, const MxPlan& pl, const Walk& w, int64_t i, const Routing& rt,
                                        int lane, bool report) {
    Item it;
    it.b = divmod_idx(i, w.nper, it.nt);
    it.write = true;
    if (pl.pair) {
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

// Accumulator columns of one epilogue warp (its 32 lanes are rows of N; warp
// group wg takes every other slice of 16 block rows) to C, 16 x 32 values at a time through
// the warp's buffer so that C is written in 16-byte pieces.
__device__ __forceinline__ void drain(const MxGemmArgs& g, const MxPlan& pl, const Item& it, uint32_t acc, int wg,
                                      int quarter, int lane, uint8_t* stg) {
    const int esz = g.out_f32 ? 4 : 2;
    const int n0 = it.nt * kMxTileRows + quarter * 32;
    const bool wide = (int64_t)g.N * esz % 16 == 0;
    const int per = 16 / esz, pieces = 32 / per;
    const uint32_t sbase = smem_u32(stg);
    for (int j0 = wg * 16; j0 < it.rows; j0 += 32) {
        int32_t mine = -1;   // C row of block row j0 + lane
        if (lane < 16) {
            const int64_t r = it.b * pl.tok + j0 + lane;
            if (!g.sorted_ids) {
                if (r < g.a_rows) mine = (int32_t)r;
            } else if (j0 + lane < pl.tok) {
                const int32_t id = g.sorted_ids[r];
                if (id >= 0 && id < g.num_pairs) mine = id;
            }
        }
        uint32_t v[16];
        tc5::ld16(acc + ((uint32_t)(quarter * 32) << 16) + j0, v);
        tc5::wait_ld();
        if (n0 >= g.N) continue;
        if (!wide) {
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int32_t p = __shfl_sync(0xffffffffu, mine, u);
                if (p < 0 || n0 + lane >= g.N) continue;
                const int64_t o = (int64_t)p * g.N + n0 + lane;
                if (g.out_f32)
                    static_cast<float*>(g.C)[o] = __uint_as_float(v[u]);
                else
                    static_cast<__nv_bfloat16*>(g.C)[o] = __float2bfloat16_rn(__uint_as_float(v[u]));
            }
            continue;
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            const uint32_t at = sbase + (uint32_t)((u * 32 + lane) * esz);
            if (g.out_f32)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v[u]) : "memory");
            else
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(at),
                             "h"(__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[u]))))
                             : "memory");
        }
        __syncwarp();
        for (int q = lane; q < 16 * pieces; q += 32) {
            const int u = q / pieces, c = n0 + (q % pieces) * per;
            const int32_t p = __shfl_sync(0xffffffffu, mine, u);
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(sbase + (uint32_t)(q * 16))
                         : "memory");
            // N is a multiple of `per` here, so a piece lies wholly inside or outside
            if (p >= 0 && c < g.N)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.C) + ((int64_t)p * g.N + c) * esz) = w;
        }
        __syncwarp();
    }
}

__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(const MxGemmArgs g, const MxPlan pl) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* stg = smem + pl.stages * pl.stage_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(stg + kEpiWarps * kStgBytes);
    uint64_t* empty = full + pl.stages;
    uint64_t* acc_full = empty + pl.stages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);   // [0] row blocks, [1] abort, [2] skip
    // what each stage's item is, written by the producer before the stage is full:
    // rows | offset << 16, or kStop
    volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(tmem_slot + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pl.pair ? tc5::cluster_rank() : 0u;
    if (warp == kProducerWarp) tc5::alloc(tmem_slot, kTmemCols);
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
            for (int s = 0; s < pl.stages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], pl.pair ? 2 : 1);   // the CTAs that read the stage's rows
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(&acc_full[s], 1);
                mbar_init(&acc_empty[s], kEpiWarps);
            }
            fence_barrier_init();
        }
    }
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    // a pair's barriers are initialised before the other CTA's copies and commits reach them
    if (pl.pair) tc5::cluster_sync();
    const uint32_t tmem = *tmem_slot;
    const int ntiles = (g.N + kMxTileRows - 1) / kMxTileRows;
    const int kstages = (g.K + kMxTileCols - 1) / kMxTileCols;
    // a pair's item is (row block, two tiles of N); an odd last tile leaves the second CTA a
    // repeat of the first's that it does not write
    const int nper = pl.pair ? (ntiles + 1) / 2 : ntiles;
    const int64_t n_items = flags[2] ? 0 : (int64_t)flags[0] * nper;
    const int64_t first = pl.pair ? blockIdx.x >> 1 : blockIdx.x;
    const Walk wk{n_items, pl.pair ? gridDim.x >> 1 : gridDim.x, nper, ntiles, rank};
    Routing nxt = load_routing(g, pl, wk, first, lane);
    const int64_t art = mx_row_tiles(g.a_rows);

    if (warp == kProducerWarp) {
        tc5::Ring r;
        int64_t issued = 0;
        bool ok = true;
        for (int64_t i = first; i < n_items && ok; i += wk.step) {
            const Item it = item_at(g, pl, wk, i, nxt, lane, false);
            nxt = load_routing(g, pl, wk, i + wk.step, lane);
            if (it.rows == 0) continue;
            if (lane == 0) {
                const uint8_t* wt = g.w + kHeaderBytes + ((int64_t)it.e * ntiles + it.nt) * kstages * kMxTileBytes;
                // tiles of the block's rows: its own (grouped), or those of the matrix it starts in (dense)
                const int64_t t0 = g.sorted_ids ? it.b * art : it.b * pl.tok / kMxTileRows;
                const uint8_t* at = g.a + kHeaderBytes + t0 * kstages * kMxTileBytes;
                const int64_t tstride = (int64_t)kstages * kMxTileBytes;
                const int r0 = min(it.rows, kMxTileRows - it.off), r1 = it.rows - r0;
                const uint32_t bytes = kMxTileBytes + (uint32_t)it.rows * 128u + (r1 > 0 ? 2048u : 1024u);
                for (int ks = 0; ks < kstages; ++ks, ++issued, r.next(pl.stages)) {
                    if (!tc5::wait(&empty[r.slot], r.phase ^ 1u, &flags[1], g.err)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = smem + r.slot * pl.stage_bytes;
                    uint8_t* sb = st + kMxTileBytes;
                    uint8_t* ss = sb + pl.tok * 128;
                    const uint8_t* a0 = at + (int64_t)ks * kMxTileBytes;
                    uint64_t* bar = &full[r.slot];
                    info[r.slot] = (uint32_t)it.rows | (uint32_t)it.off << 16;
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_g2s(st, wt + (int64_t)ks * kMxTileBytes, kMxTileBytes, bar);
                    if (!pl.pair) {
                        bulk_g2s(sb, a0 + it.off * 128, (uint32_t)r0 * 128u, bar);
                        bulk_g2s(ss, a0 + kMxCodeBytes, 1024u, bar);
                        if (r1 > 0) {
                            bulk_g2s(sb + r0 * 128, a0 + tstride, (uint32_t)r1 * 128u, bar);
                            bulk_g2s(ss + 1024, a0 + tstride + kMxCodeBytes, 1024u, bar);
                        }
                    } else {
                        // rows [h0, h1) and scale block `rank` of every tile touched, to both CTAs
                        const int h0 = (int)rank * (it.rows / 2), h1 = h0 + it.rows / 2;
                        const uint32_t so = kMxCodeBytes + rank * kMxScaleBlock;
                        if (h0 < r0)
                            tc5::bulk_g2s_pair(sb + h0 * 128, a0 + (it.off + h0) * 128, (uint32_t)(min(h1, r0) - h0) * 128u, bar);
                        if (h1 > r0) {
                            const int s0 = max(h0, r0);
                            tc5::bulk_g2s_pair(sb + s0 * 128, a0 + tstride + (s0 - r0) * 128, (uint32_t)(h1 - s0) * 128u, bar);
                        }
                        tc5::bulk_g2s_pair(ss + rank * kMxScaleBlock, a0 + so, kMxScaleBlock, bar);
                        if (r1 > 0) tc5::bulk_g2s_pair(ss + 1024 + rank * kMxScaleBlock, a0 + tstride + so, kMxScaleBlock, bar);
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        if (lane == 0 && ok && tc5::wait(&empty[r.slot], r.phase ^ 1u, &flags[1], g.err)) {
            info[r.slot] = kStop;
            mbar_arrive(&full[r.slot]);
            ++issued;
            r.next(pl.stages);
        }
        // leave only after every copy issued here has landed
        if (lane == 0) {
            for (int k = 0; k < pl.stages && k < issued; ++k) {
                r.slot = r.slot == 0 ? pl.stages - 1 : r.slot - 1;
                if (r.slot == pl.stages - 1) r.phase ^= 1u;
                if (!mbar_wait(&full[r.slot], r.phase)) set_error(g.err, CHORD_DEV_TIMEOUT);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // Slot, its address and parity; barriers as shared-memory addresses.
        struct Pos {
            uint32_t slot, st, parity;
        };
        const uint32_t base = smem_u32(smem), full_a = smem_u32(full), empty_a = smem_u32(empty);
        const uint32_t stages = (uint32_t)pl.stages, stage_bytes = (uint32_t)pl.stage_bytes, tok128 = (uint32_t)pl.tok * 128u;
        auto next = [&](Pos p) {
            return p.slot + 1 == stages ? Pos{0, base, p.parity ^ 1u} : Pos{p.slot + 1, p.st + stage_bytes, p.parity};
        };
        const uint32_t sf_base = tmem + 2u * (uint32_t)pl.tok, sf_end = sf_base + (uint32_t)pl.sf_slots * 24u;
        const bool sf_short = pl.sf_slots < pl.stages;
        Pos p{0, base, 0};
        uint32_t nitem = 0, g_stage = 0, sfa = sf_base;
        uint32_t last_bar = 0, last_parity = 0;
        bool ok = true;
        while (ok) {
            if (!tc5::wait(full_a + p.slot * 8, p.parity, &flags[1], g.err)) break;
            const uint32_t inf = __shfl_sync(0xffffffffu, info[p.slot], 0);
            if (inf == kStop) break;
            const uint32_t rows = inf & 0xffffu, off = inf >> 16, buf = nitem & 1u;
            if (!tc5::wait(smem_u32(&acc_empty[buf]), ((nitem >> 1) & 1u) ^ 1u, &flags[1], g.err)) break;
            tc5::fence_after();
            const uint32_t acc = tmem + buf * (uint32_t)pl.tok;
            const uint32_t id0 = tc5::idesc_mxf4((int)rows, 0), id2 = tc5::idesc_mxf4((int)rows, 2);
            const bool two = off + rows > (uint32_t)kMxTileRows;
            // One stage: scales of its two 128-column halves to the slot's columns, then its
            // instructions.  (A slot is reused only after the instructions that read it.)
            auto stage = [&](const Pos& q, uint32_t sf, int ks) {
                const uint64_t dsa = tc5::desc_scales(q.st + kMxCodeBytes);
                const uint64_t dsb = tc5::desc_scales(q.st + kMxTileBytes + tok128);
                const uint64_t da = tc5::desc_sw128(q.st), db = tc5::desc_sw128(q.st + kMxTileBytes);
                const int nk = min(4, (g.K - ks * kMxTileCols + 63) / 64);
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    tc5::cp_scales(sf + 4u * h, dsa + h * (kMxScaleBlock >> 4));
                    tc5::cp_scales(sf + 8u + 8u * h, dsb + h * (kMxScaleBlock >> 4));
                    if (two) tc5::cp_scales(sf + 12u + 8u * h, dsb + (1024u >> 4) + h * (kMxScaleBlock >> 4));
                }
#pragma unroll
                for (uint32_t kk = 0; kk < 4; ++kk)
                    if ((int)kk < nk)
                        tc5::mma_mxf4(acc, da + 2u * kk, db + 2u * kk, kk & 1 ? id2 : id0, sf + 4u * (kk >> 1),
                                      sf + 8u + 8u * (kk >> 1) + (off >> 5), ks > 0 || kk > 0 ? 1u : 0u);
                if (pl.pair)
                    tc5::commit_pair(empty_a + q.slot * 8);
                else
                    tc5::commit(empty_a + q.slot * 8);
                if (ks == kstages - 1) tc5::commit(smem_u32(&acc_full[buf]));
            };
            // instructions of the stage that used this stage's scale slot are done
            auto sf_free = [&](uint32_t st) {
                if (!sf_short || st < (uint32_t)pl.sf_slots) return true;
                const uint32_t old = st - (uint32_t)pl.sf_slots;
                return tc5::wait(empty_a + (old % stages) * 8, (old / stages) & 1u, &flags[1], g.err);
            };
            for (int ks = 0; ks < kstages; ks += 2) {
                const bool second = ks + 1 < kstages;
                const Pos q = next(p);
                const uint32_t sfb = sfa + 24u == sf_end ? sf_base : sfa + 24u;
                ok = (ks == 0 || tc5::wait(full_a + p.slot * 8, p.parity, &flags[1], g.err)) && sf_free(g_stage);
                if (!sf_short) ok = ok && (!second || tc5::wait(full_a + q.slot * 8, q.parity, &flags[1], g.err));
                if (!ok) break;
                if (!sf_short) {
                    if (tc5::elect()) {
                        stage(p, sfa, ks);
                        if (second) stage(q, sfb, ks + 1);
                    }
                } else {
                    if (tc5::elect()) stage(p, sfa, ks);
                    __syncwarp();
                    if (second) {
                        ok = tc5::wait(full_a + q.slot * 8, q.parity, &flags[1], g.err) && sf_free(g_stage + 1);
                        if (!ok) break;
                        if (tc5::elect()) stage(q, sfb, ks + 1);
                    }
                }
                __syncwarp();
                last_bar = empty_a + (second ? q.slot : p.slot) * 8;
                last_parity = second ? q.parity : p.parity;
                g_stage += second ? 2u : 1u;
                sfa = second ? (sfb + 24u == sf_end ? sf_base : sfb + 24u) : sfb;
                p = second ? next(q) : q;
            }
            ++nitem;
        }
        // the last instructions are done before the tensor memory is released
        if (last_bar) tc5::wait(last_bar, last_parity, &flags[1], g.err);
        __syncwarp();
    } else {
        const int wg = warp >> 2, quarter = warp & 3;
        int64_t nitem = 0;
        for (int64_t i = first; i < n_items; i += wk.step) {
            const Item it = item_at(g, pl, wk, i, nxt, lane, warp == 0);
            nxt = load_routing(g, pl, wk, i + wk.step, lane);
            if (it.rows == 0) continue;
            const int buf = (int)(nitem & 1);
            if (!tc5::wait<true>(&acc_full[buf], (uint32_t)((nitem >> 1) & 1), &flags[1], g.err)) break;
            tc5::fence_after();
            if (it.write) drain(g, pl, it, tmem + (uint32_t)(buf * pl.tok), wg, quarter, lane, stg + warp * kStgBytes);
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
            ++nitem;
        }
    }
    tc5::fence_before();
    __syncthreads();
    if (pl.pair) tc5::cluster_sync();   // the other CTA's copies and commits into this one are done
    tc5::fence_after();
    if (warp == kProducerWarp) tc5::dealloc(tmem, kTmemCols);
}

cudaError_t launch_mx_gemm(const MxGemmArgs& g, cudaStream_t st) {
    MxPlan pl;
    // Dense blocks: 192 rows (two accumulators and the scales fill the tensor
    // memory), fewer when the matrix is shorter.
    pl.tok = g.sorted_ids ? (int)g.a_rows : (g.a_rows > 128 ? 192 : (g.a_rows > 64 ? 128 : 64));
    const int tiles = (pl.tok + 64 + kMxTileRows - 1) / kMxTileRows;   // row tiles a block may touch
    pl.stage_bytes = kMxTileBytes + pl.tok * 128 + 1024 * tiles;
    const size_t fixed = 1024 + kEpiWarps * kStgBytes + 128 + 4 * kMaxStages;
    pl.stages = (int)((kSmemBudget - fixed) / (pl.stage_bytes + 16));
    if (pl.stages > kMaxStages) pl.stages = kMaxStages;
    if (pl.stages < 2) return cudaErrorInvalidConfiguration;
    pl.sf_slots = (int)((kTmemCols - 2 * pl.tok) / 24);
    if (pl.sf_slots > pl.stages) pl.sf_slots = pl.stages;
    // one CTA per SM: it takes the whole tensor memory (the ring is larger than half the shared memory)
    const size_t smem = fixed + (size_t)pl.stages * (pl.stage_bytes + 16);
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(mx_gemm_kernel), kSmemBudget);
    if (e != cudaSuccess) return e;
    const int64_t ntiles = (g.N + kMxTileRows - 1) / kMxTileRows;
    const int64_t blocks = g.sorted_ids ? g.a_groups : (g.a_rows + pl.tok - 1) / pl.tok;
    const int64_t sms = device_info().sm_count;
    pl.pair = pl.tok >= kPairRows && ntiles > 1;
    const int64_t items = pl.pair ? blocks * ((ntiles + 1) / 2) : blocks * ntiles, ctas = pl.pair ? sms / 2 : sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items < ctas ? items : ctas) * (pl.pair ? 2 : 1)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pl.pair) {
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
    return cudaLaunchKernelEx(&cfg, mx_gemm_kernel, g, pl);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMxMaxBlockM = 224;

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
    const double tok_e = (double)T * (double)(topk > 0 ? topk : 1) / (double)eg;
    // rows that an expert rarely exceeds (mean + 3 sd of a Poisson count), in
    // as few equal blocks as the kernel's largest allows
    const double need = tok_e + 3.0 * sqrt(tok_e) + 1.0;
    const double blocks = ceil(need / kMxMaxBlockM);
    const int bm = (int)ceil(need / blocks / 32.0) * 32;
    return bm > kMxMaxBlockM ? kMxMaxBlockM : bm;
}

chord_status chord_mxfp4_moe_gemm(const void* Aq, size_t aq_bytes, const void* packed, size_t packed_bytes, int E,
                                  int N, int K, const int32_t* sorted_ids, const int32_t* expert_ids,
                                  const int32_t* num_tokens_padded, int64_t capacity, int block_m, int64_t num_pairs,
                                  void* C, int c_dtype, const chord_opts* opts, void* stream) {
    if (E <= 0 || N <= 0 || K <= 0 || block_m <= 0 || capacity < 0 || num_pairs < 0) return CHORD_ERR_INVALID_ARG;
    if (K % kGroup || block_m % 32 || block_m > kMxMaxBlockM || num_pairs >= INT32_MAX || capacity >= INT32_MAX)
        return CHORD_ERR_UNSUPPORTED;
    if (capacity % block_m || (c_dtype != CHORD_DTYPE_BF16 && c_dtype != CHORD_DTYPE_F32)) return CHORD_ERR_INVALID_ARG;
    if (packed_bytes != chord_mxfp4_bytes(E, N, K) || aq_bytes != chord_mxfp4_rows_bytes(capacity, block_m, K))
        return CHORD_ERR_LAYOUT_MISMATCH;
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
