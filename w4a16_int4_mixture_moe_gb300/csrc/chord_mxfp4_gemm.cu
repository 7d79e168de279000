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
//   * a scale warp's lane copies the stage's scales to tensor memory;
//   * an issuing lane issues the stage's four K = 64 instructions into one of two FP32
//     accumulators and commits the stage back to the producer (with the scale
//     copies in the same lane a stage took about 900 cycles, paced by that lane);
//   * eight warps read the finished accumulator and write C while the next item
//     is computed into the other one.
// Every wait is bounded; the grid is persistent (static round robin).
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1, kScaleWarp = kEpiWarps + 2;
constexpr int kThreads = (kEpiWarps + 3) * 32;
constexpr int kMaxStages = 12;
constexpr int kStgBytes = 2048;          // one epilogue warp's buffer: 16 rows x 32 columns x FP32
constexpr uint32_t kTmemCols = 512;
constexpr size_t kSmemBudget = 227 * 1024;

struct MxPlan {
    int tok;        // rows of a block (dense: a multiple of 64)
    int stages;     // shared-memory ring
    int sf_slots;   // tensor-memory scale ring
    int stage_bytes;
};

struct Item {
    int64_t b;      // row block
    int nt;         // 128-row tile of N
    int e;          // expert
    int rows;       // rows of the block that hold pairs (a prefix), rounded up to 16; 0: nothing to do
    int off;        // first row inside its 128-row tile (dense blocks of 64 or 192: 0 or 64)
};

// Facts of item i, computed identically by every warp from the same arrays.
__device__ __forceinline__ Item item_at(const MxGemmArgs& g, const MxPlan& pl, int64_t i, int ntiles, int lane,
                                        bool report) {
    Item it;
    it.b = divmod_idx(i, ntiles, it.nt);
    it.e = 0;
    it.off = 0;
    if (!g.sorted_ids) {
        const int64_t r0 = it.b * pl.tok;
        const int64_t n = min((int64_t)pl.tok, g.a_rows - r0);
        it.rows = (int)((n + 15) / 16 * 16);
        it.off = (int)(r0 % kMxTileRows);
        return it;
    }
    it.e = g.expert_ids[it.b];
    int32_t ids[7];
#pragma unroll
    for (int k = 0; k < 7; ++k) {
        const int r = lane + 32 * k;
        ids[k] = r < pl.tok ? g.sorted_ids[it.b * pl.tok + r] : (int32_t)g.num_pairs;
    }
    it.rows = 0;
    if (it.e < 0 || it.e >= g.E) {
        if (report && lane == 0) set_error(g.err, CHORD_DEV_BAD_EXPERT);
        return it;
    }
    int last = 0;
#pragma unroll
    for (int k = 0; k < 7; ++k) {
        const bool ok = ids[k] >= 0 && ids[k] < g.num_pairs;
        if (report && !ok && ids[k] != g.num_pairs) set_error(g.err, CHORD_DEV_BAD_ROW);
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
    uint64_t* sf_full = empty + pl.stages;
    uint64_t* acc_full = sf_full + pl.sf_slots;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);   // [0] row count, [1] abort, [2] skip

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        bool ok = mx_header_ok(g.a, g.a_groups, g.a_rows, g.K) && mx_header_ok(g.w, g.E, g.N, g.K);
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
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < pl.sf_slots; ++s) mbar_init(&sf_full[s], 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], kEpiWarps);
        }
        fence_barrier_init();
    }
    __syncthreads();
    if (flags[2]) return;
    if (warp == kProducerWarp) tc5::alloc(tmem_slot, kTmemCols);
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tmem = *tmem_slot;
    const int ntiles = (g.N + kMxTileRows - 1) / kMxTileRows;
    const int kstages = (g.K + kMxTileCols - 1) / kMxTileCols;
    const int64_t n_items = (int64_t)flags[0] * ntiles;
    const int64_t art = mx_row_tiles(g.a_rows);

    if (warp == kProducerWarp) {
        tc5::Ring r;
        int64_t issued = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < n_items && ok; i += gridDim.x) {
            const Item it = item_at(g, pl, i, ntiles, lane, false);
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
                    mbar_arrive_expect_tx(&full[r.slot], bytes);
                    bulk_g2s(st, wt + (int64_t)ks * kMxTileBytes, kMxTileBytes, &full[r.slot]);
                    bulk_g2s(sb, a0 + it.off * 128, (uint32_t)r0 * 128u, &full[r.slot]);
                    bulk_g2s(ss, a0 + kMxCodeBytes, 1024u, &full[r.slot]);
                    if (r1 > 0) {
                        bulk_g2s(sb + r0 * 128, a0 + tstride, (uint32_t)r1 * 128u, &full[r.slot]);
                        bulk_g2s(ss + 1024, a0 + tstride + kMxCodeBytes, 1024u, &full[r.slot]);
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
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
    } else if (warp == kScaleWarp) {
        tc5::Ring r, sf;
        uint32_t g_stage = 0;
        bool ok = true;
        const uint32_t sf_base = tmem + 2u * (uint32_t)pl.tok;
        for (int64_t i = blockIdx.x; i < n_items && ok; i += gridDim.x) {
            const Item it = item_at(g, pl, i, ntiles, lane, false);
            if (it.rows == 0) continue;
            const bool two = it.off + it.rows > kMxTileRows;
            for (int ks = 0; ks < kstages; ++ks, ++g_stage, r.next(pl.stages), sf.next(pl.sf_slots)) {
                // the slot was last read by the instructions of sf_slots stages ago
                if (g_stage >= (uint32_t)pl.sf_slots) {
                    const uint32_t old = g_stage - (uint32_t)pl.sf_slots;
                    ok = tc5::wait(&empty[old % pl.stages], (old / pl.stages) & 1u, &flags[1], g.err);
                }
                ok = ok && tc5::wait(&full[r.slot], r.phase, &flags[1], g.err);
                if (!ok) break;
                tc5::fence_after();
                const uint32_t st = smem_u32(smem) + (uint32_t)(r.slot * pl.stage_bytes);
                const uint32_t sfa = sf_base + (uint32_t)sf.slot * 24u, sfb = sfa + 8u;
                const uint64_t dsa = tc5::desc_scales(st + kMxCodeBytes);
                const uint64_t dsb = tc5::desc_scales(st + kMxTileBytes + (uint32_t)pl.tok * 128u);
                if (tc5::elect()) {
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        tc5::cp_scales(sfa + 4u * h, dsa + h * (kMxScaleBlock >> 4));
                        tc5::cp_scales(sfb + 8u * h, dsb + h * (kMxScaleBlock >> 4));
                        if (two) tc5::cp_scales(sfb + 8u * h + 4u, dsb + (1024u >> 4) + h * (kMxScaleBlock >> 4));
                    }
                    tc5::commit(&sf_full[sf.slot]);
                }
                __syncwarp();
            }
        }
    } else if (warp == kMmaWarp) {
        tc5::Ring r, sf;
        uint32_t nitem = 0;
        uint64_t* last_bar = nullptr;
        uint32_t last_parity = 0;
        bool ok = true;
        const uint32_t sf_base = tmem + 2u * (uint32_t)pl.tok;
        for (int64_t i = blockIdx.x; i < n_items && ok; i += gridDim.x) {
            const Item it = item_at(g, pl, i, ntiles, lane, false);
            if (it.rows == 0) continue;
            const uint32_t buf = nitem & 1u;
            if (!tc5::wait(&acc_empty[buf], ((nitem >> 1) & 1u) ^ 1u, &flags[1], g.err)) break;
            tc5::fence_after();
            const uint32_t acc = tmem + buf * (uint32_t)pl.tok;
            const uint32_t id0 = tc5::idesc_mxf4(it.rows, 0), id2 = tc5::idesc_mxf4(it.rows, 2);
            for (int ks = 0; ks < kstages; ++ks, r.next(pl.stages), sf.next(pl.sf_slots)) {
                if (!tc5::wait(&full[r.slot], r.phase, &flags[1], g.err) ||
                    !tc5::wait(&sf_full[sf.slot], sf.phase, &flags[1], g.err)) {
                    ok = false;
                    break;
                }
                tc5::fence_after();
                const uint32_t st = smem_u32(smem) + (uint32_t)(r.slot * pl.stage_bytes);
                const uint32_t sfa = sf_base + (uint32_t)sf.slot * 24u, sfb = sfa + 8u + (uint32_t)(it.off >> 5);
                const uint64_t da = tc5::desc_sw128(st), db = tc5::desc_sw128(st + kMxTileBytes);
                const int nk = min(4, (g.K - ks * kMxTileCols + 63) / 64);
                if (tc5::elect()) {
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        if ((int)kk < nk)
                            tc5::mma_mxf4(acc, da + 2u * kk, db + 2u * kk, kk & 1 ? id2 : id0, sfa + 4u * (kk >> 1),
                                          sfb + 8u * (kk >> 1), ks > 0 || kk > 0 ? 1u : 0u);
                    tc5::commit(&empty[r.slot]);
                    if (ks == kstages - 1) tc5::commit(&acc_full[buf]);
                }
                __syncwarp();
                last_bar = &empty[r.slot];
                last_parity = r.phase;
            }
            ++nitem;
        }
        // the last instructions are done before the tensor memory is released
        if (last_bar) mbar_wait(last_bar, last_parity);
        __syncwarp();
    } else {
        const int wg = warp >> 2, quarter = warp & 3;
        int64_t nitem = 0;
        for (int64_t i = blockIdx.x; i < n_items; i += gridDim.x) {
            const Item it = item_at(g, pl, i, ntiles, lane, warp == 0);
            if (it.rows == 0) continue;
            const int buf = (int)(nitem & 1);
            if (!tc5::wait(&acc_full[buf], (uint32_t)((nitem >> 1) & 1), &flags[1], g.err)) break;
            tc5::fence_after();
            drain(g, pl, it, tmem + (uint32_t)(buf * pl.tok), wg, quarter, lane, stg + warp * kStgBytes);
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
            ++nitem;
        }
    }
    tc5::fence_before();
    __syncthreads();
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
    const size_t fixed = 1024 + kEpiWarps * kStgBytes + 128 + 8 * kMaxStages;
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
    const int64_t items = blocks * ntiles;
    const int64_t sms = device_info().sm_count;
    mx_gemm_kernel<<<(unsigned)(items < sms ? items : sms), kThreads, smem, st>>>(g, pl);
    return cudaGetLastError();
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
