// Weight rows times activation rows (chord_rows.cuh): the weight rows are the matrix instruction's M side, so
// a block of 37 rows of x costs an N = 48 instruction and an adapter of rank 16 the first sixteen
// rows of an M = 128 one (the others multiply whatever lies behind them in shared memory, their sums are
// not read).  A CTA computes one K slice of one item; the slices of an item are a cluster and
// join their sums through distributed shared memory in rank order.  Roles: a producer warp (a
// stage of 64 columns: one box of the weights for every 128 rows, and either one box of
// consecutive rows of x or, gathered, four rows a copy, each lane its own), an issuing warp, eight warps that
// read the accumulators.  The matrix instructions' additions chop, so a chain of them is kept to
// kChain stages (16 instructions); the eight warps add the chains up in registers, one accumulator being read
// while the other one is filled (K = 7168 in chains of 224: relative error 3.8e-6, of 16: 3e-7, FP32
// products and sums in PyTorch: 9e-7).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chord_internal.h"
#include "chord_rows.cuh"
#include "chord_tcgen05.cuh"

namespace chord {
namespace {

constexpr int kStepCols = 64;           // columns of a stage: 128 bytes, the swizzle's row
constexpr int kTileRows = 128;
constexpr int kRowsThreads = 320;
constexpr int kChain = 4;               // stages
constexpr int kMaxStages = 12;
constexpr long long kLandCycles = 4000000;   // about 2 ms
constexpr size_t kFixed = 1024;         // alignment
constexpr size_t kSmemMost = 226 * 1024;   // dynamic; the barriers are static
constexpr size_t kOverrun = kTileRows * 128;   // an M = 128 operand may reach past the last stage

struct RowsMaps {
    CUtensorMap w, x;
};

struct RowsPlan {
    int tiles;        // M tiles
    int w_rows;       // weight rows of a box
    int stage, stages;
    uint32_t tmem_cols;
};

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A box of a 2-D tensor map at (column, row).
__device__ __forceinline__ void box_g2s(uint32_t dst, const void* map, int col, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(col), "r"(row), "r"(bar)
        : "memory");
}
// Four rows of a tensor map whose box is one row.
__device__ __forceinline__ void gather4_g2s(uint32_t dst, const void* map, int col, int r0, int r1, int r2, int r3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(map), "r"(col), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// G2: groups of 16 accumulator columns that each of the eight warps adds up, half of an item's.
template <bool GATHER, int G2>
__global__ void __launch_bounds__(kRowsThreads, G2 <= 4 ? 2 : 1) rows_kernel(const RowsArgs a, const RowsPlan pl, const __grid_constant__ RowsMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int flag[1];   // abort
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* aborted = flag;
    if (warp == 1) tc5::alloc<false>(&tmem_slot, pl.tmem_cols);
    if (threadIdx.x == 0) {
        for (int s = 0; s < pl.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 8);
        }
        flag[0] = 0;
        fence_barrier_init();
    }
    pdl_trigger();
    pdl_wait();
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tmem = tmem_slot;
    const int S = a.splits;
    const int rank = S > 1 ? (int)tc5::cluster_rank() : 0;
    const int64_t item = blockIdx.x / S;
    const int steps1 = (a.K + kStepCols - 1) / kStepCols, steps = steps1 * a.parts;
    const int k0 = (int)((int64_t)rank * steps / S), k1 = (int)((int64_t)(rank + 1) * steps / S);
    // the item: its first weight row, its rows of x
    int w0 = 0, n = 0;
    int64_t t0 = 0;
    const int32_t* list = nullptr;
    bool live = true;
    if constexpr (GATHER) {
        int sub;
        const int64_t block = divmod_idx(item, a.block_rows / a.nb, sub);
        live = block < *a.nblocks;
        if (live) {
            const int slot = a.block_slot[block];
            live = slot >= 0;
            w0 = slot * a.R;
            list = a.rows + block * a.block_rows + sub * a.nb;
        }
        if (live) {
            // rows of a block are a prefix
            for (int j = lane; j < a.nb; j += 32)
                if (list[j] >= 0) n = j + 1;
            n = __reduce_max_sync(0xffffffffu, n);
            live = n > 0;
        }
    } else {
        int g;
        t0 = divmod_idx(item, a.groups, g) * a.nb;
        w0 = g * a.R;
        const int64_t left = a.x_rows - t0;
        n = left < a.nb ? (int)left : a.nb;
    }
    const int n16 = (n + 15) / 16 * 16;
    const uint32_t base = smem_u32(smem);
    bool ok = true;
    if (live && warp == 0) {
        // ---- producer: the lanes of a gathered block copy four rows each
        int r[4];
        if constexpr (GATHER) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = 4 * lane + q;
                const int p = list[j < n ? j : 0];
                r[q] = a.div == 1 ? p : p / a.div;
            }
        }
        const uint32_t x_rows = GATHER ? (uint32_t)(n + 3) / 4 * 4 : (uint32_t)a.nb;
        const uint32_t bytes = (uint32_t)(pl.tiles * pl.w_rows) * 128u + x_rows * 128u;
        tc5::Ring ring;
        int part = k0 / steps1, k = k0 % steps1;
        for (int s = k0; s < k1; ++s) {
            // fills of a slot after the first wait for the instructions that read it
            if (s - k0 >= pl.stages) ok = tc5::wait(&empty[ring.slot], ring.phase ^ 1u, aborted, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t st = base + (uint32_t)ring.slot * (uint32_t)pl.stage, bar = smem_u32(&full[ring.slot]);
            const uint32_t xs = st + (uint32_t)(pl.tiles * pl.w_rows) * 128u;
            if (lane == 0) {
                tc5::arrive_expect_tx(bar, bytes);
                // the part with the smallest numbers first
                const int row = (a.parts - 1 - part) * a.part_rows + w0;
                for (int m = 0; m < pl.tiles; ++m)
                    box_g2s(st + (uint32_t)(m * pl.w_rows) * 128u, &maps.w, k * kStepCols, row + m * pl.w_rows, bar);
                if (!GATHER) box_g2s(xs, &maps.x, k * kStepCols, (int)t0, bar);
            }
            __syncwarp();
            if constexpr (GATHER)
                if (4 * lane < n) gather4_g2s(xs + (uint32_t)lane * 512u, &maps.x, k * kStepCols, r[0], r[1], r[2], r[3], bar);
            ring.next(pl.stages);
            if (++k == steps1) k = 0, ++part;
        }
        // leave only after every copy issued here has been read, or had time to land (below)
    } else if (live && warp == 1) {
        // ---- issuing warp
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n16 >> 3) << 17) | ((uint32_t)(kTileRows >> 4) << 24);
        tc5::Ring ring;
        for (int s = k0; s < k1; ++s) {
            const uint32_t chain = (uint32_t)(s - k0) / kChain, buf = chain & 1u;
            const bool first = (s - k0) % kChain == 0;
            // the second use of an accumulator on: it has been read
            if (first && chain >= 2) ok = tc5::wait(&acc_empty[buf], ((chain >> 1) & 1u) ^ 1u, aborted, a.err);
            ok = ok && tc5::wait(&full[ring.slot], ring.phase, aborted, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc5::fence_after();
            const uint32_t st = base + (uint32_t)ring.slot * (uint32_t)pl.stage, acc = tmem + buf * (uint32_t)(pl.tiles * a.nb);
            const uint64_t db = tc5::desc_sw128(st + (uint32_t)(pl.tiles * pl.w_rows) * 128u);
            if (tc5::elect()) {
                for (int m = 0; m < pl.tiles; ++m) {
                    const uint64_t da = tc5::desc_sw128(st + (uint32_t)(m * pl.w_rows) * 128u);
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        mma_f16(acc + (uint32_t)(m * a.nb), da + 2u * kk, db + 2u * kk, idesc, !first || kk > 0 ? 1u : 0u);
                }
                tc5::commit<false, false>(smem_u32(&empty[ring.slot]));
                if (s + 1 == k1 || (s + 1 - k0) % kChain == 0) tc5::commit<false, false>(smem_u32(&acc_full[buf]));
            }
            __syncwarp();
            ring.next(pl.stages);
        }
    }
    // ---- the sums: group g of the accumulator's columns is 16 rows of x and one tile of weight rows
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int per = a.nb / 16, groups = pl.tiles * per;
    float sum[G2][16];
    if (live && warp >= 2) {
#pragma unroll
        for (int i = 0; i < G2; ++i)
#pragma unroll
            for (int u = 0; u < 16; ++u) sum[i][u] = 0.0f;
        const int chains = (k1 - k0 + kChain - 1) / kChain;
        for (int c = 0; c < chains; ++c) {
            const int buf = c & 1;
            ok = tc5::wait(&acc_full[buf], (uint32_t)((c >> 1) & 1), aborted, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc5::fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * pl.tiles * a.nb);
#pragma unroll
            for (int i = 0; i < G2; ++i) {
                const int g = 2 * i + half;
                if (g >= groups || g % per * 16 >= n || g / per * kTileRows + quarter * 32 >= a.R) continue;
                uint32_t v[16];
                tc5::ld16(acc + (uint32_t)(g * 16), v);
                tc5::wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u) sum[i][u] += __uint_as_float(v[u]);
            }
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
    }
    auto put = [&](int j, int r, float v) {   // sum of weight row r and row j, complete
        if constexpr (GATHER)
            a.out[(int64_t)list[j] * a.R + r] = v;
        else if (w0 + r < a.E)
            a.out[(t0 + j) * a.E + w0 + r] = v;
    };
    // the sums of rows first(q) .. first(q + 1) are joined by CTA q, its shared memory holds
    // [slice][row][R] over the ring
    __shared__ uint32_t goes_to[kTileRows];   // cluster address of row j's sums of this slice
    auto first = [&](int q) { return n * q / S; };
    const int cols = (n + S - 1) / S;
    if (S > 1 && (int)threadIdx.x < n) {
        const int j = threadIdx.x;
        int q = j * S / n;
        while (j >= first(q + 1)) ++q;   // fewer rows than slices: some own none
        goes_to[j] = tc5::at_cta(base + (uint32_t)((rank * cols + j - first(q)) * a.R * 4), (uint32_t)q);
    }
    tc5::fence_before();
    __syncthreads();
    // A role that gave up: what is still in flight (copies into this CTA's shared memory, instructions
    // on its tensor memory) gets its time here, before either is handed to the next CTA.
    if (aborted[0])
        for (const long long c0 = clock64(); clock64() - c0 < kLandCycles;) __nanosleep(1000);
    tc5::fence_after();
    if (warp == 1) tc5::dealloc<false>(tmem, pl.tmem_cols);
    if (S > 1) tc5::cluster_sync();   // nobody's ring is in use any more
    if (live && !aborted[0] && warp >= 2) {
#pragma unroll
        for (int i = 0; i < G2; ++i) {
            const int g = 2 * i + half, r = g / per * kTileRows + quarter * 32 + lane, j0 = g % per * 16;
            if (g >= groups || r >= a.R) continue;
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int j = j0 + u;
                if (j >= n) break;
                if (S == 1)
                    put(j, r, sum[i][u]);
                else
                    st_cluster(goes_to[j] + (uint32_t)r * 4u, sum[i][u]);
            }
        }
    }
    __syncwarp();
    if (S > 1) {
        tc5::cluster_sync();
        if (live && !aborted[0]) {
            const float* got = reinterpret_cast<const float*>(smem);
            const int j0 = first(rank), mine = first(rank + 1) - j0, slice = cols * a.R;
            for (int j = warp; j < mine; j += kRowsThreads / 32)
                for (int r = lane; r < a.R; r += 32) {
                    float v = got[j * a.R + r];
                    for (int s = 1; s < S; ++s) v += got[s * slice + j * a.R + r];   // in rank order
                    put(j0 + j, r, v);
                }
        }
    }
}

// K-major boxes of 64 columns with the 128-byte swizzle; what lies outside the matrix reads as 0.
bool rows_map(CUtensorMap* map, const void* p, int64_t rows, int cols, int64_t stride, int box_rows) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess;
        return reinterpret_cast<Encode>(ok && r == cudaDriverEntryPointSuccess ? f : nullptr);
    }();
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {kStepCols, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory that a CTA may take: two to an SM where two stages of it fit the half.
size_t ring_room(int stage) {
    const size_t half = 112 * 1024, all = kSmemMost;
    return (kFixed + kOverrun + 3 * (size_t)stage <= half ? half : all) - kFixed - kOverrun;
}

int rows_stage(int R, int nb) { return (R + nb) * 128; }

}  // namespace

int rows_block(int R) {
    const int tiles = (R + kTileRows - 1) / kTileRows;
    return tiles == 1 ? 128 : tiles <= 3 ? 64 : 32;
}

int rows_splits(int R, int nb, int steps, int64_t items, int want) {
    int s = 1;
    while (s < 8 && items * s * 2 <= want && steps / (s * 2) >= 4) s *= 2;
    return (size_t)R * (nb + 8) * 4 <= ring_room(rows_stage((R + 127) / 128 * 128, nb)) ? s : 1;
}

cudaError_t launch_rows(const RowsArgs& a, bool pdl, cudaStream_t st) {
    const bool gather = a.nblocks != nullptr;
    RowsPlan pl{};
    pl.tiles = (a.R + kTileRows - 1) / kTileRows;
    pl.w_rows = pl.tiles > 1 ? kTileRows : (a.R + 7) / 8 * 8;
    pl.stage = rows_stage(pl.tiles * pl.w_rows, a.nb);
    const size_t room = ring_room(pl.stage);
    pl.stages = (int)(room / pl.stage);
    if (pl.stages > kMaxStages) pl.stages = kMaxStages;
    if (pl.stages < 2) return cudaErrorInvalidConfiguration;
    pl.tmem_cols = 32;
    while (pl.tmem_cols < (uint32_t)(2 * pl.tiles * a.nb)) pl.tmem_cols *= 2;
    const int groups = pl.tiles * a.nb / 16;
    if (groups > 12) return cudaErrorInvalidConfiguration;
    size_t ring = (size_t)pl.stages * pl.stage;
    const size_t join = a.splits > 1 ? (size_t)a.R * (a.nb + 8) * 4 : 0;
    if (join > room) return cudaErrorInvalidConfiguration;
    if (ring + kOverrun < join) ring = join - kOverrun;
    const size_t smem = kFixed + kOverrun + ring;
    RowsMaps maps{};
    if (!rows_map(&maps.w, a.W, a.w_rows, a.K, a.K, pl.w_rows) || !rows_map(&maps.x, a.x, a.x_rows, a.K, a.x_stride, gather ? 1 : a.nb))
        return cudaErrorInvalidValue;
    void (*kern)(RowsArgs, RowsPlan, RowsMaps) = groups <= 8 ? (gather ? rows_kernel<true, 4> : rows_kernel<false, 4>)
                                                             : (gather ? rows_kernel<true, 6> : rows_kernel<false, 6>);
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kSmemMost);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.items * a.splits));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (a.splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)a.splits;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, a, pl, maps);
}

}  // namespace chord
