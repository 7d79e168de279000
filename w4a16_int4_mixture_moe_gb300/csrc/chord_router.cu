// Router logits: bf16 activations times the router's weights, FP32 sums and result.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "chord_common.cuh"
#include "chord_internal.h"
#include "chord_tcgen05.cuh"
#include "chord_thin.cuh"

namespace chord {
namespace {

struct LogitArgs {
    const __nv_bfloat16* x;
    int64_t stride;
    int T;
    const __nv_bfloat16* W;   // [parts, E, H]
    int parts, E, H;
    float* out;
};

// ---- few tokens: thin products (chord_thin.cuh) -------------------------------------------
// A CTA takes a tile of tokens and experts and a slice of K (of all parts, one behind the other, the smallest
// numbers first); the slices of a tile are a cluster.
// Up to 16 tokens, 16 experts (16 tokens of 7168 columns, 384 experts: 4.2 us in a graph, staged as below 6.9).
using ThinWarp = thin::Warp<2>;

__global__ void __launch_bounds__(thin::kThreads) logits_thin_kernel(const LogitArgs a, int splits) {
    using Warp = ThinWarp;
    constexpr int kTile = Warp::kRows * Warp::kCols;
    extern __shared__ __align__(16) float red[];   // [kWarps][kTile], then the shares
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
    pdl_trigger();
    pdl_wait();
    const int rank = splits > 1 ? (int)tc5::cluster_rank() : 0, e0 = (int)(blockIdx.x / splits) * Warp::kCols;
    const int steps1 = (a.H + thin::kStep - 1) / thin::kStep;
    const int64_t steps = (int64_t)steps1 * a.parts;
    const int k0 = (int)(rank * steps / splits), k1 = (int)((rank + 1) * steps / splits);
    float* mine = red + warp * kTile;
    Warp w;
    bool more = false;
    for (int part = k0 / steps1; part * steps1 < k1; ++part) {
#pragma unroll
        for (int j = 0; j < 2; ++j) w.x[j] = reinterpret_cast<const uint4*>(a.x + min(j * 8 + gr, a.T - 1) * a.stride) + c;
#pragma unroll
        for (int j = 0; j < Warp::kCols / 8; ++j)
            w.w[j] = reinterpret_cast<const uint4*>(a.W + ((int64_t)(a.parts - 1 - part) * a.E + min(e0 + j * 8 + gr, a.E - 1)) * a.H) + c;
        w.run(max(k0 - part * steps1, 0) + warp, min(k1 - part * steps1, steps1), a.H / 8, mine, more);
        more = true;
    }
    __syncthreads();
    thin::join_slices<kTile>(
        splits, red + thin::kWarps * kTile, [&](int i) { return thin::joined(red, kTile, i); },
        [&](int i, float v) {
            const int t = i / Warp::kCols, e = e0 + i % Warp::kCols;
            if (t < a.T && e < a.E) a.out[(int64_t)t * a.E + e] = v;
        });
}

// 64 tokens, 32 experts.  Bound by its copies to shared memory and their latency (48 tokens of 7168 columns, 384 experts in
// three parts: 10.9 us in a graph, 16.5 MB of weights).
using LogitTile = thin::Staged<4>;
constexpr int kLogitTile = LogitTile::kRows * LogitTile::kCols;

__global__ void __launch_bounds__(thin::kThreads, 2) logits_staged_kernel(const LogitArgs a, int splits) {
    extern __shared__ __align__(128) uint8_t smem[];   // the tile's ring, then the shares
    pdl_trigger();
    pdl_wait();
    const int rank = splits > 1 ? (int)tc5::cluster_rank() : 0;
    int et;
    const int64_t t0 = divmod_idx(blockIdx.x / splits, (a.E + LogitTile::kCols - 1) / LogitTile::kCols, et) * LogitTile::kRows;
    const int e0 = et * LogitTile::kCols, row = threadIdx.x >> 3, piece = threadIdx.x & 7;
    LogitTile tile;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t t = t0 + row + 32 * h;
        tile.x[h] = t < a.T ? a.x + t * a.stride + piece * 8 : nullptr;
        tile.w[h] = h == 0 && e0 + row < a.E ? a.W + (int64_t)(e0 + row) * a.H + piece * 8 : nullptr;
    }
    const int64_t steps = (int64_t)((a.H + LogitTile::kTileCols - 1) / LogitTile::kTileCols) * a.parts;
    tile.run(smem, (int)(rank * steps / splits), (int)((rank + 1) * steps / splits), a.H, a.parts, (int64_t)a.E * a.H);
    const float* sums = reinterpret_cast<const float*>(smem);
    thin::join_slices<kLogitTile>(
        splits, reinterpret_cast<float*>(smem + LogitTile::kBytes), [&](int i) { return LogitTile::joined(sums, i); },
        [&](int i, float v) {
            const int64_t t = t0 + i / LogitTile::kCols;
            const int e = e0 + i % LogitTile::kCols;
            if (t < a.T && e < a.E) a.out[t * a.E + e] = v;
        });
}

// tiles x slices CTAs: as many slices as leave two CTAs to an SM, of `least` steps at least.  Sixteen, more than a
// cluster may have everywhere, need the kernel to be allowed that once on each device, and pay only where their
// clusters find SMs of their own (384 experts in FP32, 48 tokens: eight slices 13.9 us, sixteen 10.9; 64 experts, 512
// tokens: eight 6.8, sixteen 8.6).
template <void (*KERN)(LogitArgs, int)>
cudaError_t launch_tiles(const LogitArgs& a, int64_t tiles, int64_t steps, int least, size_t smem, cudaStream_t st) {
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(KERN), smem);
    if (e != cudaSuccess) return e;
    int splits = 1;
    const int64_t sms = device_info().sm_count;
    while (splits < 16 && tiles * splits * 2 <= (splits < 8 ? 2 * sms : sms + sms / 3) && steps >= (int64_t)least * 2 * splits) splits *= 2;
    if (splits > 8) {
        static std::atomic<uint64_t> allowed{0};   // a bit for each device
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        const uint64_t bit = 1ull << (dev & 63);
        if (!(allowed.load(std::memory_order_relaxed) & bit)) {
            e = cudaFuncSetAttribute(reinterpret_cast<const void*>(KERN), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            if (dev < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    if (tiles * splits > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * splits));
    cfg.blockDim = dim3(thin::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)splits;
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
    return cudaLaunchKernelEx(&cfg, KERN, a, splits);
}

cudaError_t launch_thin(const LogitArgs& a, cudaStream_t st) {
    using Warp = ThinWarp;
    const size_t smem = (size_t)(thin::kWarps + 1) * Warp::kRows * Warp::kCols * 4;
    // a slice keeps two steps for each warp
    return launch_tiles<logits_thin_kernel>(a, (a.E + Warp::kCols - 1) / Warp::kCols, ceil_div64(a.H, thin::kStep) * a.parts, 2 * thin::kWarps,
                        smem, st);
}

int64_t staged_tiles(const LogitArgs& a) { return ceil_div64(a.T, LogitTile::kRows) * ((a.E + LogitTile::kCols - 1) / LogitTile::kCols); }

cudaError_t launch_staged(const LogitArgs& a, cudaStream_t st) {
    const size_t smem = LogitTile::kBytes + (size_t)kLogitTile * 4;
    return launch_tiles<logits_staged_kernel>(a, staged_tiles(a), ceil_div64(a.H, LogitTile::kTileCols) * a.parts, 2, smem, st);
}

// ---- many tokens: tcgen05 -------------------------------------------------------------------
// A pair of CTAs computes 256 tokens times N experts (cta_group::2, M = 256): each CTA copies its 128
// tokens and half of the experts' rows, so a CTA's copies are 128 + N / 2 rows for 128 x N sums.  Roles
// in each CTA: a copying warp (stages of 128 columns, two swizzled tiles of 64; both CTAs' bytes
// are counted on the first one's barrier), in the first CTA an issuing warp, and eight warps that read the
// accumulators.  The instructions' additions chop, so a chain is 256 columns (16 instructions) and
// the eight warps add the chains up in registers, one accumulator being read while the other is filled
// (relative error of a K = 7168 sum: 3.8e-6 in chains of 224, 2.5e-7 so, 9e-7 of PyTorch's FP32).
// 8192 tokens of 7168 columns, 384 experts: 36 us in a graph, 1.25 PFLOP/s, the tensor pipe 71 % busy in the CTAs that run.
constexpr int kReaders = 8, kWideThreads = (kReaders + 2) * 32;
constexpr int kHalfCols = 64, kStageCols = 2 * kHalfCols;
constexpr int kPairTokens = 256;
// The staged tiles copy 96 rows of K columns for 64 x 32 sums, the wide ones 128 + N / 2 for 128 x N, where a step of 128
// columns takes 0.25 us at least.  Staged and wide, us in a graph (E, H: tiles):
//   bf16  384, 7168: 72 12.3, 19.6; 96 19.6, 19.6; 192 31.9, 20.1.  161, 2088: 72 8.6, 10.3; 96 11.5, 10.2.  64, 4096: 64 9.3,
//         12.8; 94 13.5, 13.1.
//   FP32  384, 7168: 72 26.5, 52.0; 96 46.7, 52.2; 144 47.0, 52.2; 192 86.4, 52.6.  161, 2088: 72 14.1, 23.5; 96 22.7, 23.5; 192 37.5,
//         23.9.  64, 4096: 64 17.3, 31.2; 94 29.3, 31.4.
// One rule for both types: from 91 to about 150 tiles an FP32 router loses up to a tenth by it.
constexpr int64_t kStagedTiles = 90;
constexpr int kChainStages = 2;
constexpr int kMaxWideStages = 6;
constexpr long long kLandCycles = 4000000;   // about 2 ms
constexpr size_t kWideSmem = 225 * 1024;     // dynamic, 1 KB of it alignment; the barriers are static

struct WideMaps {
    CUtensorMap x, w;
};

struct WidePlan {
    int groups, N;   // groups of N experts
    int stages;
};

__device__ __forceinline__ void box_g2s_pair(uint32_t dst, const void* map, int col, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(col), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// G: groups of 16 accumulator columns that each reading warp adds up.
template <int G>
__global__ void __launch_bounds__(kWideThreads, 1) logits_wide_kernel(const LogitArgs a, const WidePlan pl, int* err, const __grid_constant__ WideMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw) + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMaxWideStages], empty[kMaxWideStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int flag[1];   // abort
    volatile int* aborted = flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc5::cluster_rank();
    // All of an SM's tensor memory, before the wait: no CTA of an earlier kernel that still has to allocate its own can be on
    // the SM, since 181 KB at least of shared memory here leave less than 47 KB, and the kernels that use tensor memory take more.
    if (warp == kReaders) tc5::alloc<true>(&tmem_slot, 512);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxWideStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 2 * kReaders);
        }
        flag[0] = 0;
        fence_barrier_init();
    }
    pdl_wait();
    tc5::fence_before();
    __syncthreads();
    tc5::cluster_sync();   // the barriers are initialised before the other CTA's arrivals reach them
    tc5::fence_after();
    pdl_trigger();         // not before this CTA has its tensor memory
    const uint32_t tmem = tmem_slot;
    int grp;
    const int64_t t0 = divmod_idx(blockIdx.x >> 1, pl.groups, grp) * kPairTokens + rank * 128;
    const int e0 = grp * pl.N, N = pl.N;
    const int steps1 = (a.H + kStageCols - 1) / kStageCols, steps = steps1 * a.parts;
    const uint32_t w_half = (uint32_t)(N / 2) * 128u, x_half = 128u * 128u, stage = 2u * (x_half + w_half);
    bool ok = true;
    if (warp == kReaders) {
        tc5::Ring ring;
        int part = 0, k = 0;
        for (int s = 0; s < steps; ++s) {
            if (s >= pl.stages) ok = tc5::wait<false, true>(&empty[ring.slot], ring.phase ^ 1u, aborted, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t st = base + (uint32_t)ring.slot * stage, bar = smem_u32(&full[ring.slot]);
            // the part with the smallest numbers first
            const int row = (a.parts - 1 - part) * a.E + e0 + (int)rank * (N / 2), col = k * kStageCols;
            if (tc5::elect()) {
                if (!rank) tc5::arrive_expect_tx(bar, 2u * stage);
                const uint32_t on = tc5::at_cta(bar, 0);
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    box_g2s_pair(st + h * x_half, &maps.x, col + (int)h * kHalfCols, (int)t0, on);
                    box_g2s_pair(st + 2u * x_half + h * w_half, &maps.w, col + (int)h * kHalfCols, row, on);
                }
            }
            __syncwarp();
            ring.next(pl.stages);
            if (++k == steps1) k = 0, ++part;
        }
    } else if (warp == kReaders + 1 && !rank) {
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kPairTokens >> 4) << 24);
        tc5::Ring ring;
        for (int s = 0; s < steps; ++s) {
            const int chain = s / kChainStages, buf = chain & 1;
            const bool first = s % kChainStages == 0, last = s + 1 == steps || (s + 1) % kChainStages == 0;
            // the second use of an accumulator on: it has been read
            if (first && chain >= 2) ok = tc5::wait<false, true>(&acc_empty[buf], ((uint32_t)(chain >> 1) & 1u) ^ 1u, aborted, err);
            ok = ok && tc5::wait<false, true>(&full[ring.slot], ring.phase, aborted, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc5::fence_after();
            const uint32_t st = base + (uint32_t)ring.slot * stage, acc = tmem + (uint32_t)(buf * 256);
            const uint64_t dx = tc5::desc_sw128(st), dw = tc5::desc_sw128(st + 2u * x_half);
            if (tc5::elect()) {
#pragma unroll
                for (uint32_t kk = 0; kk < 8; ++kk)
                    mma_pair(acc, dx + (kk / 4) * (x_half >> 4) + 2u * (kk % 4), dw + (uint64_t)(kk / 4) * (w_half >> 4) + 2u * (kk % 4), idesc,
                             !first || kk > 0 ? 1u : 0u);
                tc5::commit<true, true>(smem_u32(&empty[ring.slot]));
                if (last) tc5::commit<true, true>(smem_u32(&acc_full[buf]));
            }
            __syncwarp();
            ring.next(pl.stages);
        }
    } else if (warp < kReaders) {
        const int quarter = warp & 3, half = warp >> 2, groups = N / 16;
        float sum[G][16];
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int u = 0; u < 16; ++u) sum[i][u] = 0.0f;
        const int chains = (steps + kChainStages - 1) / kChainStages;
        for (int c = 0; c < chains; ++c) {
            const int buf = c & 1;
            ok = tc5::wait<false, true>(&acc_full[buf], (uint32_t)(c >> 1) & 1u, aborted, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc5::fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * 256);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int g = 2 * i + half;
                if (g >= groups) continue;
                uint32_t v[16];
                tc5::ld16(acc + (uint32_t)(g * 16), v);
                tc5::wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u) sum[i][u] += __uint_as_float(v[u]);
            }
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) tc5::arrive_relaxed_at(smem_u32(&acc_empty[buf]), 0);
        }
        // Through the warp's part of the ring, which nobody uses any more, so that 16 lanes write 64 bytes of a row.
        float* stg = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw))) + warp * (32 * 17);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int g = 2 * i + half;
            if (!ok || g >= groups) continue;
#pragma unroll
            for (int u = 0; u < 16; ++u) stg[lane * 17 + u] = sum[i][u];
            __syncwarp();
            const int e = e0 + g * 16 + (lane & 15);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int r = 2 * k + (lane >> 4);
                const int64_t t = t0 + quarter * 32 + r;
                if (t < a.T && e < a.E) a.out[t * a.E + e] = stg[r * 17 + (lane & 15)];
            }
            __syncwarp();
        }
        __syncwarp();
    }
    tc5::fence_before();
    __syncthreads();
    // A role that gave up has made the others' last waits return at once: what is still in flight
    // (copies into this CTA's shared memory, instructions on its tensor memory) gets its time here,
    // before either is handed to the next CTA.
    if (aborted[0])
        for (const long long c0 = clock64(); clock64() - c0 < kLandCycles;) __nanosleep(1000);
    tc5::cluster_sync();   // the pair's instructions, and arrivals on the other CTA's barriers, are done
    tc5::fence_after();
    if (warp == kReaders) tc5::dealloc<true>(tmem, 512);
}

// K-major boxes of 64 columns with the 128-byte swizzle; what lies outside the matrix reads as 0.
bool rows_map(CUtensorMap* map, const void* p, int64_t rows, int cols, int64_t stride, int box) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess;
        return reinterpret_cast<Encode>(found && r == cudaDriverEntryPointSuccess ? f : nullptr);
    }();
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {kHalfCols, (cuuint32_t)box}, ones[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Groups of experts (N a multiple of 32, at most 256, as cta_group::2 takes it): rounds of pairs times the rows a CTA copies in one.
WidePlan wide_plan(int64_t T, int E, int pairs) {
    WidePlan best{};
    int64_t least = INT64_MAX;
    for (int g = (E + 255) / 256; g <= (E + 31) / 32; ++g) {
        const int n = ((E + g - 1) / g + 31) / 32 * 32;
        const int64_t items = ceil_div64(T, kPairTokens) * g, cost = ceil_div64(items, pairs) * (128 + n / 2);
        if (cost < least) {
            least = cost;
            best.groups = g;
            best.N = n;
        }
    }
    best.stages = (int)((kWideSmem - 1024) / ((128 + best.N / 2) * 256));
    if (best.stages > kMaxWideStages) best.stages = kMaxWideStages;
    return best;
}

cudaError_t launch_wide(const LogitArgs& a, int* err, cudaStream_t st) {
    const WidePlan pl = wide_plan(a.T, a.E, device_info().sm_count / 2);
    const int64_t items = ceil_div64(a.T, kPairTokens) * pl.groups;
    WideMaps maps{};
    if (items > INT32_MAX / 2 || !rows_map(&maps.x, a.x, a.T, a.H, a.stride, 128) ||
        !rows_map(&maps.w, a.W, (int64_t)a.parts * a.E, a.H, a.H, pl.N / 2))
        return cudaErrorInvalidValue;
    auto* kern = pl.N <= 128 ? logits_wide_kernel<4> : pl.N <= 192 ? logits_wide_kernel<6> : logits_wide_kernel<8>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kWideSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * 2));
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = 1024 + (size_t)pl.stages * (128 + pl.N / 2) * 256;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, pl, err, maps);
}

// Eight significant bits a part, cut off towards zero: the three parts add up to the number
// exactly (down to 2^-110, where the last part's bits end), and none overflows.  Of a number of fewer
// bits the last part that is not 0 is dealt out over the ones behind it (1 is 1/2 + 1/4 + 1/4): no part of a
// number is 0 then, so that an infinite activation times the parts is an infinity and not a NaN.  An
// infinity or NaN is the first part alone.
__global__ void __launch_bounds__(256) split_kernel(const float* __restrict__ w, int64_t n, __nv_bfloat16* __restrict__ parts) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const float v = w[i];
        const bool finite = fabsf(v) <= 3.4028235e38f;
        float p0 = v, p1 = 0.0f, p2 = 0.0f;
        if (finite) {
            p0 = __bfloat162float(__float2bfloat16_rz(v));
            p1 = __bfloat162float(__float2bfloat16_rz(v - p0));
            p2 = v - p0 - p1;
            if (p2 == 0.0f && fabsf(v) >= 0x1p-110f) {   // halves and quarters are exact
                if (p1 == 0.0f) p0 = 0.5f * v, p1 = 0.5f * v;
                p1 = p2 = 0.5f * p1;
            }
        }
        parts[i] = __float2bfloat16_rn(p0);
        parts[n + i] = __float2bfloat16_rn(p1);
        parts[2 * n + i] = __float2bfloat16_rz(p2);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

chord_status chord_router_split_weights(const float* W, int64_t n, void* parts, void* stream) {
    if (n < 0 || (n > 0 && (!W || !parts || (reinterpret_cast<uintptr_t>(W) & 3) || (reinterpret_cast<uintptr_t>(parts) & 1))))
        return CHORD_ERR_INVALID_ARG;
    if (n > INT64_MAX / 8) return CHORD_ERR_UNSUPPORTED;
    if (n == 0) return CHORD_OK;
    const int64_t blocks = ceil_div64(n, 256);
    split_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        W, n, static_cast<__nv_bfloat16*>(parts));
    return cudaGetLastError() == cudaSuccess ? CHORD_OK : CHORD_ERR_CUDA;
}

chord_status chord_router_logits(const void* x, int64_t x_stride, int T, const void* W, int parts, int E, int H, float* logits,
                                 const chord_opts* opts, void* stream) {
    if (T < 0 || E <= 0 || H <= 0 || x_stride < (T > 1 ? H : 0)) return CHORD_ERR_INVALID_ARG;
    if ((parts != 1 && parts != 3) || E > 1024 || H % 8 || (T > 1 && x_stride % 8)) return CHORD_ERR_UNSUPPORTED;
    if (!W || !aligned16(W)) return CHORD_ERR_INVALID_ARG;
    if (T > 0 && (!x || !aligned16(x) || !logits || (reinterpret_cast<uintptr_t>(logits) & 3))) return CHORD_ERR_INVALID_ARG;
    if (T == 0) return CHORD_OK;
    LogitArgs a{static_cast<const __nv_bfloat16*>(x), x_stride, T, static_cast<const __nv_bfloat16*>(W), parts, E, H, logits};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    const cudaError_t e = T <= 16                                                   ? launch_thin(a, st)
                          : staged_tiles(a) <= kStagedTiles || H < kStageCols ? launch_staged(a, st)
                                                                                    : launch_wide(a, di.err, st);
    if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return CHORD_ERR_CUDA;
    if (!opts || !opts->validate) return CHORD_OK;
    int32_t code = 0;
    const chord_status s = chord_get_device_error(stream, &code);
    if (s != CHORD_OK) return s;
    if (code == CHORD_DEV_TIMEOUT) return CHORD_ERR_TIMEOUT;
    return code ? CHORD_ERR_DEVICE_VALIDATION : CHORD_OK;
}

}  // extern "C"
