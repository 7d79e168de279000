// Low-rank adapters of many requests beside a projection that they share:
//   v[p] = A[a, e] x[p / div],   y[p] = base[p] + scale[a] * B[a, e] v[p]
// A slot is an adapter of an expert, a * E + e; the pairs of one slot are taken together, in blocks, so a slot's
// weights are read once a block.
// Up to kFewPairs pairs: one launch (adapter_few_kernel), in which every CTA finds the blocks, of 16 rows, itself.  Bound by
//   latency (one token of 7168 columns, 4096 outputs, rank 16: 6.2 us in a graph; rank 32 8.3), above rank 32 also by the
//   registers: two CTAs to an SM leave 128 a thread, and what the first half holds for 64 rows of A spills 404 to 476 bytes (28 to 168
//   for 8 to 32 rows; rank 64 13.3 us, rank 128, which takes A in two passes, 21.3).
// More pairs: three launches.
//   plan   blocks of 64 rows by a counting sort of the pairs by slot: 5.5 to 8.5 us for 8192 pairs.
//   down   v, a block's rows times the slot's A, staged products (chord_thin.cuh); an item is (block, up to 64 rows of A,
//          K slice).  A cluster takes an item while there are few blocks; beyond, K slices are partial sums in the
//          workspace, as many as fill the GPU.  Bound by the copies to shared memory, x's and A's (3584 pairs of 7168
//          columns, rank 64: 22 us, 2.3 TB/s of x; 7168 pairs of 2048, rank 16: 12).
//   up     y = base + scale B v.  The slices of v are added in order, scaled and split into three bf16 parts of eight bits
//          each, so the tensor cores multiply all of an FP32 v.  A tile's columns are dealt so that a lane ends with whole
//          16-byte pieces of its rows of base and y.  Ranks up to 16 are bound by base's and y's bytes (8192 pairs of 7168
//          FP32 columns, rank 16: 100 us, 4.7 TB/s; a copy in the same pattern 84), larger ones by latency between
//          instructions at 12 warps an SM, which is what v's fragments leave room for (4096 rows of 4096 columns,
//          rank 64: 26 us, tensor pipe 48 % busy).
// Warp-level instructions: a block's rows are gathered, which TMA does at 46 ns for four rows, and a rank of 8 to 128 leaves
// tcgen05 nothing to gain from.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "chord_common.cuh"
#include "chord_internal.h"
#include "chord_tcgen05.cuh"
#include "chord_thin.cuh"

namespace chord {
namespace {

// One launch up to these.  One and three launches, us in a graph, rank 16: 256 pairs of 8 adapters 11.5, 16.4; of 16 adapters
// of 8 experts (111 blocks, two rounds of clusters) 28.7, 22.9, but 128 pairs 15.3, 19.4, and the blocks are not known before the launch.
constexpr int kFewPairs = 256;
constexpr int kFewRows = 16, kManyRows = 64;   // rows of a block
constexpr int kThreads = thin::kThreads, kWarps = thin::kWarps;
constexpr int kMaxSplit = 16;
constexpr int64_t kSplitRows = 16384;          // K slices times pairs, at most, where there is more than one slice
constexpr int kMaxPairs = 1 << 30;             // positions in the plan, padded, stay below 2^31
constexpr int kNone = -2;                      // slot of a pair that is not touched; -1: its row of y is base's

struct AdapterArgs {
    const __nv_bfloat16* x;
    int64_t x_stride;
    int div;
    const int32_t* adapter_ids;   // [T]
    const int32_t* topk_ids;      // [T, topk], null: one projection
    int P, topk, S, E;
    const __nv_bfloat16* A;       // [S, E, R, K]
    const __nv_bfloat16* B;       // [S, E, N, rank]
    const float* scale;           // [S], null: 1
    int rank, parts, R, N, K;     // R = parts * rank
    const void* base;
    void* y;
    int64_t base_stride, y_stride;
    int copy;                     // rows without an adapter are copied from base
    int units;                    // items of a block and K slice
    int cluster;                  // CTAs that share an item of the first half, each a part of its K slice
    int max_splits, resident;     // K slices at most; clusters of the first half that run at once
    float* v;                     // [slices, P, R]
    // the plan, for more than kFewPairs pairs
    int32_t* nblocks;             // [4]: blocks, sixteens, blocks without an adapter (the first ones), K slices
    int32_t* block_slot;
    int32_t* block_count;         // rows of each block
    int32_t* rows;                // [blocks, kManyRows]
    int32_t* sixteens;            // up to 16 rows of a block that hold any: 4 block + place
    int* err;
};

__device__ __forceinline__ int slot_of(const AdapterArgs& g, int p, bool report) {
    // The adapter is looked at first, so that a bad one is reported wherever the pair's expert lives.
    const int a = g.adapter_ids[g.topk == 1 ? p : p / g.topk], e = g.topk_ids ? g.topk_ids[p] : 0;
    const bool none = a < 0 || a >= g.S;
    if (none && a != -1 && report) set_error(g.err, CHORD_DEV_BAD_ADAPTER);
    if (e < 0 || e >= g.E) return kNone;
    if (none) return g.copy ? -1 : kNone;
    return a * g.E + e;
}

// ---- blocks of few pairs ------------------------------------------------------
struct FewBlocks {
    alignas(16) int slot[kFewPairs];   // of each pair
    int leader[kFewPairs];             // first pair of each block
    int rank[kFewPairs];               // pairs of the same slot before each
    int counts[kWarps];
    int n;
};

// Every thread of the CTA; thread p is pair p.
__device__ __forceinline__ void find_blocks(const AdapterArgs& g, FewBlocks& f, bool report) {
    const int p = threadIdx.x;
    const int s = p < g.P ? slot_of(g, p, report) : kNone;
    f.slot[p] = s;
    __syncthreads();
    int rank = 0;   // pairs of the same slot before this one
    if (s != kNone) {
        const int4* four = reinterpret_cast<const int4*>(f.slot);
        for (int q = 0; q < p / 4; ++q) {
            const int4 o = four[q];
            rank += (o.x == s) + (o.y == s) + (o.z == s) + (o.w == s);
        }
        for (int q = p & ~3; q < p; ++q) rank += f.slot[q] == s;
    }
    const bool lead = s != kNone && rank % kFewRows == 0;
    const unsigned m = __ballot_sync(0xffffffffu, lead);
    f.rank[p] = rank;
    if ((p & 31) == 0) f.counts[p >> 5] = __popc(m);
    __syncthreads();
    int before = __popc(m & ((1u << (p & 31)) - 1u)), n = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < (p >> 5)) before += f.counts[w];
        n += f.counts[w];
    }
    if (lead) f.leader[before] = p;
    if (p == 0) f.n = n;
    __syncthreads();
}

// The rows of block b (MB entries, -1: none) and its slot, by every thread of the CTA.
template <bool FEW, int MB>
__device__ __forceinline__ int block_rows(const AdapterArgs& g, const FewBlocks* f, int b, int32_t* rows) {
    __syncthreads();
    int slot;
    if constexpr (FEW) {
        const int p = threadIdx.x, lead = f->leader[b];
        slot = f->slot[lead];
        if (p < MB) rows[p] = -1;
        __syncthreads();
        const int at = f->rank[p] - f->rank[lead];
        if (f->slot[p] == slot && at >= 0 && at < MB) rows[at] = p;
    } else {
        slot = g.block_slot[b];
        if (threadIdx.x < MB) rows[threadIdx.x] = threadIdx.x < g.block_count[b] ? g.rows[(int64_t)b * MB + threadIdx.x] : -1;
    }
    __syncthreads();
    return slot;
}

// ---- v = A x --------------------------------------------------------------------
template <int NT>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 3 : 2) adapter_down_kernel(const AdapterArgs g) {
    using Tile = thin::Staged<NT>;
    constexpr int NB = Tile::kCols;
    static_assert(Tile::kRows == kManyRows, "a block of the plan is a tile");
    extern __shared__ __align__(128) uint8_t smem[];   // the tile's ring, then the cluster's shares
    __shared__ int32_t rows[kManyRows];
    pdl_trigger();
    pdl_wait();
    const int rank = g.cluster > 1 ? (int)tc5::cluster_rank() : 0;
    const int first = g.nblocks[2], n = g.nblocks[0] - first, splits = g.nblocks[3], chunks = (g.R + NB - 1) / NB, per = chunks * splits;
    const int steps = (g.K + Tile::kTileCols - 1) / Tile::kTileCols;
    for (int64_t i = blockIdx.x / g.cluster; i < (int64_t)n * per; i += gridDim.x / g.cluster) {
        int q;
        const int b = first + (int)divmod_idx(i, per, q), split = q % splits, r0 = q / splits * NB;
        const int slot = block_rows<false, kManyRows>(g, nullptr, b, rows);
        Tile tile;
        const int row = threadIdx.x >> 3, piece = threadIdx.x & 7;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int p = rows[row + 32 * h], r = row + 32 * h;
            tile.x[h] = p < 0 ? nullptr : g.x + (int64_t)(g.div == 1 ? p : p / g.div) * g.x_stride + piece * 8;
            tile.w[h] = r < NB && r0 + r < g.R ? g.A + ((int64_t)slot * g.R + r0 + r) * g.K + piece * 8 : nullptr;
        }
        const int cut = splits * g.cluster, at = split * g.cluster + rank;
        tile.run(smem, (int)((int64_t)at * steps / cut), (int)((int64_t)(at + 1) * steps / cut), g.K, 1, 0);
        const float* sums = reinterpret_cast<const float*>(smem);
        thin::join_slices<kManyRows * NB>(
            g.cluster, reinterpret_cast<float*>(smem + Tile::kBytes), [&](int u) { return Tile::joined(sums, u); },
            [&](int u, float v) {
                const int p = rows[u / NB], r = r0 + u % NB;
                if (p >= 0 && r < g.R) g.v[((int64_t)split * g.P + p) * g.R + r] = v;
            });
    }
}

// ---- y = base + scale * B v --------------------------------------------------------
// Eight neighbouring numbers of base's or y's type.
template <bool F32>
struct Eight;
template <>
struct Eight<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = a;
        q[1] = b;
    }
    __device__ __forceinline__ void add(const float (&d)[8]) {
        a.x += d[0], a.y += d[1], a.z += d[2], a.w += d[3];
        b.x += d[4], b.y += d[5], b.z += d[6], b.w += d[7];
    }
};
template <>
struct Eight<false> {
    uint4 a;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    }
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = a;
    }
    __device__ __forceinline__ static uint32_t pair(uint32_t o, float d0, float d1) {
        const float2 f = __bfloat1622float2(u32_as_bf2(o));
        return bf2_as_u32(__floats2bfloat162_rn(f.x + d0, f.y + d1));
    }
    __device__ __forceinline__ void add(const float (&d)[8]) {
        a.x = pair(a.x, d[0], d[1]), a.y = pair(a.y, d[2], d[3]);
        a.z = pair(a.z, d[4], d[5]), a.w = pair(a.w, d[6], d[7]);
    }
};

// Two FP32 numbers as three pairs of bf16 numbers of eight significant bits each, cut off towards zero, whose sums
// they are (exactly, down to 2^-110): the upper half of a number is its first part.  An infinity or NaN is the
// first part alone.
__device__ __forceinline__ void split3(float v0, float v1, uint32_t& h0, uint32_t& h1, uint32_t& h2) {
    auto upper = [](float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); };
    auto rest = [](float a) { return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u); };
    h0 = upper(v0, v1);
    v0 = fabsf(v0) <= 3.4028235e38f ? rest(v0) : 0.0f;
    v1 = fabsf(v1) <= 3.4028235e38f ? rest(v1) : 0.0f;
    h1 = upper(v0, v1);
    h2 = upper(rest(v0), rest(v1));
}

// ---- few pairs: one launch ---------------------------------------------------------------
// A cluster of CTAs takes an item (block, part, group of columns): each CTA a slice of K for v (chord_thin.cuh), all
// slices read by each through distributed shared memory and added in rank order, then each its share of
// the columns.  Where there are few blocks, several clusters compute the same v for columns of their own: A
// comes from L2 then, and one launch is what a call of one token costs.  Clusters are of eight CTAs while all
// blocks find one at once, of four beyond (eight and four: one token of rank 16 6.3, 7.2, of rank 64 13.3, 17.2; 64 pairs of 128 slots
// 17.8, 14.8).

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
// The two halves of tc5::cluster_sync.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int kFewCtas, int NT, bool F32>
__global__ void __launch_bounds__(kThreads, 2) adapter_few_kernel(const AdapterArgs g) {
    using Warp = thin::Warp<NT>;
    constexpr int NB = Warp::kCols;
    extern __shared__ __align__(16) float red[];             // [kWarps][16][NB], then v [16][rank] and its fragments
    __shared__ int32_t rows[kFewRows];
    __shared__ FewBlocks few;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
    float* v = red + kWarps * kFewRows * NB;
    uint4* frag = reinterpret_cast<uint4*>(v + kFewRows * g.rank);   // [k steps][3][32]
    pdl_trigger();
    pdl_wait();
    const int cta = (int)tc5::cluster_rank();
    find_blocks(g, few, blockIdx.x == 0);
    const int n = few.n, steps = (g.K + thin::kStep - 1) / thin::kStep, k0 = steps * cta / kFewCtas, k1 = steps * (cta + 1) / kFewCtas;
    const int Np = g.N / g.parts, tiles = (Np + 31) / 32, ksp = (g.rank + 15) / 16;
    const int clusters = (int)gridDim.x / kFewCtas, cluster = (int)blockIdx.x / kFewCtas;
    // groups of columns: clusters that would have nothing take some, as long as every CTA has a tile
    const int groups = max(1, min(clusters / max(n * g.parts, 1), tiles / kFewCtas));
    // column of lane group gr in tile j of a matrix instruction: the eight columns of one lane's results are 8 c ... 8 c + 7
    const int bc = 8 * (gr >> 1) + (gr & 1);
    bool reading = false;
    for (int i = cluster; i < n * g.parts * groups; i += clusters) {
        const int b = i / (g.parts * groups), q = i - b * g.parts * groups, part = q / groups, group = q - part * groups;
        const int slot = block_rows<true, kFewRows>(g, &few, b, rows);
        const int share = group * kFewCtas + cta, shares = groups * kFewCtas;
        const int t0 = (int)((int64_t)tiles * share / shares), t1 = (int)((int64_t)tiles * (share + 1) / shares);
        const __nv_bfloat16* B = g.B + ((int64_t)max(slot, 0) * g.N + part * Np) * g.rank;
        if (slot >= 0) {
            // B on its way to L2 while v is computed
            for (int64_t u = (int64_t)t0 * 32 * g.rank + threadIdx.x * 64, e = (int64_t)min(t1 * 32, Np) * g.rank; u < e; u += kThreads * 64)
                prefetch(B + u);
            if (reading) cluster_wait();   // the slices of the item before have been read
            for (int r0 = 0; r0 < g.rank; r0 += NB) {
                Warp w;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int p = rows[j * 8 + gr] < 0 ? rows[0] : rows[j * 8 + gr];
                    w.x[j] = reinterpret_cast<const uint4*>(g.x + (int64_t)(g.div == 1 ? p : p / g.div) * g.x_stride) + c;
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    w.w[j] = reinterpret_cast<const uint4*>(g.A + ((int64_t)slot * g.R + part * g.rank + min(r0 + j * 8 + gr, g.rank - 1)) * g.K) + c;
                w.run(k0 + warp, k1, g.K / 8, red + warp * kFewRows * NB, false);
                __syncthreads();
                for (int u = threadIdx.x; u < kFewRows * NB; u += kThreads)
                    if (r0 + u % NB < g.rank) v[u / NB * g.rank + r0 + u % NB] = thin::joined(red, kFewRows * NB, u);
                __syncthreads();
            }
            tc5::cluster_sync();
            // v as the fragments of the instruction's A side: lane (g, c) has rows g and g + 8, of each k
            // step the four columns 4 c ... (B's side likewise)
            const float scale = g.scale ? g.scale[slot / g.E] : 1.0f;
            for (int u = threadIdx.x; u < ksp * 32; u += kThreads) {
                const int l = u & 31, s = u >> 5, k = 16 * s + 4 * (l & 3);
                uint32_t r[3][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 f = make_float4(0, 0, 0, 0);
                    if (rows[h * 8 + (l >> 2)] >= 0 && k < g.rank) {
                        const uint32_t at = smem_u32(v + (h * 8 + (l >> 2)) * g.rank + k);
                        float4 o[kFewCtas];
#pragma unroll
                        for (int z = 0; z < kFewCtas; ++z) o[z] = ld_cluster4(tc5::at_cta(at, (uint32_t)z));
#pragma unroll
                        for (int z = 0; z < kFewCtas; ++z) f.x += o[z].x, f.y += o[z].y, f.z += o[z].z, f.w += o[z].w;
                    }
                    split3(f.x * scale, f.y * scale, r[0][h], r[1][h], r[2][h]);
                    split3(f.z * scale, f.w * scale, r[0][2 + h], r[1][2 + h], r[2][2 + h]);
                }
#pragma unroll
                for (int t = 0; t < 3; ++t) frag[(s * 3 + t) * 32 + l] = make_uint4(r[t][0], r[t][1], r[t][2], r[t][3]);
            }
            __syncthreads();
            cluster_arrive();   // waited for where v is written next, or the kernel ends
            reading = true;
        }
        int64_t from[2], to[2];
        bool live[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int p = rows[j * 8 + gr];
            live[j] = p >= 0;
            from[j] = p * g.base_stride + part * Np + 8 * c;
            to[j] = p * g.y_stride + part * Np + 8 * c;
        }
        for (int t = t0 + warp; t < t1; t += kWarps) {
            const int n0 = t * 32;
            const bool in = 8 * c < Np - n0;
            Eight<F32> o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (in && live[j]) o[j].load(g.base, from[j] + n0);
            if (slot >= 0) {
                const __nv_bfloat16* bt[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) bt[j] = B + (int64_t)(n0 + bc + 2 * j) * g.rank + 4 * c;
                const bool bin = bc < Np - n0;
                float d[4][4] = {};
#pragma unroll 4
                for (int s = 0; s < ksp; ++s) {
                    uint2 w[4];
                    const bool kin = bin && 16 * s + 4 * c < g.rank;
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = kin ? *reinterpret_cast<const uint2*>(bt[j] + 16 * s) : make_uint2(0, 0);
#pragma unroll
                    for (int t3 = 2; t3 >= 0; --t3) {
                        const uint4 a = frag[(s * 3 + t3) * 32 + lane];
#pragma unroll
                        for (int j = 0; j < 4; ++j) thin::mma(d[j], a.x, a.y, a.z, a.w, w[j].x, w[j].y);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float e[8];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        e[2 * u] = d[u][j * 2];
                        e[2 * u + 1] = d[u][j * 2 + 1];
                    }
                    o[j].add(e);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (in && live[j]) o[j].store(g.y, to[j] + n0);
        }
    }
    if (reading) cluster_wait();   // nobody reads this CTA's v any more
}

// Many pairs.  A warp has 16 rows of a block, its rows of v in registers as fragments of the instruction's A side (KS k
// steps of 16), and takes 32 columns at a time, base's pieces of the next tile on their way in registers.
// Row i of the instruction's 8-column tile j is this one of the 32 columns, so that lane (g, c) ends with whole
// 16-byte pieces of its rows: bf16 columns 8 c .. 8 c + 7, FP32 columns 4 c .. 4 c + 3 and 16 more.
template <bool F32>
__device__ __forceinline__ int column_of(int j, int i) {
    return F32 ? 16 * (j >> 1) + 4 * (i >> 1) + 2 * (j & 1) + (i & 1) : 8 * (i >> 1) + 2 * j + (i & 1);
}

constexpr int kUpThreads = 128;

template <int KS, bool F32>
struct UpRows {
    using Out = typename std::conditional<F32, float, __nv_bfloat16>::type;
    static constexpr int kY = F32 ? 2 : 1, kFirst = F32 ? 4 : 8;   // 16-byte pieces of a row that a lane has; elements of one
    struct Y {
        uint4 y[2][kY];
    };
    uint32_t a[KS][3][4];
    const Out* from[2];
    Out* to[2];
    bool live[2], adds;

    // Rows p[0] and p[1] of y (-1: not there, reads row `other` and writes nothing) in this part's columns.
    __device__ __forceinline__ void begin(const AdapterArgs& g, const int (&p)[2], int other, int slot, int part, int Np, int splits) {
        const int c = threadIdx.x & 3;
        adds = slot >= 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            live[h] = p[h] >= 0;
            const int q = live[h] ? p[h] : other;
            from[h] = static_cast<const Out*>(g.base) + q * g.base_stride + part * Np + kFirst * c;
            to[h] = static_cast<Out*>(g.y) + q * g.y_stride + part * Np + kFirst * c;
        }
        if (!adds) return;
        // v: slices added in order, scaled, in three parts; of each k step the columns 2 c, 2 c + 1 and 8 more.  All of a
        // slice's loads are in flight together.
        const float scale = g.scale ? g.scale[slot / g.E] : 1.0f;
        float2 f[KS][2][2] = {};
        const float* v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) v[h] = g.v + (int64_t)(live[h] ? p[h] : other) * g.R + part * g.rank + 2 * c;
        for (int z = 0; z < splits; ++z) {
            float2 o[KS][2][2];
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < 2; ++u)   // no branch: what is not there is read elsewhere and left out
                        o[s][h][u] = *reinterpret_cast<const float2*>(v[h] + (16 * s + 8 * u < g.rank ? 16 * s + 8 * u : 0));
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const bool in = live[h] && 16 * s + 8 * u < g.rank;
                        f[s][h][u].x += in ? o[s][h][u].x : 0.0f;
                        f[s][h][u].y += in ? o[s][h][u].y : 0.0f;
                    }
            v[0] += (int64_t)g.P * g.R;
            v[1] += (int64_t)g.P * g.R;
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    split3(f[s][h][u].x * scale, f[s][h][u].y * scale, a[s][0][2 * u + h], a[s][1][2 * u + h], a[s][2][2 * u + h]);
    }
    __device__ __forceinline__ void load(Y& x, int n0, int Np) const {
        const int c = threadIdx.x & 3;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int z = 0; z < kY; ++z)
                if (n0 + z * 16 + kFirst * c < Np) x.y[h][z] = *reinterpret_cast<const uint4*>(from[h] + n0 + z * 16);
    }
    // One k step; instructions on one accumulator are four apart.
    __device__ __forceinline__ void multiply(float (&d)[4][4], int s, const uint32_t (&w)[4][2]) const {
#pragma unroll
        for (int t3 = 2; t3 >= 0; --t3)
#pragma unroll
            for (int j = 0; j < 4; ++j) thin::mma(d[j], a[s][t3][0], a[s][t3][1], a[s][t3][2], a[s][t3][3], w[j][0], w[j][1]);
    }
    __device__ __forceinline__ void store(const Y& x, const float (&d)[4][4], int n0, int Np) const {
        const int c = threadIdx.x & 3;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int z = 0; z < kY; ++z) {
                if (!live[h] || n0 + z * 16 + kFirst * c >= Np) continue;
                uint4 o = x.y[h][z];
                if (adds) {
                    if constexpr (F32) {
                        o.x = __float_as_uint(__uint_as_float(o.x) + d[2 * z][2 * h]);
                        o.y = __float_as_uint(__uint_as_float(o.y) + d[2 * z][2 * h + 1]);
                        o.z = __float_as_uint(__uint_as_float(o.z) + d[2 * z + 1][2 * h]);
                        o.w = __float_as_uint(__uint_as_float(o.w) + d[2 * z + 1][2 * h + 1]);
                    } else {
                        o.x = Eight<false>::pair(o.x, d[0][2 * h], d[0][2 * h + 1]);
                        o.y = Eight<false>::pair(o.y, d[1][2 * h], d[1][2 * h + 1]);
                        o.z = Eight<false>::pair(o.z, d[2][2 * h], d[2][2 * h + 1]);
                        o.w = Eight<false>::pair(o.w, d[3][2 * h], d[3][2 * h + 1]);
                    }
                }
                *reinterpret_cast<uint4*>(to[h] + n0 + z * 16) = o;
            }
    }
};

// Ranks up to 16: the work of all rows, sixteen at a time, is dealt to the warps in equal ranges (blocks hold 1 to 64
// rows), B's pieces come straight from global memory a tile ahead, nothing is shared and no warp waits for another.  (8192
// pairs of rank 16, whole calls, with this kernel and with the next: FP32 126, 149; bf16 the same.)
template <bool F32>
__global__ void __launch_bounds__(kUpThreads, 4) adapter_up_small_kernel(const AdapterArgs g) {
    using Rows = UpRows<1, F32>;
    const int lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
    pdl_wait();
    const int splits = g.nblocks[3];
    const int Np = g.N / g.parts, tiles = (Np + 31) / 32;
    const int64_t total = (int64_t)g.nblocks[1] * g.parts * tiles, warps = (int64_t)gridDim.x * (kUpThreads / 32);
    const int64_t warp = (int64_t)blockIdx.x * (kUpThreads / 32) + (threadIdx.x >> 5), end = total * (warp + 1) / warps;
    for (int64_t at = total * warp / warps; at < end;) {
        int t0, part;
        const int u = (int)divmod_idx(divmod_idx(at, tiles, t0), g.parts, part), t1 = (int)min((int64_t)tiles, t0 + (end - at));
        at += t1 - t0;
        const int where = g.sixteens[u], b = where >> 2, r0 = (where & 3) * 16, count = g.block_count[b], slot = g.block_slot[b];
        const int32_t* rows = g.rows + (int64_t)b * kManyRows + r0;
        const int p[2] = {r0 + gr < count ? rows[gr] : -1, r0 + gr + 8 < count ? rows[gr + 8] : -1};
        struct Tile {
            typename Rows::Y y;
            uint32_t w[4][2];
        } x, y;
        Rows r;
        const __nv_bfloat16* bw = g.B + ((int64_t)max(slot, 0) * g.N + part * Np) * g.rank + 2 * c;
        auto load = [&](Tile& z, int t) {
            r.load(z.y, t * 32, Np);
            if (slot < 0) return;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = t * 32 + column_of<F32>(j, gr);
                const __nv_bfloat16* from = bw + (int64_t)col * g.rank;
                z.w[j][0] = col < Np ? *reinterpret_cast<const uint32_t*>(from) : 0u;
                z.w[j][1] = col < Np && g.rank > 8 ? *reinterpret_cast<const uint32_t*>(from + 8) : 0u;
            }
        };
        auto finish = [&](Tile& z, int t) {
            float d[4][4] = {};
            if (slot >= 0) r.multiply(d, 0, z.w);
            r.store(z.y, d, t * 32, Np);
        };
        r.begin(g, p, rows[0], slot, part, Np, splits);
        load(x, t0);
        for (int t = t0; t < t1; t += 2) {
            if (t + 1 < t1) load(y, t + 1);
            finish(x, t);
            if (t + 1 >= t1) break;
            if (t + 2 < t1) load(x, t + 2);
            finish(y, t + 1);
        }
    }
}

// Larger ranks: B's bytes and the instructions weigh as much as base and y, so the four warps of a CTA take the rows of a
// block and share B, 128 columns a stage, that cp.async copies two stages ahead.
template <int KS>
struct UpStage {
    static constexpr int kCols = 128, kStages = 3;
    static constexpr int kPitch = KS * 32 + 16;                 // padded: neighbouring rows lie in other banks
    static constexpr int kBytes = kCols * kPitch;
    static constexpr int kPieces = kCols * KS * 2 / kUpThreads; // 16-byte pieces a thread copies
};

template <int KS, bool F32>
__global__ void __launch_bounds__(kUpThreads, KS <= 4 ? 3 : 2) adapter_up_kernel(const AdapterArgs g) {
    using T = UpStage<KS>;
    using Rows = UpRows<KS, F32>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int32_t rows[kManyRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2;
    pdl_wait();
    const int n = g.nblocks[0], splits = g.nblocks[3];
    const int Np = g.N / g.parts, chunks = (Np + T::kCols - 1) / T::kCols;
    const uint32_t base = smem_u32(smem);
    // Columns are stored in the order of the instruction's rows.  ldmatrix: matrix j of two 8-column tiles is k half j & 1
    // of tile j >> 1.
    const uint32_t b_at = (uint32_t)(((lane >> 4) * 8 + (lane & 7)) * T::kPitch + ((lane >> 3) & 1) * 16);
    int b_col[T::kPieces], b_to[T::kPieces];
#pragma unroll
    for (int h = 0; h < T::kPieces; ++h) {
        const int u = threadIdx.x + h * kUpThreads, row = u / (g.rank / 8), k = u - row * (g.rank / 8);
        b_col[h] = row < T::kCols ? row : INT32_MAX;
        const int w = row & 31;   // column w of 32 is row i of tile j
        const int j = F32 ? (w >> 4) * 2 + (w >> 1 & 1) : w >> 1 & 3, i = F32 ? (w >> 2 & 3) * 2 + (w & 1) : (w >> 3) * 2 + (w & 1);
        b_to[h] = ((row & ~31) + j * 8 + i) * T::kPitch + k * 16;
    }
    const int64_t total = (int64_t)n * g.parts * chunks, end = total * (blockIdx.x + 1) / gridDim.x;
    for (int64_t at = total * blockIdx.x / gridDim.x; at < end;) {
        int c0, part;
        const int b = (int)divmod_idx(divmod_idx(at, chunks, c0), g.parts, part), c1 = (int)min((int64_t)chunks, c0 + (end - at));
        at += c1 - c0;
        const int slot = block_rows<false, kManyRows>(g, nullptr, b, rows);
        const __nv_bfloat16* src = g.B + ((int64_t)max(slot, 0) * g.N + part * Np) * g.rank + threadIdx.x * 8;
        int next = c0, slot_in = 0, slot_out = 0;
        auto issue = [&]() {
            if (next < c1 && slot >= 0) {
                const int n0 = next * T::kCols;
                const uint32_t st = base + (uint32_t)(slot_in * T::kBytes);
#pragma unroll
                for (int h = 0; h < T::kPieces; ++h)
                    if (b_col[h] < Np - n0) cp_async16(st + (uint32_t)b_to[h], src + (int64_t)n0 * g.rank + h * kUpThreads * 8);
            }
            ++next;
            cp_async_commit();
            if (++slot_in == T::kStages) slot_in = 0;
        };
        // a rank that ends inside a k step: zeros behind it, in every stage
        if (g.rank % 16)
            for (int u = threadIdx.x; u < T::kStages * T::kCols; u += kUpThreads)
                *reinterpret_cast<uint4*>(smem + u * T::kPitch + g.rank * 2) = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < T::kStages - 1; ++k) issue();
        const int r0 = warp * 16, p[2] = {rows[r0 + gr], rows[r0 + gr + 8]};
        const bool busy = rows[r0] >= 0;   // rows of a block are a prefix
        Rows r;
        typename Rows::Y y[2];
        if (busy) {
            r.begin(g, p, rows[r0], slot, part, Np, splits);
            r.load(y[0], c0 * T::kCols, Np);
        }
        for (int ch = c0; ch < c1; ++ch) {
            cp_async_wait<T::kStages - 2>();
            __syncthreads();   // the stage is there for all, and the one before has been read by all
            issue();
            const uint32_t st = base + (uint32_t)(slot_out * T::kBytes) + b_at;
            if (++slot_out == T::kStages) slot_out = 0;
            if (!busy) continue;
            const int end_col = min(Np, (ch + 1) * T::kCols);
#pragma unroll
            for (int q = 0; q < T::kCols / 32; ++q) {
                const int n0 = ch * T::kCols + q * 32;
                if (n0 >= end_col) break;
                if (n0 + 32 < Np && (ch + 1 < c1 || q + 1 < T::kCols / 32)) r.load(y[(q + 1) & 1], n0 + 32, Np);
                float d[4][4] = {};
                if (slot >= 0) {
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        if (16 * s >= g.rank) break;
                        uint32_t w[2][4];
                        thin::ldsm4(w[0], st + (uint32_t)(q * 32 * T::kPitch + s * 32));
                        thin::ldsm4(w[1], st + (uint32_t)((q * 32 + 16) * T::kPitch + s * 32));
                        const uint32_t v[4][2] = {{w[0][0], w[0][1]}, {w[0][2], w[0][3]}, {w[1][0], w[1][1]}, {w[1][2], w[1][3]}};
                        r.multiply(d, s, v);
                    }
                }
                r.store(y[q & 1], d, n0, Np);
            }
        }
        cp_async_wait<0>();
    }
}

// ---- the plan ------------------------------------------------------------------------
// A counting sort of the pairs by slot (index slot + 1, so that rows without an adapter come first).
// Which of a slot's pairs come first depends on timing; what a row of y becomes does not.
struct PlanArgs {
    AdapterArgs g;
    int nslots;        // S * E + 1
    int32_t* counts;   // [nslots], then the next free position of each
};

constexpr int kPlanThreads = 1024;
// A cluster of kPlanCtas CTAs plans up to these, as many as its threads hold; beyond, three kernels over the GPU (a call of 512
// pairs 12.3 us with the one, 18.5 with the three; of 16384 19.5, 27.4).
constexpr int kPlanCtas = 8, kPlanPerThread = 2, kPlanPairs = kPlanCtas * kPlanPerThread * kPlanThreads, kPlanSlots = 16384;

// Exclusive sum over the threads of the CTA; every thread gets the total too.
__device__ __forceinline__ int block_scan(int v, int& total) {
    __shared__ int sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        sums[lane] = s;
    }
    __syncthreads();
    total = sums[31];
    return x - v + (warp ? sums[warp - 1] : 0);
}

// The n pairs of a slot: blocks from b on, sixteens from u on.
__device__ __forceinline__ void lay_out(const AdapterArgs& g, int slot, int n, int& b, int& u) {
    for (int k = 0; k < n; k += kManyRows, ++b) {
        const int here = min(n - k, kManyRows);
        g.block_slot[b] = slot;
        g.block_count[b] = here;
        for (int j = 0; j < here; j += 16) g.sixteens[u++] = 4 * b + j / 16;
    }
}
__device__ __forceinline__ int blocks_for(int n) { return (n + kManyRows - 1) / kManyRows; }
// n / 64 full blocks of four sixteens and the rest's
__device__ __forceinline__ int sixteens_for(int n) { return (n + 15) / 16; }

// K slices of the first half for so many blocks, by a whole warp: the fewest rounds of clusters times what a round takes, its
// stages and about five more to fill the ring and to add the sums up, and one for a slice, which the second half reads.  (As many slices as
// make an item for every CTA, whatever is left for a second round: 4096 rows of 8 adapters, K 4096, rank 128, 76 us for 70; 4096 pairs
// of 64 experts, K 7168, rank 16, 103 for 95.)
__device__ __forceinline__ int slices_for(const AdapterArgs& g, int blocks) {
    const int s = (threadIdx.x & 31) + 1, steps = (g.K + thin::Staged<8>::kTileCols - 1) / thin::Staged<8>::kTileCols;
    if (g.max_splits == 1) return 1;   // more than one only where all of this fits 32 bits
    const int rounds = (blocks * g.units * s + g.resident - 1) / g.resident, cut = s * g.cluster;
    const unsigned cost = s <= g.max_splits ? (unsigned)(rounds * ((steps + cut - 1) / cut + 5) + s) : 0xffffffffu, least = __reduce_min_sync(0xffffffffu, cost);
    return __ffs(__ballot_sync(0xffffffffu, cost == least));
}

// Counts to first positions; the blocks and sixteens.
__device__ __forceinline__ void plan_scan(const PlanArgs& a, int32_t* counts) {
    const int per = (a.nslots + kPlanThreads - 1) / kPlanThreads;
    const int s0 = threadIdx.x * per, s1 = min(s0 + per, a.nslots);
    const int none = blocks_for(counts[0]);   // read by all before anyone's positions overwrite it
    int blocks = 0, sixteens = 0, total_b, total_u;
    for (int s = s0; s < s1; ++s) {
        blocks += blocks_for(counts[s]);
        sixteens += sixteens_for(counts[s]);
    }
    int b = block_scan(blocks, total_b);
    __syncthreads();
    int u = block_scan(sixteens, total_u);
    for (int s = s0; s < s1; ++s) {
        const int n = counts[s];
        counts[s] = b * kManyRows;
        lay_out(a.g, s - 1, n, b, u);
    }
    if (threadIdx.x < 32) {
        const int splits = slices_for(a.g, total_b - none);
        if (threadIdx.x == 0) {
            a.g.nblocks[0] = total_b;
            a.g.nblocks[1] = total_u;
            a.g.nblocks[2] = none;
            a.g.nblocks[3] = splits;
        }
    }
}

// This pair's place among those of its slot; the lanes of a warp with one slot for all (the tokens of a
// prompt) make one addition.  A pair of kNone takes no part.
__device__ __forceinline__ int take_place(int32_t* counts, int slot) {
    const int lane = threadIdx.x & 31;
    if (__all_sync(0xffffffffu, slot == __shfl_sync(0xffffffffu, slot, 0))) {
        if (slot == kNone) return 0;
        int base = 0;
        if (lane == 0) base = atomicAdd(&counts[slot + 1], 32);
        return __shfl_sync(0xffffffffu, base, 0) + lane;
    }
    return slot == kNone ? 0 : atomicAdd(&counts[slot + 1], 1);
}

__device__ __forceinline__ int32_t ld_cluster(uint32_t addr) {
    int32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Each CTA counts its share of the pairs; each then takes a share of the slots, adds up the CTAs'
// counts, and hands every CTA the position of its first pair of each slot.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads) adapter_plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t counts_s[];
    __shared__ int32_t before[kPlanCtas];   // blocks of each CTA's slots, and sixteens in the upper half (below 2^15 both)
    __shared__ int32_t none;                // blocks of rows without an adapter, in the first CTA
    pdl_trigger();
    const int rank = (int)tc5::cluster_rank();
    int slot[kPlanPerThread], place[kPlanPerThread];
#pragma unroll
    for (int i = 0; i < kPlanPerThread; ++i) {
        const int p = (i * kPlanCtas + rank) * kPlanThreads + threadIdx.x;
        slot[i] = p < a.g.P ? slot_of(a.g, p, true) : kNone;
    }
    for (int s = threadIdx.x; s < a.nslots; s += kPlanThreads) counts_s[s] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPlanPerThread; ++i) place[i] = take_place(counts_s, slot[i]);
    tc5::cluster_sync();
    const int share = (a.nslots + kPlanCtas - 1) / kPlanCtas, per = (share + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(rank * share + (int)threadIdx.x * per, a.nslots), s1 = min(min(s0 + per, (rank + 1) * share), a.nslots);
    auto counts_of = [&](int cta, int s) { return tc5::at_cta(smem_u32(counts_s + s), (uint32_t)cta); };
    int mine = 0, total;
    for (int s = s0; s < s1; ++s) {
        int n = 0;
#pragma unroll
        for (int z = 0; z < kPlanCtas; ++z) n += ld_cluster(counts_of(z, s));
        mine += blocks_for(n) + (sixteens_for(n) << 16);
        if (s == 0) none = blocks_for(n);
    }
    int first = block_scan(mine, total);
    if (threadIdx.x < kPlanCtas) st_cluster(tc5::at_cta(smem_u32(before + rank), threadIdx.x), total);
    tc5::cluster_sync();
    int all = 0;
    for (int z = 0; z < kPlanCtas; ++z) {
        if (z < rank) first += before[z];
        all += before[z];
    }
    if (rank == 0 && threadIdx.x >= kPlanThreads - 32) {   // the last slots' warp has the least to lay out
        const int splits = slices_for(a.g, (all & 0xffff) - none);
        if (threadIdx.x == kPlanThreads - 1) {
            a.g.nblocks[0] = all & 0xffff;
            a.g.nblocks[1] = all >> 16;
            a.g.nblocks[2] = none;
            a.g.nblocks[3] = splits;
        }
    }
    int b = first & 0xffff, u = first >> 16;
    for (int s = s0; s < s1; ++s) {
        int n = 0;
#pragma unroll
        for (int z = 0; z < kPlanCtas; ++z) {
            const uint32_t at = counts_of(z, s);
            const int here = ld_cluster(at);
            st_cluster(at, b * kManyRows + n);
            n += here;
        }
        lay_out(a.g, s - 1, n, b, u);
    }
    tc5::cluster_sync();
#pragma unroll
    for (int i = 0; i < kPlanPerThread; ++i)
        if (slot[i] != kNone) a.g.rows[counts_s[slot[i] + 1] + place[i]] = (i * kPlanCtas + rank) * kPlanThreads + threadIdx.x;
}

__global__ void __launch_bounds__(256) adapter_count_kernel(const PlanArgs a) {
    for (int64_t p0 = (int64_t)blockIdx.x * 256; p0 < a.g.P; p0 += (int64_t)gridDim.x * 256) {
        const int64_t p = p0 + threadIdx.x;
        take_place(a.counts, p < a.g.P ? slot_of(a.g, (int)p, true) : kNone);
    }
}
__global__ void __launch_bounds__(kPlanThreads) adapter_scan_kernel(const PlanArgs a) { plan_scan(a, a.counts); }
__global__ void __launch_bounds__(256) adapter_place_kernel(const PlanArgs a) {
    for (int64_t p0 = (int64_t)blockIdx.x * 256; p0 < a.g.P; p0 += (int64_t)gridDim.x * 256) {
        const int64_t p = p0 + threadIdx.x;
        const int s = p < a.g.P ? slot_of(a.g, (int)p, false) : kNone;
        const int at = take_place(a.counts, s);
        if (s != kNone) a.g.rows[at] = (int32_t)p;
    }
}

// ---- host ---------------------------------------------------------------------------------
struct Layout {
    int max_splits;
    int64_t blocks;   // at most
    size_t v, nblocks, block_slot, block_count, rows, sixteens, counts, bytes;
};

Layout layout_of(int64_t P, int64_t slots, int R) {
    Layout l{};
    const bool few = P <= kFewPairs;   // needs no workspace
    const int64_t mb = few ? kFewRows : kManyRows;
    l.blocks = P / mb + (P < slots + 1 ? P : slots + 1) + 1;
    const int64_t s = P > 0 ? kSplitRows / P : 1;
    l.max_splits = (int)(s > kMaxSplit ? kMaxSplit : s < 1 ? 1 : s);
    auto take = [&](size_t n) {
        const size_t at = l.bytes;
        l.bytes += (n + 255) / 256 * 256;
        return at;
    };
    if (!few) {
        // Room for what a smaller call may take too, whose slices are more (16384 / P of them, at most 16): the largest
        // batch's workspace is enough for every other.
        const int64_t rows = kMaxSplit * P < kSplitRows ? kMaxSplit * P : kSplitRows;
        l.v = take((size_t)(rows > P ? rows : P) * R * 4);
        l.nblocks = take(16);
        l.block_slot = take((size_t)l.blocks * 4);
        l.block_count = take((size_t)l.blocks * 4);
        l.rows = take((size_t)l.blocks * kManyRows * 4);
        l.sixteens = take((size_t)(l.blocks + P / 16) * 4);
        l.counts = take((size_t)(slots + 1) * 4);
    }
    return l;
}

// Rows of A that an item of the first half takes.
int down_cols(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : R <= 32 ? 32 : 64; }

struct DownKernel {
    void (*kern)(AdapterArgs);
    size_t smem;
    int ctas;   // to an SM
};

template <int NT>
DownKernel down_kernel_as() {
    return {adapter_down_kernel<NT>, thin::Staged<NT>::kBytes + kManyRows * NT * 8 * 4, 0};
}

cudaError_t down_kernel(int R, DownKernel& k) {
    const int cols = down_cols(R);
    k = cols == 8 ? down_kernel_as<1>() : cols == 16 ? down_kernel_as<2>() : cols == 32 ? down_kernel_as<4>() : down_kernel_as<8>();
    return kernel_ctas_per_sm(reinterpret_cast<const void*>(k.kern), kThreads, k.smem, k.smem, &k.ctas);
}

cudaError_t launch_down(const AdapterArgs& g, const DownKernel& k, int64_t blocks, cudaStream_t st) {
    const int64_t items = blocks * g.units * g.max_splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items < g.resident ? items : g.resident) * g.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = k.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (g.cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)g.cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl_for(g.P)) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, k.kern, g);
}

template <int CTAS, int NT, bool F32>
cudaError_t launch_few_as(const AdapterArgs& g, int64_t blocks, cudaStream_t st) {
    auto* kern = adapter_few_kernel<CTAS, NT, F32>;
    const size_t smem = ((size_t)kWarps * kFewRows * NT * 8 + (size_t)kFewRows * g.rank) * 4 + (size_t)((g.rank + 15) / 16) * 3 * 512;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), 64 * 1024);   // at most 52 KB
    if (e != cudaSuccess) return e;
    // clusters for the blocks' parts, or to share the columns of few; two CTAs to an SM
    const int tiles = (g.N / g.parts + 31) / 32, most = 2 * device_info().sm_count / CTAS;
    const int64_t want = blocks * g.parts * ((tiles + CTAS - 1) / CTAS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((want < most ? want : most) * CTAS));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CTAS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, g);
}

template <int CTAS, bool F32>
cudaError_t launch_few_of(const AdapterArgs& g, int64_t blocks, cudaStream_t st) {
    switch (down_cols(g.rank)) {
        case 8: return launch_few_as<CTAS, 1, F32>(g, blocks, st);
        case 16: return launch_few_as<CTAS, 2, F32>(g, blocks, st);
        case 32: return launch_few_as<CTAS, 4, F32>(g, blocks, st);
        default: return launch_few_as<CTAS, 8, F32>(g, blocks, st);
    }
}

template <bool F32>
cudaError_t launch_few(const AdapterArgs& g, int64_t blocks, cudaStream_t st) {
    return blocks * g.parts * 8 <= 2 * device_info().sm_count ? launch_few_of<8, F32>(g, blocks, st) : launch_few_of<4, F32>(g, blocks, st);
}

cudaError_t launch_up_as(void (*kern)(AdapterArgs), const AdapterArgs& g, size_t smem, cudaStream_t st) {
    int ctas = 0;
    cudaError_t e = kernel_ctas_per_sm(reinterpret_cast<const void*>(kern), kUpThreads, smem, smem, &ctas);
    if (e != cudaSuccess) return e;
    return launch_pdl(pdl_for(g.P), kern, dim3((unsigned)(device_info().sm_count * ctas)), dim3(kUpThreads), smem, st, g);
}

template <bool F32>
cudaError_t launch_up(const AdapterArgs& g, cudaStream_t st) {
    if (g.rank <= 16) return launch_up_as(adapter_up_small_kernel<F32>, g, 0, st);
    if (g.rank <= 32) return launch_up_as(adapter_up_kernel<2, F32>, g, UpStage<2>::kStages * UpStage<2>::kBytes, st);
    if (g.rank <= 64) return launch_up_as(adapter_up_kernel<4, F32>, g, UpStage<4>::kStages * UpStage<4>::kBytes, st);
    return launch_up_as(adapter_up_kernel<8, F32>, g, UpStage<8>::kStages * UpStage<8>::kBytes, st);
}

cudaError_t launch_plan(const AdapterArgs& g, int64_t slots, int32_t* counts, cudaStream_t st) {
    PlanArgs a{g, (int)slots + 1, counts};
    if (g.P <= kPlanPairs && slots < kPlanSlots) {
        const size_t smem = (size_t)a.nslots * 4;
        cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(adapter_plan_kernel), (size_t)kPlanSlots * 4);
        if (e != cudaSuccess) return e;
        adapter_plan_kernel<<<kPlanCtas, kPlanThreads, smem, st>>>(a);
        return cudaGetLastError();
    }
    cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)a.nslots * 4, st);
    if (e != cudaSuccess) return e;
    const int64_t blocks = ceil_div64(g.P, 256), most = 8 * (int64_t)device_info().sm_count;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    adapter_count_kernel<<<grid, 256, 0, st>>>(a);
    adapter_scan_kernel<<<1, kPlanThreads, 0, st>>>(a);
    adapter_place_kernel<<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// n rows of `width` bytes, `pitch` apart (at least a width).
struct Rows2D {
    const void* at;
    int64_t n, pitch, width;
};

// The rows have a byte in common.  Rows of the same distance may lie between one another, columns of one buffer; of
// different distances, the ranges from first to last byte decide.
bool overlap(const Rows2D& a, const Rows2D& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    if (x >= y + (uintptr_t)((b.n - 1) * b.pitch + b.width) || y >= x + (uintptr_t)((a.n - 1) * a.pitch + a.width)) return false;
    if (a.n > 1 && b.n > 1 && a.pitch != b.pitch) return true;
    // a single row meets the other ones as any of their distance would
    const int64_t pitch = a.n > 1 ? a.pitch : b.pitch, d = (int64_t)(y - x) % pitch, off = d < 0 ? d + pitch : d;   // of b's rows behind a's
    return off < a.width || off + b.width > pitch;
}

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

size_t chord_adapter_workspace_bytes(int64_t T, int topk, int adapters, int E, int rank, int parts) {
    if (T < 0 || topk <= 0 || adapters <= 0 || E <= 0 || rank <= 0 || parts <= 0 || rank > 128 || parts > 4) return 0;
    if (T > (kMaxPairs - 1) / topk || adapters > 65536 / E) return 0;
    const size_t bytes = layout_of(T * topk, (int64_t)adapters * E, rank * parts).bytes;
    return bytes ? bytes : 256;
}

chord_status chord_adapter_add(const void* x, int64_t x_rows, int64_t x_stride, int a_row_divisor, const int32_t* adapter_ids,
                               const int32_t* topk_ids, int T, int topk, int adapters, int E, const void* A, const void* B,
                               const float* scale, int rank, int parts, int N, int K, const void* base, int64_t base_stride,
                               void* y, int64_t y_stride, int y_dtype, void* workspace, size_t workspace_bytes,
                               const chord_opts* opts, void* stream) {
    if (T < 0 || topk <= 0 || adapters <= 0 || E <= 0 || rank <= 0 || parts <= 0 || N <= 0 || K <= 0 || a_row_divisor <= 0 ||
        x_rows < 0 || (y_dtype != CHORD_DTYPE_BF16 && y_dtype != CHORD_DTYPE_F32))
        return CHORD_ERR_INVALID_ARG;
    const int64_t P = (int64_t)T * topk;
    const int per = y_dtype == CHORD_DTYPE_F32 ? 4 : 8;
    if (P >= kMaxPairs || adapters > 65536 / E || rank % 8 || rank > 128 || parts > 4 || N % (8 * parts) || K % 8)
        return CHORD_ERR_UNSUPPORTED;
    if (!topk_ids && E != 1) return CHORD_ERR_INVALID_ARG;
    if (P == 0) return CHORD_OK;
    if ((P - 1) / a_row_divisor >= x_rows) return CHORD_ERR_INVALID_ARG;
    // the stride of a single row is not used
    if (P <= a_row_divisor) x_stride = K;
    if (P == 1) base_stride = y_stride = N;
    if (x_stride < K || base_stride < N || y_stride < N) return CHORD_ERR_INVALID_ARG;
    if (x_stride % 8 || base_stride % per || y_stride % per) return CHORD_ERR_UNSUPPORTED;
    if (!x || !aligned16(x) || !adapter_ids || !A || !aligned16(A) || !B || !aligned16(B) || !base || !aligned16(base) || !y ||
        !aligned16(y) || !workspace || !aligned16(workspace))
        return CHORD_ERR_INVALID_ARG;
    const int64_t esize = 16 / per;
    const Rows2D xs{x, (P - 1) / a_row_divisor + 1, x_stride * 2, (int64_t)K * 2}, bases{base, P, base_stride * esize, N * esize},
        ys{y, P, y_stride * esize, N * esize};
    if (overlap(ys, xs) || (base == y ? base_stride != y_stride : overlap(ys, bases))) return CHORD_ERR_INVALID_ARG;
    if (workspace_bytes < chord_adapter_workspace_bytes(T, topk, adapters, E, rank, parts)) return CHORD_ERR_BUFFER_TOO_SMALL;
    const DeviceInfo& di = device_info();
    if (!di.err) return CHORD_ERR_CUDA;
    const int64_t slots = (int64_t)adapters * E;
    const bool few = P <= kFewPairs, f32 = y_dtype == CHORD_DTYPE_F32;
    const Layout l = layout_of(P, slots, rank * parts);
    const int cols = down_cols(rank * parts), units = (rank * parts + cols - 1) / cols;
    const int most = (K + thin::kStep * kWarps - 1) / (thin::kStep * kWarps);   // slices of 256 columns: a step for every warp
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    AdapterArgs g{static_cast<const __nv_bfloat16*>(x), x_stride, a_row_divisor, adapter_ids, topk_ids, (int)P, topk, adapters, E,
                  static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B), scale, rank, parts, rank * parts, N, K,
                  base, y, base_stride, y_stride, base != y, units, 1, 1, 0,
                  reinterpret_cast<float*>(ws + l.v),
                  reinterpret_cast<int32_t*>(ws + l.nblocks), reinterpret_cast<int32_t*>(ws + l.block_slot),
                  reinterpret_cast<int32_t*>(ws + l.block_count), reinterpret_cast<int32_t*>(ws + l.rows),
                  reinterpret_cast<int32_t*>(ws + l.sixteens), di.err};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (few) {
        e = f32 ? launch_few<true>(g, l.blocks, st) : launch_few<false>(g, l.blocks, st);
    } else {
        DownKernel down;
        e = down_kernel(g.R, down);
        // Few blocks: clusters join their sums before the second half reads them, which it does once for each of its CTAs.  As large
        // as all blocks find a place at once, by the most there can be (without and with clusters: 512 rows of rank 16 18.3 and
        // 15.4 us, 2048 rows of rank 64 41.0, 35.7; 4096 pairs of 512 slots 95, 128).
        const int splits = l.max_splits < most ? l.max_splits : most, resident = di.sm_count * down.ctas;
        g.cluster = 1;
        while (g.cluster < 4 && 2 * g.cluster <= splits && l.blocks * units * 2 * g.cluster <= resident) g.cluster *= 2;
        g.max_splits = splits / g.cluster;
        g.resident = resident / g.cluster;
        if (e == cudaSuccess) e = launch_plan(g, slots, reinterpret_cast<int32_t*>(ws + l.counts), st);
        if (e == cudaSuccess) e = launch_down(g, down, l.blocks, st);
        if (e == cudaSuccess) e = f32 ? launch_up<true>(g, st) : launch_up<false>(g, st);
    }
    if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return CHORD_ERR_CUDA;
    if (!opts || !opts->validate) return CHORD_OK;
    int32_t code = 0;
    const chord_status s = chord_get_device_error(stream, &code);
    if (s != CHORD_OK) return s;
    if (code == CHORD_DEV_TIMEOUT) return CHORD_ERR_TIMEOUT;
    return code ? CHORD_ERR_DEVICE_VALIDATION : CHORD_OK;
}

}  // extern "C"
