// One mixture-of-experts layer for a few tokens (at most CHORD_FEW_MAX_TOKENS),
// expert weights in 4 bits:
//   h[t, e]   = topk_w[t, e] * SiLU(W13[e][:I] x_t) * (W13[e][I:] x_t)
//   out[t]    = bf16( sum over the token's local experts of W2[e] h[t, e] )
// in two launches: gate_up with the activation and the routing weight, then
// the down projection with the sum over the experts.
//
// The used experts' weight bytes bound the layer, next to them the instructions that
// turn codes into bf16.  Both kernels are the same stream: a producer lane copies K
// stages of 128 weight rows (and the tokens' activations for those columns) into
// a ring with cp.async.bulk; four consumer warps take 32 rows each, dequantise in registers
// and multiply on the warp-level tensor cores with up to eight tokens on the B side.  A
// 16 x 128 tile is a warp's A operand: lane (g, c) holds rows g and g + 8 and the
// 32-column group c, one 16-byte load and one scale per row; the MMA's k order
// inside a tile is whatever puts a lane's own 32 columns into its slots, the same for A
// and B.  An expert with more than eight tokens is taken in several passes.
//   gate_up: an item is 64 gate rows and their 64 up rows of one expert, so a lane
//     ends with a gate sum and its up sum.  h keeps its FP32 number as three bf16 parts of
//     eight bits each, so the tensor cores multiply all of it (with two parts,
//     16 bits, 2.4 of 1000 outputs were another bf16 number than the exact sum's for that
//     reason alone; 16 tokens TP8 88.3 us for 87.7, 32 with MXFP4 168 for 159).  Few items: a cluster
//     of CTAs splits K and joins the sums through distributed shared memory in rank order.
//   down: several CTAs share 128 output rows for all experts: each takes a slice of
//     the (pass, K stage) list, and the last one to finish adds the FP32 sums in
//     slice order, so there is no combine pass and no order that changes a result.  The
//     kernel is launched early (programmatic dependent launch) and its weights are on
//     the way while gate_up still runs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "chord_internal.h"
#include "chord_mxfp4.cuh"
#include "chord_tcgen05.cuh"

namespace chord {
namespace {

constexpr int kConsumers = 4;                      // warps, 32 weight rows each
constexpr int kThreads = (kConsumers + 1) * 32;    // and the producer warp
constexpr int kPassTokens = 8;                     // tokens of one pass over an expert (MMA N)
constexpr int kZeroBytes = 256;                    // covers a token's 128-column unit
// The matrix instructions' FP32 additions chop, so a long chain of them on one accumulator ends
// up a little too small, every time.  Chains are kept to 48 instructions and their sums added in
// FP32 with rounding: kChainCols columns of gate_up's K (two chains of 32), down_chain_cols of the
// down projection's.  With the 7168 columns of 16 tokens TP8 in one chain, 3.3 of 1000 outputs were
// another bf16 number than the exact sum's, now 0.5 (FP32 products and sums in PyTorch: 0.25),
// for 0.5 us of gate_up's 54; with I = 1984 in one chain of the down projection 2.1, now below 1.
constexpr int kChainCols = 1024;
constexpr size_t kSmemMax = 96 * 1024;             // dynamic; a ring never takes more than a third of an SM

struct FewArgs {
    const uint16_t* x;
    const int32_t* ids;
    const float* wts;
    int T, topk, E, H, I;
    const uint8_t* w13;
    const uint8_t* w2;
    uint16_t* h;         // [3][T * topk, Ip]: an FP32 number as the sum of three bf16 parts; a row per (expert, token) in use
    int Ip;              // I rounded up to whole stages
    uint16_t* out;
    int* err;
    int validate;        // report ids outside [-1, E)
    int slot_cap;        // most passes a call can need
    int cluster;         // CTAs that share an item (gate_up, a cluster) or an output tile (down, list slices)
    float4* part;        // down, slices that are not a cluster: their sums
    int* joined;         // down: CTAs of each output tile that have left theirs
    int depth;           // stages of the ring
    int stage_bytes;
};

// ---- passes: which experts are used, by which tokens -----------------------
struct Route {
    int slots;                 // passes: (expert, up to eight of its tokens), experts ascending
    const uint16_t* expert;
    const uint32_t* tokens;    // bit t: token t
    const uint16_t* first;     // row of h of the pass's first token
};

__host__ __device__ __forceinline__ size_t route_bytes(int E, int P, int slot_cap) {
    return ((size_t)E * 4 + (size_t)P * 8 + (size_t)slot_cap * 8 + 127) / 128 * 128;
}

// What both kernels keep beside their ring of stages.
struct Shared {
    uint64_t full[16], empty[16];
    int flags;        // check_headers
    int abort_flag;
    int slots;
    int last;         // down: this CTA joins its tile
    uint32_t sums[kThreads / 32];
    __align__(16) uint32_t zeros[kZeroBytes / 4];   // what lanes without a token read
};

// Headers of both blobs, a word per lane of one warp: bit 0 they fit the call, bit 1 w13 is in
// the gate/up-interleaved layout, bit 2 the one-FMA dequantisation fits w13, bit 3
// it fits w2.
template <bool MX>
__device__ __forceinline__ int check_headers(const FewArgs& a) {
    const int lane = threadIdx.x & 31, i = lane & 15;
    const bool second = lane >= 16;
    const int N = second ? a.H : 2 * a.I, K = second ? a.I : a.H;
    const uint32_t v = i < 12 ? __ldg(reinterpret_cast<const uint32_t*>(second ? a.w2 : a.w13) + i) : 0u;
    const uint64_t stride = MX ? (uint64_t)mx_group_bytes(N, K) : (uint64_t)N * (uint64_t)K * 9ull / 16ull;
    uint32_t want = 0;
    switch (i) {
        case 0: want = kMagic; break;
        case 1: want = 1u; break;
        case 2: want = MX ? CHORD_LAYOUT_MXFP4 : CHORD_LAYOUT_TCGEN05; break;
        case 3: want = kGroup; break;
        case 4: want = (uint32_t)a.E; break;
        case 5: want = (uint32_t)N; break;
        case 6: want = (uint32_t)K; break;
        case 7: want = v; break;
        case 8: want = (uint32_t)stride; break;
        case 9: want = (uint32_t)(stride >> 32); break;
        case 10: want = (uint32_t)kHeaderBytes; break;
        default: break;
    }
    const bool inter = !MX && lane == 2 && v == (uint32_t)CHORD_LAYOUT_GATE_UP_INTERLEAVED;
    const bool ok = __all_sync(0xffffffffu, v == want || inter);
    const uint32_t ones = __ballot_sync(0xffffffffu, v == 1u);
    return (ok ? 1 : 0) | (__any_sync(0xffffffffu, inter) ? 2 : 0) | (ones >> kHdrScaleRangeWord & 1u ? 4 : 0) |
           (ones >> (16 + kHdrScaleRangeWord) & 1u ? 8 : 0);
}

// Barriers, header check and the passes, built in shared memory by all threads;
// the ids and weights are left there too.  Every global load is issued first.
template <bool MX>
__device__ Route prologue(const FewArgs& a, Shared& sh, uint8_t* sm, int32_t*& s_ids, float*& s_w, bool report) {
    const int P = a.T * a.topk, tid = threadIdx.x;
    uint32_t* mask = reinterpret_cast<uint32_t*>(sm);
    s_ids = reinterpret_cast<int32_t*>(mask + a.E);
    s_w = reinterpret_cast<float*>(s_ids + P);
    uint32_t* tokens = reinterpret_cast<uint32_t*>(s_w + P);
    uint16_t* expert = reinterpret_cast<uint16_t*>(tokens + a.slot_cap);
    uint16_t* first = expert + a.slot_cap;
    const int32_t id0 = tid < P ? __ldg(a.ids + tid) : 0;
    const float w0 = tid < P ? __ldg(a.wts + tid) : 0.0f;
    if (tid >= kConsumers * 32) {
        const int f = check_headers<MX>(a);
        if (tid == kConsumers * 32) sh.flags = f;
    }
    for (int e = tid; e < a.E; e += kThreads) mask[e] = 0;
    for (int i = tid; i < kZeroBytes / 4; i += kThreads) sh.zeros[i] = 0u;
    if (tid == 0) {
        sh.abort_flag = 0;
        for (int s = 0; s < a.depth; ++s) {
            mbar_init(&sh.full[s], 1 + 32);   // the bulk copies' bytes, and every producer lane's own copies
            mbar_init(&sh.empty[s], kConsumers);
        }
        fence_barrier_init();
    }
    __syncthreads();
    for (int p = tid; p < P; p += kThreads) {
        const int32_t e = p == tid ? id0 : a.ids[p];
        s_ids[p] = e;
        s_w[p] = p == tid ? w0 : a.wts[p];
        if (e >= 0 && e < a.E) {
            atomicOr(&mask[e], 1u << (p / a.topk));
        } else if (report && e != -1) {
            set_error(a.err, CHORD_DEV_BAD_EXPERT);
        }
    }
    __syncthreads();
    // Each thread takes `per` consecutive experts: an exclusive scan of (passes << 16 |
    // rows of h) over the threads, then the passes.
    const int per = (a.E + kThreads - 1) / kThreads, e0 = tid * per, e1 = min(e0 + per, a.E);
    uint32_t mine = 0;
    for (int e = e0; e < e1; ++e) {
        const int n = __popc(mask[e]);
        mine += (uint32_t)((n + kPassTokens - 1) / kPassTokens) << 16 | (uint32_t)n;
    }
    uint32_t at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, at, o);
        if ((tid & 31) >= o) at += v;
    }
    if ((tid & 31) == 31) sh.sums[tid >> 5] = at;
    at -= mine;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < (tid >> 5)) at += sh.sums[w];
    }
    if (tid == kThreads - 1) sh.slots = (int)((at + mine) >> 16);
    for (int e = e0; e < e1; ++e) {
        uint32_t left = mask[e];
        while (left) {
            uint32_t part = left;
            if (__popc(left) > kPassTokens) {
                part = 0;
                for (int k = 0; k < kPassTokens; ++k) {
                    part |= left & (0u - left);
                    left &= left - 1;
                }
            } else {
                left = 0;
            }
            expert[at >> 16] = (uint16_t)e;
            tokens[at >> 16] = part;
            first[at >> 16] = (uint16_t)at;
            at += (1u << 16) + __popc(part);
        }
    }
    __syncthreads();
    return Route{sh.slots, expert, tokens, first};
}

// Position of the n-th set bit of m (n below their number; mostly 0 or 1 here).
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
    for (; n > 0; --n) m &= m - 1;
    return __ffs(m) - 1;
}

// ---- stages -----------------------------------------------------------------
// INT4: 128 columns.  The blob's four (64-column chunk, 32-column half) blocks of
//   codes go 32 bytes further apart than they are long, so that the four lanes of a
//   quad read different banks; then the scale words, row r of chunk h at 512 h + 4 r.
// MXFP4: 256 columns, 128-byte swizzled rows as in the blob, then the scale blocks.
// After the weights: the activations, one row per token of the pass.
template <bool MX>
struct Stage {
    static constexpr int kCols = MX ? 256 : 128;
    static constexpr int kUnits = kCols / 128;
    static constexpr int kBlock = 2048 + 32;                  // INT4
    static constexpr int kScale = MX ? 16384 : 4 * kBlock;    // offset of the scales
    static constexpr int kUpWeights = kScale + (MX ? 4096 : 1024);
    static constexpr int kDownWeights = kScale + 1024;
    static constexpr int kUpRow = kCols * 2 + 16;             // activations of a token, gate_up
    static constexpr int kDownPart = kCols * 2 + 64;          // one of the three parts of an activation row, down
    static constexpr int kDownRow = 3 * kDownPart;
    // a stage with room for the activations of `tokens`, 128-byte aligned
    static __host__ __device__ int up_bytes(int tokens) { return (kUpWeights + tokens * kUpRow + 127) / 128 * 128; }
    static __host__ __device__ int down_bytes(int tokens) { return (kDownWeights + tokens * kDownRow + 127) / 128 * 128; }
};

// MXFP4 rows are 128 bytes apart and swizzled by row mod 8: with MMA row g taken
// from row (g & 1) * 4 + g / 2 the eight lanes of a load phase hit different banks.
template <bool MX>
__device__ __forceinline__ int phys_row(int g) {
    return MX ? ((g & 1) << 2) | (g >> 1) : g;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// The scale of a lane's group, ready for the dequantisation in use.
//   INT4, every scale in the one-FMA range (dequant_row8_fma): (s * 2^129, -8 s, -s / 2).
//     A nibble at bits 4..7 of a half-word is q * 2^-129 and becomes (q - 8) s; one at bits
//     0..3 is q * 2^-133 and becomes (q - 8) s / 16 with the same multiplier, so two of a
//     word's four pairs need no shift; their products are summed apart and join times 16
//     (mma16816).  A sixteenth of a weight is exact unless it is subnormal, so units with a
//     scale below 2^-118 (`odd`) shift instead and take -8 s.  Else: (s, s).
//   MXFP4: a code's three magnitude bits at bits 6..8 of a half-word are the bf16
//   number value * 2^-126 (subnormal 0.5 included), so one multiply by
//   2^(b - 1) gives the weight exactly; it fits bf16 for b <= 128, and larger scales
//   (`odd` units) take two multiplies, 2^126 and 2^(b - 127).  n: b itself.
struct Scale {
    uint32_t m, n, o;
};

template <bool MX, bool FAST>
__device__ __forceinline__ Scale make_scale(uint32_t word, int c) {
    Scale s;
    if constexpr (MX) {
        const uint32_t b = (word >> (8 * c)) & 255u;
        s.m = b * 0x00800080u + 0x3F003F00u;   // twice 2^(b - 1), for b up to 128
        s.n = b;
    } else {
        const uint32_t sp = prmt(word, c & 1 ? 0x3232u : 0x1010u);
        s.m = sp;
        s.n = s.o = 0;
        if constexpr (FAST) {
            fma_scale_pair(sp, s.m, s.n);
            s.o = bf2_as_u32(__hmul2(u32_as_bf2(sp), u32_as_bf2(0xBF00BF00u)));   // times -1/2
        }
    }
    return s;
}

// Eight codes to four bf16 pairs.  ODD: the unit has a scale that the short form does not
// cover (see Scale).  Pairs 0 and 2 of a FAST, not ODD word are sixteenths.
template <bool MX, bool FAST, bool ODD>
__device__ __forceinline__ void dequant8(uint32_t w, const Scale& s, uint32_t (&o)[4]) {
    if constexpr (MX) {
        uint32_t v[4];
        // a code n at bits 0..3 of a half-word times 2^6 + 2^12 has its magnitude at bits 6..8
        // and its sign at bit 15 (the other copies are masked away); at bits 4..7, times a
        // sixteenth of that: two logical operations and a multiplication, on different pipes
        const uint32_t t = w >> 8;
        v[0] = ((w & 0x000F000Fu) * 4160u) & 0x81C081C0u;   // columns 0, 4
        v[1] = ((w & 0x00F000F0u) * 260u) & 0x81C081C0u;    // 1, 5
        v[2] = ((t & 0x000F000Fu) * 4160u) & 0x81C081C0u;   // 2, 6
        v[3] = ((t & 0x00F000F0u) * 260u) & 0x81C081C0u;    // 3, 7
        if constexpr (ODD) {
            const __nv_bfloat162 big = u32_as_bf2(0x7E807E80u);        // 2^126
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s.n > 128u) v[i] = bf2_as_u32(__hmul2(u32_as_bf2(v[i]), big));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = bf2_as_u32(__hmul2(u32_as_bf2(v[i]), u32_as_bf2(s.m)));
    } else if constexpr (FAST && ODD) {
        dequant_row8_fma(w, s.m, s.n, o);
    } else if constexpr (FAST) {
        const uint32_t t = w >> 8;
        const __nv_bfloat162 m = u32_as_bf2(s.m), n = u32_as_bf2(s.n), h = u32_as_bf2(s.o);
        o[0] = bf2_as_u32(__hfma2(u32_as_bf2(w & 0x000F000Fu), m, h));   // columns +0, +1, a sixteenth
        o[1] = bf2_as_u32(__hfma2(u32_as_bf2(w & 0x00F000F0u), m, n));   // +2, +3
        o[2] = bf2_as_u32(__hfma2(u32_as_bf2(t & 0x000F000Fu), m, h));   // +4, +5, a sixteenth
        o[3] = bf2_as_u32(__hfma2(u32_as_bf2(t & 0x00F000F0u), m, n));   // +6, +7
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

// Where column `col` of an h row is kept: by 128-column unit, then (8-column piece
// of the group, group), so that a quad's loads of one piece are contiguous, in b_order.
template <bool MX>
__device__ __forceinline__ int h_pos(int col) {
    const int e = MX ? ((col & 3) << 1) | ((col >> 2) & 1) : col & 7;
    return (col & ~127) | ((col >> 3) & 3) << 5 | ((col >> 5) & 3) << 3 | e;
}

// 16 rows x 32 columns (eight of each lane) times eight tokens.  d: two sums, so that
// consecutive instructions do not wait on one another: d[0] of pairs 0 and 2, which may be
// sixteenths (whole: they are not, and go to d[1]), d[1] of pairs 1 and 3.
template <bool WHOLE>
__device__ __forceinline__ void mma16816(float (&d)[2][4], const uint32_t (&r0)[4], const uint32_t (&r1)[4], const uint4& b) {
    float(&e)[4] = d[WHOLE ? 1 : 0];
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(e[0]), "+f"(e[1]), "+f"(e[2]), "+f"(e[3])
        : "r"(r0[0]), "r"(r1[0]), "r"(r0[2]), "r"(r1[2]), "r"(b.x), "r"(b.z));
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[1][0]), "+f"(d[1][1]), "+f"(d[1][2]), "+f"(d[1][3])
        : "r"(r0[1]), "r"(r1[1]), "r"(r0[3]), "r"(r1[3]), "r"(b.y), "r"(b.w));
}

// The two sums joined.
template <bool SIXTEENTH>
__device__ __forceinline__ float4 both(const float (&d)[2][4]) {
    constexpr float f = SIXTEENTH ? 16.0f : 1.0f;
    return make_float4(fmaf(d[0][0], f, d[1][0]), fmaf(d[0][1], f, d[1][1]), fmaf(d[0][2], f, d[1][2]), fmaf(d[0][3], f, d[1][3]));
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// To the same shared-memory address of CTA `cta` of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t cta, float4 v) {
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(cta));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(ra), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

struct Ring {
    uint64_t *full, *empty;
    volatile int* abort_flag;
    uint32_t base, zero;      // stage 0, the zeros
    uint8_t* ptr;
};

// A lane's weight addresses inside a stage: tile i's first row at off + i * d_tile, its
// second row d_row further on (the same for the scale words).
struct LaneRows {
    uint32_t off, d_row, d_tile;
    uint32_t soff, sd_row, sd_tile;
};

struct NoMore {
    __device__ uint4 operator()(int, int) const { return uint4{}; }
};

// One 128-column unit of a stage: 32 rows of this warp times eight columns.  b(j): this
// lane's piece j of its column's activations; MORE: `extra` (one or two) more operands for the
// same columns, more(j, e).
template <bool MX, bool FAST, bool MORE, typename LoadB, typename LoadMore>
__device__ __forceinline__ void unit_mma(uint32_t st, const LaneRows& lr, uint32_t code_xor, uint32_t scale_add, bool on, int c,
                                         float (&acc)[2][2][4], LoadB&& b, int extra, LoadMore&& more) {
    uint4 q[2][2];
    Scale s[2][2];
    const uint32_t codes = st + (lr.off ^ code_xor);   // (MXFP4: d_tile and d_row are multiples of 1024)
    uint32_t least = 0xffffffffu;   // INT4: least scale - 1 (a scale of 0 stands for no column)
    uint32_t most = 0;              // MXFP4: largest scale
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            q[i][h] = lds128(codes + i * lr.d_tile + h * lr.d_row);
            uint32_t w = lds32(st + lr.soff + i * lr.sd_tile + h * lr.sd_row + scale_add);
            if (!MX && !on) w = 0;   // columns past K: codes left in the stage, times 0
            s[i][h] = make_scale<MX, FAST>(w, c);
            if constexpr (MX)
                most = max(most, s[i][h].n);
            else if constexpr (FAST)
                least = min(least, prmt(w, c & 1 ? 0x3232u : 0x1010u) - 1u);
        }
    const bool odd = MX ? most > 128u : FAST && least < 0x04800480u - 1u;   // INT4: below 2^-118
    auto columns = [&](auto is_odd) {
        constexpr bool kOdd = decltype(is_odd)::value;
        constexpr bool kWhole = !MX && FAST && kOdd;
        if constexpr (MX && kOdd) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                Scale& v = s[k >> 1][k & 1];
                if (v.n > 128u) v.m = v.n == 255u ? 0x7FC07FC0u : v.n * 0x00800080u;
            }
        }
#pragma unroll(MX && kOdd ? 1 : 4)   // rare: kept short, the instruction cache is
        for (int j = 0; j < 4; ++j) {
            const uint4 v = b(j);
            uint4 r0, r1;   // loaded ahead of the dequantisation (one operand after the other: 8 experts of
                            // 4096 x 3584, 16 tokens 71.6 us, 69.5 so)
            if constexpr (MORE) {
                r0 = more(j, 0);
                r1 = more(j, extra - 1);
            }
            uint32_t x[2][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                dequant8<MX, FAST, kOdd>(word(q[i][0], j), s[i][0], x[i][0]);
                dequant8<MX, FAST, kOdd>(word(q[i][1], j), s[i][1], x[i][1]);
                mma16816<kWhole>(acc[i], x[i][0], x[i][1], v);
            }
            if constexpr (MORE) {
#pragma unroll
                for (int i = 0; i < 2; ++i) mma16816<kWhole>(acc[i], x[i][0], x[i][1], r0);
                if (extra > 1) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) mma16816<kWhole>(acc[i], x[i][0], x[i][1], r1);
                }
            }
        }
    };
    if ((MX || FAST) && __any_sync(0xffffffffu, odd))
        columns(std::true_type{});
    else
        columns(std::false_type{});
}

// After the last stage: every copy that was issued has landed.
__device__ __forceinline__ void drain_ring(const FewArgs& a, const Ring& rg, tc5::Ring r, int issued) {
    for (int k = 0; k < a.depth && k < issued; ++k) {
        if (r.slot == 0) {
            r.slot = a.depth - 1;
            r.phase ^= 1u;
        } else {
            --r.slot;
        }
        if (!mbar_wait(&rg.full[r.slot], r.phase)) set_error(a.err, CHORD_DEV_TIMEOUT);
    }
}

// ---- gate_up ----------------------------------------------------------------
// h of one lane's gate and up sums (column col; tokens 2c and 2c + 1 of the pass).
template <bool MX>
__device__ __forceinline__ void store_h(const FewArgs& a, const Route& rt, int slot, const int32_t* s_ids, const float* s_w,
                                        int col, int c, float4 s) {
    if (col >= a.I) return;
    const uint32_t tokens = rt.tokens[slot];
    const int n = __popc(tokens), e = rt.expert[slot];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = 2 * c + i;
        if (j >= n) continue;
        const int t = nth_bit(tokens, j);
        float wt = 0.0f;
        for (int k = 0; k < a.topk; ++k)
            if (s_ids[t * a.topk + k] == e) wt += s_w[t * a.topk + k];
        const float h = wt * silu_times(i ? s.y : s.x, i ? s.w : s.z);
        // Three bf16 parts, each what is left cut to eight bits, so that a finite number has
        // finite parts and their sum is h; infinities and NaN have the first one only.
        const int64_t plane = (int64_t)a.T * a.topk * a.Ip;
        uint16_t* to = a.h + (int64_t)(rt.first[slot] + j) * a.Ip + h_pos<MX>(col);
        float rest = h;
#pragma unroll
        for (int k = 0; k < 3; ++k, to += plane) {
            const __nv_bfloat16 part = __float2bfloat16_rz(rest);
            *to = __bfloat16_as_ushort(part);
            rest -= __bfloat162float(part);
            if (!isfinite(rest)) rest = 0.0f;
        }
    }
}

// The weights' code blocks go through cp.async.bulk, a block per lane; what comes in
// short pieces (scale words, activation rows) through 16-byte cp.async of all
// lanes: bulk copies of a few hundred bytes hold up the ones behind them.  The warp
// shares its scheduler with consumers, so a stage costs it few instructions: every
// address is a running pointer.
template <bool MX>
__device__ __forceinline__ void up_producer(const FewArgs& a, const Route& rt, const Ring& rg, bool inter, int items, int mt,
                                            int ks0, int ks1) {
    using S = Stage<MX>;
    const int lane = threadIdx.x & 31;
    constexpr int kPieces = S::kCols / 8;   // 16-byte pieces of an activation row
    constexpr int kStep = MX ? kMxTileBytes : 9216;
    // lane l copies block l of a stage: `bytes` to `to`, from `from` of the item
    const int blocks = MX || !inter ? 8 : 4;
    uint32_t bytes, to;
    if constexpr (MX) {   // codes, then scale blocks, of 32 rows each: gate, gate, up, up
        bytes = lane < 4 ? 4096u : 1024u;
        to = lane < 4 ? lane * 4096u : S::kScale + (lane - 4) * 1024u;
    } else {              // (chunk, half) blocks of 128 rows, or of 64 gate and 64 up rows
        bytes = inter ? 2048u : 1024u;
        to = inter ? lane * S::kBlock : (lane >> 1) * S::kBlock + (lane & 1) * 1024u;
    }
    const uint32_t total = MX ? 16384u + 4096u : 8192u;
    tc5::Ring r;
    int issued = 0;
    bool ok = true;
    for (int item = blockIdx.x / a.cluster; item < items; item += gridDim.x / a.cluster) {
        const int slot = item / mt, m = item - slot * mt, e = rt.expert[slot];
        const uint32_t tokens = rt.tokens[slot];
        const uint8_t *from, *scales = nullptr;
        if constexpr (MX) {
            const uint8_t* base = a.w13 + kHeaderBytes + (uint64_t)e * mx_group_bytes(2 * a.I, a.H);
            const int gi = lane & 3, row = (gi >> 1) * a.I + m * 64 + (gi & 1) * 32;   // 32 rows never cross a tile
            from = base + ((int64_t)(row >> 7) * mx_col_tiles(a.H) + ks0) * kStep + (lane < 4 ? (row & 127) * 128 : kMxCodeBytes);
        } else {
            const uint8_t* base = a.w13 + kHeaderBytes + (uint64_t)e * ((uint64_t)(2 * a.I) * a.H * 9ull / 16ull) + (int64_t)ks0 * kStep;
            const int64_t band = (int64_t)(a.H / 64) * 4608;
            const int q = inter ? lane : lane >> 1, row = inter ? m * 128 : (lane & 1) * a.I + m * 64;   // I % 64 == 0
            from = base + (row >> 7) * band + ((q >> 1) & 1) * 4608 + (q & 1) * 2048 + (row & 127) * 16;
            const int srow = inter ? m * 128 : (lane >> 4) * a.I + m * 64;
            scales = base + (srow >> 7) * band + 4096 + (inter ? lane * 16 : (srow & 127) * 4 + (lane & 15) * 16);
        }
        const uint16_t* x = a.x + ks0 * S::kCols + lane * 8;
        int left = a.H - ks0 * S::kCols - lane * 8;   // columns from this lane's piece on
        for (int ks = ks0; ks < ks1 && ok; ++ks) {
            ok = tc5::wait(&rg.empty[r.slot], r.phase ^ 1u, rg.abort_flag, a.err);
            if (!ok) break;
            const uint32_t bar = smem_u32(&rg.full[r.slot]), st = rg.base + r.slot * a.stage_bytes;
            if (lane == 0) tc5::arrive_expect_tx(bar, total);
            if (lane < blocks) tc5::bulk_g2s(st + to, from, bytes, bar);
            if constexpr (!MX) {
                cp_async16(st + S::kScale + lane * 16, scales);
                cp_async16(st + S::kScale + 512 + lane * 16, scales + 4608);
                scales += kStep;
            }
            if (lane < kPieces && left > 0) {
                uint32_t xs = st + S::kUpWeights + lane * 16;
                for (uint32_t mk = tokens; mk; mk &= mk - 1, xs += S::kUpRow) cp_async16(xs, x + (int64_t)(__ffs(mk) - 1) * a.H);
            }
            cp_async_arrive_noinc(&rg.full[r.slot]);
            from += kStep;
            x += S::kCols;
            left -= S::kCols;
            ++issued;
            r.next(a.depth);
        }
        __syncwarp();
        if (a.cluster > 1) cluster_sync_all();
    }
    cp_async_wait<0>();
    drain_ring(a, rg, r, issued);
    __syncwarp();
}

template <bool MX, bool FAST>
__device__ __forceinline__ void up_consumer(const FewArgs& a, const Route& rt, const Ring& rg, float4* part, bool inter,
                                            const int32_t* s_ids, const float* s_w, int items, int mt, int rank, int ks0, int ks1) {
    using S = Stage<MX>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, p = phys_row<MX>(g);
    LaneRows lr;
    if constexpr (MX) {
        const uint32_t row = 16 * warp + p;    // of the 64 gate rows
        lr = LaneRows{row * 128 + ((c ^ (row & 7)) << 4), 8192, 1024, 0, 2048, 128};
    } else {
        const uint32_t row = inter ? 32 * warp + g : 16 * warp + g;
        lr = LaneRows{(uint32_t)c * S::kBlock + row * 16, inter ? 128u : 1024u, inter ? 256u : 128u,
                      (uint32_t)S::kScale + (c >> 1) * 512 + row * 4, inter ? 32u : 256u, inter ? 64u : 32u};
    }
    tc5::Ring r;
    bool ok = true;
    int nitem = 0;
    for (int item = blockIdx.x / a.cluster; item < items; item += gridDim.x / a.cluster, ++nitem) {
        const int slot = item / mt, m = item - slot * mt, n = __popc(rt.tokens[slot]);
        uint32_t quad[2] = {0, 0};
        if constexpr (MX) {
            // scale words of row R of the 64: block R / 32, word (absolute row / 32) mod 4
            lr.soff = S::kScale + (warp >> 1) * 1024 + ((16 * warp + p) & 31) * 16;
            quad[0] = (((uint32_t)(m * 64) >> 5) + (warp >> 1)) & 3;
            quad[1] = (((uint32_t)(a.I + m * 64) >> 5) + (warp >> 1)) & 3;
            lr.soff += quad[0] * 4;
            lr.sd_row = 2048 + quad[1] * 4 - quad[0] * 4;
        }
        float acc[2][2][4] = {};
        float4 sum[2] = {};   // of finished chains
        for (int ks = ks0; ks < ks1 && ok;) {
            for (const int end = min(ks + kChainCols / S::kCols, ks1); ks < end; ++ks, r.next(a.depth)) {
                ok = tc5::wait(&rg.full[r.slot], r.phase, rg.abort_flag, a.err);
                if (!ok) break;
                const uint32_t st = rg.base + r.slot * a.stage_bytes;
                const uint32_t xs = st + S::kUpWeights + g * S::kUpRow + c * 64;
#pragma unroll
                for (int u = 0; u < S::kUnits; ++u) {
                    const bool on = ks * S::kCols + u * 128 + c * 32 < a.H;
                    const uint32_t xb = g < n && on ? xs + u * 256 : rg.zero;
                    unit_mma<MX, FAST, false>(st, lr, u * 64, u * kMxScaleBlock, on, c, acc,
                                              [&](int j) { return b_order<MX>(lds128(xb + j * 16)); }, 0, NoMore{});
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&rg.empty[r.slot]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 v = both<!MX && FAST>(acc[i]);
                sum[i].x += v.x, sum[i].y += v.y, sum[i].z += v.z, sum[i].w += v.w;
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[i][k >> 2][k & 3] = 0.0f;
            }
        }
        const int col0 = m * 64 + 16 * warp + p;
        if (a.cluster == 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (ok) store_h<MX>(a, rt, slot, s_ids, s_w, col0 + 8 * i, c, sum[i]);
            continue;
        }
        // join the cluster's K ranges: tile q = 2 warp + i belongs to CTA q mod cluster, which
        // is sent every CTA's sums ([tile of its own][rank][lane]) and adds them in rank order.
        // Buffers alternate, so one barrier an item is enough, and after the last nobody
        // touches another CTA's memory.
        const uint32_t own = 8u / (uint32_t)a.cluster;   // tiles of a CTA
        float4* buf = part + (nitem & 1) * 256;
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
            const uint32_t q = (uint32_t)warp * 2 + i;
            st_cluster(smem_u32(buf + ((q / a.cluster) * a.cluster + rank) * 32 + lane), q % a.cluster, sum[i]);
        }
        __syncwarp();
        cluster_sync_all();
        if (ok && (uint32_t)warp < own) {
            const float4* mine = buf + warp * a.cluster * 32 + lane;
            float4 s = mine[0];
            for (int r = 1; r < a.cluster; ++r) {
                const float4 v = mine[r * 32];
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            store_h<MX>(a, rt, slot, s_ids, s_w, m * 64 + 8 * (warp * a.cluster + rank) + p, c, s);
        }
    }
}

// One token on 8 experts of 2 x 256 x 7168 is latency: 3 us to the first weights' copies, 2 to
// their arrival, then 16.5 MB.  More tokens: the weights' stream, with instruction issue
// close behind (8 tokens, 57 experts: 117 MB at 5.0 TB/s; 16 tokens INT4 issue 2.1 of 4
// instructions a cycle; MXFP4 codes take 17 operations for eight against 9).
template <bool MX>
__global__ void __launch_bounds__(kThreads, 4) few_gate_up_kernel(const FewArgs a) {
    using S = Stage<MX>;
    pdl_trigger();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const Ring rg{sh.full, sh.empty, &sh.abort_flag, smem_u32(smem), smem_u32(sh.zeros), smem};
    float4* part = reinterpret_cast<float4*>(smem + a.depth * a.stage_bytes);
    int32_t* s_ids;
    float* s_w;
    const Route rt = prologue<MX>(a, sh, reinterpret_cast<uint8_t*>(part + (a.cluster > 1 ? 512 : 0)), s_ids, s_w,
                                  a.validate && blockIdx.x == 0);
    if (blockIdx.x == 0)   // for the down kernel
        for (int i = threadIdx.x; i < (a.H + 127) / 128; i += kThreads) a.joined[i] = 0;
    if (!(sh.flags & 1)) {   // the same in every CTA
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, CHORD_DEV_BAD_HEADER);
        return;
    }
    if (a.cluster > 1) cluster_sync_all();   // every CTA runs before another one's sums arrive
    const int stages = (a.H + S::kCols - 1) / S::kCols, mt = (a.I + 63) / 64, items = rt.slots * mt;
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    const int ks0 = rank * stages / a.cluster, ks1 = (rank + 1) * stages / a.cluster;
    const bool inter = (sh.flags & 2) != 0;
    if (threadIdx.x >= kConsumers * 32)
        up_producer<MX>(a, rt, rg, inter, items, mt, ks0, ks1);
    else if (MX || (sh.flags & 4))
        up_consumer<MX, true>(a, rt, rg, part, inter, s_ids, s_w, items, mt, rank, ks0, ks1);
    else
        up_consumer<MX, false>(a, rt, rg, part, inter, s_ids, s_w, items, mt, rank, ks0, ks1);
}

// ---- down -------------------------------------------------------------------
// Entries [v0, v1) of the list, entry v = (pass v / kst, K stage v % kst).
template <bool MX>
__device__ __forceinline__ void down_producer(const FewArgs& a, const Route& rt, const Ring& rg, int tile, int v0, int v1, int kst) {
    using S = Stage<MX>;
    constexpr int kPieces = S::kCols / 8;   // 16-byte pieces of a part of a row
    const int lane = threadIdx.x & 31;
    struct At {
        int sl, ks;
        __device__ void next(int kst) {
            if (++ks == kst) {
                ks = 0;
                ++sl;
            }
        }
    };
    const uint64_t expert_bytes = MX ? mx_group_bytes(a.H, a.I) : (uint64_t)a.H * a.I * 9ull / 16ull;
    const uint8_t* tile_base = a.w2 + kHeaderBytes + (MX ? (int64_t)tile * mx_col_tiles(a.I) * kMxTileBytes
                                                        : (int64_t)tile * (a.I / 64) * 4608);
    auto weights = [&](const At& at, int slot) {
        const uint32_t bar = smem_u32(&rg.full[slot]), st = rg.base + slot * a.stage_bytes;
        const uint8_t* t = tile_base + (uint64_t)rt.expert[at.sl] * expert_bytes;
        if constexpr (MX) {
            if (lane == 0) {
                tc5::arrive_expect_tx(bar, kMxTileBytes);
                tc5::bulk_g2s(st, t + (int64_t)at.ks * kMxTileBytes, kMxTileBytes, bar);
            }
        } else {
            const int chunks = a.I / 64 - 2 * at.ks >= 2 ? 2 : 1;
            t += (int64_t)at.ks * 9216;
            if (lane == 0) tc5::arrive_expect_tx(bar, (uint32_t)chunks * 4096u);
            if (lane < 2 * chunks) tc5::bulk_g2s(st + lane * S::kBlock, t + (lane >> 1) * 4608 + (lane & 1) * 2048, 2048, bar);
            cp_async16(st + S::kScale + lane * 16, t + 4096 + lane * 16);
            if (chunks == 2) cp_async16(st + S::kScale + 512 + lane * 16, t + 4608 + 4096 + lane * 16);
        }
    };
    const int64_t plane = (int64_t)a.T * a.topk * a.Ip;
    const int64_t second = MX ? plane : plane - kPieces * 8;   // INT4: lanes 16 .. 31 take the second part
    auto activations = [&](const At& at, int slot) {
        const int n = __popc(rt.tokens[at.sl]);
        uint32_t hs = smem_u32(rg.ptr + slot * a.stage_bytes + S::kDownWeights) + lane * 16;
        const uint16_t* src = a.h + (int64_t)rt.first[at.sl] * a.Ip + at.ks * S::kCols + lane * 8;
        if (!MX && lane >= kPieces) src += second, hs += S::kDownPart - kPieces * 16;
        for (int j = 0; j < n; ++j, hs += S::kDownRow, src += a.Ip) {
            cp_async16(hs, src);
            if constexpr (MX) {
                cp_async16(hs + S::kDownPart, src + second);
                cp_async16(hs + 2 * S::kDownPart, src + 2 * second);
            } else {
                if (lane < kPieces) cp_async16(hs + 2 * S::kDownPart, src + 2 * plane);
            }
        }
        cp_async_arrive_noinc(&rg.full[slot]);
    };
    // the first stages' weights do not depend on the gate_up kernel
    const int n = v1 - v0;
    At w{v0 / kst, v0 % kst}, act = w;
    int pre = 0;
    for (; pre < n && pre < a.depth; ++pre, w.next(kst)) weights(w, pre);
    pdl_wait();   // h of the gate_up kernel is complete from here on
    tc5::Ring r;
    int issued = 0;
    for (; issued < n; ++issued, r.next(a.depth), act.next(kst)) {
        if (issued >= pre) {
            if (!tc5::wait(&rg.empty[r.slot], r.phase ^ 1u, rg.abort_flag, a.err)) break;
            weights(act, r.slot);
        }
        activations(act, r.slot);
    }
    cp_async_wait<0>();
    drain_ring(a, rg, r, issued);
}

// Where the three parts of a pass's activations go among the eight columns.
//   kOne: up to two tokens, one instruction: token j's parts in columns 4 j, 4 j + 1, 4 j + 2
//   kTwo: up to four, two instructions: first parts in columns 0 .. 3, second ones in 4 .. 7;
//     third ones in 0 .. 3
//   kThree: a column a token, an instruction a part
// The enumerator is the number of instructions after the first.
enum Spread { kOne = 0, kTwo = 1, kThree = 2 };
// Columns of a chain: 48 instructions on each of its two sums.
__device__ __forceinline__ int down_chain_cols(Spread s) { return s == kOne ? 1536 : s == kTwo ? 768 : 512; }

// A pass's sums into the sums by token (lane (g, c), tile nt: tokens 8 nt + 2c and + 1).
template <int NT, bool SIXTEENTH>
__device__ __forceinline__ void add_pass(float (&sum)[2][NT][4], float (&chains)[2][2][4], uint32_t tokens, Spread spread, int c) {
    float p[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i >> 2][i & 3] = fmaf(chains[i >> 2][0][i & 3], SIXTEENTH ? 16.0f : 1.0f, chains[i >> 2][1][i & 3]);
        chains[i >> 2][0][i & 3] = chains[i >> 2][1][i & 3] = 0.0f;
    }
    auto add = [&](int ta, int tb, const float (&va)[4], const float (&vb)[4]) {   // tokens and their sums by (tile, row half)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && (ta >> 3) != nt && (tb >> 3) != nt) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = 8 * nt + 2 * c + k;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (t == ta) sum[i >> 1][nt][(i & 1) * 2 + k] += va[i];
                    if (t == tb) sum[i >> 1][nt][(i & 1) * 2 + k] += vb[i];
                }
            }
        }
    };
    if (spread == kOne) {   // lanes c = 0, 1: the first token's parts, 2, 3: the second one's
        float va[4], vb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = p[i >> 1][(i & 1) * 2] + p[i >> 1][(i & 1) * 2 + 1];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            va[i] = __shfl_sync(0xffffffffu, v, 0, 4);
            vb[i] = __shfl_sync(0xffffffffu, v, 2, 4);
        }
        const int ta = __ffs(tokens) - 1, tb = __ffs(tokens & (tokens - 1)) - 1;
        add(ta, tb, va, vb);
        return;
    }
    if (spread == kTwo) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] += __shfl_xor_sync(0xffffffffu, p[i >> 2][i & 3], 2);
    }
    for (int jj = 0; tokens; ++jj) {   // columns 2 jj and 2 jj + 1
        const int ta = __ffs(tokens) - 1;
        tokens &= tokens - 1;
        const int tb = __ffs(tokens) - 1;   // -1: no such column
        tokens &= tokens - 1;
        float va[4], vb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            va[i] = __shfl_sync(0xffffffffu, p[i >> 1][(i & 1) * 2], jj, 4);
            vb[i] = __shfl_sync(0xffffffffu, p[i >> 1][(i & 1) * 2 + 1], jj, 4);
        }
        add(ta, tb, va, vb);
    }
}

template <bool MX, int NT, bool ONE, bool FAST>
__device__ __forceinline__ void down_consumer(const FewArgs& a, const Route& rt, const Ring& rg, int v0, int v1, int kst,
                                              float (&sum)[2][NT][4]) {
    using S = Stage<MX>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t row = 32 * warp + phys_row<MX>(g);
    const LaneRows lr = MX ? LaneRows{row * 128 + ((c ^ (row & 7)) << 4), 1024, 2048,
                                      (uint32_t)S::kScale + (row & 31) * 16 + (row >> 5) * 4, 128, 256}
                           : LaneRows{(uint32_t)c * S::kBlock + row * 16, 128, 256,
                                      (uint32_t)S::kScale + (c >> 1) * 512 + row * 4, 32, 64};
    tc5::Ring r;
    int sl = v0 / kst, ks = v0 - sl * kst;
    float pass[2][2][4] = {};
    for (int left = v1 - v0; left > 0;) {
        const uint32_t tokens = rt.tokens[sl];
        const int n = __popc(tokens);
        const Spread spread = ONE || n <= 2 ? kOne : n <= 4 ? kTwo : kThree;
        const int j = spread == kOne ? g >> 2 : spread == kTwo ? g & 3 : g;            // this lane's token of the pass
        const int part = spread == kOne ? g & 3 : spread == kTwo ? g >> 2 : 0;
        const uint32_t h0 = j < n && part < 3 ? S::kDownWeights + (uint32_t)j * S::kDownRow + c * 16 + part * S::kDownPart : 0u;
        const uint32_t h1 = j < n && part < 1 ? h0 + S::kDownPart * (spread == kTwo ? 2 : 1) : 0u;   // of the instructions after
        const int end = min(min(kst, ks + left), ks + down_chain_cols(spread) / S::kCols);
        left -= end - ks;
        for (; ks < end; ++ks, r.next(a.depth)) {
            if (!tc5::wait(&rg.full[r.slot], r.phase, rg.abort_flag, a.err)) return;
            const uint32_t st = rg.base + r.slot * a.stage_bytes;
#pragma unroll
            for (int u = 0; u < S::kUnits; ++u) {
                const bool on = ks * S::kCols + u * 128 + c * 32 < a.I;
                const uint32_t hb = h0 && on ? st + h0 + u * 256 : rg.zero;
                if (ONE || spread == kOne) {
                    unit_mma<MX, FAST, false>(st, lr, u * 64, u * kMxScaleBlock, on, c, pass,
                                              [&](int j) { return lds128(hb + j * 64); }, 0, NoMore{});
                } else {
                    const uint32_t more = h1 && on ? st + h1 + u * 256 : rg.zero, step = h1 && on ? S::kDownPart : 0;
                    unit_mma<MX, FAST, true>(st, lr, u * 64, u * kMxScaleBlock, on, c, pass,
                                             [&](int j) { return lds128(hb + j * 64); }, spread,
                                             [&](int j, int e) { return lds128(more + j * 64 + e * step); });
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&rg.empty[r.slot]);
        }
        add_pass<NT, !MX && FAST>(sum, pass, tokens, ONE ? kOne : spread, c);
        if (ks == kst) {
            ++sl;
            ks = 0;
        }
    }
}

// What the slices of a cluster send one another, beside the ring: a CTA's share of the
// (16 rows, 8 tokens) tiles, from every slice.
__host__ __device__ __forceinline__ size_t down_part_bytes(int nt, int cluster) {
    return (size_t)((kConsumers * 2 * nt + cluster - 1) / cluster) * cluster * 512;
}

// gridDim.x = output tiles of 128 rows x a.cluster list slices (slice fastest).  Short
// lists: the slices are a cluster and exchange their FP32 sums through distributed shared
// memory.  Long ones, whose rings leave room for three CTAs per SM (51 clusters of eight, and
// 56 tiles of 7168 rows would take a second wave): each CTA leaves its sums in the workspace
// and the tile's last one adds them.  Always in slice order, so the result does not depend
// on which CTA is last.
// Bound as gate_up is: 8 tokens, 57 experts of 7168 x 256: 58 MB in 12 us once its first
// weights are there; before that 5 us pass between gate_up's last stage and this kernel's
// first (its end, this one's routing, a ring's fill), half of it hidden where this kernel's
// CTAs fit beside gate_up's.  (Both halves in one cooperative launch, the ring filled
// ahead of a grid barrier, measured the same: 8 tokens 58.6 us against 58.5, 16 tokens 93
// against 89.)
// ONE: no pass has more than two tokens, so the code for more of them is not there (one token
// TP8 with its weights in L2 18.7 us, with it 19.9).
// CLUSTERED: four CTAs per SM.  Else three, so up to 128 registers a thread: with 96 the eight
// tokens of MXFP4 TP8 (59 experts) take 65.3 us instead of 64.6.
template <bool MX, int NT, bool ONE, bool CLUSTERED>
__global__ void __launch_bounds__(kThreads, CLUSTERED ? 4 : 3) few_down_kernel(const FewArgs a) {
    using S = Stage<MX>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const Ring rg{sh.full, sh.empty, &sh.abort_flag, smem_u32(smem), smem_u32(sh.zeros), smem};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* s_ids;
    float* s_w;
    const Route rt = prologue<MX>(a, sh, smem + a.depth * a.stage_bytes + (CLUSTERED ? down_part_bytes(NT, a.cluster) : 0), s_ids,
                                  s_w, false);
    if (!(sh.flags & 1)) {   // the same in every CTA; the gate_up kernel reported it
        pdl_wait();          // what follows in the stream comes after both kernels, also here
        return;
    }
    if (CLUSTERED) cluster_sync_all();   // every CTA runs before another one's sums arrive
    const int rank = blockIdx.x % a.cluster, tile = blockIdx.x / a.cluster;
    const int kst = (a.I + S::kCols - 1) / S::kCols, total = rt.slots * kst;
    const int v0 = (int)((int64_t)rank * total / a.cluster), v1 = (int)((int64_t)(rank + 1) * total / a.cluster);
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2 * NT * 4; ++i) acc[i / (NT * 4)][i / 4 % NT][i % 4] = 0.0f;
    if (warp == kConsumers)
        down_producer<MX>(a, rt, rg, tile, v0, v1, kst);
    else if (MX || (sh.flags & 8))
        down_consumer<MX, NT, ONE, true>(a, rt, rg, v0, v1, kst, acc);
    else
        down_consumer<MX, NT, ONE, false>(a, rt, rg, v0, v1, kst, acc);
    __syncwarp();
    constexpr int kTiles = kConsumers * 2 * NT;      // (16 rows, 8 tokens) tiles of a CTA, q = (2 warp + i) NT + nt
    constexpr int kPer = kTiles * 32;                // float4 of a CTA: [tile][lane]
    auto write = [&](int q, float4 s) {
        const int row = tile * 128 + (q / NT) * 16 + phys_row<MX>(lane >> 2), t = 8 * (q % NT) + 2 * (lane & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int tk = t + (k & 1), n = row + (k >> 1) * 8;
            const float v = k == 0 ? s.x : k == 1 ? s.y : k == 2 ? s.z : s.w;
            // + 0.0f: a sum of nothing, or of zeros of either sign, is +0
            if (tk < a.T && n < a.H) a.out[(int64_t)tk * a.H + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v + 0.0f));
        }
    };
    auto sum_of = [&](int i, int nt) { return make_float4(acc[i][nt][0], acc[i][nt][1], acc[i][nt][2], acc[i][nt][3]); };
    if (a.cluster == 1) {
        if (warp == kConsumers) return;
        pdl_wait();   // (an empty list has waited for nothing yet)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) write((2 * warp + i) * NT + nt, sum_of(i, nt));
        return;
    }
    if constexpr (CLUSTERED) {
        // short lists: tile q belongs to CTA q mod cluster, which is sent every slice's sums
        float4* buf = reinterpret_cast<float4*>(smem + a.depth * a.stage_bytes);   // [tile of its own][slice][lane]
        if (warp < kConsumers) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int q = (2 * warp + i) * NT + nt;
                    st_cluster(smem_u32(buf + ((q / a.cluster) * a.cluster + rank) * 32 + lane), (uint32_t)(q % a.cluster), sum_of(i, nt));
                }
        }
        __syncwarp();
        cluster_sync_all();
        if (warp == kConsumers) return;
        for (int j = warp; j * a.cluster + rank < kTiles; j += kConsumers) {
            const float4* from = buf + j * a.cluster * 32 + lane;
            float4 s = from[0];
            for (int r = 1; r < a.cluster; ++r) {
                const float4 v = from[r * 32];
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            write(j * a.cluster + rank, s);
        }
        return;
    }
    pdl_wait();   // (threads that read nothing of the gate_up kernel) its zeroed counters
    float4* mine = a.part + (int64_t)blockIdx.x * kPer;
    if (warp < kConsumers) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mine[((2 * warp + i) * NT + nt) * 32 + lane] = sum_of(i, nt);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();   // the CTA's sums (ordered before it by the barrier) before the count
        sh.last = atomicAdd(a.joined + tile, 1) == a.cluster - 1;
        __threadfence();
    }
    __syncthreads();
    if (!sh.last || warp == kConsumers) return;
    // slices in order, eight at a time, the loads of all column tiles of a row tile before
    // their sums
    const float4* from = a.part + (int64_t)tile * a.cluster * kPer + warp * 2 * NT * 32 + lane;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float4 s[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt] = make_float4(0, 0, 0, 0);
        for (int r0 = 0; r0 < a.cluster; r0 += 8) {
            float4 v[NT][8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    v[nt][r] = r0 + r < a.cluster && 8 * nt < a.T ? __ldcg(from + (int64_t)(r0 + r) * kPer + (i * NT + nt) * 32)
                                                                  : make_float4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[nt].x += v[nt][r].x, s[nt].y += v[nt][r].y, s[nt].z += v[nt][r].z, s[nt].w += v[nt][r].w;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) write((2 * warp + i) * NT + nt, s[nt]);
    }
}

// List slices per output tile of the down kernel: three CTAs per SM of a GB300 (152
// SMs; host arithmetic, the workspace depends on it), at most 16, one for every list entry.
int down_slices(int H, int64_t list) {
    const int tiles = (H + 127) / 128;
    int n = 152 * 3 / tiles;
    n = n > 16 ? 16 : (n < 1 ? 1 : n);
    return list < n ? (int)(list < 1 ? 1 : list) : n;
}

// Stages of a ring: what fits, but no more than a CTA will use (a small ring lets the
// down kernel's CTAs in beside the gate_up kernel's).
int ring_depth(size_t room, int stage_bytes, int64_t used) {
    int64_t d = (int64_t)(room / (size_t)stage_bytes);
    if (d > used) d = used;
    return d > 16 ? 16 : (d < 2 ? 2 : (int)d);
}

template <typename Kern>
cudaError_t launch(Kern kern, const FewArgs& a, unsigned groups, size_t smem, bool cluster, bool pdl, cudaStream_t st) {
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(groups * (unsigned)a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster && a.cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)a.cluster;
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
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool MX, int NT, bool ONE>
cudaError_t launch_few_nt(FewArgs a, cudaStream_t st) {
    using S = Stage<MX>;
    const int sms = device_info().sm_count;
    const size_t route = route_bytes(a.E, a.T * a.topk, a.slot_cap);
    // gate_up: three CTAs per SM while the items of an even routing then run in one wave
    // (they spread evenly: the layer for 16 tokens TP8, 436 items, 88 us against 92.5 with four per
    // SM), else four (32 tokens EP8, 22 experts of 32 items each: 138 us against 143).  Where they
    // would leave half of the GPU idle, a cluster shares each item's K range, three stages or
    // more a CTA (4 tokens, top-2 of 16 experts of 2 x 1024 x 1024, eight stages: in twos 17.2 us, in
    // fours 18.5).  Every pair counts as local: on an expert-parallel share fewer items come than
    // are planned for, and clusters are smaller than they might be.
    const int mt = (a.I + 63) / 64, stages = (a.H + S::kCols - 1) / S::kCols;
    const int64_t items = (int64_t)a.slot_cap * mt;
    const double pairs = (double)a.T * a.topk, hit = a.E * (1.0 - pow(1.0 - 1.0 / a.E, pairs));   // experts with a token
    const double passes = hit * fmax(1.0, pairs / hit / kPassTokens + 0.5), even = passes * mt;
    a.cluster = 8;
    while (a.cluster > 1 && (even * a.cluster > 4.0 * sms || a.cluster * 3 > stages)) a.cluster >>= 1;
    const int per_sm = a.cluster == 1 && even <= 3.0 * sms ? 3 : 4;
    const int64_t resident = (int64_t)sms * per_sm / a.cluster;
    const size_t third = 72 * 1024, up_room = per_sm == 3 ? third : 53 * 1024, beside = route + (a.cluster > 1 ? 8192 : 0);
    const int tokens = a.T < kPassTokens ? a.T : kPassTokens;
    a.stage_bytes = S::up_bytes(tokens);
    a.depth = ring_depth(up_room - beside, a.stage_bytes, items > resident ? 16 : (stages + a.cluster - 1) / a.cluster);
    size_t smem = (size_t)a.depth * a.stage_bytes + beside;
    // a plain launch: the down kernel reads ids, weights and blobs before its wait (see pdl_wait)
    cudaError_t e = launch(few_gate_up_kernel<MX>, a, (unsigned)(items < resident ? items : resident), smem, true, false, st);
    if (e != cudaSuccess) return e;
    // down: the (pass, K stage) list of an output tile in slices, as many as fill the GPU
    // once at three CTAs per SM
    const int64_t list = (int64_t)a.slot_cap * ((a.I + S::kCols - 1) / S::kCols);
    const int tiles = (a.H + 127) / 128;
    const int slices = down_slices(a.H, list);
    a.stage_bytes = S::down_bytes(tokens);
    // in clusters of up to eight where the ring then leaves room for four CTAs per SM (16
    // tokens of a layer of 8 experts, 256 x 128: 12.5 us, joined by the last CTA 14.4)
    a.cluster = slices < 8 ? slices : 8;
    a.depth = ring_depth(third - route, a.stage_bytes, (list + a.cluster - 1) / a.cluster);
    smem = (size_t)a.depth * a.stage_bytes + route + down_part_bytes(NT, a.cluster);
    const bool clustered = a.cluster > 1 && smem <= 53 * 1024;
    if (!clustered) {
        a.cluster = slices;
        a.depth = ring_depth(third - route, a.stage_bytes, (list + a.cluster - 1) / a.cluster);
        smem = (size_t)a.depth * a.stage_bytes + route;
    }
    const unsigned groups = (unsigned)tiles;
    return clustered ? launch(few_down_kernel<MX, NT, ONE, true>, a, groups, smem, true, pdl_enabled(), st)
                     : launch(few_down_kernel<MX, NT, ONE, false>, a, groups, smem, false, pdl_enabled(), st);
}

cudaError_t launch_few(const FewArgs& a, bool mx, cudaStream_t st) {
    if (a.T <= 2) return mx ? launch_few_nt<true, 1, true>(a, st) : launch_few_nt<false, 1, true>(a, st);
    if (a.T <= 8) return mx ? launch_few_nt<true, 1, false>(a, st) : launch_few_nt<false, 1, false>(a, st);
    if (a.T <= 16) return mx ? launch_few_nt<true, 2, false>(a, st) : launch_few_nt<false, 2, false>(a, st);
    return mx ? launch_few_nt<true, 4, false>(a, st) : launch_few_nt<false, 4, false>(a, st);
}

// Workspace: h (three parts), the down kernel's slices and its counters.
struct FewWs {
    size_t part, joined, total;
};
FewWs few_ws(int T, int topk, int H, int I) {
    FewWs w;
    w.part = (size_t)T * (size_t)topk * (((size_t)I + 255) / 256 * 256) * 6;
    const size_t tiles = ((size_t)H + 127) / 128, nt = T <= 8 ? 1 : (T <= 16 ? 2 : 4);
    w.joined = w.part + tiles * (size_t)down_slices(H, INT32_MAX) * kConsumers * 2 * nt * 512;
    w.total = w.joined + (tiles * 4 + 255) / 256 * 256;
    return w;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

size_t chord_moe_few_workspace_bytes(int T, int topk, int E, int H, int I) {
    if (T < 0 || topk <= 0 || E <= 0 || H <= 0 || I <= 0) return 0;
    return few_ws(T, topk, H, I).total;
}

chord_status chord_moe_layer_few(const void* x, const int32_t* topk_ids, const float* topk_w, int T, int topk, int E,
                                 int H, int I, int weights, const void* packed_w13, size_t w13_bytes,
                                 const void* packed_w2, size_t w2_bytes, void* workspace, size_t workspace_bytes,
                                 void* out, const chord_opts* opts, void* stream) {
    if (T < 0 || topk <= 0 || E <= 0 || H <= 0 || I <= 0) return CHORD_ERR_INVALID_ARG;
    if (weights != CHORD_WEIGHTS_INT4 && weights != CHORD_WEIGHTS_MXFP4) return CHORD_ERR_INVALID_ARG;
    if (T > CHORD_FEW_MAX_TOKENS || topk > 32 || E > 1024 || H > (1 << 20) || I > (1 << 20))
        return CHORD_ERR_UNSUPPORTED;
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
    a.Ip = (I + 255) / 256 * 256;
    const FewWs ws = few_ws(T, topk, H, I);
    a.part = reinterpret_cast<float4*>(static_cast<uint8_t*>(workspace) + ws.part);
    a.joined = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + ws.joined);
    // every used expert's tokens in passes of eight
    const int P = T * topk, many = E + P / kPassTokens;
    a.slot_cap = P < many ? P : many;
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
