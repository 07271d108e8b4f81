// F8 products on the block-scaled tensor cores: f8_gemm and f8_gemm_experts.
//
//   Y[t][o] = sum_g 2^(ex[t][g] - 127) 2^(ew[o / 128][g] - 127) sum_{i in group g} x[t][i] w[o][i]
//
// with e4m3 codes x, w and scale bytes ex (one per 128 values of a row), ew (one per
// 128 x 128 block).  tcgen05.mma of kind mxf8f6f4 multiplies both operands' scales into the
// products itself: it takes one scale byte per operand row and 32 values of K, picked out
// of a 32-bit word in tensor memory by a byte index in the instruction descriptor.  The
// four instructions of a 128-value group name the same byte, so a word as it stands in
// memory (the bytes of four groups) serves sixteen instructions, and no value passes
// through a register before the epilogue.
//
// The weight rows are the M = 128 side (lanes of tensor memory), so the scale of a tile's
// 128 rows is one byte; the tokens are the N side, in steps of 16, so a ragged tile costs
// what its rows cost.
//
// One persistent CTA per SM.  Warp roles:
//   warps 0-7   epilogue: tcgen05.ld of a lane quarter, through shared memory to whole output
//               rows of 128 columns, gated unit, store; two groups of four warps take
//               alternate pieces of 16 tokens
//   warps 8-11  scales: words of both operands to shared memory, four groups ahead
//   warp 12     copies: per stage 128 weight rows and the tile's token rows, 128 bytes of K
//   warp 13     tcgen05.cp of the scale words to tensor memory, tcgen05.mma (four per stage, K = 32
//               each); allocates tensor memory
// Tensor memory: two fp32 accumulators of BT columns (the epilogue of a tile overlaps the
// next main loop), then a few buffers of scale words.
// Every mbarrier wait is bounded, and begins after the dependent-launch wait: it never counts the
// time of the kernel before.  On expiry the CTA raises the device error word, waits for what
// it has in flight (again bounded), frees its tensor memory and returns.
//
// What bounds it, measured on one GB300:
//   few tokens   the weights' bytes: 1x128256x4096 78 us (6.7 TB/s, the copy rate), 1x8192x28672
//                36.6 us; 32 rows over 24 experts of 4096x4096 65 us (6.2 TB/s).  A stage costs the
//                issuing thread about 420 cycles (two waits, the scale copies, four MMAs, two
//                commits), half of the 800 that its 18 KB take at the memory's rate.  Small
//                matrices are bound by the launch and one pipeline fill: 1x4096x4096 5.2 us.
//   many tokens  the power limit: 2048x28672x8192 with N(0,1) operands runs at 3.5 PFLOP/s for the
//                first milliseconds and 3.0 to 3.1 at the 1.4 to 1.5 GHz that 1400 W leave
//                (bf16 library product, same shape: 2.0 and 1.7): 0.86 to 0.89 of the tensor rate
//                at that clock (16384 operations a cycle and SM).  Calls at K = 8192 fit 256 + h
//                cycles for a stage of h rows, of which the tensor work alone is 2 h: what is left
//                at few rows is shared memory.

#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tensor_core.cuh"

namespace cq {
namespace {

constexpr int kRows = 128;              // weight rows per tile (MMA M, lanes)
constexpr int kKB = 128;                // K per stage: one scale group, one swizzle row
constexpr int kEpiWarps = 8;            // two groups of four, one warp per lane quarter
constexpr int kScaleWarp0 = kEpiWarps;
constexpr int kCopyWarp = kScaleWarp0 + 4;
constexpr int kMmaWarp = kCopyWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kScaleSlots = 4;          // groups of scale words in shared memory, one per scale warp
constexpr int kEpiRows = 8;             // tokens per step of the epilogue
constexpr int kTmem = 512;
constexpr int kSmemMax = 227 * 1024;

// Tile configuration of one kernel instance.
//   BT       tokens per tile at most
//   EXPERTS  rows grouped by expert
//   PAIR     two CTAs share a tile of 256 weight rows: each holds 128 of them and half of the
//            tokens, and one tcgen05.mma (cta_group::2) reads both halves, so a stage brings
//            half the token bytes into each SM for the same work
//   SPLIT    the CTAs of a cluster (2, 4 or 8) share a tile along K: each holds a partial sum
//            of a range of K, and adds up its share of the tokens through the others'
//            shared memory, in rank order.  For few tiles, where whole rows would leave SMs
//            without work
template <int BT_, bool EXPERTS_, bool PAIR_ = false, bool SPLIT_ = false>
struct F8Cfg {
    static constexpr int BT = BT_;
    static constexpr bool EXPERTS = EXPERTS_;
    static constexpr bool PAIR = PAIR_;
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int CTAS = PAIR ? 2 : 1;            // CTAs that share an instruction
    static constexpr int XROWS = BT / CTAS;              // token rows of a CTA's stage
    static constexpr int XBOX = XROWS % 56 == 0 ? 56 : PAIR ? 64 : XROWS < 32 ? XROWS : 32;   // token rows per copy
    static constexpr int STAGE = (kRows + XROWS) * kKB;
    static constexpr int STMEM = PAIR ? 2 : 4;           // buffers of scale words in tensor memory
    static constexpr int XCHUNKS = (BT + 127) / 128;     // 128 token rows of scale words each
    static constexpr int SCOLS = 4 + 4 * XCHUNKS;
    // Tensor memory: two accumulators, then the scale words.  256 tokens a tile leave them 480
    // columns: they share 32 (224 .. 255), which the epilogue reads first, so the next tile's
    // MMAs wait for those alone.
    static constexpr bool SHARED = BT == 256;
    static constexpr int ACC1 = SHARED ? 224 : BT;       // first column of the second accumulator
    static constexpr int SCOL0 = ACC1 + BT;
    static constexpr int SSLOT = 512 + 512 * XCHUNKS;    // scale words of a group: weights, tokens
    static constexpr int TABLE = EXPERTS ? (2 * CQ_MOE_MAX_EXPERTS + 2) * 4 + 2 * CQ_MOE_MAX_EXPERTS : 0;
    // output rows: one step of each epilogue group, or the partial rows of a whole tile
    static constexpr int ROWS = (SPLIT ? BT : 2 * kEpiRows) * kRows * 4;
    // alignment, output rows, scale words, barriers, expert tables
    static constexpr int FIXED = 1024 + ROWS + kScaleSlots * SSLOT + 512 + TABLE;
    static constexpr int STAGES = (kSmemMax - FIXED) / STAGE < 12 ? (kSmemMax - FIXED) / STAGE : 12;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static_assert(BT % 16 == 0 && XROWS % XBOX == 0 && XBOX % 8 == 0 && BT <= 256, "MMA N and copy boxes");
    static_assert(SCOL0 + STMEM * SCOLS <= kTmem, "tensor memory budget");
    static_assert(SMEM <= kSmemMax, "shared memory budget");
    static_assert((2 * STAGES + 2 * kScaleSlots + 7) * 8 + 16 <= 512, "barrier block");
    static_assert(!(PAIR && SPLIT), "one use of the cluster");
};

struct F8Params {
    CUtensorMap wmap;          // weight codes [E][N][Kp], box 128 x 128 x 1
    CUtensorMap xmap;          // token codes [R][Kp], box 128 x XBOX
    const uint8_t* ws;         // [E][ceil(N / 128)][Ks]
    const uint8_t* xs;         // [R][Ks]
    const int32_t* offsets;    // [E + 1] (experts)
    void* Y;                   // [R][cols]
    int E, N, R;
    int kb;                    // groups of 128 along K
    int Ks;                    // scale bytes per row
    int tn;                    // blocks of 128 along N
    int bt;                    // tokens per tile at most: BT, or less
    int split;                 // CTAs that share a tile along K
    int segs;                  // runs of K with an accumulator of their own
    int gated;
    int f32;                   // output type
    unsigned int* err;
    unsigned long long timeout_ns;
};

// Tensor copies into this CTA's shared memory that complete on barrier `bar` (a shared::cluster
// address).  PAIR: the barrier may be the other CTA's.
template <bool PAIR>
__device__ __forceinline__ void copy_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z),
            "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z),
            "r"(bar)
            : "memory");
}
// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The completion of every MMA issued so far by this thread arrives on `bar`: on this CTA's, or
// on both CTAs' of a pair.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else umma_commit(bar);
}
// the same on this CTA's barrier alone
template <bool PAIR>
__device__ __forceinline__ void umma_commit_one(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
    else umma_commit(bar);
}

// Instruction descriptor, kind mxf8f6f4: fp32 accumulator, A and B e4m3, both K-major, scale
// bytes as powers of two.  The byte indexes of the scales are added per group.
__device__ __forceinline__ uint32_t idesc_mxf8(int m, int n) {
    return ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27);
}
__device__ __forceinline__ uint32_t idesc_byte(int j) { return ((uint32_t)j << 4) | ((uint32_t)j << 29); }

template <bool PAIR>
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                          uint32_t sb, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}
// 32 rows of 16 bytes from shared memory (unswizzled, 8-row groups 128 bytes apart) to four
// columns of tensor memory, the same in every lane quarter
__device__ __forceinline__ uint64_t smem_desc_rows16(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}
template <bool PAIR>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// waits for the load of r: the values are named so that nothing that uses them moves above
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}

// One output tile of a CTA: weight rows 128 nb .. of matrix e, token rows [t0, t0 + n).
struct F8Tile {
    int e, nb, t0, n;
};

// Height of the `tm` token tiles of `rows` rows: about equal, at most bt, and (tm - 1) h < rows.
__device__ __forceinline__ int tile_height(int rows, int tm) { return ((rows + tm - 1) / tm + 15) & ~15; }

// What the kernel knows of the experts, in shared memory.
struct F8Experts {
    int* off;           // [E + 1] row offsets
    int* first;         // [E + 1] tile number at which each place of the order starts
    uint16_t* order;    // [E] experts in the order of their tiles
};

// The tiles of a CTA or cluster: its number, + the number of clusters, ...  Token tiles of a
// weight tile are neighbours.
template <class C>
struct TileWalk {
    const F8Params& p;
    const F8Experts& x;
    int tile, step, end, e, rank;
    __device__ TileWalk(const F8Params& p_, const F8Experts& x_, int rank_, int size)
        : p(p_), x(x_), tile((int)blockIdx.x / size), step((int)gridDim.x / size), e(0), rank(C::PAIR ? rank_ : 0) {
        end = C::EXPERTS ? x.first[p.E] : (p.R + p.bt - 1) / p.bt * weight_tiles(p);
    }
    __device__ static int weight_tiles(const F8Params& p) { return (p.tn + C::CTAS - 1) / C::CTAS; }
    __device__ bool more() const { return tile < end; }
    __device__ bool next(F8Tile& t) {
        if (tile >= end) return false;
        int local = tile, r0 = 0, r1 = p.R;
        t.e = 0;
        if constexpr (C::EXPERTS) {
            while (x.first[e + 1] <= tile) ++e;
            local = tile - x.first[e];
            t.e = x.order[e];
            r0 = x.off[t.e];
            r1 = x.off[t.e + 1];
        }
        const int rows = r1 - r0, tm = (rows + p.bt - 1) / p.bt;
        const int h = tile_height(rows, tm);
        const int nt = local / tm;
        t.nb = nt * C::CTAS + rank;
        t.t0 = r0 + (local - nt * tm) * h;
        t.n = min(h, r1 - t.t0);
        tile += step;
        return true;
    }
};

// Fills F8Experts from the caller's offsets.  All threads of the CTA call it; they synchronise
// after it.  Pairs (tiles bound by their MMAs) take the experts with the highest tiles first:
// dealt in turn, tiles in descending order leave no cluster more than one tile ahead, where the
// caller's order left the busiest of 76 pairs 4 to 8 % above its share (64 experts of uneven
// popularity, 32768 rows).  Beyond 256 experts the counting of ranks would take longer.
// Runs of tiles per cluster, which balance as well, were twice as slow: all experts are then
// in flight at once, and their rows leave the L2 cache before the next weight tile needs them.
template <class C>
__device__ __forceinline__ void plan_experts(const F8Params& p, const F8Experts& x) {
    const int tid = threadIdx.x, lane = tid & 31;
    // held inside [0, R] and ascending whatever the caller's array says
    for (int e = tid; e <= p.E; e += kThreads) x.off[e] = min(max(__ldg(p.offsets + e), 0), p.R);
    __syncthreads();
    if (tid < 32) {
        int low = x.off[0];
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int hi = e < p.E ? x.off[e + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, hi, o);
                if (lane >= o) hi = max(hi, u);
            }
            hi = max(hi, low);
            if (e < p.E) x.off[e + 1] = hi;
            low = __shfl_sync(0xffffffffu, hi, 31);
        }
    }
    __syncthreads();
    auto height = [&](int e) {   // 0 for an expert without rows
        const int rows = x.off[e + 1] - x.off[e];
        return rows > 0 ? tile_height(rows, (rows + p.bt - 1) / p.bt) : 0;
    };
    if (C::PAIR && p.E <= 256) {
        for (int e = tid; e < p.E; e += kThreads) x.first[e] = height(e);
        __syncthreads();
        for (int e = tid; e < p.E; e += kThreads) {
            const int h = x.first[e];
            int place = 0;
            for (int i = 0; i < p.E; ++i) place += x.first[i] > h || (x.first[i] == h && i < e) ? 1 : 0;
            x.order[place] = (uint16_t)e;
        }
    } else {
        for (int e = tid; e < p.E; e += kThreads) x.order[e] = (uint16_t)e;
    }
    __syncthreads();
    if (tid < 32) {
        int run = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            int tiles = 0;
            if (e0 + lane < p.E) {
                const int e = x.order[e0 + lane];
                tiles = (x.off[e + 1] - x.off[e] + p.bt - 1) / p.bt * TileWalk<C>::weight_tiles(p);
            }
            int inc = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            if (e0 + lane < p.E) x.first[e0 + lane] = run + inc - tiles;
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) x.first[p.E] = run;
    }
}

__device__ __forceinline__ float rcp_approx(float x) {   // 1 ulp; 0 for infinity
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// g / (1 + exp(-g)) * u, with h = exp(-|g| / 2):  g u / (1 + h^2) for g >= 0, (g h) (u h) / (1 + h^2)
// below.  The square root keeps h a normal number down to g = -174, where h^2 no longer is, so
// that a result that a large u makes a normal number is right; from there on h = 0, an error
// of at most 2^-240 |u|.  h = 2^-t with t + lo = |g| / 2 log2(e), log2(e) in two pieces, so the
// rounding of t does not grow with |g|.  Within 17 * 2^-24 of the result: h twice (ex2 4, the
// product 1), rcp 2, and five roundings.  g = -infinity gives NaN, as the formula does.
__device__ __forceinline__ float silu_mul(float g, float u) {
    constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453;
    constexpr float kHi = (float)(0.5 * kLog2e), kLo = (float)(0.5 * kLog2e - (double)kHi);
    const float c = fminf(fabsf(g), 1024.0f);   // h is 0 long before
    const float t = kHi * c;
    const float lo = fmaf(kLo, c, fmaf(kHi, c, -t));
    float h;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(-t));
    h = fmaf(h, lo * (float)-kLn2, h);
    const float w = g < 0.0f ? h : 1.0f;
    return g * w * rcp_approx(fmaf(h, h, 1.0f)) * (u * w);
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void put(float* y, float v) { *y = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put2(float* y, float a, float b) { *reinterpret_cast<float2*>(y) = make_float2(a, b); }
__device__ __forceinline__ void put2(__nv_bfloat16* y, float a, float b) { *reinterpret_cast<uint32_t*>(y) = bf16x2(a, b); }
__device__ __forceinline__ void put4(float* y, float4 v) { *reinterpret_cast<float4*>(y) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16* y, float4 v) {
    *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
}
// Four consecutive products of a token (weight rows o .., `left` of them up to N), or the two
// gated values they make, to y.  VEC: N is a multiple of 4, so a store is a whole vector.
template <typename TO, bool GATED, bool VEC>
__device__ __forceinline__ void store4(uint8_t* at, float4 v, int left) {
    TO* y = reinterpret_cast<TO*>(at);
    if constexpr (GATED) {
        const float a = silu_mul(v.x, v.y), b = silu_mul(v.z, v.w);
        if constexpr (VEC) {
            put2(y, a, b);
        } else {
            put(y, a);
            if (left > 2) put(y + 1, b);
        }
    } else if constexpr (VEC) {
        put4(y, v);
    } else {
        put(y, v.x);
        if (left > 1) put(y + 1, v.y);
        if (left > 2) put(y + 2, v.z);
        if (left > 3) put(y + 3, v.w);
    }
}
// Two rows at once: one choice of the kind, two independent chains.
template <typename TO, bool GATED, bool VEC>
__device__ __forceinline__ void store_rows(uint8_t* ya, float4 va, bool a, uint8_t* yb, float4 vb, bool b, int left) {
    if (a) store4<TO, GATED, VEC>(ya, va, left);
    if (b) store4<TO, GATED, VEC>(yb, vb, left);
}
// Where a lane's four columns of a tile go.
struct F8Out {
    uint8_t* y;       // of the tile's first token
    int64_t pitch;    // bytes per token
    int left;         // weight rows from the lane's first one to N
    int kind;         // float32, gated, odd N: bits 0, 1, 2
    __device__ __forceinline__ F8Out(const F8Params& p, const F8Tile& t, int lane) {
        const int o = t.nb * kRows + 4 * lane;
        const int sh = p.f32 ? 2 : 1;
        pitch = (int64_t)(p.gated ? p.N >> 1 : p.N) << sh;
        left = p.N - o;
        kind = (p.f32 ? 1 : 0) | (p.gated ? 2 : 0) | ((p.N & 3) ? 4 : 0);
        y = static_cast<uint8_t*>(p.Y) + (int64_t)t.t0 * pitch + ((int64_t)(p.gated ? o >> 1 : o) << sh);
    }
    // what an earlier run of K left at y (float32, not gated), as far as the row goes
    __device__ __forceinline__ float4 before(const uint8_t* y, bool there) const {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!there || left <= 0) return v;
        const float* f = reinterpret_cast<const float*>(y);
        if (!(kind & 4)) return *reinterpret_cast<const float4*>(f);
        v.x = f[0];
        if (left > 1) v.y = f[1];
        if (left > 2) v.z = f[2];
        if (left > 3) v.w = f[3];
        return v;
    }
    __device__ __forceinline__ void rows(uint8_t* ya, float4 va, bool a, uint8_t* yb, float4 vb, bool b) const {
        using bf16 = __nv_bfloat16;
        a = a && left > 0;
        b = b && left > 0;
        if (kind == 0) store_rows<bf16, false, true>(ya, va, a, yb, vb, b, left);
        else if (kind == 2) store_rows<bf16, true, true>(ya, va, a, yb, vb, b, left);
        else if (kind == 1) store_rows<float, false, true>(ya, va, a, yb, vb, b, left);
        else if (kind == 3) store_rows<float, true, true>(ya, va, a, yb, vb, b, left);
        else if (kind == 4) store_rows<bf16, false, false>(ya, va, a, yb, vb, b, left);
        else if (kind == 6) store_rows<bf16, true, false>(ya, va, a, yb, vb, b, left);
        else if (kind == 5) store_rows<float, false, false>(ya, va, a, yb, vb, b, left);
        else store_rows<float, true, false>(ya, va, a, yb, vb, b, left);
    }
};

// whether all epilogue warps say yes (also their barrier)
__device__ __forceinline__ bool epilogue_agree(bool yes) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n"
        " selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)yes), "n"(kEpiWarps * 32)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + group) : "memory");
}
// a word to another CTA's shared memory; four bytes less to wait for on its barrier
__device__ __forceinline__ void store_async(uint32_t addr, uint32_t v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(addr), "r"(v),
                 "r"(bar)
                 : "memory");
}
template <class C>
__global__ void __launch_bounds__(kThreads, 1) f8_gemm_kernel(const __grid_constant__ F8Params p) {
    constexpr int kStages = C::STAGES;
    constexpr bool kPair = C::PAIR, kSplit = C::SPLIT, kCluster = kPair || kSplit;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* rows = reinterpret_cast<float*>(ring + kStages * C::STAGE);   // output rows of 128
    uint8_t* slots = ring + kStages * C::STAGE + C::ROWS;                // scale words
    uint64_t* full = reinterpret_cast<uint64_t*>(slots + kScaleSlots * C::SSLOT);   // copies landed
    uint64_t* empty = full + kStages;                  // stage read by the MMA
    uint64_t* sf_full = empty + kStages;               // scale words written
    uint64_t* sf_empty = sf_full + kScaleSlots;        // scale words read
    uint64_t* acc_full = sf_empty + kScaleSlots;       // [2] accumulator complete
    uint64_t* acc_empty = acc_full + 2;                // [2] accumulator read
    uint64_t* part_full = acc_empty + 2;               // the partial rows of all CTAs are here (split)
    uint64_t* part_empty = part_full + 1;              // every CTA has read its partial rows (split)
    uint64_t* drain = part_empty + 1;                  // used only when a wait ran out
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    F8Experts experts;
    experts.off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 512);
    experts.first = experts.off + CQ_MOE_MAX_EXPERTS + 1;
    experts.order = reinterpret_cast<uint16_t*>(experts.first + CQ_MOE_MAX_EXPERTS + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // pair: CTA 0 issues the MMAs; full, sf_full and acc_empty count on its copy of the barriers
    const uint32_t rank = kCluster ? cluster_rank() : 0u;
    const int size = kSplit ? p.split : C::CTAS;
    pdl_trigger();
    if (tid < 32) {   // one barrier of each kind per lane
        if (lane < kStages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < kScaleSlots) {
            mbar_init(&sf_full[lane], C::CTAS);
            mbar_init(&sf_empty[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&acc_full[lane], 1);
            mbar_init(&acc_empty[lane], kEpiWarps * C::CTAS);
        }
        if (lane == 0) {
            mbar_init(part_full, 1);
            mbar_init(part_empty, kEpiWarps * (uint32_t)size);
            *abort_flag = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (C::EXPERTS && warp == kCopyWarp && lane == 0) {   // dense: the first copies go out at once
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.wmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.xmap)) : "memory");
    }
    if (warp == kMmaWarp) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(kTmem));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(kTmem));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kCluster) cluster_sync();   // the barriers of all CTAs are set up
    tc_fence_after();
    if constexpr (C::EXPERTS) {
        pdl_wait();
        plan_experts<C>(p, experts);
        __syncthreads();
    }
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t* b, uint32_t parity) {
        return mbar_wait_until<kCluster>(b, parity, abort_flag, p.err, p.timeout_ns);
    };
    // arrive on CTA 0's copy of a barrier
    auto arrive0 = [&](uint64_t* b) {
        if constexpr (kPair) cluster_arrive(cluster_addr(b, 0u));
        else mbar_arrive(b);
    };
    // the whole warp waits, and gives up together
    auto wait_warp = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
    TileWalk<C> walk(p, experts, (int)rank, size);
    F8Tile t;
    // this CTA's groups of 128 along K
    const int k0 = kSplit ? (int)((int64_t)p.kb * rank / (uint32_t)size) : 0;
    const int k1 = kSplit ? (int)((int64_t)p.kb * (rank + 1) / (uint32_t)size) : p.kb;
    // where its run `seg` of them begins
    auto run_begin = [&](int seg) { return k0 + (int)((int64_t)(k1 - k0) * seg / p.segs); };
    int issued = 0;   // stages that this thread has issued copies for (copy warp)

    if (warp < kEpiWarps) {
        // ------------------------------ epilogue ----------------------------------
        // Pieces of 16 tokens, alternating between two groups of four warps, in steps of eight.
        // Each warp of a group brings its 32 weight rows of a step to shared memory; then it
        // reads two of the step's rows of 128 products, four to a lane, and stores them.
        if constexpr (!C::EXPERTS) pdl_wait();
        const int quarter = warp & 3, group = warp >> 2;
        const uint32_t lane0 = tmem + ((uint32_t)(quarter * 32) << 16);
        // this group's step in shared memory: where this lane puts its weight row, and finds four
        float* put_at = rows + group * (kEpiRows * kRows) + quarter * 32 + lane;
        const float4* get_at = reinterpret_cast<const float4*>(rows + (group * kEpiRows + quarter) * kRows) + lane;
        bool ok = true;
        for (int it = 0, seg = 0; ok; ++it, seg = seg + 1 < p.segs ? seg + 1 : 0) {
            if (seg == 0 && !walk.next(t)) break;
            const int buf = it & 1;
            const uint32_t col0 = lane0 + (uint32_t)(buf * C::ACC1);
            const int pieces = (t.n + 15) / 16;
            const F8Out out(p, t, lane);
            const int64_t half = 4 * out.pitch;
            auto read_done = [&] {   // the accumulator (or the shared part of it) is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive0(&acc_empty[C::SHARED ? 0 : buf]);
            };
            ok = wait_warp(&acc_full[buf], (uint32_t)((it >> 1) & 1));
            if constexpr (kSplit) {
                if (!ok) break;
            }
            tc_fence_after();
            if constexpr (!kSplit) {
                // this group's pieces: group, group + 2, ...; in a tile of more than 14 whose last
                // columns are the shared ones, 14 + group comes first
                constexpr int kLast = 14;
                const bool turned = C::SHARED && buf == 0 && pieces > kLast;
                const int upto = turned ? kLast : pieces;
                const int head = turned && kLast + group < pieces ? kLast + group : group;
                auto after = [&](int c) { return c >= upto ? group : c + 2; };   // >= upto: no more
                uint32_t r[2][16];
                int c = head;
                const bool any = ok && c < pieces;
                if (any) tmem_ld16_async(col0 + (uint32_t)(16 * c), r[0]);
                if (C::SHARED && any) tmem_wait_ld16(r[0]);
                if (C::SHARED || !any) read_done();   // first of all: the next tile's MMAs wait for it
                ok = epilogue_agree(ok);
                if (!ok) {
                    if (any) tmem_wait_ld16(r[0]);
                    break;
                }
                // an earlier run's sums of this warp's four rows of a piece, on their way a piece ahead
                auto sums_of = [&](int c, float4 (&o)[4]) {
                    const uint8_t* ya = out.y + (16 * c + quarter) * out.pitch;
                    const int left = t.n - 16 * c - quarter;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = out.before(ya + i * half, left > 4 * i);
                };
                float4 sums[2][4];
                auto piece = [&](auto adds, uint32_t (&cur)[16], uint32_t (&nxt)[16], const float4 (&sum)[4],
                                 float4 (&next_sum)[4]) {
                    constexpr bool kAdd = decltype(adds)::value;   // to an earlier run's sum
                    tmem_wait_ld16(cur);
                    const int next = after(c);
                    // 16 columns a load: its issue takes 70 to 300 cycles, whatever the width
                    if (next < upto) tmem_ld16_async(col0 + (uint32_t)(16 * next), nxt);
                    if (!C::SHARED && next >= upto) read_done();
                    if constexpr (kAdd) {
                        if (next < upto) sums_of(next, next_sum);
                    }
                    uint8_t* ya = out.y + (16 * c + quarter) * out.pitch;
                    int left = t.n - 16 * c - quarter;   // tokens from this warp's row on
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h && 16 * c + 8 >= t.n) break;
                        group_sync(group);   // the group has read its previous step
#pragma unroll
                        for (int j = 0; j < kEpiRows; ++j) put_at[j * kRows] = __uint_as_float(cur[8 * h + j]);
                        group_sync(group);
                        float4 va = get_at[0], vb = get_at[kRows];   // rows quarter and quarter + 4
                        if constexpr (kAdd) {
                            const float4 oa = sum[2 * h], ob = sum[2 * h + 1];
                            va = make_float4(va.x + oa.x, va.y + oa.y, va.z + oa.z, va.w + oa.w);
                            vb = make_float4(vb.x + ob.x, vb.y + ob.y, vb.z + ob.z, vb.w + ob.w);
                        }
                        out.rows(ya, va, left > 0, ya + half, vb, left > 4);
                        ya += 2 * half;
                        left -= kEpiRows;
                    }
                    c = next;
                    return next < upto;
                };
                if (any && seg == 0) {
                    while (piece(std::false_type(), r[0], r[1], sums[0], sums[1]) &&
                           piece(std::false_type(), r[1], r[0], sums[1], sums[0])) {}
                } else if (any) {
                    sums_of(c, sums[0]);
                    while (piece(std::true_type(), r[0], r[1], sums[0], sums[1]) &&
                           piece(std::true_type(), r[1], r[0], sums[1], sums[0])) {}
                }
            } else {
                // Token i of the tile belongs to CTA i % size: every CTA sends its partial row there,
                // to row (rank, i / size) of the owner's shared memory.  The owner's barrier
                // counts the bytes; it adds the partial rows in rank order.
                const int lg = __ffs(size) - 1, per = C::BT >> lg;   // rows of each rank
                const uint32_t ph = (uint32_t)(it & 1);
                const int own = t.n > (int)rank ? ((t.n - 1 - (int)rank) >> lg) + 1 : 0;
                if (tid == 0) mbar_arrive_tx(part_full, (uint32_t)(own * size * kRows * 4));
                if (!wait_warp(part_empty, ph ^ 1u)) break;          // the last tile's have been read
                const uint32_t at = smem_u32(rows) + (uint32_t)(((int)rank * per * kRows + quarter * 32 + lane) * 4);
                for (int c = group; c < pieces; c += 2) {
                    uint32_t r[16];
                    tmem_ld16_async(col0 + (uint32_t)(16 * c), r);
                    tmem_wait_ld16(r);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int i = 16 * c + j;
                        if (i < t.n) {
                            const uint32_t to = (uint32_t)(i & (size - 1));
                            store_async(map_rank(at + (uint32_t)((i >> lg) * (kRows * 4)), to), r[j],
                                        cluster_addr(part_full, to));
                        }
                    }
                }
                read_done();
                if (!wait_warp(part_full, ph)) break;
                for (int i = warp; i < own; i += kEpiWarps) {
                    const float4* row = reinterpret_cast<const float4*>(rows + i * kRows) + lane;
                    uint8_t* y = out.y + ((i << lg) + (int)rank) * out.pitch;
                    const float4 o = out.before(y, seg > 0);
                    float4 v = row[0];
                    for (int k = 1; k < size; ++k) {
                        const float4 w = row[k * per * (kRows / 4)];
                        v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
                    }
                    if (seg > 0) v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
                    out.rows(y, v, true, y, v, false);
                }
                // not after the last tile: a CTA that has its partial rows may then leave
                if (walk.more() || seg + 1 < p.segs) {
                    __syncwarp();
                    if (lane < size) cluster_arrive(cluster_addr(part_empty, (uint32_t)lane));
                }
            }
        }
    } else if (warp < kCopyWarp) {
        // ------------------------------ scales ------------------------------------
        // each warp takes every fourth group of scale words, into a slot of its own: row
        // 128 c + 32 j + i of an operand is word j of the 16 bytes of row i of chunk c, the
        // order in which the MMA reads the words from lane i of columns 4 c + j
        if constexpr (!C::EXPERTS) pdl_wait();
        const int sw = warp - kScaleWarp0;
        uint32_t* slot = reinterpret_cast<uint32_t*>(slots + sw * C::SSLOT);
        int it = 0, used = 0;
        bool ok = true;
        while (ok && walk.next(t)) {
            const bool wok = t.nb < p.tn;   // the second CTA of a pair may have no weight rows
            for (int seg = 0; ok && seg < p.segs; ++seg) {
                const int q0 = run_begin(seg) >> 2, quads = ((run_begin(seg + 1) - 1) >> 2) - q0 + 1;
                const uint32_t* wsrc =
                    reinterpret_cast<const uint32_t*>(p.ws + ((int64_t)t.e * p.tn + (wok ? t.nb : 0)) * p.Ks) + q0;
                for (int q = (sw - it) & 3; q < quads; q += 4, ++used) {
                    const uint32_t w = wok ? __ldg(wsrc + q) : 0x7F7F7F7Fu;
                    uint4 x[C::XCHUNKS];
#pragma unroll
                    for (int c = 0; c < C::XCHUNKS; ++c) {
                        uint32_t* xw = reinterpret_cast<uint32_t*>(&x[c]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 128 * c + 32 * j + lane;
                            xw[j] = r < t.n ? __ldg(reinterpret_cast<const uint32_t*>(p.xs + (int64_t)(t.t0 + r) * p.Ks) +
                                                    q0 + q)
                                            : 0x7F7F7F7Fu;
                        }
                    }
                    if (!wait_warp(&sf_empty[sw], (uint32_t)(used & 1) ^ 1u)) { ok = false; break; }
                    reinterpret_cast<uint4*>(slot)[lane] = make_uint4(w, w, w, w);
#pragma unroll
                    for (int c = 0; c < C::XCHUNKS; ++c) reinterpret_cast<uint4*>(slot + 128 * (c + 1))[lane] = x[c];
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the tensor core reads them
                    __syncwarp();
                    if (lane == 0) arrive0(&sf_full[sw]);
                }
                it += quads;
            }
        }
    } else if (warp == kCopyWarp) {
        // ------------------------------ copies ------------------------------------
        if (elect_lane()) {
            int s = 0;
            uint32_t ph = 0;
            // one stage: the weight rows, and this CTA's token rows, all of the tile's or its half
            // of them (rounded to the MMA's N); whole boxes, rows past the tile are not used
            auto boxes_of = [&](const F8Tile& t) {
                return (((t.n + 15) & ~15) / C::CTAS + C::XBOX - 1) / C::XBOX;
            };
            auto bar_of = [&](int s) { return kPair ? cluster_addr(&full[s], 0u) : smem_u32(&full[s]); };
            auto copy_w = [&](const F8Tile& t, int k, int s) {
                if (rank == 0 || !kPair)
                    mbar_arrive_tx(&full[s], (uint32_t)(C::CTAS * (kRows + boxes_of(t) * C::XBOX) * kKB));
                copy_3d<kPair>(smem_u32(ring + s * C::STAGE), &p.wmap, k * kKB, t.nb * kRows, t.e, bar_of(s));
            };
            auto copy_x = [&](const F8Tile& t, int k, int s) {
                const int x0 = t.t0 + (kPair ? (int)rank * (((t.n + 15) & ~15) / 2) : 0);
                for (int b = 0; b < boxes_of(t); ++b)
                    copy_2d<kPair>(smem_u32(ring + s * C::STAGE) + (uint32_t)((kRows + b * C::XBOX) * kKB), &p.xmap,
                                   k * kKB, x0 + b * C::XBOX, bar_of(s));
            };
            bool any = walk.next(t);
            int k = k0;
            if constexpr (!C::EXPERTS) {
                // the first stages' weights do not depend on the kernel before this one, but for one
                // that ends with weights_written() (after the wait: 1x4096x4096 5.8 -> 6.1 us)
                if (any)
                    for (; k < k1 && issued < kStages; ++k, ++issued) copy_w(t, k, issued);
                pdl_wait();
                for (int i = 0; i < issued; ++i) copy_x(t, k0 + i, i);
                s = issued % kStages;
                ph = issued == kStages ? 1u : 0u;
            }
            while (any) {
                for (; k < k1; ++k) {
                    if (!wait(&empty[s], ph ^ 1u)) break;
                    copy_w(t, k, s);
                    copy_x(t, k, s);
                    ++issued;
                    if (++s == kStages) { s = 0; ph ^= 1u; }
                }
                if (k < k1) break;
                k = k0;
                any = walk.next(t);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------ MMA ---------------------------------------
        // elect.sync, not a test of the lane: the compiler then keeps the operands in uniform
        // registers (four MMAs issue in 60 cycles instead of 316)
        if ((rank == 0 || !kPair) && elect_lane()) {
            if constexpr (!C::EXPERTS) pdl_wait();   // its inputs come no sooner, and its waits are bounded
            int s = 0, g = 0;   // stage, group of scale words
            uint32_t ph = 0, sa = 0;
            bool ok = true;
            const uint64_t sdesc0 = smem_desc_rows16(smem_u32(slots));
            const uint64_t desc0 = smem_desc_sw128(smem_u32(ring));
            for (int it = 0, seg = 0; ok; ++it, seg = seg + 1 < p.segs ? seg + 1 : 0) {
                if (seg == 0 && !walk.next(t)) break;
                const int buf = it & 1;
                if constexpr (C::SHARED) {
                    // the previous tile's shared columns have been read, and so has all of the one
                    // before it (the same warps read them in turn)
                    if (it > 0 && !wait(&acc_empty[0], (uint32_t)((it - 1) & 1))) { ok = false; break; }
                } else if (!wait(&acc_empty[buf], (uint32_t)((it >> 1) & 1) ^ 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * C::ACC1);
                const uint32_t idesc = idesc_mxf8(kRows * C::CTAS, (t.n + 15) & ~15);
                const int b0 = run_begin(seg), b1 = run_begin(seg + 1);
                for (int k = b0; k < b1; ++k) {
                    if ((k & 3) == 0 || k == b0) {
                        // the tensor-memory buffer's previous words have been used ...
                        const int u = g - C::STMEM;
                        if (u >= 0 && !wait(&sf_empty[u % kScaleSlots], (uint32_t)((u / kScaleSlots) & 1))) {
                            ok = false;
                            break;
                        }
                        // ... and the new ones are in their slot; copies and MMAs run in order
                        if (!wait(&sf_full[g % kScaleSlots], (uint32_t)((g / kScaleSlots) & 1))) { ok = false; break; }
                        tc_fence_after();
                        sa = tmem + (uint32_t)(C::SCOL0 + g % C::STMEM * C::SCOLS);
                        const uint64_t sd = sdesc0 + (uint64_t)(g % kScaleSlots * C::SSLOT >> 4);
#pragma unroll
                        for (int c = 0; c <= C::XCHUNKS; ++c)
                            tmem_copy_scales<kPair>(sa + 4u * c, sd + (uint64_t)(512 * c >> 4));
                    }
                    if (!wait(&full[s], ph)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t a = desc0 + (uint64_t)((s * C::STAGE) >> 4);
                    const uint64_t b = a + (uint64_t)((kRows * kKB) >> 4);
                    const uint32_t id = idesc + idesc_byte(k & 3);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // 32 bytes of K: +2 in the 16-byte address field
                        umma_mxf8<kPair>(d, a + 2u * kk, b + 2u * kk, id, sa, sa + 4u, k != b0 || kk != 0 ? 1u : 0u);
                    commit<kPair>(&empty[s]);
                    if (++s == kStages) { s = 0; ph ^= 1u; }
                    if ((k & 3) == 3 || k == b1 - 1) {
                        commit<kPair>(&sf_empty[g % kScaleSlots]);
                        ++g;
                    }
                }
                if (ok) commit<kPair>(&acc_full[buf]);
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a wait ran out, in whichever role: what this CTA has in flight ends before its memory is
        // given back.  (Else the epilogue has waited for every MMA, and those for every copy.)
        volatile int none = 0;
        for (int i = issued > kStages ? issued - kStages : 0; i < issued && (rank == 0 || !kPair); ++i)
            (void)mbar_wait_until<kCluster>(&full[i % kStages], (uint32_t)((i / kStages) & 1), &none, p.err,
                                            100000000ull);
        if (warp == kMmaWarp && (rank == 0 || !kPair) && elect_lane()) {
            mbar_init(drain, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            umma_commit_one<kPair>(drain);
            (void)mbar_wait_until<false>(drain, 0u, &none, p.err, 100000000ull);
        }
        __syncwarp();
    }
    // No CTA's memory is touched by another any more: a pair waits for that; the partial rows of a
    // split tile have all arrived, unless a wait ran out somewhere
    if (kPair || (kSplit && *abort_flag)) cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        if constexpr (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
    }
}

// ---------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------
static __device__ unsigned int g_f8_err;

std::mutex g_f8_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_f8_encode = nullptr;
unsigned int* g_f8_err_ptr[64] = {nullptr};

int g_f8_fit[64][4] = {};   // clusters of 1, 2, 4, 8 CTAs that the device runs at once

template <class C>
cudaLaunchConfig_t f8_config(int grid, int cluster, cudaStream_t cs, cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = cs;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C::PAIR || C::SPLIT ? 2 : 1;
    return cfg;
}

template <class C>
cudaError_t set_smem() {
    return cudaFuncSetAttribute(f8_gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
}

// Every instance holds a whole SM, so one of them says how many clusters of a size fit.
using F8FitCfg = F8Cfg<16, false, false, true>;
cudaError_t fit_clusters(int dev) {
    for (int lg = 0; lg < 4; ++lg) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = f8_config<F8FitCfg>(sm_count() >> lg << lg, 1 << lg, nullptr, attr);
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&g_f8_fit[dev][lg], f8_gemm_kernel<F8FitCfg>, &cfg);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Once per device: the tensor-map encoder, the error word's address, the kernels' shared memory.
cq_status f8_setup(unsigned int** err) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) { set_last_cuda_error((int)e); return CQ_ERR_CUDA; }
    if (dev < 0 || dev >= 64) return CQ_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_f8_mu);
    if (!g_f8_encode) {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) {
            set_last_cuda_error((int)e);
            return CQ_ERR_UNSUPPORTED;
        }
        g_f8_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    if (!g_f8_err_ptr[dev]) {
        void* pe = nullptr;
        e = cudaGetSymbolAddress(&pe, g_f8_err);
        if (e == cudaSuccess) e = set_smem<F8Cfg<16, false>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<32, false>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<64, false>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<128, false>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<224, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<256, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<16, false, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<32, false, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<64, false, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<128, false, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<32, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<64, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<128, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<224, true, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<32, true, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<64, true, false, true>>();
        if (e == cudaSuccess) e = set_smem<F8Cfg<128, true, false, true>>();
        if (e == cudaSuccess) e = fit_clusters(dev);
        if (e != cudaSuccess) { set_last_cuda_error((int)e); return CQ_ERR_CUDA; }
        g_f8_err_ptr[dev] = static_cast<unsigned int*>(pe);
    }
    *err = g_f8_err_ptr[dev];
    return CQ_OK;
}

cq_status code_map(CUtensorMap* map, const void* base, int rank, uint64_t Kp, uint64_t rows, uint64_t mats, int box) {
    cuuint64_t dims[3] = {(cuuint64_t)Kp, (cuuint64_t)rows, (cuuint64_t)mats};
    cuuint64_t strides[2] = {(cuuint64_t)Kp, (cuuint64_t)(Kp * rows)};
    cuuint32_t boxes[3] = {(cuuint32_t)kKB, (cuuint32_t)box, 1u};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUresult r = g_f8_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims,
                                   strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) { set_last_cuda_error((int)r); return CQ_ERR_CUDA; }
    return CQ_OK;
}

// Clusters of `size` CTAs (a power of two) that run at once on the current device.
int f8_fit(int size) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    return g_f8_fit[dev][size == 8 ? 3 : size == 4 ? 2 : size == 2 ? 1 : 0];
}

struct F8Args {
    const uint8_t *wc, *ws, *xc, *xs;
    const int32_t* offsets;
    int64_t E, N, K, R;
    cq_act act;
    void* Y;
    cq_dtype yt;
    cudaStream_t cs;
};

// Output tiles of `rows` weight-row blocks x BT tokens at most: every expert may end in a partial one.
int64_t f8_tiles(const F8Args& a, int BT, int rows) {
    const int64_t tn = (a.N + kRows - 1) / kRows;
    return ((a.R + BT - 1) / BT + (a.offsets ? a.E : 0)) * ((tn + rows - 1) / rows);
}

// Runs of K with an accumulator of their own.  The tensor core cuts off what does not fit the
// accumulator's 24 bits at each of its K / 32 additions, an error that grows with K: up to 1.1e-6 of
// the result (2-norm) at K = 3300 and 3.7e-6 at 15000.  A float32 result keeps runs of at most
// 2048 values apart and adds them with rounding (2e-7 as a rule, at most 1e-6 in ten thousand random
// cases; a float32 product 0.7e-7), a bfloat16 one (2e-3) does not.  A gated one
// needs the whole sum before it is written: f8_least_split spreads its K over a cluster instead.
constexpr int kRunGroups = 16, kGatedRunGroups = 20;   // groups of 128
int f8_runs(const F8Args& a, int kb, int split) {
    if (a.yt != CQ_F32 || a.act != CQ_ACT_NONE) return 1;
    const int per = (kb + split - 1) / split;   // groups of 128 of one CTA
    return (per + kRunGroups - 1) / kRunGroups;
}

template <class C>
cq_status f8_launch(const F8Args& a, int split, int bt = C::BT) {
    F8Params p;
    p.kb = (int)((a.K + kKB - 1) / kKB);
    p.Ks = (p.kb + 3) / 4 * 4;
    p.tn = (int)((a.N + kRows - 1) / kRows);
    unsigned int* err = nullptr;
    cq_status st = f8_setup(&err);
    if (st != CQ_OK) return st;
    const uint64_t Kp = (uint64_t)p.kb * kKB;
    st = code_map(&p.wmap, a.wc, 3, Kp, (uint64_t)a.N, (uint64_t)a.E, kRows);
    if (st == CQ_OK) st = code_map(&p.xmap, a.xc, 2, Kp, (uint64_t)a.R, 1, C::XBOX);
    if (st != CQ_OK) return st;
    p.ws = a.ws; p.xs = a.xs; p.offsets = a.offsets; p.Y = a.Y;
    p.E = (int)a.E; p.N = (int)a.N; p.R = (int)a.R;
    p.bt = bt;
    p.split = split;
    p.segs = f8_runs(a, p.kb, split);
    p.gated = a.act == CQ_ACT_SWIGLU;
    p.f32 = a.yt == CQ_F32;
    p.err = err;
    p.timeout_ns = 2000000000ull;   // 2 s per wait
    const int64_t most = f8_tiles(a, bt, C::CTAS);
    const int size = C::SPLIT ? split : C::CTAS;
    const int fit = f8_fit(size);
    if (fit < 1) return CQ_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = f8_config<C>((int)(most < fit ? most : fit) * size, size, a.cs, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, f8_gemm_kernel<C>, p);
    if (e != cudaSuccess) { set_last_cuda_error((int)e); return CQ_ERR_CUDA; }
    return check_launch();
}

// The fewest CTAs per tile along K: for a gated float32 result as many as leave each at most
// kGatedRunGroups groups, up to the 8 of a cluster.
int f8_least_split(const F8Args& a) {
    const int64_t kb = (a.K + kKB - 1) / kKB;
    int S = 1;
    if (a.yt == CQ_F32 && a.act == CQ_ACT_SWIGLU)
        while (S < 8 && S * kGatedRunGroups < kb) S *= 2;
    return S;
}

// How a call is cut: tokens per tile, CTAs per tile along K, pairs of CTAs or single ones, and the
// cycles that takes.
struct F8Plan {
    int64_t cycles = INT64_MAX;
    int bt = 0, split = 1;
    bool pairs = false;
};

// Cycles that the epilogue of a tile of h rows takes.
int64_t f8_epilogue(const F8Args& a, int64_t h) { return (a.act == CQ_ACT_SWIGLU ? 27 : 18) * h; }

// The best split of tiles of bt rows, of which h are used.  The costs fit times of single calls in
// a graph, 4 to 64 groups along K, 4 to 300 tiles, splits 1 to 8:
//   a stage (128 values of K)       300 cycles up to 32 rows, 360 at 64, 390 at 128 (there 650 when
//                                   split: the exchange buffer takes half of the ring)
//   from a CTA's tile to the next   1400, and no less than the epilogue
//   the exchange of partial sums    1300 + 18 a row
//   beyond half of the SMs          300 max(4, split): the next call's CTAs cannot start early
// 64 tokens, N x K, us, CTAs per tile 1 / 2 / 4 / 8:
//   4096 x 4096, 64 rows   9.2  8.2  7.4 10.2     32 rows   8.3  7.6  8.1 13.0
//   1024 x 8192, 64 rows  14.6 10.3  7.3  5.9     32 rows  13.3  9.2  6.5  7.1
//   1536 x 512,  64 rows   3.9  5.0  4.6    -     32 rows   3.4  4.2  4.4    -
F8Plan f8_narrow_plan(const F8Args& a, int bt, int64_t h, int64_t tiles) {
    const int64_t kb = (a.K + kKB - 1) / kKB, epi = f8_epilogue(a, h), ctas = f8_fit(1);
    F8Plan best;
    for (int S = f8_least_split(a); S <= 8 && S <= kb; S *= 2) {
        const int64_t fit = f8_fit(S);
        if (fit < 1) break;
        const int64_t stages = (kb + S - 1) / S * (bt <= 32 ? 300 : bt <= 64 ? 360 : S > 1 ? 650 : 390) + 300;
        int64_t cycles = stages + (tiles - 1) / fit * (std::max(stages, epi) + 1400) + epi;
        if (S > 1) cycles += 1300 + 18 * h;
        if (2 * tiles * S > ctas) cycles += 300 * std::max(4, S);
        if (cycles < best.cycles) {
            best.cycles = cycles;
            best.bt = bt;
            best.split = S;
        }
    }
    return best;
}

// Cycles of a call of pairs with tiles of h rows: coefficients that fit the times of whole calls at
// K = 8192 and order them rightly, not the times of single stages.  256 + h a stage up to 224 rows
// (its four MMAs read, and its copies write, 64 + h / 4 cycles' worth of shared memory each; the
// tensor work alone is 2 h).  Taller ones fit 228 + h (below the 512 of the tensor work at 256
// rows) with 4000 from tile to tile, in which the next one's MMAs wait for the shared columns.
// A call of pairs fits 6000 more than one of single CTAs, which therefore win while one wave of
// them is enough: 8192 x 8192, 192 tokens, 17.9 us against 19.2; 384 tokens, 35.4 against 23.5.
int64_t f8_pair_cycles(const F8Args& a, int64_t h, int64_t tiles, int64_t fit) {
    const int64_t kb = (a.K + kKB - 1) / kKB;
    const int64_t tile = h > 224 ? kb * (228 + h) + 4000 : kb * (256 + h) + 300;
    return (tiles + fit - 1) / fit * tile + 20 * h + (h > 224 ? 4000 : 6000);
}

// Token rows per tile (a multiple of 16, up to 256) for pairs on one matrix, as equal as can be.
F8Plan f8_pair_plan(const F8Args& a) {
    const int64_t tn = (a.N + 2 * kRows - 1) / (2 * kRows), fit = f8_fit(2);
    F8Plan best;
    if (fit < 1) return best;
    best.pairs = true;
    const int64_t tm0 = (a.R + 255) / 256;
    for (int64_t tm = tm0; tm < tm0 + 8; ++tm) {
        const int64_t h = ((a.R + tm - 1) / tm + 15) / 16 * 16;
        if (h < 64 && tm > tm0) break;
        const int64_t cycles = f8_pair_cycles(a, h, (a.R + h - 1) / h * tn, fit);
        if (cycles < best.cycles) {
            best.cycles = cycles;
            best.bt = (int)h;
        }
    }
    return best;
}

// Tokens per tile.  Measured in a graph, us, weights in turn beyond the L2 cache:
//   N x K        M     16     32     64    128   pairs
//   8192 x 8192  1   13.3   13.5   14.0   15.0   21.0
//                32  14.3   13.6   13.7   15.4   17.2
//                128 44.7   24.9   15.9   18.2   18.5
//                192    -      -   24.2   17.9   19.2
//                384    -      -   38.9   35.4   23.5
//   4096 x 4096  129    -      -    9.1    9.8   10.9
//                384    -      -   15.3   11.1   12.0
//   11008 x 4096 128    -      -   20.2   12.5      -
//   28672 x 8192 64     -   40.9   39.3   43.4   43.0
//                128    -      -   44.7   46.5   45.2
//                192    -      -      -   50.9   47.7
// A wider tile has a shallower ring of weights and a longer epilogue; narrower ones are more,
// down to where they no longer fit the SMs at once.  The fewest estimated cycles win.
F8Plan f8_dense_plan(const F8Args& a) {
    const int64_t tn = (a.N + kRows - 1) / kRows;
    F8Plan best;
    best.split = f8_least_split(a);
    if (best.split == 1 && a.R > 64) best = f8_pair_plan(a);   // 28672 x 8192, 64 tokens: 43.0 us, single CTAs 39.3
    for (int bt = 16; bt <= 128; bt *= 2) {
        const F8Plan plan = f8_narrow_plan(a, bt, std::min<int64_t>(bt, (a.R + 15) / 16 * 16), (a.R + bt - 1) / bt * tn);
        if (plan.cycles < best.cycles) best = plan;
    }
    return best;
}

// Tokens per tile, by the rows an expert has on average.  Measured in a graph, us, 32 experts of
// 4096 x 4096 of uneven popularity:
//   rows each    32     64    128   pairs
//   1          55.8   55.6   57.7   61.2
//   4          76.9   77.6   80.4   84.0
//   32         90.6   87.4   86.2   90.0
//   48         96.8   87.2   87.7   90.7
//   96          149    106   95.6   97.3
//   128         193    120    101   99.8
//   192         264    158    124    111
// and 8 experts of 1092 x 1544: 75 rows each 9.4, 7.0, 7.7, 9.8; 384 rows 21.7, 16.4, 11.8, 15.9.
// The fewest estimated cycles win.  The offsets are on the device: the number of tiles is
// estimated, half a tile lost per expert.
F8Plan f8_experts_plan(const F8Args& a) {
    const int64_t used = a.R < a.E ? a.R : a.E;   // experts that have rows, at most
    const auto tiles = [&](int64_t bt, int64_t n) { return (a.N + n - 1) / n * std::max(used, a.R / bt + used / 2); };
    const int64_t fit = f8_fit(2);
    F8Plan best;
    best.split = f8_least_split(a);
    best.pairs = best.split == 1 && fit > 0;
    best.bt = 224;
    if (best.pairs) best.cycles = f8_pair_cycles(a, best.bt, tiles(best.bt, 2 * kRows), fit);
    for (int bt = 32; bt <= 128; bt *= 2) {
        const F8Plan plan = f8_narrow_plan(a, bt, bt, tiles(bt, kRows));
        if (plan.cycles < best.cycles) best = plan;
    }
    return best;
}

template <int BT, bool EXPERTS>
cq_status f8_narrow(const F8Args& a, int split) {
    return split > 1 ? f8_launch<F8Cfg<BT, EXPERTS, false, true>>(a, split) : f8_launch<F8Cfg<BT, EXPERTS>>(a, 1);
}

cq_status f8_check_sizes(const F8Args& a) {
    if (a.E < 1 || a.N < 1 || a.K < 1 || a.R < 1 || !cq_dtype_valid(a.yt)) return CQ_ERR_INVALID_ARG;
    if (a.act != CQ_ACT_NONE && a.act != CQ_ACT_SWIGLU) return CQ_ERR_INVALID_ARG;
    if (a.act == CQ_ACT_SWIGLU && a.N % 2 != 0) return CQ_ERR_INVALID_ARG;
    if (a.E > CQ_MOE_MAX_EXPERTS || a.N > CQ_F8_MAX_N || a.K > CQ_F8_MAX_K || a.R > CQ_F8_MAX_ROWS)
        return CQ_ERR_UNSUPPORTED;
    return f8_tiles(a, 16, 1) > (1 << 30) ? CQ_ERR_UNSUPPORTED : CQ_OK;   // 32-bit tile numbers
}

cq_status f8_check(const F8Args& a) {
    if (!a.wc || !a.ws || !a.xc || !a.xs || !a.Y) return CQ_ERR_INVALID_ARG;
    const cq_status st = f8_check_sizes(a);
    if (st != CQ_OK) return st;
    if (!aligned16(a.wc) || !aligned16(a.ws) || !aligned16(a.xc) || !aligned16(a.xs) || !aligned16(a.Y))
        return CQ_ERR_ALIGNMENT;
    return CQ_OK;
}

}  // namespace

__global__ void bounded_wait_probe_f8_kernel(unsigned int* err, unsigned long long timeout_ns) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (threadIdx.x == 0) (void)mbar_wait_until<false>(&bar, 0u, &abort_flag, err, timeout_ns);
}

cq_status probe_f8_wait(unsigned long long timeout_ns, cudaStream_t st) {
    unsigned int* err = nullptr;
    const cq_status se = f8_setup(&err);
    if (se != CQ_OK) return se;
    bounded_wait_probe_f8_kernel<<<1, 32, 0, st>>>(err, timeout_ns);
    return check_launch();
}

unsigned int* f8_error_word(int dev) {
    if (dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(g_f8_mu);
    return g_f8_err_ptr[dev];
}

}  // namespace cq

using namespace cq;

extern "C" cq_status f8_gemm(const uint8_t* wcodes, const uint8_t* wscales, int64_t N, int64_t K,
                             const uint8_t* xcodes, const uint8_t* xscales, int64_t M, cq_act act, void* Y,
                             cq_dtype yt, void* stream) {
    const F8Args a = {wcodes, wscales, xcodes, xscales, nullptr, 1, N, K, M, act, Y, yt, as_stream(stream)};
    unsigned int* err = nullptr;
    cq_status st = f8_check(a);
    if (st == CQ_OK) st = f8_setup(&err);
    if (st != CQ_OK) return st;
    const F8Plan best = f8_dense_plan(a);
    if (best.pairs)
        return best.bt > 224 ? f8_launch<F8Cfg<256, false, true>>(a, 1, best.bt)
                             : f8_launch<F8Cfg<224, false, true>>(a, 1, best.bt);
    switch (best.bt) {
        case 16: return f8_narrow<16, false>(a, best.split);
        case 32: return f8_narrow<32, false>(a, best.split);
        case 64: return f8_narrow<64, false>(a, best.split);
        default: return f8_narrow<128, false>(a, best.split);
    }
}

extern "C" cq_status f8_gemm_experts(const uint8_t* wcodes, const uint8_t* wscales, int64_t E, int64_t N, int64_t K,
                                     const int32_t* offsets, const uint8_t* xcodes, const uint8_t* xscales, int64_t R,
                                     cq_act act, void* Y, cq_dtype yt, void* stream) {
    const F8Args a = {wcodes, wscales, xcodes, xscales, offsets, E, N, K, R, act, Y, yt, as_stream(stream)};
    if (!offsets) return CQ_ERR_INVALID_ARG;
    unsigned int* err = nullptr;
    cq_status st = f8_check(a);
    if (st == CQ_OK && !aligned16(offsets)) st = CQ_ERR_ALIGNMENT;
    if (st == CQ_OK) st = f8_setup(&err);
    if (st != CQ_OK) return st;
    const F8Plan best = f8_experts_plan(a);
    if (best.pairs) return f8_launch<F8Cfg<224, true, true>>(a, 1);
    switch (best.bt) {
        case 32: return f8_narrow<32, true>(a, best.split);
        case 64: return f8_narrow<64, true>(a, best.split);
        default: return f8_narrow<128, true>(a, best.split);
    }
}

extern "C" cq_status f8_gemm_plan(int64_t E, int64_t N, int64_t K, int64_t R, cq_act act, cq_dtype yt, int32_t* plan) {
    if (!plan || E < 0) return CQ_ERR_INVALID_ARG;
    F8Args a = {};
    a.offsets = E ? plan : nullptr;   // experts or not; not read
    a.E = E ? E : 1;
    a.N = N; a.K = K; a.R = R; a.act = act; a.yt = yt;
    unsigned int* err = nullptr;
    cq_status st = f8_check_sizes(a);
    if (st == CQ_OK) st = f8_setup(&err);
    if (st != CQ_OK) return st;
    const F8Plan best = E ? f8_experts_plan(a) : f8_dense_plan(a);
    plan[0] = best.bt;
    plan[1] = best.pairs ? 2 : 1;
    plan[2] = best.split;
    return CQ_OK;
}
