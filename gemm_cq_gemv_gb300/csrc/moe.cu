// The two ends of an expert layer: moe_route (softmax top-k of the router's logits and the
// order of the rows by expert) and moe_combine (the weighted sum of each token's rows).
//
// Measured on one GB300, in a graph: moe_route of 1 token over 64 experts, k = 8, 2.3 us, 64
// tokens 3.5 us, 512 tokens 7.5 us; 16384 tokens over 256 experts 18 us, the selection's
// instructions (about 490 a token) and two more launches, where the logits' bytes take 2.5 us.
// moe_combine of 8192 x 8 rows of 4096 bfloat16 columns 104 us, 5.8 TB/s: the memory (a gather
// of as many rows by the library runs at 5.2 TB/s).

#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"

namespace cq {
namespace {

constexpr int kChunk = 64;            // tokens per CTA of the selection at most: one bit each in a mask
constexpr int kSelThreads = 512;
constexpr int kMaxCluster = 8;        // CTAs of the selection that finish the order among themselves
static_assert(CQ_MOE_ONE_LAUNCH == kMaxCluster * kChunk, "tokens of one cluster");

// Order-preserving integer of a logit: larger float, larger key.  -0 counts as 0 and NaN as
// -infinity, whose key is above 0, the key of "not there".
__device__ __forceinline__ uint32_t logit_key(float x) {
    const uint32_t b = __float_as_uint(fmaxf(x, -__int_as_float(0x7F800000)) + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// exp(l - max), with 1 for the maximum itself (also an infinite one)
__device__ __forceinline__ float softmax_term(float l, float best) { return l == best ? 1.0f : expf(l - best); }

struct RouteParams {
    const float* logits;   // [T][E]
    int64_t T;
    int E, k;
    int normalize;
    int32_t* ids;          // [T][k]
    float* weights;        // [T][k]
    int32_t* offsets;      // [E + 1]
    int32_t* rows;         // [T k]
    int32_t* pos;          // [T][k]
    int32_t* counts;       // [chunks][E]: rows per expert of a chunk, then of the chunks before it
    int32_t* totals;       // [E]
    int64_t chunks;
    int chunk;             // tokens of each
};

// The logits of a token, one warp: experts VPT lane .. VPT lane + VPT - 1 in this lane.
template <int VPT>
__device__ __forceinline__ void load_logits(float (&l)[VPT], const RouteParams& p, int64_t t, int lane) {
    const float* row = p.logits + t * p.E;
    const int e0 = VPT * lane;
    if (VPT >= 4 && (p.E & 3) == 0) {   // rows and quads on 16-byte boundaries
#pragma unroll
        for (int i = 0; i + 3 < VPT; i += 4) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (e0 + i < p.E) v = __ldg(reinterpret_cast<const float4*>(row + e0 + i));
            l[i] = v.x; l[i + 1] = v.y; l[i + 2] = v.z; l[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) l[i] = e0 + i < p.E ? __ldg(row + e0 + i) : 0.0f;
    }
}

// The k largest logits of one token, one warp, experts VPT lane .. in this lane; writes the
// choices and the weights and marks the token in the experts' masks.
//  1. The k-th largest of the lanes' maxima (equal ones counted once) is a bound that no choice is
//     below.
//  2. The logits at or above the bound, usually k to 2 k of them, move to one lane each, as the
//     key above the expert's complement: equal logits in the order of their experts.
//  3. Each counts how many are larger: its place.
// Where more than 32 reach the bound (many equal logits), k rounds search all logits instead.
// About 490 instructions at VPT = 8, k = 8, half of them before and after the choice itself.
template <int VPT>
__device__ __forceinline__ void select_token(const RouteParams& p, int64_t t, const float (&l)[VPT], int lane,
                                             uint64_t* mask, int bit, uint64_t* scratch) {
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    uint32_t key[VPT], head = 0u;
#pragma unroll
    for (int i = 0; i < VPT; ++i) key[i] = logit_key(l[i]);
    if (VPT * lane + VPT > p.E) {   // past the last expert
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (VPT * lane + i >= p.E) key[i] = 0u;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) head = max(head, key[i]);
    uint32_t bound = __reduce_max_sync(kAll, head);
    const float best = key_logit(bound);
    for (int j = 1; j < p.k; ++j) {
        if (head == bound) head = 0u;
        bound = __reduce_max_sync(kAll, head);
    }
    bound = max(bound, 1u);
    int total = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const bool in = key[i] >= bound;
        const uint32_t who = __ballot_sync(kAll, in);
        const int at = total + __popc(who & ((1u << lane) - 1u));
        if (in && at < 32) scratch[at] = (uint64_t)key[i] << 32 | (uint32_t)~(VPT * lane + i);
        total += __popc(who);
    }
    if (lane >= total) scratch[lane] = 0ull;
    __syncwarp();
    uint32_t my_key = 0;
    int my_id = 0, place = p.k;   // place p.k and above: not chosen
    if (total <= 32) {
        const uint64_t c = scratch[lane];
        place = lane < total ? 0 : p.k;
        for (int j = 0; j < total; j += 4) {
            const ulonglong2 a = reinterpret_cast<const ulonglong2*>(scratch + j)[0];
            const ulonglong2 b = reinterpret_cast<const ulonglong2*>(scratch + j)[1];
            place += (a.x > c ? 1 : 0) + (a.y > c ? 1 : 0) + (b.x > c ? 1 : 0) + (b.y > c ? 1 : 0);
        }
        my_key = (uint32_t)(c >> 32);
        my_id = (int)~(uint32_t)c;
    } else {
        for (int j = 0; j < p.k; ++j) {
            uint32_t most = key[0];
            int slot = 0;
#pragma unroll
            for (int i = 1; i < VPT; ++i)
                if (key[i] > most) { most = key[i]; slot = i; }
            const uint32_t top = __reduce_max_sync(kAll, most);
            const int from = __ffs(__ballot_sync(kAll, most == top)) - 1;
            const int id = __shfl_sync(kAll, VPT * lane + slot, from);
            if (lane == j) { my_id = id; my_key = top; place = j; }
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (id == VPT * lane + i) key[i] = 0u;
        }
    }
    __syncwarp();   // the scratch is the next token's
    const float w = place < p.k ? softmax_term(key_logit(my_key), best) : 0.0f;
    float all = w;
    if (!p.normalize) {
        all = 0.0f;
        if (fabsf(best) < __int_as_float(0x7F800000)) {
            // the terms of the sum by ex2: an error of |l - max| 2^-24 of a term exp(l - max).  A NaN
            // is -infinity here as in its key
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const float x = (fmaxf(l[i], -__int_as_float(0x7F800000)) - best) * 1.44269504088896341f;
                float e;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
                if (VPT * lane + i < p.E) all += e;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (VPT * lane + i < p.E) all += softmax_term(key_logit(logit_key(l[i])), best);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(kAll, all, o);
    if (place < p.k) {
        p.ids[t * p.k + place] = my_id;
        // a token whose every expert is masked takes the lowest ones with weight 0
        p.weights[t * p.k + place] = __float_as_uint(best) == 0xFF800000u ? 0.0f : w / all;
        atomicOr(reinterpret_cast<unsigned int*>(mask + my_id) + (bit >> 5), 1u << (bit & 31));   // little-endian halves
    }
}

// Exclusive prefix of v over the threads of the CTA (all of them call it); `total` gets the sum.
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int s = lane < nwarps ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    *total = warp_sums[31];
    return inc - v + (warp ? warp_sums[warp - 1] : 0);
}

__device__ __forceinline__ uint64_t cluster_load64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// One chunk of tokens per CTA: the choices, and each choice's rank among the chunk's rows of
// its expert.  A 64-bit mask per expert holds the chunk's tokens that chose it, so the rank
// is the number of set bits below the token's own: the same whatever order the warps ran in.
// ONE: the grid is one cluster, whose CTAs read each other's masks and write the offsets and
// the final rows here too (512 tokens, 8 of 64: one launch instead of three).
template <int VPT, bool ONE>
__global__ void __launch_bounds__(kSelThreads) route_select_kernel(const __grid_constant__ RouteParams p) {
    __shared__ uint64_t mask[CQ_MOE_MAX_EXPERTS];
    __shared__ int first[ONE ? CQ_MOE_MAX_EXPERTS : 1];
    __shared__ int warp_sums[32];
    __shared__ __align__(16) uint64_t candidates[kSelThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0ull;
    pdl_trigger();
    __syncthreads();
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    const int n = (int)max((int64_t)0, min((int64_t)p.chunk, p.T - t0));
    const int warps = blockDim.x >> 5;
    float l[VPT];
    if constexpr (VPT <= 16) {   // the next token's logits on their way; more do not fit the registers
        float next[VPT];
        if (warp < n) load_logits<VPT>(next, p, t0 + warp, lane);
        for (int i = warp; i < n; i += warps) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) l[j] = next[j];
            if (i + warps < n) load_logits<VPT>(next, p, t0 + i + warps, lane);
            select_token<VPT>(p, t0 + i, l, lane, mask, i, candidates[warp]);
        }
    } else {
        for (int i = warp; i < n; i += warps) {
            load_logits<VPT>(l, p, t0 + i, lane);
            select_token<VPT>(p, t0 + i, l, lane, mask, i, candidates[warp]);
        }
    }
    if constexpr (ONE) {
        // every CTA's masks are complete (a cluster barrier takes a microsecond: not for one CTA)
        if (gridDim.x > 1) cluster_sync();
        else __syncthreads();
        const uint32_t me = cluster_rank();
        int base = 0;
        for (int e0 = 0; e0 < p.E; e0 += blockDim.x) {
            const int e = e0 + threadIdx.x;
            int rows = 0, before = 0, total;
            if (e < p.E)
                for (uint32_t c = 0; c < gridDim.x; ++c) {
                    const int there = __popcll(cluster_load64(cluster_addr(&mask[e], c)));
                    rows += there;
                    before += c < me ? there : 0;
                }
            const int at = base + block_exclusive(rows, warp_sums, &total);
            if (e < p.E) {
                first[e] = at + before;
                if (me == 0) p.offsets[e] = at;
            }
            base += total;
            __syncthreads();
        }
        if (me == 0 && threadIdx.x == 0) p.offsets[p.E] = base;
    } else {
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += blockDim.x)
            p.counts[(int64_t)blockIdx.x * p.E + e] = __popcll(mask[e]);
    }
    for (int i = threadIdx.x; i < n * p.k; i += blockDim.x) {
        const int t = i / p.k;
        const int e = p.ids[t0 * p.k + i];
        const int rank = __popcll(mask[e] & ((1ull << t) - 1ull));
        if constexpr (ONE) {
            p.pos[t0 * p.k + i] = first[e] + rank;
            p.rows[first[e] + rank] = (int32_t)t0 + t;
        } else {
            p.pos[t0 * p.k + i] = rank;
        }
    }
    if (ONE && gridDim.x > 1) cluster_sync();   // no CTA's masks are read any more
}

// counts [chunks][E] -> how many rows of the expert the chunks before this one have; totals [E].
// 32 experts a CTA, their chunks in 32 segments.
__global__ void __launch_bounds__(1024) route_scan_kernel(const __grid_constant__ RouteParams p) {
    __shared__ int seg[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, s = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int64_t per = (p.chunks + 31) / 32;
    const int64_t c0 = min((int64_t)s * per, p.chunks), c1 = min(c0 + per, p.chunks);
    int32_t* col = p.counts + e;
    int sum = 0;
    if (e < p.E) {
#pragma unroll 8
        for (int64_t c = c0; c < c1; ++c) sum += col[c * p.E];
    }
    seg[s][lane] = sum;
    __syncthreads();
    const int mine = seg[lane][s];   // warp s: the segments of expert s of the CTA
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    seg[lane][s] = inc - mine;
    if (lane == 31 && blockIdx.x * 32 + s < p.E) p.totals[blockIdx.x * 32 + s] = inc;
    __syncthreads();
    int at = seg[s][lane];
    if (e < p.E) {
        for (int64_t c = c0; c < c1; c += 8) {   // eight loads before their stores
            int n[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) n[j] = c + j < c1 ? col[(c + j) * p.E] : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (c + j < c1) col[(c + j) * p.E] = at;
                at += n[j];
            }
        }
    }
}

constexpr int kPlaceThreads = 512;
constexpr int kPlacePer = 4;   // choices per thread

// offsets from the totals (every CTA for itself), then the row of each choice.
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const __grid_constant__ RouteParams p) {
    __shared__ int first[CQ_MOE_MAX_EXPERTS];
    __shared__ int warp_sums[32];
    pdl_trigger();
    pdl_wait();
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += kPlaceThreads) {
        const int e = e0 + threadIdx.x;
        int total;
        const int at = base + block_exclusive(e < p.E ? p.totals[e] : 0, warp_sums, &total);
        if (e < p.E) {
            first[e] = at;
            if (blockIdx.x == 0) p.offsets[e] = at;
        }
        base += total;
        __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.E] = base;
    const int64_t i0 = (int64_t)blockIdx.x * (kPlaceThreads * kPlacePer) + threadIdx.x, n = p.T * p.k;
    int e[kPlacePer], at[kPlacePer];   // every load before the first store
    uint32_t t[kPlacePer];
#pragma unroll
    for (int j = 0; j < kPlacePer; ++j) {
        const int64_t i = i0 + j * kPlaceThreads;
        e[j] = i < n ? p.ids[i] : 0;
        at[j] = i < n ? p.pos[i] : 0;
    }
#pragma unroll
    for (int j = 0; j < kPlacePer; ++j) {
        const int64_t i = i0 + j * kPlaceThreads;
        t[j] = (uint32_t)i / (uint32_t)p.k;   // T k is at most 2^30
        if (i < n) at[j] += first[e[j]] + p.counts[(int64_t)(t[j] / (uint32_t)p.chunk) * p.E + e[j]];
    }
#pragma unroll
    for (int j = 0; j < kPlacePer; ++j) {
        const int64_t i = i0 + j * kPlaceThreads;
        if (i < n) {
            p.pos[i] = at[j];
            p.rows[at[j]] = (int32_t)t[j];
        }
    }
}

template <int VPT>
cq_status launch_select(const RouteParams& p, bool one, cudaStream_t cs) {
    const unsigned n = (unsigned)p.chunks;
    constexpr int kWarps = kSelThreads / 32;
    const int rounds = (p.chunk + kWarps - 1) / kWarps;   // no warp has a token more than another
    const dim3 threads(32u * (unsigned)((p.chunk + rounds - 1) / rounds));
    return one ? launch_pdl_cluster(route_select_kernel<VPT, true>, dim3(n), threads, 0, n, cs, p)
               : launch_pdl(route_select_kernel<VPT, false>, dim3(n), threads, 0, cs, p);
}

// ---- combine ----------------------------------------------------------------------
template <typename T, bool VEC>
__device__ __forceinline__ void get8(float (&v)[8], const T* y, int64_t n, int64_t N) {
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = n + i < N ? (float)y[n + i] : 0.0f;
    } else if constexpr (sizeof(T) == 2) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(y + n));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 a = __ldg(reinterpret_cast<const float4*>(y + n));
        const float4 b = __ldg(reinterpret_cast<const float4*>(y + n + 4));
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}
template <bool VEC>
__device__ __forceinline__ void put8(float* o, const float (&v)[8], int64_t n, int64_t N) {
    if constexpr (VEC) {
        *reinterpret_cast<float4*>(o + n) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(o + n + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < N) o[n + i] = v[i];
    }
}
template <bool VEC>
__device__ __forceinline__ void put8(__nv_bfloat16* o, const float (&v)[8], int64_t n, int64_t N) {
    if constexpr (VEC) {
        uint4 a;
        uint32_t* w = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(o + n) = a;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < N) o[n + i] = __float2bfloat16_rn(v[i]);
    }
}

// One thread per eight columns of a token; the k rows are added in the order of the choices.
template <typename TY, typename TO, bool VEC>
__global__ void __launch_bounds__(256)
moe_combine_kernel(const TY* __restrict__ Y, int64_t R, int64_t N, const int32_t* __restrict__ pos,
                   const float* __restrict__ weights, int64_t T, int k, TO* __restrict__ out) {
    pdl_trigger();
    pdl_wait();
    const int64_t per = (N + 7) / 8;
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= T * per) return;
    const int64_t t = u / per, n = (u - t * per) * 8;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
        const int64_t r = __ldg(pos + t * k + j);
        const float w = __ldg(weights + t * k + j);
        if (r < 0 || r >= R || w == 0.0f) continue;   // dropped, or masked: its row is not read
        float v[8];
        get8<TY, VEC>(v, Y + r * N, n, N);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
    put8<VEC>(out + t * N, acc, n, N);
}

template <typename TY, typename TO>
cq_status launch_combine(const void* Y, int64_t R, int64_t N, const int32_t* pos, const float* weights, int64_t T,
                         int k, void* out, cudaStream_t cs) {
    const int64_t grid = (T * ((N + 7) / 8) + 255) / 256;
    if (grid > 0x7FFFFFFF) return CQ_ERR_UNSUPPORTED;
    const dim3 gd((unsigned)grid), bd(256);
    const TY* y = static_cast<const TY*>(Y);
    TO* o = static_cast<TO*>(out);
    return N % 8 == 0 ? launch_pdl(moe_combine_kernel<TY, TO, true>, gd, bd, 0, cs, y, R, N, pos, weights, T, k, o)
                      : launch_pdl(moe_combine_kernel<TY, TO, false>, gd, bd, 0, cs, y, R, N, pos, weights, T, k, o);
}

}  // namespace
}  // namespace cq

using namespace cq;

// Tokens per CTA of the selection: one for every warp, as long as a cluster (or two CTAs per
// SM, beyond a cluster's worth of tokens) holds them all, else what makes that many CTAs.  152
// SMs as a constant: the workspace's size must not depend on the current device.
static int route_chunk(int64_t T) {
    const int64_t ctas = T <= CQ_MOE_ONE_LAUNCH ? kMaxCluster : 2 * 152;
    const int64_t even = (T + ctas - 1) / ctas;
    return (int)std::min<int64_t>(kChunk, std::max<int64_t>(kSelThreads / 32, even));
}

extern "C" size_t moe_route_workspace_bytes(int64_t T, int64_t E) {
    if (T < 1 || E < 1) return 0;
    if (T <= CQ_MOE_ONE_LAUNCH) return 0;
    const size_t chunk = (size_t)route_chunk(T), chunks = ((size_t)T + chunk - 1) / chunk;
    return ((chunks + 1) * (size_t)E * sizeof(int32_t) + 255u) & ~(size_t)255u;
}

extern "C" cq_status moe_route(const float* logits, int64_t T, int64_t E, int k, int normalize, int32_t* ids,
                               float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* workspace,
                               size_t workspace_bytes, void* stream) {
    if (!logits || !ids || !weights || !offsets || !rows || !pos) return CQ_ERR_INVALID_ARG;
    if (T < 1 || E < 1 || k < 1 || k > E) return CQ_ERR_INVALID_ARG;
    if (E > CQ_MOE_MAX_EXPERTS || k > CQ_MOE_MAX_K || T > CQ_F8_MAX_ROWS / k) return CQ_ERR_UNSUPPORTED;
    if (!aligned16(logits) || !aligned16(ids) || !aligned16(weights) || !aligned16(offsets) || !aligned16(rows) ||
        !aligned16(pos) || !aligned16(workspace))
        return CQ_ERR_ALIGNMENT;
    const size_t need = moe_route_workspace_bytes(T, E);
    if (need && (!workspace || workspace_bytes < need)) return CQ_ERR_WORKSPACE;
    RouteParams p;
    p.logits = logits; p.T = T; p.E = (int)E; p.k = k; p.normalize = normalize;
    p.ids = ids; p.weights = weights; p.offsets = offsets; p.rows = rows; p.pos = pos;
    p.counts = static_cast<int32_t*>(workspace);
    const bool one = T <= CQ_MOE_ONE_LAUNCH;
    p.chunk = route_chunk(T);
    p.chunks = (T + p.chunk - 1) / p.chunk;
    p.totals = p.counts + p.chunks * E;
    const cudaStream_t cs = as_stream(stream);
    cq_status st;
    if (E <= 32) st = launch_select<1>(p, one, cs);
    else if (E <= 64) st = launch_select<2>(p, one, cs);
    else if (E <= 128) st = launch_select<4>(p, one, cs);
    else if (E <= 256) st = launch_select<8>(p, one, cs);
    else if (E <= 512) st = launch_select<16>(p, one, cs);
    else st = launch_select<32>(p, one, cs);
    if (st != CQ_OK || one) return st;
    st = launch_pdl(route_scan_kernel, dim3((unsigned)((E + 31) / 32)), dim3(1024), 0, cs, p);
    if (st != CQ_OK) return st;
    constexpr int kPerCta = kPlaceThreads * kPlacePer;
    return launch_pdl(route_place_kernel, dim3((unsigned)((T * k + kPerCta - 1) / kPerCta)), dim3(kPlaceThreads), 0, cs, p);
}

extern "C" cq_status moe_combine(const void* Y, cq_dtype yt, int64_t R, int64_t N, const int32_t* pos,
                                 const float* weights, int64_t T, int k, void* out, cq_dtype ot, void* stream) {
    if (!Y || !pos || !weights || !out || R < 1 || N < 1 || T < 1 || k < 1) return CQ_ERR_INVALID_ARG;
    if (!cq_dtype_valid(yt) || !cq_dtype_valid(ot)) return CQ_ERR_INVALID_ARG;
    if (k > CQ_MOE_MAX_K || T > CQ_F8_MAX_ROWS || R > CQ_F8_MAX_ROWS || N > CQ_F8_MAX_N) return CQ_ERR_UNSUPPORTED;
    if (!aligned16(Y) || !aligned16(pos) || !aligned16(weights) || !aligned16(out)) return CQ_ERR_ALIGNMENT;
    const cudaStream_t cs = as_stream(stream);
    if (yt == CQ_F32)
        return ot == CQ_F32 ? launch_combine<float, float>(Y, R, N, pos, weights, T, k, out, cs)
                            : launch_combine<float, __nv_bfloat16>(Y, R, N, pos, weights, T, k, out, cs);
    return ot == CQ_F32 ? launch_combine<__nv_bfloat16, float>(Y, R, N, pos, weights, T, k, out, cs)
                        : launch_combine<__nv_bfloat16, __nv_bfloat16>(Y, R, N, pos, weights, T, k, out, cs);
}
