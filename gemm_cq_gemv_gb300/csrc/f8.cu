// F8 quantizers: e4m3 codes with one power-of-two scale per 128 values of a row
// (activations) or per 128 x 128 block (weights).
//
// The scale of a block is the smallest s = 2^(e - 127), e in 0..254, with
// max |x| <= 448 s (448 = 1.75 * 2^8, the largest e4m3 value); the codes are e4m3(x / s),
// rounded to nearest even.  A power of two makes x / s exact, so there is one rounding and
// the codes are the same in any precision; e is what the block-scaled tensor-core product
// takes as it stands.
//
// Measured on one GB300: 8192 x 4096 bfloat16 values 18.7 us, float32 27.9 us (5.4 and 6.0 TB/s);
// bound by the memory.  The same rows to 8 experts each 63 us for 337 MB, of which 270 MB are
// writes: a plain fill of as many bytes takes 74 us.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace cq {
namespace {

constexpr int kQuantCtas = 4;   // CTAs of 256 threads per SM: what the registers of either type allow

// The bits of max |x| of a block (as an unsigned integer, in which NaN > infinity > every
// finite value) -> scale byte.  1.m * 2^(E - 127) <= 1.75 * 2^8 * 2^(e - 127) gives
// e = E - 8, one more when 1.m > 1.75; below 2^-126 (E = 0, or e < 0) the smallest scale.
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t amax_bits) {
    if (amax_bits == 0u) return kF8One;
    if (amax_bits >= 0x7F800000u) return kF8NaN;
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(e, 0);
}
// 2^(127 - e) for a finite block's scale byte (at most 248: the result is a normal number);
// 0 for a non-finite block, whose codes are written as zeros.
__device__ __forceinline__ float f8_inverse(uint32_t e) {
    return e == kF8NaN ? 0.0f : __uint_as_float((254u - e) << 23);
}

// Four e4m3 codes, a in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// x * inv, 0 in a non-finite block (where x * 0 could be NaN)
__device__ __forceinline__ float scaled(float x, float inv) { return inv == 0.0f ? 0.0f : x * inv; }

// Sixteen consecutive values of a row, as loaded: float32 words or bfloat16 pairs.
template <typename T>
struct Values16;
template <>
struct Values16<float> {
    uint32_t w[16];
    __device__ __forceinline__ uint32_t amax_bits() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ uint32_t codes4(int i, float inv) const {
        return e4m3x4(__uint_as_float(w[4 * i]) * inv, __uint_as_float(w[4 * i + 1]) * inv,
                      __uint_as_float(w[4 * i + 2]) * inv, __uint_as_float(w[4 * i + 3]) * inv);
    }
};
template <>
struct Values16<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ uint32_t amax_bits() const {
        uint32_t m = 0;   // two 16-bit maxima
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return max(m & 0xFFFF0000u, m << 16);
    }
    // the products by a power of two are exact in bfloat16 down to 2^-126, far below half of the
    // smallest code
    __device__ __forceinline__ uint32_t codes4(int i, float inv) const {
        const __nv_bfloat162 f = __float2bfloat162_rn(inv);
        uint32_t p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * i + j]), f);
            p[j] = *reinterpret_cast<const uint32_t*>(&x);
        }
        return e4m3x4(__uint_as_float(p[0] << 16), __uint_as_float(p[0] & 0xFFFF0000u), __uint_as_float(p[1] << 16),
                      __uint_as_float(p[1] & 0xFFFF0000u));
    }
};

// Columns k .. k + 15 of a row of K values, zero past K.  VEC: whole 16-byte loads (rows start
// on 16-byte boundaries and K is a multiple of 16 bytes' worth of values).
template <bool VEC, typename T>
__device__ __forceinline__ void load16(Values16<T>& v, const T* row, int64_t k, int64_t K) {
    constexpr int kPer = 16 / (int)sizeof(T);   // values per 16 bytes
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 16 / kPer; ++i) {
            uint4 a = make_uint4(0u, 0u, 0u, 0u);
            if (k + kPer * i < K) a = __ldg(reinterpret_cast<const uint4*>(row + k) + i);
            v.w[4 * i] = a.x; v.w[4 * i + 1] = a.y; v.w[4 * i + 2] = a.z; v.w[4 * i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (sizeof(T) == 4) {
                v.w[i] = k + i < K ? __float_as_uint(__ldg(row + k + i)) : 0u;
            } else {
                const uint32_t h = k + i < K ? __bfloat16_as_ushort(row[k + i]) : 0u;
                v.w[i >> 1] = i & 1 ? v.w[i >> 1] | h << 16 : h;
            }
        }
    }
}

// A quad of four groups of a row (512 columns) in one warp: eight lanes a group, 16 values a
// lane, so a group needs three shuffles and one scale, a lane's codes are one 16-byte word
// vector and the quad's scale bytes one word.  Codes of groups past the row are not there.
struct Quad {
    uint4 codes;
    uint32_t scales;
    bool there;
};
template <typename T>
__device__ __forceinline__ Quad quantize_quad(const Values16<T>& v, int q, int groups, int lane, bool inside) {
    uint32_t m = v.amax_bits();
#pragma unroll
    for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    Quad d;
    d.there = 4 * q + (lane >> 3) < groups;
    const uint32_t e = inside || !d.there ? f8_scale_byte(m) : kF8NaN;
    const float inv = f8_inverse(e);
    const uint32_t keep = e == kF8NaN ? 0u : 0xFFFFFFFFu;   // a NaN block's codes are zero
    d.codes = make_uint4(keep & v.codes4(0, inv), keep & v.codes4(1, inv), keep & v.codes4(2, inv),
                         keep & v.codes4(3, inv));
    d.scales = e << (lane & 24);   // byte lane / 8; padding groups: all zero, byte 127
    d.scales |= __shfl_xor_sync(0xffffffffu, d.scales, 8);
    d.scales |= __shfl_xor_sync(0xffffffffu, d.scales, 16);
    return d;
}

// Each output row from its own source row.  A warp takes up to `per` quads of a row one after the
// other and loads the next before it works on the present one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, kQuantCtas)
f8_quantize_kernel(const T* __restrict__ X, int64_t M, int64_t K, const int32_t* __restrict__ rows, int64_t R,
                   uint8_t* __restrict__ codes, uint32_t* __restrict__ scales, int quads, int per, int segs) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int groups = (int)((K + kGroup - 1) / kGroup);
    const int64_t units = R * segs, warps = (int64_t)gridDim.x * 8;
    for (int64_t u = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5; u < units; u += warps) {
        const int64_t r = segs == 1 ? u : u / segs;
        const int q0 = (int)(u - r * segs) * per, q1 = min(q0 + per, quads);
        const int64_t src = rows ? (int64_t)__ldg(rows + r) : r;
        const bool inside = src >= 0 && src < M;   // a row outside X becomes a NaN row
        const int64_t cols = inside ? K : 0;
        const T* x = X + (inside ? src * K : 0);
        uint8_t* out = codes + r * groups * kGroup + 16 * lane;
        Values16<T> v, next;
        load16<VEC>(next, x, (int64_t)q0 * (4 * kGroup) + 16 * lane, cols);
        for (int q = q0; q < q1; ++q) {
            v = next;
            if (q + 1 < q1) load16<VEC>(next, x, (int64_t)(q + 1) * (4 * kGroup) + 16 * lane, cols);
            const Quad d = quantize_quad(v, q, groups, lane, inside);
            if (d.there) *reinterpret_cast<uint4*>(out + (int64_t)q * (4 * kGroup)) = d.codes;
            if (lane == 0) scales[r * quads + q] = d.scales;
        }
    }
}

// Gathers with repeated source rows: each source row is quantized once for up to 32 output rows
// that name it.  With 8 rows of each of 8192 tokens of 4096 bfloat16 values the kernel above
// is bound by its arithmetic, done eight times (120 us; the bytes: 50 us).
//
// Room for the output rows of a source row: half as many again as a source row has on average.
// Those beyond it, and those of a row outside X, go on one list of their own and are
// quantized one by one as above: whatever the indexes are, no warp has more than 32 rows
// (2^18 rows of one of 4000 sources: 0.10 ms, walked as one list 29 ms).
struct Lists {
    int32_t* count;   // [M] output rows that name the source row, [1] rows on `alone`
    int32_t* slots;   // [M][cap] the first of them
    int32_t* alone;   // [R]
    int cap;
};
__host__ __device__ __forceinline__ int64_t list_cap(int64_t M, int64_t R) {
    const int64_t each = (R + M - 1) / M;
    return each + (each + 1) / 2;
}
//  1. Which row takes which place depends on the order of the atomics; the outputs do not.  Lanes
//     that name the same source share an atomic.
__global__ void __launch_bounds__(256)
f8_list_kernel(const int32_t* __restrict__ rows, int64_t M, int64_t R, Lists l) {
    pdl_trigger();
    pdl_wait();
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int32_t src = r < R ? __ldg(rows + r) : -1;
    const bool inside = src >= 0 && src < M;
    const uint32_t peers = __match_any_sync(kAll, inside ? src : -1);
    const int first = __ffs(peers) - 1;
    int at = 0;
    if (inside && lane == first) at = atomicAdd(l.count + src, __popc(peers));
    at = __shfl_sync(kAll, at, first) + __popc(peers & below);
    const bool listed = inside && at < l.cap;
    if (listed) l.slots[(int64_t)src * l.cap + at] = (int32_t)r;
    const bool alone = r < R && !listed;
    const uint32_t who = __ballot_sync(kAll, alone);
    if (!who) return;
    int base = 0;
    if (lane == 0) base = atomicAdd(l.count + M, __popc(who));
    base = __shfl_sync(kAll, base, 0);
    if (alone) l.alone[base + __popc(who & below)] = (int32_t)r;
}
//  2. A warp takes up to `per` quads of a source row for up to 32 rows of its list (`parts` of
//     them), or of the source of one row of `alone`.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, kQuantCtas)
f8_quantize_lists_kernel(const T* __restrict__ X, int64_t M, int64_t K, const int32_t* __restrict__ rows, Lists l,
                         uint8_t* __restrict__ codes, uint32_t* __restrict__ scales, int quads, int per, int segs,
                         int parts) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int groups = (int)((K + kGroup - 1) / kGroup);
    const int64_t listed = M * parts, units = (listed + l.count[M]) * segs, warps = (int64_t)gridDim.x * 8;
    for (int64_t u = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5; u < units; u += warps) {
        const int64_t w = segs == 1 ? u : u / segs;
        const int q0 = (int)(u - w * segs) * per, q1 = min(q0 + per, quads);
        int64_t src;
        int32_t mine = 0;   // the output row of lane 0 .. n - 1
        int n = 1;
        bool inside = true;
        if (w < listed) {
            src = parts == 1 ? w : w / parts;
            const int i0 = (int)(w - src * parts) * 32;
            n = min(min(l.count[src], l.cap) - i0, 32);
            if (n <= 0) continue;
            if (lane < n) mine = l.slots[src * l.cap + i0 + lane];
        } else {
            mine = l.alone[w - listed];
            src = __ldg(rows + mine);
            inside = src >= 0 && src < M;   // a row outside X becomes a NaN row
        }
        const T* x = X + (inside ? src * K : 0);
        const int64_t cols = inside ? K : 0;
        Values16<T> v, next;
        load16<VEC>(next, x, (int64_t)q0 * (4 * kGroup) + 16 * lane, cols);
        for (int q = q0; q < q1; ++q) {
            v = next;
            if (q + 1 < q1) load16<VEC>(next, x, (int64_t)(q + 1) * (4 * kGroup) + 16 * lane, cols);
            const Quad d = quantize_quad(v, q, groups, lane, inside);
            if (lane < n) scales[(int64_t)mine * quads + q] = d.scales;
            for (int i = 0; i < n; ++i) {
                const int64_t to = __shfl_sync(0xffffffffu, mine, i);
                if (d.there)   // streamed: 8192 x 4096 bfloat16 to 8 experts 62.8 us, 65.3 otherwise
                    __stcs(reinterpret_cast<uint4*>(codes + (to * groups + 4 * q) * kGroup + 16 * lane), d.codes);
            }
        }
    }
}

// One CTA per 128 x 128 block (and per padding byte of the scale rows): warp w takes rows
// w, w + 8, ..., a lane four columns.  Offline.
template <typename T>
__global__ void __launch_bounds__(256)
f8_quantize_weights_kernel(const T* __restrict__ W, int64_t N, int64_t K, int64_t nblk, int64_t sbytes,
                           int64_t blocks, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    __shared__ uint32_t warp_max[8];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t groups = (K + kGroup - 1) / kGroup;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t g = b % sbytes, nb = (b / sbytes) % nblk, e = b / sbytes / nblk;
        if (g >= groups) {
            if (threadIdx.x == 0) scales[b] = kF8One;
            continue;
        }
        float v[16][4];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t n = nb * kGroup + warp + 8 * i;
            const T* row = W + (e * N + n) * K;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t k = g * kGroup + 4 * lane + j;
                v[i][j] = n < N && k < K ? (float)row[k] : 0.0f;
                m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        __syncthreads();
        if (lane == 0) warp_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, warp_max[w]);
        const uint32_t sb = f8_scale_byte(m);
        const float inv = f8_inverse(sb);
        if (threadIdx.x == 0) scales[b] = (uint8_t)sb;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t n = nb * kGroup + warp + 8 * i;
            if (n < N)
                *reinterpret_cast<uint32_t*>(codes + ((e * N + n) * groups + g) * kGroup + 4 * lane) =
                    e4m3x4(scaled(v[i][0], inv), scaled(v[i][1], inv), scaled(v[i][2], inv), scaled(v[i][3], inv));
        }
    }
    weights_written();
}

}  // namespace
}  // namespace cq

using namespace cq;

// Whether a gather of R rows from M is worth the two launches that build the lists: rows repeat,
// and the 16 M values and more take longer than those launches.
static bool f8_use_lists(int64_t M, int64_t K, int64_t R) { return R >= 2 * M && R * K >= ((int64_t)1 << 24); }

extern "C" size_t f8_quantize_workspace_bytes(int64_t M, int64_t K, int64_t R) {
    if (M < 1 || K < 1 || R < 1 || M > CQ_F8_MAX_ROWS || K > CQ_F8_MAX_K || R > CQ_F8_MAX_ROWS) return 0;
    if (!f8_use_lists(M, K, R)) return 0;
    return (((size_t)M * (size_t)(1 + list_cap(M, R)) + 1u + (size_t)R) * sizeof(int32_t) + 255u) & ~(size_t)255u;
}

extern "C" cq_status f8_quantize(const void* X, cq_dtype xt, int64_t M, int64_t K, const int32_t* rows,
                                 int64_t R, uint8_t* codes, uint8_t* scales, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    if (!X || !codes || !scales || M < 1 || K < 1 || R < 1 || !cq_dtype_valid(xt)) return CQ_ERR_INVALID_ARG;
    if (!rows && R != M) return CQ_ERR_INVALID_ARG;
    if (M > CQ_F8_MAX_ROWS || R > CQ_F8_MAX_ROWS || K > CQ_F8_MAX_K) return CQ_ERR_UNSUPPORTED;
    if (!aligned16(X) || (rows && !aligned16(rows)) || !aligned16(codes) || !aligned16(scales) ||
        !aligned16(workspace))
        return CQ_ERR_ALIGNMENT;
    const int groups = (int)((K + kGroup - 1) / kGroup), quads = (groups + 3) / 4;
    if (R > ((int64_t)1 << 34) / quads) return CQ_ERR_UNSUPPORTED;
    const size_t space = rows ? f8_quantize_workspace_bytes(M, K, R) : 0;
    if (space && (!workspace || workspace_bytes < space)) return CQ_ERR_WORKSPACE;
    const cudaStream_t cs = as_stream(stream);
    uint32_t* words = reinterpret_cast<uint32_t*>(scales);
    Lists l = {};
    int64_t from = R;   // pieces of work of a row each, at most
    int parts = 1;
    if (space) {
        l.cap = (int)list_cap(M, R);
        l.count = static_cast<int32_t*>(workspace);
        l.slots = l.count + M + 1;
        l.alone = l.slots + M * l.cap;
        parts = (l.cap + 31) / 32;
        from = M * parts;
        const cudaError_t e = cudaMemsetAsync(l.count, 0, ((size_t)M + 1) * sizeof(int32_t), cs);
        if (e != cudaSuccess) { set_last_cuda_error((int)e); return CQ_ERR_CUDA; }
        const cq_status st = launch_pdl(f8_list_kernel, dim3((unsigned)((R + 255) / 256)), dim3(256), 0, cs, rows, M, R, l);
        if (st != CQ_OK) return st;
    }
    // whole rows where they give every warp several, else as many segments as fill the warps
    const int64_t fill = (int64_t)sm_count() * kQuantCtas * 8, want = space ? 4 * fill : fill;
    int64_t segs64 = from >= want ? 1 : (want + from - 1) / from;
    if (segs64 > quads) segs64 = quads;
    const int per = (quads + (int)segs64 - 1) / (int)segs64;
    const int segs = (quads + per - 1) / per;
    const int64_t need = ((from > R ? from : R) * segs + 7) / 8;
    const dim3 gd((unsigned)(need < fill / 8 ? need : fill / 8)), bd(256);
    auto launch = [&](auto direct, auto lists, auto x) {
        return space ? launch_pdl(lists, gd, bd, 0, cs, x, M, K, rows, l, codes, words, quads, per, segs, parts)
                     : launch_pdl(direct, gd, bd, 0, cs, x, M, K, rows, R, codes, words, quads, per, segs);
    };
    using bf16 = __nv_bfloat16;
    if (xt == CQ_F32) {
        const float* x = static_cast<const float*>(X);
        return K % 4 == 0 ? launch(f8_quantize_kernel<float, true>, f8_quantize_lists_kernel<float, true>, x)
                          : launch(f8_quantize_kernel<float, false>, f8_quantize_lists_kernel<float, false>, x);
    }
    const bf16* x = static_cast<const bf16*>(X);
    return K % 8 == 0 ? launch(f8_quantize_kernel<bf16, true>, f8_quantize_lists_kernel<bf16, true>, x)
                      : launch(f8_quantize_kernel<bf16, false>, f8_quantize_lists_kernel<bf16, false>, x);
}

extern "C" cq_status f8_quantize_weights(const void* W, cq_dtype wt, int64_t E, int64_t N, int64_t K,
                                         uint8_t* codes, uint8_t* scales, void* stream) {
    if (!W || !codes || !scales || E < 1 || N < 1 || K < 1 || !cq_dtype_valid(wt)) return CQ_ERR_INVALID_ARG;
    if (E > CQ_MOE_MAX_EXPERTS || N > CQ_F8_MAX_N || K > CQ_F8_MAX_K) return CQ_ERR_UNSUPPORTED;
    if (!aligned16(W) || !aligned16(codes) || !aligned16(scales)) return CQ_ERR_ALIGNMENT;
    const int64_t nblk = (N + kGroup - 1) / kGroup;
    const int64_t sbytes = (K + 4 * kGroup - 1) / (4 * kGroup) * 4;
    const int64_t blocks = E * nblk * sbytes;
    const int64_t cap = (int64_t)sm_count() * 16;
    const dim3 gd((unsigned)(blocks < cap ? blocks : cap)), bd(256);
    const cudaStream_t cs = as_stream(stream);
    if (wt == CQ_F32)
        return launch_pdl(f8_quantize_weights_kernel<float>, gd, bd, 0, cs, static_cast<const float*>(W), N, K, nblk,
                          sbytes, blocks, codes, scales);
    return launch_pdl(f8_quantize_weights_kernel<__nv_bfloat16>, gd, bd, 0, cs,
                      static_cast<const __nv_bfloat16*>(W), N, K, nblk, sbytes, blocks, codes, scales);
}
