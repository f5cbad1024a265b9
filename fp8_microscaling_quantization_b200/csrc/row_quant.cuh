// row_quant.cuh -- block-scaled codes of values that a kernel holds in
// registers, shared by the kernels that quantize what they compute (norm.cu,
// swiglu.cu).  A lane holds chunks of 8 consecutive elements of a row; a block
// of 16 or 32 spans 2 or 4 adjacent lanes.
#pragma once

#include <mutex>

#include "common.cuh"
#include "overlap.h"

namespace bsq {

// Largest row of the kernels that keep a row in one CTA's registers:
// 1024 threads x 4 chunks x 8 elements.
constexpr int64_t kMaxRowElems = 32768;
constexpr int kMaxRowSmem = 226 * 1024;  // dynamic shared memory of a CTA at most (1 KiB is static)

static inline int fmt_block(bsq_format f) { return f == BSQ_NVFP4 ? 16 : 32; }

static inline bsq_status check_quant_format(const char* fn, bsq_format f) {
    if (f != BSQ_NVFP4 && f != BSQ_MXFP4 && f != BSQ_MXFP8)
        return fail(BSQ_ERR_UNSUPPORTED, "%s: format must be NVFP4, MXFP4 or MXFP8", fn);
    return BSQ_OK;
}

// Sums and maxima over the threads of a CTA, one barrier each: consecutive
// reductions of a kernel alternate between two 32-float halves of `buf`, so a
// thread that still reads one half is behind the barrier of the next before
// that half is written again.  Warps add up their lanes by shuffles, then
// every thread adds the warps' values in order (up to 8 of them as two 16-byte
// reads), so the order of a sum depends on the CTA's size alone.
struct RowReduce {
    float* buf;  // 64 floats of shared memory, 16-byte aligned
    int half = 0;
    __device__ __forceinline__ explicit RowReduce(float* b) : buf(b) {
        if (threadIdx.x < 64) b[threadIdx.x] = 0.0f;  // warps that the CTA does not have
        if (blockDim.x < 64) b[threadIdx.x + 32] = 0.0f;
        __syncthreads();
    }
    template <typename OP>
    __device__ __forceinline__ float across(float v, OP op) {
        if (blockDim.x == 32) return v;
        float* b = buf + 32 * half;
        half ^= 1;
        if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
        __syncthreads();
        const float4* q = reinterpret_cast<const float4*>(b);
        float4 x = q[0], y = q[1];
        v = op(op(op(x.x, x.y), op(x.z, x.w)), op(op(y.x, y.y), op(y.z, y.w)));
        for (int i = 2; i < (int)(blockDim.x + 127) / 128; ++i) {
            x = q[i];
            v = op(v, op(op(x.x, x.y), op(x.z, x.w)));
        }
        return v;
    }
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return across(v, [](float a, float b) { return a + b; });
    }
    __device__ __forceinline__ float max_nonneg(float v) {
        return across(warp_max_nonneg(v), [](float a, float b) { return fmaxf(a, b); });
    }
};

static __device__ __noinline__ uint32_t e2m1x8_by_division(float v0, float v1, float v2, float v3, float v4, float v5, float v6,
                                                    float v7, float d) {
    const float q[8] = {__fdiv_rn(v0, d), __fdiv_rn(v1, d), __fdiv_rn(v2, d), __fdiv_rn(v3, d),
                        __fdiv_rn(v4, d), __fdiv_rn(v5, d), __fdiv_rn(v6, d), __fdiv_rn(v7, d)};
    return e2m1x8_encode_hw(q);
}

// e2m1 codes of RN(v[j] / d), d > 0.  With r = RN(1 / d), v * r * (1 -+ 2**-21)
// enclose RN(v / d) (r, its two products and the quotient round by 2**-24
// each), and e2m1 rounding is monotone: where both ends give the same codes,
// those are the quotient's.  Else, or where d or r could be subnormal, by
// division.
__device__ __forceinline__ uint32_t e2m1x8_by_brackets(const float v[8], float d) {
    if (d >= 2.3509887e-38f /* 2**-125 */ && d <= 4.2535296e37f /* 2**125 */) {
        const float r = __frcp_rn(d);
        const float2 rlo = make_float2(__fmul_rn(r, 0.99999952f), __fmul_rn(r, 0.99999952f));
        const float2 rhi = make_float2(__fmul_rn(r, 1.00000048f), __fmul_rn(r, 1.00000048f));
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 a = make_float2(v[j], v[j + 1]);
            const float2 l = mul_f32x2(a, rlo), u = mul_f32x2(a, rhi);
            lo[j] = l.x; lo[j + 1] = l.y;
            hi[j] = u.x; hi[j + 1] = u.y;
        }
        const uint32_t c = e2m1x8_encode_hw(lo);
        if (c == e2m1x8_encode_hw(hi)) return c;
    }
    return e2m1x8_by_division(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], d);
}

// Codes and scale byte of one chunk (8 values) whose block maximum is amax_b.
// g and rg: row scale and nv_recip_or_zero(g) (NVFP4 only).  The code word is
// 4 bytes of e2m1 (low word) or 8 bytes of e4m3.
template <int FMT>
__device__ __forceinline__ uint2 chunk_codes(const float v[8], float amax_b, float g, float rg, uint32_t* scale) {
    if (FMT == BSQ_NVFP4) {
        if (g == 0.0f) {
            *scale = 0u;
            return make_uint2(0u, 0u);
        }
        const uint32_t s = nv_scale_code(amax_b, g, rg);
        *scale = s;
        return make_uint2(e2m1x8_by_brackets(v, __fmul_rn(e4m3x2_decode_hw(s).x, g)), 0u);
    }
    const int e = (FMT == BSQ_MXFP4) ? mx_exponent(amax_b) : mx8_exponent(amax_b);
    *scale = (uint32_t)(e + 127);
    const float inv = exp2_int(-e);  // v * 2**-e == v / 2**e exactly
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = v[j] * inv;
    if (FMT == BSQ_MXFP4) return make_uint2(e2m1x8_encode_hw(q), 0u);
    return make_uint2(e4m3x2_encode_hw(q[0], q[1]) | (e4m3x2_encode_hw(q[2], q[3]) << 16),
                      e4m3x2_encode_hw(q[4], q[5]) | (e4m3x2_encode_hw(q[6], q[7]) << 16));
}

// Quantize a row held as NCH chunks per thread (chunk i of a thread is chunk
// threadIdx.x + i * blockDim.x of the row; values past the row's end are not
// used: blocks do not straddle it).
// codes and scales point at the row's first byte.  Returns the NVFP4 row scale.
template <int FMT, int NCH>
__device__ __forceinline__ float quantize_row(float (&y)[NCH][8], int nchunks, uint8_t* codes, uint8_t* scales,
                                              RowReduce& red) {
    constexpr int L = (FMT == BSQ_NVFP4) ? 2 : 4;  // lanes per block
    float am[NCH], top = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        am[i] = group_max<L>(amax8(y[i]));
        if ((int)(threadIdx.x + i * blockDim.x) < nchunks) top = fmaxf(top, am[i]);
    }
    float g = 0.0f, rg = 0.0f;
    if (FMT == BSQ_NVFP4) {
        g = __fdiv_rn(red.max_nonneg(top), kNvGlobalDiv);
        rg = nv_recip_or_zero(g);
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nchunks) {
            uint32_t s;
            const uint2 w = chunk_codes<FMT>(y[i], am[i], g, rg, &s);
            if (FMT == BSQ_MXFP8) reinterpret_cast<uint2*>(codes)[c] = w;
            else reinterpret_cast<uint32_t*>(codes)[c] = w.x;
            if ((threadIdx.x % L) == 0) scales[c / L] = (uint8_t)s;
        }
    }
    return g;
}

// v[j] * w[j] and v[j] * f of 8 values, by packed binary32 multiplies.
__device__ __forceinline__ void mul8(float v[8], const float w[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 p = mul_f32x2(make_float2(v[j], v[j + 1]), make_float2(w[j], w[j + 1]));
        v[j] = p.x;
        v[j + 1] = p.y;
    }
}
__device__ __forceinline__ void mul8(float v[8], float f) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 p = mul_f32x2(make_float2(v[j], v[j + 1]), make_float2(f, f));
        v[j] = p.x;
        v[j + 1] = p.y;
    }
}
// v[j] = a[j] * b + c[j]
__device__ __forceinline__ void fma8(float v[8], const float a[8], float b, const float c[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 p = fma_f32x2(make_float2(a[j], a[j + 1]), make_float2(b, b), make_float2(c[j], c[j + 1]));
        v[j] = p.x;
        v[j + 1] = p.y;
    }
}
// s + sum of a[j] * b[j], kept as two running sums (even and odd j)
__device__ __forceinline__ float2 dot8(const float a[8], const float b[8], float2 s) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) s = fma_f32x2(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), s);
    return s;
}

// CTAs of KERNEL that one SM holds at `threads` threads and `smem` bytes of
// dynamic shared memory (0 where it may not be given that many), from the
// occupancy calculator; the latest kResidentKept answers are kept.
constexpr int kResidentKept = 64;
template <auto KERNEL>
static inline int resident_rows(int threads, int smem = 0) {
    struct Entry {
        int dev, threads, smem, n;  // n + 1; 0: none yet
    };
    static Entry kept[kResidentKept] = {};
    static int next = 0;
    static std::mutex mu;
    int dev = -1;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& e : kept) {
        if (e.n == 0) break;
        if (e.dev == dev && e.threads == threads && e.smem == smem) return e.n - 1;
    }
    int n = 0;
    if ((smem > 0 && cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRowSmem) != cudaSuccess) ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, threads, smem) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = smem > 0 ? 0 : 1;
    }
    kept[next] = {dev, threads, smem, n + 1};
    next = (next + 1) % kResidentKept;
    return n;
}

// One wave of CTAs, a row each at a time.
template <auto KERNEL, typename... A>
static inline void launch_rows(int64_t rows, int threads, cudaStream_t st, A... args) {
    const int64_t cap = (int64_t)sm_count() * resident_rows<KERNEL>(threads);
    KERNEL<<<(int)std::min<int64_t>(rows, cap), threads, 0, st>>>(args...);
}

}  // namespace bsq
