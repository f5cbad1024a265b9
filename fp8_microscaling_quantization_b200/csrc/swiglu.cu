// swiglu.cu -- the gated activation of a feed-forward layer, quantized for
// the down product, and its backward pass.
//
// x [rows, 2F] is the fused gate/up product: the gate half g in columns
// [0, F), the up half u in [F, 2F).
//   y  = silu(g) * u,   silu(g) = g * s,  s = 1 / (1 + exp(-g))
// in binary32, quantized without being stored.  Backward (the codes' rounding
// passed straight through):
//   grad_g = gy * u * s * (1 + g * (1 - s)),   grad_u = gy * g * s
//
// Both passes read and write every tensor once and are bound by HBM.
#include <algorithm>

#define BSQ_DBG_FILE 9
#include "debug.cuh"
#include "row_quant.cuh"

namespace bsq {

// s = 1 / (1 + exp(-g)), of the backward pass: HBM bounds that either way
// (16384 x 2048 bf16 55.5 us, with the hardware's approximations 56).
__device__ __forceinline__ float sigmoid(float g) { return __frcp_rn(1.0f + expf(-g)); }

// silu(g) * u of 8 elements, into g.  The division is the hardware's reciprocal
// (1 last place off); where 1 + exp(-g) passes 2**126, at g < -87.3, it gives 0.
//
// bf16: a rounded product g * log2(e) would put |g| * 2**-23 of error into the
// power, so it is split.  With H = log2(e) to 16 bits, t = -g * H is exact (8
// bits times 16) and p = 2**t is the hardware's (2 last places off); the rest
// of log2(e) makes the power p exp(-q), q = g * c, and with |q| < 5e-4 that is
// p (1 - q), give or take q**2 / 2.  (16384 x 2048 bf16 to MXFP8 31.4 us, to
// NVFP4 36.9, with the rounded product 31.1 and 37.0; with expf 41 and 45.)
__device__ __forceinline__ void swiglu8(float g[8], const float u[8], const uint16_t*) {
    constexpr float kH = 1.44268798828125f;  // 47274 / 2**15
    constexpr float kC = 4.8884951e-06f;     // (log2(e) - kH) ln(2)
    const float2 h = make_float2(-kH, -kH), c = make_float2(-kC, -kC), one = make_float2(1.0f, 1.0f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 v = make_float2(g[j], g[j + 1]), t = mul_f32x2(v, h);
        float2 p, s;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(t.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(t.y));
        p = fma_f32x2(p, fma_f32x2(v, c, one), one);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(p.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(p.y));
        const float2 y = mul_f32x2(v, s);
        g[j] = y.x;
        g[j + 1] = y.y;
    }
    mul8(g, u);
}
// fp32: HBM hides expf (16384 x 2048 to MXFP8 51.8 us, without it 51.5).
__device__ __forceinline__ void swiglu8(float g[8], const float u[8], const float*) {
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = 1.0f + expf(-g[j]);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[j]) : "f"(x));
    }
    mul8(g, s);
    mul8(g, u);
}

// NVFP4: a CTA holds a row, whose maximum gives the row scale.
template <typename T, int NCH, int MAXT>
__global__ void __launch_bounds__(MAXT) swiglu_quant_kernel(const T* __restrict__ x, int64_t rows, int F, uint8_t* __restrict__ codes,
                                    uint8_t* __restrict__ scales, float* __restrict__ row_scale) {
    __shared__ __align__(16) float buf[64];
    RowReduce red(buf);
    const int nchunks = F / 8;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* xr = x + row * 2 * F;
        Raw8<T> rg[NCH], ru[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            rg[i].zero();
            ru[i].zero();
            if (c < nchunks && BSQ_DOK(F + c * 8 + 8 <= 2 * F)) {
                rg[i].load_cs(xr + c * 8);
                ru[i].load_cs(xr + F + c * 8);
            }
        }
        float y[NCH][8];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            float g[8], u[8];
            rg[i].get(g);
            ru[i].get(u);
            swiglu8(g, u, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[i][j] = g[j];
        }
        const int64_t base = row * F;
        const float g = quantize_row<BSQ_NVFP4, NCH>(y, nchunks, codes + base / 2, scales + base / 16, red);
        if (threadIdx.x == 0) row_scale[row] = g;
    }
}

// The formats without a row scale: chunks of all rows in one stream.  One
// chunk per thread at a time, at full occupancy: the loads of other warps
// cover a warp's arithmetic (16384 x 2048 bf16 to MXFP8 31.4 us, 82% of the
// HBM copy rate; two or four chunks in flight per thread 35 us).
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads, 8) swiglu_flat_kernel(const T* __restrict__ x, FastDiv row_chunks, int64_t nchunks,
                                                                  int F, uint8_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    // whole warps loop together: a block's scale is found by its lanes
    for (int64_t base = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); base < nchunks; base += stride) {
        const int64_t c = min(base + lane, nchunks - 1);  // lanes past the end stand in for the last chunk
        const uint32_t row = fdiv((uint32_t)c, row_chunks);
        const int64_t at = (int64_t)row * 2 * F + (c - (int64_t)row * row_chunks.d) * 8;
        Raw8<T> rg, ru;
        if (BSQ_DOK(at + F + 8 <= nchunks * 16)) {
            rg.load_cs(x + at);
            ru.load_cs(x + at + F);
        }
        float g[8], u[8];
        rg.get(g);
        ru.get(u);
        swiglu8(g, u, x);
        uint32_t s;
        const uint2 w = chunk_codes<FMT>(g, group_max<4>(amax8(g)), 0.0f, 0.0f, &s);
        if (base + lane < nchunks) {
            if (FMT == BSQ_MXFP8) reinterpret_cast<uint2*>(codes)[c] = w;
            else reinterpret_cast<uint32_t*>(codes)[c] = w.x;
            if ((lane & 3) == 0) scales[c >> 2] = (uint8_t)s;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 6) swiglu_bwd_kernel(const T* __restrict__ gy, const T* x,
                                                                 FastDiv row_chunks, int64_t nchunks, int F,
                                                                 T* gx) {  // gx may be x
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < nchunks; c += stride) {
        const uint32_t row = fdiv((uint32_t)c, row_chunks);
        const int64_t at = (int64_t)row * 2 * F + (c - (int64_t)row * row_chunks.d) * 8;
        if (!BSQ_DOK(at + F + 8 <= nchunks * 16)) continue;
        Raw8<T> rd, rg, ru;
        rd.load_cs(gy + c * 8);
        rg.load_cs(x + at);
        ru.load_cs(x + at + F);
        float d[8], g[8], u[8];
        rd.get(d);
        rg.get(g);
        ru.get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid(g[j]), gs = g[j] * s;
            u[j] = d[j] * u[j] * (s + gs * (1.0f - s));
            d[j] = d[j] * gs;
        }
        store8(gx + at, u);
        store8(gx + at + F, d);
    }
}

template <typename T>
static void launch_swiglu_nvfp4(const T* x, int64_t rows, int64_t F, uint8_t* codes, uint8_t* scales, float* row_scale,
                                cudaStream_t st) {
    const int64_t n = F / 8;
    auto threads = [&](int nch) { return (int)((n + 32 * nch - 1) / (32 * nch) * 32); };
    if (n <= 128) launch_rows<swiglu_quant_kernel<T, 1, 128>>(rows, threads(1), st, x, rows, (int)F, codes, scales, row_scale);
    else if (n <= 1024) launch_rows<swiglu_quant_kernel<T, 4, 256>>(rows, threads(4), st, x, rows, (int)F, codes, scales, row_scale);
    else if (n <= 2048) launch_rows<swiglu_quant_kernel<T, 4, 512>>(rows, threads(4), st, x, rows, (int)F, codes, scales, row_scale);
    else launch_rows<swiglu_quant_kernel<T, 4, 1024>>(rows, threads(4), st, x, rows, (int)F, codes, scales, row_scale);
}

template <typename T>
static void launch_swiglu_fmt(bsq_format fmt, const void* xv, int64_t rows, int64_t F, uint8_t* codes, uint8_t* scales,
                              float* row_scale, cudaStream_t st) {
    const T* x = (const T*)xv;
    const int64_t n = rows * F / 8;
    const FastDiv rc = make_fastdiv((uint32_t)(F / 8));
    if (fmt == BSQ_NVFP4) launch_swiglu_nvfp4<T>(x, rows, F, codes, scales, row_scale, st);
    else if (fmt == BSQ_MXFP4) launch_fit<swiglu_flat_kernel<T, BSQ_MXFP4>>(n, 1, st, x, rc, n, (int)F, codes, scales);
    else launch_fit<swiglu_flat_kernel<T, BSQ_MXFP8>>(n, 1, st, x, rc, n, (int)F, codes, scales);
}

}  // namespace bsq

using namespace bsq;

BSQ_API bsq_status bsq_swiglu_quantize(bsq_format fmt, const void* x, bsq_dtype t, int64_t rows, int64_t F,
                                       uint8_t* codes, uint8_t* scales, float* row_scale, bsq_stream_t stream) {
    const char* fn = "bsq_swiglu_quantize";
    BSQ_TRY(check_dtype(t));
    BSQ_TRY(check_quant_format(fn, fmt));
    BSQ_TRY(check_matrix(fn, x, rows, F, fmt_block(fmt)));
    if (F > kMaxRowElems) return fail(BSQ_ERR_UNSUPPORTED, "%s: rows of more than %lld elements", fn, (long long)kMaxRowElems);
    if (rows * F == 0) return BSQ_OK;
    if (!codes || !scales || (fmt == BSQ_NVFP4 && !row_scale)) return fail(BSQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(x, 16) || !aligned(codes, 8) || !aligned(row_scale, 4))
        return fail(BSQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const size_t n = (size_t)(rows * F);
    const Span outs[] = {{codes, fmt == BSQ_MXFP8 ? n : n / 2}, {scales, n / fmt_block(fmt)},
                         {fmt == BSQ_NVFP4 ? row_scale : nullptr, (size_t)rows * 4}};
    const Span read[] = {{x, 2 * n * (t == BSQ_BF16 ? 2 : 4)}};
    if (any_overlap(outs, read)) return fail(BSQ_ERR_INVALID_ARG, "%s: an output overlaps x or another output", fn);
    cudaStream_t st = (cudaStream_t)stream;
    if (t == BSQ_BF16) launch_swiglu_fmt<uint16_t>(fmt, x, rows, F, codes, scales, row_scale, st);
    else launch_swiglu_fmt<float>(fmt, x, rows, F, codes, scales, row_scale, st);
    return check_launch(fn);
}

BSQ_API bsq_status bsq_swiglu_backward(const void* grad_y, const void* x, bsq_dtype t, int64_t rows, int64_t F,
                                       void* grad_x, bsq_stream_t stream) {
    const char* fn = "bsq_swiglu_backward";
    BSQ_TRY(check_dtype(t));
    BSQ_TRY(check_matrix(fn, grad_y, rows, F, 8));
    if (rows * F == 0) return BSQ_OK;
    if (!x || !grad_x) return fail(BSQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (F > (int64_t(1) << 30)) return fail(BSQ_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (!aligned(grad_y, 16) || !aligned(x, 16) || !aligned(grad_x, 16))
        return fail(BSQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    // each thread reads its gate and up elements before it writes their gradients
    const size_t bytes = (size_t)(rows * F) * (t == BSQ_BF16 ? 2 : 4);
    if (overlap(grad_x, 2 * bytes, grad_y, bytes) || (grad_x != x && overlap(grad_x, 2 * bytes, x, 2 * bytes)))
        return fail(BSQ_ERR_INVALID_ARG, "%s: grad_x overlaps an input (it may be x itself)", fn);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t nchunks = rows * F / 8;
    const FastDiv rc = make_fastdiv((uint32_t)(F / 8));
    if (t == BSQ_BF16)
        launch_fit<swiglu_bwd_kernel<uint16_t>>(nchunks, 1, st, (const uint16_t*)grad_y, (const uint16_t*)x, rc, nchunks,
                                                   (int)F, (uint16_t*)grad_x);
    else
        launch_fit<swiglu_bwd_kernel<float>>(nchunks, 1, st, (const float*)grad_y, (const float*)x, rc, nchunks, (int)F,
                                                (float*)grad_x);
    return check_launch(fn);
}

#ifdef BSQ_DEBUG
cudaError_t bsq_dbg_take_swiglu(uint32_t* count, uint32_t* first) { return bsq::dbg_take(count, first); }
#endif
