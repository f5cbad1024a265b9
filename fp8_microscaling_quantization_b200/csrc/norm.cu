// norm.cu -- the norms around a block, fused: the RMS norm after the block
// with its gate, the residual scale and sum, the RMS norm before the next
// block and the quantization of its output; and the backward pass.
//
// Forward, per row of C elements (all in binary32):
//   v = x                              (the block's output)
//   v = v * rx * post_weight           rx = (mean(v^2) + eps)^-1/2, if post_weight
//   v = v * gate                       if gate
//   h = residual + residual_scale * v
//   y = h * rh * weight                rh = (mean(h^2) + eps)^-1/2
// h is rounded once to its dtype and stored; y, from the unrounded h, goes to
// the codes of the chosen format without ever being stored.
//
// Backward, with the codes' rounding passed straight through (gy = dL/dy, gh
// = dL/dh from the residual stream, hhat = h * rh, xhat = x * rx):
//   a  = gy * weight
//   dh = gh + rh * (a - hhat * mean(a * hhat))         = grad_residual
//   grad_weight      = sum over rows of gy * hhat
//   dv = residual_scale * dh
//   grad_gate        = dv * (xhat * post_weight)       (dv * x without post_weight)
//   du = dv * gate
//   grad_post_weight = sum over rows of du * xhat
//   grad_x           = rx * (b - xhat * mean(b * xhat)), b = du * post_weight
//                      (du without post_weight)
//
// One CTA holds a row: bound by HBM for many rows and by the barriers of the
// row's two or three reductions for few.  Rows overlap because several CTAs
// share an SM; copying a thread's part of the next row ahead with cp.async
// instead was slower, by its instructions (16384 x 7168 bf16 to MXFP8 with
// post-norm and gate: 219 us against 185 at the time).
//   Forward: up to 20480 columns the row's inputs stay in registers and every
// tensor is read once; longer rows read x a second time if there is a norm
// after the block (from L2).  Which optional operands there are is known at
// compile time from 257 to 20480 columns.
//   Backward: up to 8192 columns (bf16: 16384) the inputs stay in registers;
// longer rows read h, and with post_weight x, a second time.  The sums of the
// weight gradients over a CTA's rows, each thread's own columns, are in
// registers up to 8192 columns, then in shared memory, or, where that does not
// hold them, in the CTA's row of the scratch; a second kernel adds the CTAs'
// sums in a fixed order.  Optional operands are known at compile time from 257
// to 8192 columns.
#include <algorithm>

#define BSQ_DBG_FILE 8
#include "debug.cuh"
#include "row_quant.cuh"

namespace bsq {

template <typename T>
struct NormArgs {
    const T* x;
    const T* residual;  // NULL: 0
    const T* gate;      // NULL: 1
    int64_t rows;
    int C;
    float scale, eps;
    const float* post_weight;  // NULL: no norm after the block
    const float* weight;
    T* h;  // NULL: not stored
    uint8_t* codes;
    uint8_t* scales;
    float* row_scale;  // NVFP4
    float* rstd;
    float* post_rstd;
};

// 8 weights from element `at`.
__device__ __forceinline__ void load_weight(const float* w, uint32_t at, float v[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + at));
    const float4 b = __ldg(reinterpret_cast<const float4*>(w + at) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Which optional operands a kernel has: known at compile time, so that its
// chunks' arithmetic is one block of code (tests of the pointers split it:
// 16384 x 7168 226 against 185 us), or kAny: tested at run time, for the row
// lengths whose kernels are not worth a copy per combination.
constexpr int kAny = -1, kPost = 1, kGate = 2, kStream = 4;  // kStream: residual, or grad_h
template <int HAVE>
__device__ __forceinline__ bool have(int bit, const void* p) {
    return HAVE == kAny ? p != nullptr : (HAVE & bit) != 0;
}

// Where a thread's chunks lie in a row of C elements.  A chunk past the row's
// end stands in for the row's last one: it is loaded and computed with like
// the others (a branch around it cost more: 16384 x 7168 321 us), but adds
// nothing to sums and is not stored.
template <int NCH>
struct Chunks {
    uint32_t C;
    __device__ __forceinline__ explicit Chunks(int c) : C((uint32_t)c) {}
    __device__ __forceinline__ uint32_t raw(int i) const { return (threadIdx.x + (uint32_t)i * blockDim.x) * 8u; }
    __device__ __forceinline__ bool valid(int i) const { return raw(i) < C; }
    __device__ __forceinline__ uint32_t at(int i) const { return min(raw(i), C - 8u); }
    // whether chunk i of a row is stored
    __device__ __forceinline__ bool stored(int i, int64_t row, int64_t rows) const {
        return valid(i) && BSQ_DOK(row < rows && at(i) + 8u <= C);
    }
};

// (sum / C + eps)^-1/2, each step rounded to nearest: a row's factor is in all
// of its codes.  It is multiplied in by itself too: folded into the residual
// scale first, that product's rounding would be in all of them as well.  (The
// weights differ by column, and weight * rstd first costs nothing in accuracy
// and less time: 16384 x 7168 bf16 to NVFP4 with post-norm and gate 214 us,
// after h * rstd 224.)
__device__ __forceinline__ float rms_factor(float sum, int C, float eps) {
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)C), eps));
}

// KEEP: a thread's elements of the inputs stay in registers, all loads issued
// first; else (rows too long for that) they are read where they are used,
// again from L2 the second time.
template <typename T, int FMT, int NCH, int MAXT, int MINB, int HAVE, bool KEEP>
__global__ void __launch_bounds__(MAXT, MINB) norm_quant_kernel(NormArgs<T> p) {
    __shared__ __align__(16) float buf[64];
    RowReduce red(buf);
    constexpr int kCodeBits = (FMT == BSQ_MXFP8) ? 8 : 4, kBlock = (FMT == BSQ_NVFP4) ? 16 : 32;
    const Chunks<NCH> ch(p.C);
    const bool post_norm = have<HAVE>(kPost, p.post_weight), gated = have<HAVE>(kGate, p.gate);
    const bool summed = have<HAVE>(kStream, p.residual);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t base = row * p.C;
        const T *x = p.x + base, *residual = p.residual + base, *gate = p.gate + base;  // used if not NULL
        Raw8<T> rx[NCH], rr[NCH], rz[NCH];
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const uint32_t at = ch.at(i);
                rx[i].load_cs(x + at);
                if (summed) rr[i].load_cs(residual + at);
                if (gated) rz[i].load_cs(gate + at);
            }
        }
        float post = 1.0f;
        if (post_norm) {
            float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                float v[8];
                if (!KEEP) rx[i].load(x + ch.at(i));
                rx[i].get(v);
                ss = ch.valid(i) ? dot8(v, v, ss) : ss;
            }
            post = rms_factor(red.sum(ss.x + ss.y), p.C, p.eps);
        }
        float h[NCH][8];
        float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t at = ch.at(i);
            if (!KEEP) {
                rx[i].load(x + at);
                if (summed) rr[i].load_cs(residual + at);
                if (gated) rz[i].load_cs(gate + at);
            }
            rx[i].get(h[i]);
            if (post_norm) {
                float w[8];
                load_weight(p.post_weight, at, w);
                mul8(h[i], post);
                mul8(h[i], w);
            }
            if (gated) {
                float z[8];
                rz[i].get(z);
                mul8(h[i], z);
            }
            if (summed) {
                float r[8];
                rr[i].get(r);
                fma8(h[i], h[i], p.scale, r);
            } else {
                mul8(h[i], p.scale);
            }
            ss = ch.valid(i) ? dot8(h[i], h[i], ss) : ss;
            if (p.h && ch.stored(i, row, p.rows)) store8(p.h + base + at, h[i]);
        }
        const float rstd = rms_factor(red.sum(ss.x + ss.y), p.C, p.eps);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t at = ch.at(i);
            float w[8];
            load_weight(p.weight, at, w);
            mul8(w, rstd);
            mul8(h[i], w);
        }
        const float g = quantize_row<FMT, NCH>(h, p.C / 8, p.codes + base * kCodeBits / 8, p.scales + base / kBlock, red);
        if (threadIdx.x == 0) {
            if (FMT == BSQ_NVFP4) p.row_scale[row] = g;
            p.rstd[row] = rstd;
            if (post_norm) p.post_rstd[row] = post;
        }
    }
}

// Columns [8c, 8c + 8) of a row of sums.
__device__ __forceinline__ void put_sum(float* row, int c, const float v[8]) {
    *reinterpret_cast<float4*>(row + 8 * c) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + 8 * c + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void get_sum(const float* row, int c, float v[8]) {
    const float4 a = *reinterpret_cast<const float4*>(row + 8 * c), b = *reinterpret_cast<const float4*>(row + 8 * c + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// v[j] += a[j] * b[j]
__device__ __forceinline__ void add_products(float v[8], const float a[8], const float b[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 t = fma_f32x2(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), make_float2(v[j], v[j + 1]));
        v[j] = t.x;
        v[j + 1] = t.y;
    }
}
// The same for the sums of chunk c's columns, in registers or in a row.
template <bool REGS>
__device__ __forceinline__ void add_sum(float regs[8], float* row, int c, const float a[8], const float b[8]) {
    if (REGS) {
        add_products(regs, a, b);
    } else {
        float v[8];
        get_sum(row, c, v);
        add_products(v, a, b);
        put_sum(row, c, v);
    }
}

template <typename T>
struct NormBwdArgs {
    const T* gy;
    const T* gh;  // NULL: 0
    const T* h;
    const float* rstd;
    const float* weight;
    const T* x;     // NULL: grad_x = scale * dh needs no x
    const T* gate;  // NULL: 1
    const float* post_weight;
    const float* post_rstd;
    float scale;
    int64_t rows;
    int C;
    T* grad_residual;  // NULL: not stored
    T* grad_x;         // NULL: not stored
    T* grad_gate;
    float* partial;       // [CTAs, C] sums of grad_weight
    float* partial_post;  // [CTAs, C] sums of grad_post_weight
};

// The sums of the weight gradients over the CTA's rows are in registers
// (REGS), else in `sums`: dynamic shared memory, or the partial rows
// themselves where that does not hold them.  The next row's grad_y and h are
// requested once this row's are used, so that a CTA alone on its SM (its
// registers leave no room for a second) keeps loads in flight across the
// reductions.
template <typename T, int NCH, int MAXT, bool REGS, int HAVE, bool KEEP>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(NormBwdArgs<T> p, bool sums_in_smem) {
    extern __shared__ float4 sums[];
    __shared__ __align__(16) float buf[64];
    RowReduce red(buf);
    const int nchunks = p.C / 8;
    constexpr int NR = REGS ? NCH : 1;
    float dw[NR][8], dpw[NR][8];
    const bool post_norm = have<HAVE>(kPost, p.post_weight), gated = have<HAVE>(kGate, p.gate);
    const bool summed = have<HAVE>(kStream, p.gh), has_x = post_norm || gated;
    float* const out = p.partial + (int64_t)blockIdx.x * p.C;
    float* const out_post = p.partial_post + (int64_t)blockIdx.x * p.C;
    float* const sw = sums_in_smem ? reinterpret_cast<float*>(sums) : out;
    float* const spw = sums_in_smem ? sw + p.C : out_post;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = dpw[i][j] = 0.0f;
    if (!REGS)
        for (int c = threadIdx.x; c < nchunks; c += blockDim.x) {  // each thread its own columns
            put_sum(sw, c, dw[0]);
            if (post_norm) put_sum(spw, c, dw[0]);
        }
    const Chunks<NCH> ch(p.C);
    int64_t row = blockIdx.x;
    Raw8<T> rgy[NCH], rh[NCH];
    if (KEEP) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t at = ch.at(i);
            rgy[i].load_cs(p.gy + row * p.C + at);
            rh[i].load_cs(p.h + row * p.C + at);
        }
    }
    for (; row < p.rows; row += gridDim.x) {
        const int64_t base = row * p.C;
        const T *pgh = p.gh + base, *px = p.x + base, *pz = p.gate + base;  // used if not NULL
        Raw8<T> rgh[NCH], rx[NCH], rz[NCH];
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const uint32_t at = ch.at(i);
                if (summed) rgh[i].load_cs(pgh + at);
                if (has_x) rx[i].load_cs(px + at);
                if (gated) rz[i].load_cs(pz + at);
            }
        }
        const float rstd = p.rstd[row];
        const float post = post_norm ? p.post_rstd[row] : 1.0f;
        float d[NCH][8];  // a, then dh, then the gradient of what precedes
        float2 dot = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t at = ch.at(i);
            float w[8], hh[8];
            load_weight(p.weight, at, w);
            if (!KEEP) {
                rgy[i].load_cs(p.gy + base + at);
                rh[i].load(p.h + base + at);
            }
            rgy[i].get(d[i]);
            rh[i].get(hh);
            mul8(hh, rstd);
            if (REGS || ch.valid(i)) add_sum<REGS>(dw[REGS ? i : 0], sw, at / 8, d[i], hh);
            mul8(d[i], w);
            dot = ch.valid(i) ? dot8(d[i], hh, dot) : dot;
        }
        const float mean = __fdiv_rn(red.sum(dot.x + dot.y), (float)p.C);
        const float hm = -(rstd * mean) * rstd;  // dh = gh + rstd * a - (rstd^2 mean) h
        const int64_t next = min(row + gridDim.x, p.rows - 1);
        dot = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const uint32_t at = ch.at(i);
            float hh[8];
            if (!KEEP) {
                rh[i].load_cs(p.h + base + at);
                if (summed) rgh[i].load_cs(pgh + at);
                if (has_x) rx[i].load(px + at);
                if (gated) rz[i].load_cs(pz + at);
            }
            rh[i].get(hh);
            if (KEEP) {
                rgy[i].load_cs(p.gy + next * p.C + at);
                rh[i].load_cs(p.h + next * p.C + at);
            }
            if (summed) {
                float gh[8];
                rgh[i].get(gh);
                fma8(hh, hh, hm, gh);
            } else {
                mul8(hh, hm);
            }
            fma8(d[i], d[i], rstd, hh);
            if (p.grad_residual && ch.stored(i, row, p.rows)) store8(p.grad_residual + base + at, d[i]);
            if (has_x || p.grad_x) {
                mul8(d[i], p.scale);
                if (has_x) {
                    float x[8], w[8];
                    rx[i].get(x);
                    if (post_norm) {
                        load_weight(p.post_weight, at, w);
                        mul8(x, post);
                    }
                    if (gated) {
                        float z[8], gz[8];
                        rz[i].get(z);
#pragma unroll
                        for (int j = 0; j < 8; ++j) gz[j] = d[i][j];
                        mul8(gz, x);
                        if (post_norm) mul8(gz, w);
                        mul8(d[i], z);
                        if (ch.stored(i, row, p.rows)) store8(p.grad_gate + base + at, gz);
                    }
                    if (post_norm) {
                        if (REGS || ch.valid(i)) add_sum<REGS>(dpw[REGS ? i : 0], spw, at / 8, d[i], x);
                        mul8(d[i], w);
                        dot = ch.valid(i) ? dot8(d[i], x, dot) : dot;
                    }
                }
                if (!post_norm && ch.stored(i, row, p.rows)) store8(p.grad_x + base + at, d[i]);
            }
        }
        if (post_norm) {
            const float m = __fdiv_rn(red.sum(dot.x + dot.y), (float)p.C);
            const float xm = -(post * m) * post;  // grad_x = post * b - (post^2 mean) x
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const uint32_t at = ch.at(i);
                float x[8];
                if (!KEEP) rx[i].load_cs(px + at);
                rx[i].get(x);
                mul8(x, xm);
                fma8(d[i], d[i], post, x);
                if (ch.stored(i, row, p.rows)) store8(p.grad_x + base + at, d[i]);
            }
        }
    }
    if (REGS) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nchunks) continue;
            put_sum(out, c, dw[i]);
            if (post_norm) put_sum(out_post, c, dpw[i]);
        }
    } else if (sums_in_smem) {
        for (int c = threadIdx.x; c < nchunks; c += blockDim.x) {
            float v[8];
            get_sum(sw, c, v);
            put_sum(out, c, v);
            if (post_norm) {
                get_sum(spw, c, v);
                put_sum(out_post, c, v);
            }
        }
    }
}

// out[c] = sum over n partial rows: 32 columns (8 threads of 4) x 32 row
// slices per CTA, the slices' sums added in order.  blockIdx.y picks the
// gradient.
__global__ void __launch_bounds__(256) norm_weight_sum_kernel(const float* __restrict__ p0, float* __restrict__ o0,
                                                              const float* __restrict__ p1, float* __restrict__ o1, int n,
                                                              int C) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are written
    const float* p = blockIdx.y ? p1 : p0;
    float* o = blockIdx.y ? o1 : o0;
    const int q = threadIdx.x & 7, slice = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + 4 * q;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < C) {
#pragma unroll 8
        for (int r = slice; r < n; r += 32) {
            // each read once: from L2, past L1
            const float4 t = __ldcg(reinterpret_cast<const float4*>(p + (int64_t)r * C + c));
            v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
        }
    }
    s[slice][4 * q] = v.x; s[slice][4 * q + 1] = v.y; s[slice][4 * q + 2] = v.z; s[slice][4 * q + 3] = v.w;
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < C) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
        o[blockIdx.x * 32 + threadIdx.x] = a;
    }
}

// Threads for a row of nchunks chunks at NCH chunks per thread.
static inline int row_threads(int64_t nchunks, int nch) { return (int)((nchunks + 32 * nch - 1) / (32 * nch) * 32); }

template <typename T, int FMT, int NCH, int MAXT, int MINB, int HAVE = 0>
static void launch_norm_have(int have, const NormArgs<T>& p, cudaStream_t st) {
    if constexpr (HAVE < 8) {
        if (have != HAVE) return launch_norm_have<T, FMT, NCH, MAXT, MINB, HAVE + 1>(have, p, st);
        launch_rows<norm_quant_kernel<T, FMT, NCH, MAXT, MINB, HAVE, true>>(p.rows, row_threads(p.C / 8, NCH), st, p);
    }
}

// Four chunks to a thread spread a row's reductions (some 30 instructions per
// warp each) over 32 elements (16384 x 7168 bf16 to MXFP8 with post-norm and
// gate 188 us; with two chunks and 512 threads 16 us more, with three and 384
// threads 2).  An SM's registers are to hold three CTAs of 256 threads; two for
// fp32 rows, which take twice the registers in flight.  us with two, three and
// four CTAs:
//   16384 x 7168 bf16 to MXFP8, post-norm and gate 214, 188, 197, neither 163, 139, 137
//   4096 x 7168 fp32 to MXFP8, post-norm and gate 89, 122, 127, neither 65, 68, 73
// One warp holds rows of up to 256 elements a chunk per lane; longer rows take
// more threads.
template <typename T, int FMT>
static void launch_norm(const NormArgs<T>& p, cudaStream_t st) {
    const int64_t n = p.C / 8;
    const int have = (p.post_weight ? kPost : 0) | (p.gate ? kGate : 0) | (p.residual ? kStream : 0);
    constexpr int kCtas = sizeof(T) == 4 ? 2 : 3;
    if (n <= 32) launch_rows<norm_quant_kernel<T, FMT, 1, 32, 16, kAny, true>>(p.rows, 32, st, p);
    else if (n <= 1024) launch_norm_have<T, FMT, 4, 256, kCtas>(have, p, st);
    else if (n <= 2048) launch_norm_have<T, FMT, 2, 1024, 1>(have, p, st);
    else if (n <= 2560) launch_norm_have<T, FMT, 4, 640, 1>(have, p, st);
    else launch_rows<norm_quant_kernel<T, FMT, 4, 1024, 1, kAny, false>>(p.rows, row_threads(n, 4), st, p);
}

template <typename T>
static void launch_norm_fmt(bsq_format fmt, const NormArgs<T>& p, cudaStream_t st) {
    if (fmt == BSQ_NVFP4) launch_norm<T, BSQ_NVFP4>(p, st);
    else if (fmt == BSQ_MXFP4) launch_norm<T, BSQ_MXFP4>(p, st);
    else launch_norm<T, BSQ_MXFP8>(p, st);
}

// CTAs of the backward kernel at most: each leaves one partial row per weight.
static int norm_bwd_ctas(int64_t rows, int64_t C) {
    const int per_sm = C <= 512 ? 16 : (C <= 1024 ? 8 : (C <= 2048 ? 4 : 3));
    return (int)std::min<int64_t>(rows, (int64_t)sm_count() * per_sm);
}

// Returns the number of partial rows.
template <typename T, int NCH, int MAXT, bool REGS, int HAVE, bool KEEP = true>
static int launch_norm_bwd_as(const NormBwdArgs<T>& p, int max_ctas, cudaStream_t st) {
    constexpr auto kern = norm_bwd_kernel<T, NCH, MAXT, REGS, HAVE, KEEP>;
    const int threads = row_threads(p.C / 8, NCH);
    const int want = REGS ? 0 : p.C * 4 * (p.post_weight ? 2 : 1);
    const int smem = want <= kMaxRowSmem && resident_rows<kern>(threads, want) > 0 ? want : 0;
    const int n = (int)std::min<int64_t>(max_ctas, (int64_t)sm_count() * std::max(1, resident_rows<kern>(threads, smem)));
    kern<<<n, threads, smem, st>>>(p, smem > 0);
    return n;
}

template <typename T, int HAVE>
static int launch_norm_bwd_have(int have, const NormBwdArgs<T>& p, int max_ctas, cudaStream_t st) {
    if constexpr (HAVE < 8) {
        if (have != HAVE) return launch_norm_bwd_have<T, HAVE + 1>(have, p, max_ctas, st);
        // One chunk per thread keeps more warps on an SM; with the second norm
        // its second reduction and more sums favour two chunks and half the
        // warps (4096 x 7168 bf16 with post-norm and gate 103 against 119 us;
        // without, 8192 x 4096 with a gate 88 against 115 us, 2048 x 7168 fp32
        // 44 against 57 us).
        constexpr bool kTwo = (HAVE & kPost) != 0;
        return launch_norm_bwd_as<T, kTwo ? 2 : 1, kTwo ? 512 : 1024, true, HAVE>(p, max_ctas, st);
    }
    return 0;
}

template <typename T>
static int launch_norm_bwd(const NormBwdArgs<T>& p, int max_ctas, cudaStream_t st) {
    const int64_t n = p.C / 8;
    const int have = (p.post_weight ? kPost : 0) | (p.gate ? kGate : 0) | (p.gh ? kStream : 0);
    if (n <= 32) return launch_norm_bwd_as<T, 1, 32, true, kAny>(p, max_ctas, st);
    if (n <= 1024) return launch_norm_bwd_have<T, 0>(have, p, max_ctas, st);
    if (n <= 2048) return launch_norm_bwd_as<T, 2, 1024, false, kAny, sizeof(T) == 2>(p, max_ctas, st);
    if (n <= 2560) return launch_norm_bwd_as<T, 4, 640, false, kAny, false>(p, max_ctas, st);
    return launch_norm_bwd_as<T, 4, 1024, false, kAny, false>(p, max_ctas, st);
}

}  // namespace bsq

using namespace bsq;

static bsq_status check_row_size(const char* fn, int64_t C) {
    if (C > kMaxRowElems) return fail(BSQ_ERR_UNSUPPORTED, "%s: rows of more than %lld elements", fn, (long long)kMaxRowElems);
    return BSQ_OK;
}

template <typename T>
static bsq_status run_norm(bsq_format fmt, const void* x, const void* residual, const void* gate, int64_t rows, int64_t C,
                           float scale, const float* post_weight, const float* weight, float eps, void* h, uint8_t* codes,
                           uint8_t* scales, float* row_scale, float* rstd, float* post_rstd, cudaStream_t st,
                           const char* fn) {
    NormArgs<T> p;
    p.x = (const T*)x;
    p.residual = (const T*)residual;
    p.gate = (const T*)gate;
    p.rows = rows;
    p.C = (int)C;
    p.scale = scale;
    p.eps = eps;
    p.post_weight = post_weight;
    p.weight = weight;
    p.h = (T*)h;
    p.codes = codes;
    p.scales = scales;
    p.row_scale = row_scale;
    p.rstd = rstd;
    p.post_rstd = post_rstd;
    launch_norm_fmt<T>(fmt, p, st);
    return check_launch(fn);
}

BSQ_API bsq_status bsq_norm_quantize(bsq_format fmt, const void* x, const void* residual, const void* gate, bsq_dtype t,
                                     int64_t rows, int64_t C, float residual_scale, const float* post_weight,
                                     const float* weight, float eps, void* h, uint8_t* codes, uint8_t* scales,
                                     float* row_scale, float* rstd, float* post_rstd, bsq_stream_t stream) {
    const char* fn = "bsq_norm_quantize";
    BSQ_TRY(check_dtype(t));
    BSQ_TRY(check_quant_format(fn, fmt));
    BSQ_TRY(check_matrix(fn, x, rows, C, fmt_block(fmt)));
    BSQ_TRY(check_row_size(fn, C));
    if (rows * C == 0) return BSQ_OK;
    if (!weight || !codes || !scales || !rstd || (fmt == BSQ_NVFP4 && !row_scale) || (post_weight && !post_rstd))
        return fail(BSQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gate, 16) || !aligned(weight, 16) ||
        !aligned(post_weight, 16) || !aligned(h, 16) || !aligned(codes, 8) || !aligned(rstd, 4) ||
        !aligned(post_rstd, 4) || !aligned(row_scale, 4))
        return fail(BSQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    // a row's inputs are read before its h is written, by the same threads
    const size_t bytes = (size_t)(rows * C) * (t == BSQ_BF16 ? 2 : 4);
    if (overlap(h, bytes, gate, bytes) || (h != x && overlap(h, bytes, x, bytes)) ||
        (h != residual && overlap(h, bytes, residual, bytes)))
        return fail(BSQ_ERR_INVALID_ARG, "%s: h overlaps an input (it may be x or residual itself)", fn);
    const size_t n = (size_t)(rows * C), per_row = (size_t)rows * 4, per_col = (size_t)C * 4;
    const Span outs[] = {{codes, fmt == BSQ_MXFP8 ? n : n / 2}, {scales, n / fmt_block(fmt)},
                         {fmt == BSQ_NVFP4 ? row_scale : nullptr, per_row}, {rstd, per_row},
                         {post_weight ? post_rstd : nullptr, per_row}};
    const Span read[] = {{x, bytes}, {residual, bytes}, {gate, bytes}, {weight, per_col}, {post_weight, per_col}, {h, bytes}};
    if (any_overlap(outs, read) || overlap(h, bytes, weight, per_col) || overlap(h, bytes, post_weight, per_col))
        return fail(BSQ_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
    cudaStream_t st = (cudaStream_t)stream;
    return t == BSQ_BF16 ? run_norm<uint16_t>(fmt, x, residual, gate, rows, C, residual_scale, post_weight, weight, eps, h,
                                              codes, scales, row_scale, rstd, post_rstd, st, fn)
                         : run_norm<float>(fmt, x, residual, gate, rows, C, residual_scale, post_weight, weight, eps, h,
                                           codes, scales, row_scale, rstd, post_rstd, st, fn);
}

BSQ_API size_t bsq_norm_backward_scratch_bytes(int64_t rows, int64_t C, int post) {
    if (rows <= 0 || C <= 0) return 16;
    return (size_t)norm_bwd_ctas(rows, C) * (size_t)C * sizeof(float) * (post ? 2 : 1);
}

template <typename T>
static bsq_status run_norm_bwd(const void* gy, const void* gh, const void* h, const float* rstd, const float* weight,
                               const void* x, const void* gate, const float* post_weight, const float* post_rstd,
                               float scale, int64_t rows, int64_t C, void* grad_residual, void* grad_x, void* grad_gate,
                               float* grad_weight, float* grad_post_weight, float* scratch, cudaStream_t st,
                               const char* fn) {
    const int max_ctas = norm_bwd_ctas(rows, C);
    NormBwdArgs<T> p;
    p.gy = (const T*)gy;
    p.gh = (const T*)gh;
    p.h = (const T*)h;
    p.rstd = rstd;
    p.weight = weight;
    p.x = (const T*)x;
    p.gate = (const T*)gate;
    p.post_weight = post_weight;
    p.post_rstd = post_rstd;
    p.scale = scale;
    p.rows = rows;
    p.C = (int)C;
    p.grad_residual = (T*)grad_residual;
    p.grad_x = (T*)grad_x;
    p.grad_gate = (T*)grad_gate;
    p.partial = scratch;
    p.partial_post = scratch + (size_t)max_ctas * C;
    const int ctas = launch_norm_bwd<T>(p, max_ctas, st);
    BSQ_TRY(check_launch(fn));
    // a programmatic launch: it may start when the last CTA above has ended, and
    // waits itself until what that wrote is visible
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((C + 31) / 32), post_weight ? 2 : 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_weight_sum_kernel, (const float*)p.partial, grad_weight,
                                             (const float*)p.partial_post, grad_post_weight, ctas, (int)C);
    if (e != cudaSuccess) return fail(BSQ_ERR_CUDA, "%s: launch failed (%s)", fn, cudaGetErrorString(e));
    return check_launch(fn);
}

BSQ_API bsq_status bsq_norm_quantize_backward(const void* grad_y, const void* grad_h, const void* h, const float* rstd,
                                              const float* weight, const void* x, const void* gate,
                                              const float* post_weight, const float* post_rstd, float residual_scale,
                                              bsq_dtype t, int64_t rows, int64_t C, void* grad_residual, void* grad_x,
                                              void* grad_gate, float* grad_weight, float* grad_post_weight,
                                              void* scratch, size_t scratch_bytes, bsq_stream_t stream) {
    const char* fn = "bsq_norm_quantize_backward";
    BSQ_TRY(check_dtype(t));
    BSQ_TRY(check_matrix(fn, grad_y, rows, C, 8));
    BSQ_TRY(check_row_size(fn, C));
    if (C > 0 && (!grad_weight || (post_weight && !grad_post_weight)))
        return fail(BSQ_ERR_INVALID_ARG, "%s: null weight gradient", fn);
    cudaStream_t st = (cudaStream_t)stream;
    if (rows * C == 0) {
        if (C > 0) {
            cudaMemsetAsync(grad_weight, 0, (size_t)C * 4, st);
            if (post_weight) cudaMemsetAsync(grad_post_weight, 0, (size_t)C * 4, st);
        }
        return check_launch(fn);
    }
    const bool needs_x = post_weight || gate;
    if (!h || !rstd || !weight || !scratch || (post_weight && !post_rstd) || (needs_x && (!x || !grad_x)) ||
        (gate && !grad_gate) || (!grad_residual && !grad_x))
        return fail(BSQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    const void* al[] = {grad_y, grad_h, h, weight, x, gate, post_weight, grad_residual, grad_x, grad_gate, scratch};
    for (const void* q : al)
        if (!aligned(q, 16)) return fail(BSQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (!aligned(rstd, 4) || !aligned(post_rstd, 4) || !aligned(grad_weight, 4) || !aligned(grad_post_weight, 4))
        return fail(BSQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const size_t bytes = (size_t)(rows * C) * (t == BSQ_BF16 ? 2 : 4);
    const void* in[] = {grad_y, grad_h, h, needs_x ? x : nullptr, gate};
    const void* outs[] = {grad_residual, grad_x, grad_gate};
    for (const void* o : outs)
        for (const void* i : in)
            if (overlap(o, bytes, i, bytes)) return fail(BSQ_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    if (overlap(grad_residual, bytes, grad_x, bytes) || overlap(grad_residual, bytes, grad_gate, bytes) ||
        overlap(grad_x, bytes, grad_gate, bytes))
        return fail(BSQ_ERR_INVALID_ARG, "%s: two outputs overlap", fn);
    const size_t need = bsq_norm_backward_scratch_bytes(rows, C, post_weight != nullptr);
    if (scratch_bytes < need)
        return fail(BSQ_ERR_INVALID_ARG, "%s: scratch of %zu bytes, need %zu", fn, scratch_bytes, need);
    const size_t per_row = (size_t)rows * 4, per_col = (size_t)C * 4;
    const Span written[] = {{grad_residual, bytes}, {grad_x, bytes}, {grad_gate, bytes}, {grad_weight, per_col},
                            {post_weight ? grad_post_weight : nullptr, per_col}, {scratch, need}};
    const Span read[] = {{grad_y, bytes}, {grad_h, bytes}, {h, bytes}, {needs_x ? x : nullptr, bytes}, {gate, bytes},
                         {weight, per_col}, {post_weight, per_col}, {rstd, per_row}, {post_weight ? post_rstd : nullptr, per_row}};
    if (any_overlap(written, read))
        return fail(BSQ_ERR_INVALID_ARG, "%s: an output or the scratch overlaps an input or another output", fn);
    const void* xin = needs_x ? x : nullptr;
    return t == BSQ_BF16
               ? run_norm_bwd<uint16_t>(grad_y, grad_h, h, rstd, weight, xin, gate, post_weight, post_rstd, residual_scale,
                                        rows, C, grad_residual, grad_x, grad_gate, grad_weight, grad_post_weight,
                                        (float*)scratch, st, fn)
               : run_norm_bwd<float>(grad_y, grad_h, h, rstd, weight, xin, gate, post_weight, post_rstd, residual_scale,
                                     rows, C, grad_residual, grad_x, grad_gate, grad_weight, grad_post_weight,
                                     (float*)scratch, st, fn);
}

#ifdef BSQ_DEBUG
cudaError_t bsq_dbg_take_norm(uint32_t* count, uint32_t* first) { return bsq::dbg_take(count, first); }
#endif
