// scaled_mm.cu -- grouped product of two block-scaled operands on the sm_100a
// block-scaled tensor cores.
//
//   out[t, n] = ga[t] * gw[e, n] * sum_k (a[t, k] * sa[t, k / B]) * (w[e, n, k] * sw[e, n, k / B])
//
// for the tokens t of expert e (rows [offs[e-1], offs[e]) of a), with a and w
// in NVFP4 (B = 16, row scales ga and gw), MXFP4 or MXFP8 (B = 32, no row
// scales), or a in MXFP8 and w in MXFP4.  The tensor core applies the block
// scales itself (tcgen05 kind::mxf4nvf4, mxf4 and mxf8f6f4 with .block_scale)
// and accumulates in binary32; the row scales are applied to the accumulator,
// and the result is rounded once to bf16.
//
// The MMA computes the transposed product D[feature, token]: weights are the
// M operand (128 rows per CTA), an expert's tokens the N operand, rounded up
// to 16, so one decoded token costs an N = 16 MMA and no padding to 128 rows.
//
// Codes are K-major in both operands and go to shared memory by TMA with the
// 128-byte swizzle: a k-step is 128 bytes of a row (256 e2m1 or 128 e4m3
// codes), four MMAs.  e2m1 weights against e4m3 activations are widened to
// one code per byte container by the TMA load.  Scales are stored row-major
// by the quantizers and come by TMA too, in a ring of their own: 16 bytes of
// each row (two k-steps of MXFP4, four of MXFP8) or 32 (two of NVFP4, a whole
// sector).  Four warps lay them out in the stages as the tensor core reads
// them: blocks of 128 rows x 4 bytes, the bytes of row r at (r % 32) * 16 +
// (r / 32) * 4.  Scale rows that TMA cannot read, of other than a multiple of
// 16 bytes, are loaded by the four warps themselves, which costs the memory
// pipe a request per row (4096 x 4096 x 2080 against 2048: NVFP4 63 us
// against 27, MXFP8 48 against 35).  The MMA warp copies the blocks to a ring
// of tensor-memory slots and issues the k-step's MMAs.
//
// Persistent, warp-specialised CTA of 480 threads (one per SM):
//   warps 0-7  epilogue: tensor memory -> registers -> row scales -> bf16 ->
//              transposed by stmatrix into shared memory -> TMA stores of 32
//              tokens x 32 features (rows that an expert's end cuts: plain
//              stores).  Against transposing by shuffles, 16384 x 2048 x 7168
//              over 32 experts took 142 us instead of 159, and K = 256, where
//              the output is most of the work, 44 us instead of 90.
//   warps 8-11 scale producers, a warp per 128 rows of scales
//   warp 12    TMA loads of both operands
//   warp 13    tensor-memory allocation, scale copies and MMAs
//   warp 14    proxy fence between the scale producers' stores and the tensor
//              core's reads, which so never waits for their loads in flight
// The MMA warp stays converged and one elected lane issues: the instructions
// take their operands from uniform registers, and a lone thread's loop spent
// 0.9 us per k-step moving operands there (T = 1, N = 2048, K = 7168: 28.6 us
// against 16.5).
//
// Two tile shapes:
//   - pairs (cta_group::2): 256 features x up to 256 tokens, each CTA holding
//     its 128 weight rows and half of the tokens' codes.  What a k-step loads
//     from L2 per MMA bounds it, so the tile is the largest that tensor memory
//     holds beside the scales.  The accumulators of consecutive tiles lie at columns 0 and 160
//     and overlap in 96 columns: the epilogue drains those first, and the
//     next tile's MMAs run under the rest of the drain.
//   - single CTAs: 128 features x up to 32 tokens, up to eight k-steps in
//     flight: bound by the weight bytes.  Where the tiles leave SMs idle, a cluster
//     of up to 8 CTAs splits a tile's contraction and adds the partial sums
//     over distributed shared memory, in rank order.
//
// Every mbarrier wait is bounded (about a second): the thread records
// BSQ_DEVERR_TIMEOUT in the error word and raises a CTA-wide abort flag, and all
// roles leave their loops.  The MMA warp waits for its MMAs; when the roles of
// all CTAs of a pair have stopped, the loads in flight are waited for too, by
// what each role had done (pipeline_drain.h; one limit for all of them), and
// tensor memory is freed before the CTA exits.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <mutex>

#define BSQ_DBG_FILE 7
#include "debug.cuh"
#include "common.cuh"
#include "host_util.h"
#include "overlap.h"
#include "pipeline_drain.h"
#include "scaled_tc.cuh"
#include "tma_encode.h"

namespace bsq {
using namespace sm100;

namespace smm {

constexpr int WM = 128;   // features per CTA (the CTA's share of MMA M)
constexpr int BKB = 128;  // bytes of a row per k-step
constexpr int kEpiWarps = 8, kScaleWarps = 4;
constexpr int kTmaWarp = kEpiWarps + kScaleWarps;  // 12
constexpr int kMmaWarp = kTmaWarp + 1;             // 13
constexpr int kFenceWarp = kMmaWarp + 1;           // 14
constexpr int kThreads = (kFenceWarp + 1) * 32;    // 480
constexpr uint32_t kWBytes = WM * BKB;             // 16 KiB
constexpr int kMaxExperts = 1024;
constexpr int kMaxSplit = 8;
constexpr uint32_t kOutPiece = 2048;               // 32 tokens x 32 features, bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 1000000000ull;

// 4-byte scale words per row and k-step.
__host__ __device__ constexpr int scale_words(int kind) { return kind == MMA_NVFP4 ? 4 : (kind == MMA_MXFP4 ? 2 : 1); }

// Scale bytes of a row that one TMA box holds: one (NVFP4), two or four
// k-steps need 16 bytes; NVFP4 takes two k-steps at a time, a whole sector.
__host__ __device__ constexpr int raw_row_bytes(int kind) { return kind == MMA_NVFP4 ? 32 : 16; }

// Plan of a CTA group: CG = 2, a pair with tiles of up to TN = 256 tokens, or
// CG = 1, a single CTA with up to TN = 32.  RAW: scale rows come by TMA, a
// chunk of kRawBytes of each row at a time into a ring of two slots of their
// own, and are laid out in the stages from there.
template <int KIND, int CG, bool RAW>
struct Plan {
    static constexpr int NBLK = scale_words(KIND);
    static constexpr int TN = (CG == 2) ? 256 : 32;
    static constexpr int XBLK = (TN + 127) / 128;  // 128-row blocks of token scales
    static constexpr int kXRows = TN / CG;  // token rows of a CTA: one TMA box
    static constexpr uint32_t kX = kXRows * BKB;
    static constexpr uint32_t kSW = NBLK * 512, kSX = NBLK * XBLK * 512;
    static constexpr uint32_t kXOff = kWBytes, kSWOff = kXOff + kX, kSXOff = kSWOff + kSW;
    static constexpr uint32_t kStage = (kSXOff + kSX + 1023) / 1024 * 1024;
    static constexpr int kRawRow = raw_row_bytes(KIND), kRawSteps = kRawRow / (4 * NBLK);
    static constexpr uint32_t kRawSlot = RAW ? (WM + TN) * kRawRow : 0;
    static constexpr int kOutBufs = (CG == 2) ? 2 : 1;  // 2 KiB output pieces of an epilogue warp
    static constexpr uint32_t kOut = kEpiWarps * kOutBufs * kOutPiece;
    static constexpr int kRowFloats = (KIND == MMA_NVFP4) ? TN / 2 < 32 ? 32 : TN / 2 : 0;  // token row scales of an epilogue warp
    static constexpr uint32_t kMisc = 1024 /* barriers, flags */ + 4 * (2 * kMaxExperts + 2) + kEpiWarps * kRowFloats * 4;
    static constexpr int kFit = (232448 - 1024 /* alignment slack */ - 2 * kRawSlot - kOut - kMisc) / kStage;
    static constexpr int STAGES = kFit < 8 ? kFit : 8;
    static constexpr size_t kRawOff = (size_t)STAGES * kStage, kOutOff = kRawOff + 2 * kRawSlot, kBarOff = kOutOff + kOut;
    static constexpr int kNumBars = 3 * STAGES + 4 + 3;
    static constexpr size_t kSmemBytes = 1024 + kBarOff + kMisc;
    // Tensor memory.  Pairs: accumulators at 0 and 160 (256 columns each, 96
    // shared), two scale slots from 416.  Single CTAs: accumulators at 0 and
    // 32, a scale slot per stage from 64.  A slot: 16 columns of weight
    // scales, then the token scales.
    static constexpr int kAccStep = (CG == 2) ? 160 : 32;
    static constexpr int kAccShared = (CG == 2) ? TN - kAccStep : 0;
    static constexpr int kScaleCols = (CG == 2) ? 416 : 64;
    static constexpr int kSlots = (CG == 2) ? 2 : STAGES;
    static constexpr int kSlotCols = 16 + 16 * XBLK;
    static_assert(kScaleCols + kSlots * kSlotCols <= (int)kTmemCols && kAccStep + TN <= kScaleCols, "tensor memory plan");
    static_assert(kNumBars * 8 + 64 <= 1024 && kOutOff % 1024 == 0 && STAGES >= 3, "shared memory plan");
};

struct Args {
    const uint8_t *a_scales, *a_scales_end;
    const float* a_row;
    const uint8_t *w_scales, *w_scales_end;
    const float* w_row;
    const int32_t* offs;  // NULL: one expert owns every row
    uint16_t* out;
    uint32_t* err;
    uint64_t wait_ns;
    int E, T, N;
    int k_steps;
    int row_scales;  // scale bytes per row
    int split;       // CTAs of a cluster that share a tile's contraction (single CTAs)
    uint32_t w_tx;   // bytes that a weight tile counts on its barrier
    uint32_t idesc;  // instruction descriptor without N and M
};

struct Tile {
    int e, tok0, ntok, f0;
};

struct Shared {
    uint8_t* stage;
    uint8_t* raw_rows;   // [2] slots of scale rows: weights, then tokens
    uint8_t* out;        // output pieces of the epilogue warps
    uint64_t* full;
    uint64_t* empty;
    uint64_t* raw;       // a slot's scale rows are loaded
    uint64_t* raw_free;  // a slot's scale rows are read
    uint64_t* scales;    // a stage's scales are laid out, not yet fenced
    uint64_t* acc_full;  // a tile's accumulator is complete
    uint64_t* acc_free;  // what the next tile's accumulator needs of it is drained
    uint64_t* drain;
    uint32_t* tmem_slot;
    volatile int* abort;
    // what each CTA of a pair (a single CTA: [0]) had done when its roles had stopped
    int* issued;      // [2] k-steps whose codes it has loaded
    int* fenced;      // [2] k-steps whose scales it has handed over
    int* gave_up;     // [2]
    int* raw_issued;  // chunks of scale rows that this CTA has loaded
    int* tt_prefix;  // [E + 1] first token tile of each expert
    int* seg;        // [E + 1] seg[e] = first row of expert e, seg[E] = offs[E-1]
    float* row;      // [kEpiWarps][kRowFloats] row scales of the tokens that each epilogue warp drains
};

template <int KIND, int CG, bool RAW>
__device__ __forceinline__ Shared carve(uint8_t* raw) {
    using P = Plan<KIND, CG, RAW>;
    Shared s;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.stage = base;
    s.raw_rows = base + P::kRawOff;
    s.out = base + P::kOutOff;
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + P::kBarOff);
    s.full = bars;
    s.empty = bars + P::STAGES;
    s.scales = bars + 2 * P::STAGES;
    s.raw = bars + 3 * P::STAGES;
    s.raw_free = s.raw + 2;
    s.acc_full = s.raw + 4;
    s.acc_free = s.acc_full + 1;
    s.drain = s.acc_full + 2;
    s.tmem_slot = reinterpret_cast<uint32_t*>(bars + P::kNumBars);
    s.abort = reinterpret_cast<volatile int*>(s.tmem_slot + 1);
    s.issued = reinterpret_cast<int*>(s.tmem_slot + 4);
    s.fenced = s.issued + 2;
    s.gave_up = s.issued + 4;
    s.raw_issued = s.issued + 6;
    s.row = reinterpret_cast<float*>(base + P::kBarOff + 1024);
    s.tt_prefix = reinterpret_cast<int*>(s.row + kEpiWarps * P::kRowFloats);
    s.seg = s.tt_prefix + kMaxExperts + 1;
    return s;
}

// Bounded wait that also gives up as soon as another role has aborted.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const Shared& sh, const Args& a) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*sh.abort) return false;
        if (globaltimer_ns() - t0 > a.wait_ns) {
            *sh.abort = 1;
            atomicOr(a.err, (uint32_t)BSQ_DEVERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The same for a whole warp, with one outcome for its 32 lanes.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, const Shared& sh, const Args& a) {
    const bool ok = wait_bar(bar, parity, sh, a);
    return __all_sync(0xffffffffu, ok);
}

template <int CG, int TN>
__device__ __forceinline__ Tile decode_tile(int t, int f_tiles, int E, const Shared& sh) {
    const int tg = t / f_tiles;
    const int ft = t - tg * f_tiles;
    int lo = 0, hi = E - 1;  // last expert whose first token tile is <= tg
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sh.tt_prefix[mid] <= tg) lo = mid;
        else hi = mid - 1;
    }
    Tile ti;
    ti.e = lo;
    ti.tok0 = sh.seg[lo] + (tg - sh.tt_prefix[lo]) * TN;
    ti.ntok = min(TN, sh.seg[lo + 1] - ti.tok0);
    ti.f0 = ft * WM * CG;
    return ti;
}

// Tile table from offs, by one warp: seg, tt_prefix and the status words
// (abort, bad offs, token tiles).
template <int TN>
__device__ __forceinline__ void build_table(const Shared& sh, const Args& a, int lane) {
    int total = 0, prev = 0;
    bool bad = false;
    for (int base = 0; base < a.E; base += 32) {
        const int e = base + lane;
        int o = prev;
        if (a.offs == nullptr) o = a.T;  // dense: E == 1
        else if (e < a.E) o = a.offs[e];
        int before = __shfl_up_sync(0xffffffffu, o, 1);
        if (lane == 0) before = prev;
        const bool mine = e < a.E && (o < before || o > a.T);
        bad = bad || __any_sync(0xffffffffu, mine);
        const int tiles = (e < a.E && !bad) ? (o - before + TN - 1) / TN : 0;
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        if (e < a.E) {
            sh.seg[e] = before;
            sh.tt_prefix[e] = total + incl - tiles;
        }
        total += __shfl_sync(0xffffffffu, incl, 31);
        prev = __shfl_sync(0xffffffffu, o, min(31, a.E - 1 - base));
    }
    if (lane == 0) {
        sh.seg[a.E] = bad ? 0 : prev;
        sh.tt_prefix[a.E] = total;
        sh.tmem_slot[1] = 0;  // abort flag
        sh.tmem_slot[2] = bad;
        sh.tmem_slot[3] = bad ? 0 : total;
        if (bad && blockIdx.x == 0) atomicOr(a.err, (uint32_t)BSQ_DEVERR_BAD_OFFS);
    }
}

template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    if (CG == 1) mbar_arrive(bar);
    else mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
}

// ------------------------------------------------------------------ scales --

// Scale bytes of one row for a chunk of k-steps, of rows of any length and
// alignment: the aligned words around the bytes, held as loaded until they are
// stored (a value derived at the load would make the thread wait for it
// there), then cut at the row's end (bytes past it scale codes that are zero,
// but the next row's byte there may be a NaN) and shifted into place.
template <int NBLK>
struct Chunk {
    static constexpr int kSteps = 4 / NBLK;  // 16 bytes
    uint32_t v[5];
    static __device__ __forceinline__ int shift(const uint8_t* row, int off) {
        return (int)(reinterpret_cast<uintptr_t>(row + off) & 3);
    }
    // [lo, hi): the whole tensor; a word that is not all in it is left for ready()
    __device__ __forceinline__ void load(const uint8_t* row, int off, int n, const uint8_t* lo, const uint8_t* hi) {
        const uint8_t* p = row + off - shift(row, off);
#pragma unroll
        for (int i = 0; i < 5; ++i)
            if (p + 4 * i < row + n && p + 4 * i >= lo && p + 4 * i + 4 <= hi)
                v[i] = __ldg(reinterpret_cast<const uint32_t*>(p + 4 * i));
    }
    __device__ __forceinline__ void ready(const uint8_t* row, int off, int n, const uint8_t* lo, const uint8_t* hi) {
        const uint8_t* p = row + off - shift(row, off);
        if (p >= lo && p + 20 <= row + n) return;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const uint8_t* q = p + 4 * i;
            const int left = (int)(row + n - q);  // bytes of the row from this word on
            if (left <= 0) {
                v[i] = 0u;
            } else if (q < lo || q + 4 > hi) {  // the tensor's first or last word: byte by byte
                v[i] = 0u;
                for (int j = 0; j < min(left, 4); ++j)
                    if (q + j >= lo) v[i] |= (uint32_t)__ldg(q + j) << (8 * j);
            } else if (left < 4) {
                v[i] &= (1u << (8 * left)) - 1u;
            }
        }
    }
    __device__ __forceinline__ uint32_t word(int i, const uint8_t* row, int off) const {
        return __funnelshift_r(v[i], v[i + 1], 8 * shift(row, off));
    }
};

__device__ __forceinline__ void sts32(uint32_t saddr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}

// What a CTA works on: tiles t0, t0 + step, ... below num, k-steps [k0, k1) of each.
struct Work {
    int t0, step, num, f_tiles, k0, k1;
};

__device__ __forceinline__ uint32_t lds32(uint32_t saddr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(saddr) : "memory");
    return v;
}

// The scale producers, from the rows that TMA loaded, a chunk of k-steps at a
// time: a warp per block of 128 rows (one of weights, XBLK of tokens), four
// rows per thread, whose words of a block lie side by side, so that stores
// take 16 bytes without bank conflicts (16384 x 2048 x 7168 NVFP4 over 32
// experts 131.5 us; a row per thread and 4-byte stores 135.5).  (Loads by the
// threads themselves, a line of L1 per row and warp instruction, cost a fifth
// of the whole product: 4096 x 4096 x 7168 NVFP4 without an epilogue 61 us,
// with the same loads coalesced 52 us.)
template <int KIND, int CG>
__device__ __forceinline__ void lay_out_scales(const Shared& sh, const Args& args, const Work& wk) {
    using P = Plan<KIND, CG, true>;
    constexpr int NBLK = P::NBLK, XBLK = P::XBLK;
    const int warp = (threadIdx.x >> 5) - kEpiWarps, lane = threadIdx.x & 31;
    const uint32_t st_base = smem_u32(sh.stage), raw_base = smem_u32(sh.raw_rows) + (uint32_t)(warp * 128 + lane) * P::kRawRow;
    int s = 0, rs = 0;
    uint32_t ph = 1, rph = 0;
    for (int t = wk.t0; t < wk.num; t += wk.step) {
        const int ntok = decode_tile<CG, P::TN>(t, wk.f_tiles, args.E, sh).ntok;
        for (int k0 = wk.k0; k0 < wk.k1; k0 += P::kRawSteps) {
            if (!wait_bar_warp(&sh.raw[rs], rph, sh, args)) return;
#pragma unroll
            for (int k = 0; k < P::kRawSteps; ++k) {
                if (k0 + k >= wk.k1) break;
                if (!wait_bar_warp(&sh.empty[s], ph, sh, args)) return;
                const uint32_t st = st_base + s * P::kStage;
                const uint32_t from = raw_base + rs * P::kRawSlot + k * (4 * NBLK);
                // of `rows` rows, to blocks `stride` apart
                auto block = [&](uint32_t to, uint32_t stride, int rows) {
                    uint32_t v[4][4] = {};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t at = from + (uint32_t)(32 * q * P::kRawRow);
                        if (32 * q >= rows) break;
                        if (NBLK == 4) {
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(v[q][0]), "=r"(v[q][1]), "=r"(v[q][2]), "=r"(v[q][3]) : "r"(at) : "memory");
                        } else if (NBLK == 2) {
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[q][0]), "=r"(v[q][1]) : "r"(at) : "memory");
                        } else {
                            v[q][0] = lds32(at);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NBLK; ++i)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + i * stride + lane * 16),
                                     "r"(v[0][i]), "r"(v[1][i]), "r"(v[2][i]), "r"(v[3][i]) : "memory");
                };
                if (warp == 0) block(st + P::kSWOff, 512, WM);
                else if (warp <= XBLK && 128 * (warp - 1) < ntok)
                    block(st + P::kSXOff + (warp - 1) * 512, XBLK * 512, P::TN < 128 ? P::TN : 128);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.scales[s]);
                if (++s == P::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (lane == 0) mbar_arrive(&sh.raw_free[rs]);  // after the last step's __syncwarp
            rs ^= 1;
            rph ^= (uint32_t)(rs == 0);
        }
    }
}

// From rows of any length and alignment, the next chunks in flight in
// registers.  Rows outside the tile read a row inside it: their outputs are
// never stored.
template <int KIND, int CG>
__device__ __forceinline__ void produce_scales(const Shared& sh, const Args& args, const Work& wk, int rank) {
    using P = Plan<KIND, CG, false>;
    constexpr int NBLK = P::NBLK, XBLK = P::XBLK;
    using C = Chunk<NBLK>;
    // Chunks in flight: what the registers hold.  A fourth of NVFP4's spills
    // (T = 4096, N = 4096, K = 2080: 68.4 us against 62.2).
    constexpr int kAhead = C::kSteps >= 2 ? 2 : 3;
    const int r = threadIdx.x - kEpiWarps * 32, lane = threadIdx.x & 31;
    const uint32_t st_base = smem_u32(sh.stage);
    const uint32_t place = (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
    const int n = args.row_scales;
    const bool has_x = r < P::TN;  // the same for a whole warp
    struct Cursor {
        int t, ks;
        const uint8_t *w, *x[XBLK];
        int nx;  // token blocks of the tile
    };
    auto place_at = [&](Cursor& c) {
        const Tile ti = decode_tile<CG, P::TN>(c.t, wk.f_tiles, args.E, sh);
        const int f = min(ti.f0 + WM * rank + r, args.N - 1);
        c.ks = wk.k0;
        c.w = args.w_scales + ((int64_t)ti.e * args.N + f) * n;
#pragma unroll
        for (int x = 0; x < XBLK; ++x)
            c.x[x] = args.a_scales + (int64_t)(ti.tok0 + min(128 * x + r, ti.ntok - 1)) * n;
        c.nx = has_x ? (ti.ntok + 127) / 128 : 0;
    };
    auto advance = [&](Cursor& c) {
        c.ks += C::kSteps;
        if (c.ks >= wk.k1) {
            c.t += wk.step;
            if (c.t < wk.num) place_at(c);
        }
    };
    struct Item {
        C w, x[XBLK];
    };
    auto load = [&](Item& b, Cursor& c) {
        if (c.t >= wk.num) return;
        const int off = c.ks * (4 * NBLK);
        if (BSQ_DOK(off < n)) {
            b.w.load(c.w, off, n, args.w_scales, args.w_scales_end);
#pragma unroll
            for (int x = 0; x < XBLK; ++x)
                if (x < c.nx) b.x[x].load(c.x[x], off, n, args.a_scales, args.a_scales_end);
        }
        advance(c);
    };
    if (wk.t0 >= wk.num || wk.k0 >= wk.k1) return;
    Cursor ld;
    ld.t = wk.t0;
    place_at(ld);
    Cursor st = ld;
    Item buf[kAhead];
#pragma unroll
    for (int b = 0; b < kAhead; ++b) load(buf[b], ld);
    int s = 0;
    uint32_t ph = 1;  // parity of the stage's "empty" wait
    while (true) {
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
            if (st.t >= wk.num) return;
            const int off = st.ks * (4 * NBLK);
            buf[b].w.ready(st.w, off, n, args.w_scales, args.w_scales_end);
#pragma unroll
            for (int x = 0; x < XBLK; ++x)
                if (x < st.nx) buf[b].x[x].ready(st.x[x], off, n, args.a_scales, args.a_scales_end);
#pragma unroll
            for (int k = 0; k < C::kSteps; ++k) {
                if (st.ks + k >= wk.k1) break;
                if (!wait_bar_warp(&sh.empty[s], ph, sh, args)) return;
                const uint32_t ws = st_base + s * P::kStage + P::kSWOff + place;
                const uint32_t xs = st_base + s * P::kStage + P::kSXOff + place;
#pragma unroll
                for (int i = 0; i < NBLK; ++i) {
                    sts32(ws + i * 512, buf[b].w.word(k * NBLK + i, st.w, off));
#pragma unroll
                    for (int x = 0; x < XBLK; ++x)
                        if (x < st.nx) sts32(xs + (i * XBLK + x) * 512, buf[b].x[x].word(k * NBLK + i, st.x[x], off));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.scales[s]);
                if (++s == P::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
            advance(st);
            load(buf[b], ld);
        }
    }
}

// ---------------------------------------------------------------- epilogue --

// Tokens [c0, c1) of a tile (c0 a multiple of 32) from accumulator columns
// acc + c0 ... to the output, for the warp's 32 features; two warps per
// quadrant take the groups of 32 tokens in turn (half: 0 or 1).  A group is
// read as 16-lane matrix fragments (a thread holds features t / 4 + 8i of
// tokens 2 (t % 4) and the next), rounded, transposed into shared memory by
// stmatrix, 64 bytes per token with the 64-byte swizzle, and stored by TMA;
// a group that the expert's end cuts is stored by the threads.
// gw[i]: row scale of feature t / 4 + 8i; row: of the warp's tokens.
template <int KIND, int CG, bool RAW>
__device__ __forceinline__ void drain_tokens(const CUtensorMap* tmap_out, const Args& args, const Tile& ti, uint32_t acc,
                                             int c0, int c1, int half, int f0, const float (&gw)[4], const float* row,
                                             uint32_t out, int& piece, int lane) {
    using P = Plan<KIND, CG, RAW>;
#pragma unroll 1
    for (int c = c0 + 32 * (((c0 >> 5) & 1) ^ half); c < c1; c += 64) {
        uint32_t r[2][16];
        tmem_ld_16x256b_x4(acc + (uint32_t)c, r[0]);
        tmem_ld_16x256b_x4(acc + (16u << 16) + (uint32_t)c, r[1]);
        // the buffer's previous store has read it
        if (lane == 0) bulk_wait_read<P::kOutBufs - 1>();
        __syncwarp();
        const uint32_t buf = out + (uint32_t)piece * kOutPiece;
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 tokens
            float2 s = make_float2(1.0f, 1.0f);
            if (KIND == MMA_NVFP4) s = *reinterpret_cast<const float2*>(row + (c >> 6) * 32 + 8 * i + 2 * (lane & 3));
            uint32_t m[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 8 features
                float2 v = make_float2(__uint_as_float(r[j / 2][4 * i + 2 * (j & 1)]),
                                       __uint_as_float(r[j / 2][4 * i + 2 * (j & 1) + 1]));
                if (KIND == MMA_NVFP4) v = mul_f32x2(mul_f32x2(v, s), make_float2(gw[j], gw[j]));
                m[j] = pack_bf16x2(v.x, v.y);
            }
            const int t = 8 * i + (lane & 7);
            stmatrix_x4_trans(buf + t * 64 + (((lane >> 3) ^ ((t >> 1) & 3)) << 4), m);
        }
        if (f0 < args.N) {
            if (c + 32 <= ti.ntok) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && BSQ_DOK(ti.tok0 + c + 32 <= args.T)) tma_store_2d(tmap_out, buf, f0, ti.tok0 + c);
            } else {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 8 * i + (lane >> 2), f = f0 + 8 * (lane & 3);
                    if (c + t < ti.ntok && f < args.N && BSQ_DOK(ti.tok0 + c + t < args.T && f + 8 <= args.N))
                        *reinterpret_cast<uint4*>(args.out + (int64_t)(ti.tok0 + c + t) * args.N + f) =
                            lds128(buf + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
                }
                __syncwarp();
            }
        }
        if (lane == 0) bulk_commit();
        if (++piece == P::kOutBufs) piece = 0;
    }
}

// Waits, by one thread of each CTA and for a second at most, for the loads that
// are in flight when the roles of all CTAs have stopped: the codes of both CTAs
// of a pair, which count on the leader's barriers, and the CTA's own scale rows.
template <int KIND, int CG, bool RAW>
__device__ __forceinline__ void drain_loads(const Shared& sh, uint32_t bytes, int rank) {
    constexpr int S = Plan<KIND, CG, RAW>::STAGES;
    const uint64_t t0 = globaltimer_ns();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const uint64_t spent = globaltimer_ns() - t0;
        mbar_wait(bar, parity, spent < kWaitNs ? kWaitNs - spent : 0);
    };
    if (rank == 0) {
        const int first = drain_first(sh.issued, CG, S), last = drain_last(sh.issued, CG);
        for (int j = first; j < last; ++j) {
            const PhaseDebt d = phase_debt(j, sh.issued, CG, bytes, sh.fenced, CG);
            uint64_t* bar = &sh.full[j % S];
            if (d.expect) mbar_arrive_expect_tx(bar, d.expect);
            if (d.complete) mbar_complete_tx(bar, d.complete);
            if (d.arrivals) mbar_arrive_n(bar, d.arrivals);
        }
        for (int j = first; j < last; ++j) wait(&sh.full[j % S], (uint32_t)(j / S) & 1);
    }
    if (RAW)  // the thread that loads scale rows names their bytes: nothing else is owed
        for (int j = max(0, *sh.raw_issued - 2); j < *sh.raw_issued; ++j) wait(&sh.raw[j & 1], (uint32_t)(j >> 1) & 1);
}

__device__ __forceinline__ float lds_cluster_f32(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// ------------------------------------------------------------------ kernel --

template <int KIND, int CG, bool RAW>
__global__ void __launch_bounds__(kThreads, 1)
    scaled_mm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                     const __grid_constant__ CUtensorMap tmap_sx, const __grid_constant__ CUtensorMap tmap_sw,
                     const __grid_constant__ CUtensorMap tmap_out, Args args) {
    using P = Plan<KIND, CG, RAW>;
    constexpr int NBLK = P::NBLK, TN = P::TN;
    extern __shared__ uint8_t smem_raw[];
    const Shared sh = carve<KIND, CG, RAW>(smem_raw);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;  // uniform to the compiler
    const int E = args.E;
    const int f_tiles = (args.N + WM * CG - 1) / (WM * CG);
    const int split = (CG == 1) ? args.split : 1;
    const uint32_t crank = (CG == 2 || split > 1) ? cluster_ctarank() : 0u;
    const int rank = (CG == 2) ? (int)crank : 0;      // half of a pair's tile
    const int krank = (CG == 2) ? 0 : (int)crank;     // share of the contraction
    const bool leader = rank == 0;
    Work wk;
    wk.t0 = blockIdx.x / (CG * split);
    wk.step = gridDim.x / (CG * split);
    wk.f_tiles = f_tiles;
    {
        // shares of the contraction, in units of a chunk of scales
        constexpr int G = P::kRawSteps;
        const int units = (args.k_steps + G - 1) / G;
        wk.k0 = (int)((int64_t)units * krank / split) * G;
        wk.k1 = min(args.k_steps, (int)((int64_t)units * (krank + 1) / split) * G);
    }

    if (warp == 0) {
        if (lane == 0) {
            for (int s = 0; s < P::STAGES; ++s) {
                // the fence thread of each CTA, plus the leader's TMA thread
                // (its arrive carries the expected bytes)
                mbar_init(&sh.full[s], CG + 1);
                mbar_init(&sh.empty[s], 1);
                mbar_init(&sh.scales[s], kScaleWarps);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.raw[i], 1);
                mbar_init(&sh.raw_free[i], kScaleWarps);
            }
            mbar_init(sh.acc_full, 1);
            mbar_init(sh.acc_free, kEpiWarps * CG);
            mbar_init(sh.drain, 1);
            fence_barrier_init();
        }
        build_table<TN>(sh, args, lane);
    }
    if (warp == kMmaWarp) {
        if (CG == 1) {
            tmem_alloc(sh.tmem_slot, kTmemCols);
            tmem_relinquish();
        } else {
            tmem_alloc_pair(sh.tmem_slot, kTmemCols);
            tmem_relinquish_pair();
        }
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&tmap_x);
        tma_prefetch_desc(&tmap_w);
        if (RAW) {
            tma_prefetch_desc(&tmap_sx);
            tma_prefetch_desc(&tmap_sw);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();  // the peer's barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = sh.tmem_slot[0];
    const int bad = sh.tmem_slot[2];
    wk.num = bad ? 0 : sh.tmem_slot[3] * f_tiles;

    if (warp < kEpiWarps) {
        // ---------------------------------------------------------- epilogue
        if (!bad) {  // rows at or past offs[E-1] are zero
            const int vec_per_row = args.N / 8;
            for (int r = sh.seg[E] + blockIdx.x; r < args.T; r += gridDim.x) {
                uint4* dst = reinterpret_cast<uint4*>(args.out + (int64_t)r * args.N);
                for (int v = threadIdx.x; v < vec_per_row; v += kEpiWarps * 32) dst[v] = make_uint4(0, 0, 0, 0);
            }
        }
        const int q = warp & 3, half = warp >> 2;  // tensor-memory lanes of this warp = features 32q..32q+31
        const uint32_t out = smem_u32(sh.out) + (uint32_t)(warp * P::kOutBufs) * kOutPiece;
        int piece = 0;
        int tile_iter = 0;
        for (int t = wk.t0; t < wk.num; t += wk.step, ++tile_iter) {
            __syncwarp();  // the previous tile's row scales are read
            const Tile ti = decode_tile<CG, TN>(t, f_tiles, E, sh);
            const int f0 = ti.f0 + WM * rank + q * 32;
            float gw[4];
            float* row = sh.row + warp * P::kRowFloats;
            if (KIND == MMA_NVFP4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = f0 + (lane >> 2) + 8 * i;
                    gw[i] = (f < args.N) ? __ldg(args.w_row + (int64_t)ti.e * args.N + f) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < P::kRowFloats / 32; ++i) {
                    const int t = 64 * i + 32 * half + lane;
                    row[32 * i + lane] = (t < ti.ntok) ? __ldg(args.a_row + ti.tok0 + t) : 0.0f;
                }
                __syncwarp();
            }
            if (!wait_bar_warp(sh.acc_full, tile_iter & 1, sh, args)) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((tile_iter & 1) * P::kAccStep);
            auto drain = [&](int c0, int c1) {
                drain_tokens<KIND, CG, RAW>(&tmap_out, args, ti, acc, c0, c1, half, f0, gw, row, out, piece, lane);
            };
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader<CG>(sh.acc_free);
            };
            if (CG == 2) {
                // the columns that the next tile's accumulator covers first:
                // the last 96 of the one at column 0, the first of the other
                const bool high = (tile_iter & 1) == 0;
                const int a = high ? min(P::kAccStep, ti.ntok) : 0, b = high ? ti.ntok : min(P::kAccShared, ti.ntok);
                drain(a, b);
                release();
                drain(high ? 0 : b, high ? a : ti.ntok);
            } else if (split == 1) {
                // consecutive accumulators are apart: the next may start at once
                release();
                drain(0, ti.ntok);
            } else {
                // partial sums to this CTA's shared memory, [token][feature]
                // (its loads and MMAs are done: the stages are free)
                float* part = reinterpret_cast<float*>(sh.stage);
                for (int c = 16 * half; c < ti.ntok; c += 32) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(acc + (uint32_t)c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * WM + q * 32 + lane] = __uint_as_float(r[j]);
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp < kTmaWarp) {
        if (RAW) lay_out_scales<KIND, CG>(sh, args, wk);
        else produce_scales<KIND, CG>(sh, args, wk, rank);
    } else if (warp == kTmaWarp) {
        // ------------------------------------------------ codes of both operands
        // one box of weights and one of tokens per k-step; converged, as the
        // MMA warp below
        int it = 0, rit = 0;
        int s = 0, rs = 0;
        uint32_t ph = 1, rph = 1;
        bool ok = true;
        for (int t = wk.t0; t < wk.num && ok; t += wk.step) {
            const Tile ti = decode_tile<CG, TN>(t, f_tiles, E, sh);
            const int h = ((ti.ntok + 15) & ~15) / CG;  // tokens of the MMA: this CTA's share
            const int f = ti.f0 + WM * rank, tok = ti.tok0 + rank * h;
            for (int ks = wk.k0; ks < wk.k1; ++ks, ++it) {
                if (RAW && (ks - wk.k0) % P::kRawSteps == 0) {
                    if (!wait_bar_warp(&sh.raw_free[rs], rph, sh, args)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {  // each CTA loads the scales of all its tile's tokens
                        uint8_t* rw = sh.raw_rows + rs * P::kRawSlot;
                        mbar_arrive_expect_tx(&sh.raw[rs], P::kRawSlot);
                        tma_load_3d(rw, &tmap_sw, &sh.raw[rs], ks * 4 * NBLK, f, ti.e);
                        tma_load_2d(rw + WM * P::kRawRow, &tmap_sx, &sh.raw[rs], ks * 4 * NBLK, ti.tok0);
                    }
                    ++rit;
                    rs ^= 1;
                    rph ^= (uint32_t)(rs == 0);
                }
                if (!wait_bar_warp(&sh.empty[s], ph, sh, args)) {
                    ok = false;
                    break;
                }
                uint8_t* st = sh.stage + s * P::kStage;
                // the coordinate of a k-step: 128 bytes, or 128 widened codes
                if (elect_one()) {
                    if (CG == 1) {
                        mbar_arrive_expect_tx(&sh.full[s], args.w_tx + P::kX);
                        tma_load_3d(st, &tmap_w, &sh.full[s], ks * BKB, f, ti.e);
                        tma_load_2d(st + P::kXOff, &tmap_x, &sh.full[s], ks * BKB, tok);
                    } else {
                        // both CTAs' loads complete on the leader's barrier
                        if (leader) mbar_arrive_expect_tx(&sh.full[s], 2 * (args.w_tx + P::kX));
                        const uint32_t bar = mapa_shared(smem_u32(&sh.full[s]), 0);
                        tma_load_3d_pair(st, &tmap_w, bar, ks * BKB, f, ti.e);
                        tma_load_2d_pair(st + P::kXOff, &tmap_x, bar, ks * BKB, tok);
                    }
                }
                if (++s == P::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (lane == 0) {
            sh.issued[rank] = it;
            *sh.raw_issued = rit;
        }
    } else if (warp == kFenceWarp) {
        // ----------------------------- scales: generic stores -> tensor core
        if (lane == 0) {
            int my_tiles = 0;
            if (wk.num > wk.t0) my_tiles = (wk.num - 1 - wk.t0) / wk.step + 1;
            const int items = my_tiles * (wk.k1 - wk.k0);
            int s = 0, it = 0;
            uint32_t ph = 0;
            for (; it < items; ++it) {
                if (!wait_bar(&sh.scales[s], ph, sh, args)) break;
                fence_proxy_async_smem();
                arrive_leader<CG>(&sh.full[s]);
                if (++s == P::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
            sh.fenced[rank] = it;
        }
    } else if (leader) {
        // ------------------------------------------------ MMA (leader only)
        const uint32_t st_base = smem_u32(sh.stage);
        int s = 0, prev = 0;  // stage of this k-step, and of the one that last used its scale slot
        uint32_t ph = 0, pph = 0;
        int slot = 0, unused = P::kSlots, tile_iter = 0;
        bool ok = true;
        for (int t = wk.t0; t < wk.num && ok; t += wk.step, ++tile_iter) {
            const Tile ti = decode_tile<CG, TN>(t, f_tiles, E, sh);
            const uint32_t n = (uint32_t)((ti.ntok + 15) & ~15);
            const uint32_t idesc = args.idesc | idesc_scaled(WM * CG, n, 0, 0, 0);
            const uint32_t acc = tmem + (uint32_t)((tile_iter & 1) * P::kAccStep);
            if (!wait_bar_warp(sh.acc_free, (tile_iter & 1) ^ 1, sh, args)) break;
            tc_fence_after();
            for (int ks = wk.k0; ks < wk.k1; ++ks) {
                // a slot's previous scales are free once the MMAs that read
                // them are done; with a slot per stage, a full stage says so
                if (P::kSlots < P::STAGES) {
                    if (unused > 0) {
                        --unused;
                    } else {
                        if (!wait_bar_warp(&sh.empty[prev], pph, sh, args)) {
                            ok = false;
                            break;
                        }
                        if (++prev == P::STAGES) {
                            prev = 0;
                            pph ^= 1;
                        }
                    }
                }
                if (!wait_bar_warp(&sh.full[s], ph, sh, args)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ss = st_base + s * P::kStage;
                const uint32_t sw = tmem + P::kScaleCols + (uint32_t)slot * P::kSlotCols, sx = sw + 16;
                if (elect_one()) {
                    const uint64_t dw = smem_desc_plain(ss + P::kSWOff), dx = smem_desc_plain(ss + P::kSXOff);
#pragma unroll
                    for (int b = 0; b < NBLK; ++b) {
                        copy_scales<CG>(sw + b * 4, dw + b * (512 >> 4));
#pragma unroll
                        for (int x = 0; x < P::XBLK; ++x)
                            if (x == 0 || n > 128u)
                                copy_scales<CG>(sx + (b * P::XBLK + x) * 4, dx + (b * P::XBLK + x) * (512 >> 4));
                    }
                    const uint64_t ad0 = smem_desc(ss, 16, 1024), bd0 = smem_desc(ss + P::kXOff, 16, 1024);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // 32 bytes of each row per MMA: its scale block, and
                        // the byte of the scale word it starts at
                        const int blk = (KIND == MMA_NVFP4) ? j : (KIND == MMA_MXFP4 ? j / 2 : 0);
                        const uint32_t byte = (KIND == MMA_NVFP4) ? 0u : (KIND == MMA_MXFP4 ? (j & 1) * 2u : (uint32_t)j);
                        mma_scaled<KIND, CG>(acc, ad0 + 2 * j, bd0 + 2 * j, idesc | idesc_scale_byte(byte), sw + blk * 4,
                                             sx + blk * P::XBLK * 4, (ks > wk.k0 || j > 0) ? 1u : 0u);
                    }
                    if (CG == 1) mma_commit(&sh.empty[s]);
                    else mma_commit_pair_multicast(&sh.empty[s], 0x3);
                }
                if (++slot == P::kSlots) slot = 0;
                if (++s == P::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (ok && elect_one()) {
                if (CG == 1) mma_commit(sh.acc_full);
                else mma_commit_pair_multicast(sh.acc_full, 0x3);
            }
        }
        // every MMA issued here has completed once `drain` fires
        if (elect_one()) {
            if (CG == 1) mma_commit(sh.drain);
            else mma_commit_pair_multicast(sh.drain, 0x1);
            mbar_wait(sh.drain, 0, kWaitNs);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (CG == 2) {
        if (threadIdx.x == 0) {  // to the peer: what this CTA has done
            const uint32_t to = mapa_shared(smem_u32(sh.issued + rank), rank ^ 1);
            sh.gave_up[rank] = *sh.abort;
            st_cluster(to, sh.issued[rank]);
            st_cluster(to + 8, sh.fenced[rank]);
            st_cluster(to + 16, *sh.abort);
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while its peer may still touch it
    }
    if (CG == 2 ? (sh.gave_up[0] | sh.gave_up[1]) != 0 : *sh.abort != 0) {
        if (threadIdx.x == 0) drain_loads<KIND, CG, RAW>(sh, args.w_tx + P::kX, rank);
        __syncwarp();
        if (CG == 2) cluster_sync();  // the leader has waited for its peer's loads
        else __syncthreads();
    }
    if (CG == 1 && split > 1) {
        // add the cluster's partial sums in rank order, each CTA for its share
        // of the features
        cluster_sync();
        if (wk.t0 < wk.num) {
            const Tile ti = decode_tile<CG, TN>(wk.t0, f_tiles, E, sh);
            const int fr = WM / split;
            const uint32_t part = smem_u32(sh.stage);
            for (int i = threadIdx.x; i < ti.ntok * fr; i += kThreads) {
                const int tok = i / fr, fl = krank * fr + i % fr, f = ti.f0 + fl;
                if (f >= args.N) continue;
                float v = 0.0f;
                for (int p = 0; p < split; ++p) v += lds_cluster_f32(mapa_shared(part, p) + (uint32_t)(tok * WM + fl) * 4);
                if (KIND == MMA_NVFP4)
                    v = v * __ldg(args.a_row + ti.tok0 + tok) * __ldg(args.w_row + (int64_t)ti.e * args.N + f);
                const __nv_bfloat16 h = __float2bfloat16_rn(v);
                if (BSQ_DOK(ti.tok0 + tok < args.T))
                    args.out[(int64_t)(ti.tok0 + tok) * args.N + f] = *reinterpret_cast<const uint16_t*>(&h);
            }
        }
        cluster_sync();  // no CTA leaves while a peer may still read it
    }
    tc_fence_after();
    if (warp == kMmaWarp) {
        if (CG == 1) tmem_dealloc(tmem, kTmemCols);
        else tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ----------------------------------------------------------------- host -----

struct Launch {
    CUtensorMap x, w, sx, sw, out;
    Args args;
    cudaStream_t stream;
};

template <int KIND, int CG, bool RAW>
static bsq_status launch(Launch& l, int64_t max_groups, const char* fn) {
    static std::mutex mu;
    static int max_active[64][4] = {{0}};  // co-resident clusters per device, by log2 of the size (0: not yet queried)
    auto kern = scaled_mm_kernel<KIND, CG, RAW>;
    const size_t smem = Plan<KIND, CG, RAW>::kSmemBytes;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(BSQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = l.stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 1 : 0;
    int fit[4];  // clusters of 1, 2, 4 and 8 CTAs that the device holds at once (pairs: of 2)
    {
        std::lock_guard<std::mutex> lock(mu);
        const int slot = (dev >= 0 && dev < 64) ? dev : 63;
        int* have = max_active[slot];
        if (have[CG - 1] == 0 || slot != dev) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess)
                return fail(BSQ_ERR_CUDA, "%s: shared-memory opt-in failed (%s)", fn, cudaGetErrorString(e));
            have[0] = sm_count();
            for (int i = 1; i < (CG == 2 ? 2 : 4); ++i) {
                attr[0].val.clusterDim.x = 1u << i;
                cfg.numAttrs = 1;
                cfg.gridDim = dim3((unsigned)(sm_count() >> i) << i, 1, 1);
                int clusters = 0;
                if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters <= 0) {
                    cudaGetLastError();
                    clusters = CG == 2 ? sm_count() / 2 : 0;
                }
                have[i] = clusters;
            }
        }
        std::copy(have, have + 4, fit);
    }
    // Single CTAs that would leave SMs idle split each tile's contraction over
    // a cluster, a chunk of scales at least to a CTA, as long as all clusters
    // run at once (one tile per cluster then; a second wave of clusters costs
    // more than it saves: one token, N = 2048, K = 7168, 16 tiles: 13.0 us
    // unsplit, 9.2 us over 4 CTAs, 14.3 us over 8).
    l.args.split = 1;
    constexpr int G = Plan<KIND, CG, RAW>::kRawSteps;
    int lg = CG - 1;
    if (CG == 1)
        while ((2 << lg) <= kMaxSplit && max_groups <= fit[lg + 1] && l.args.k_steps >= (2 << lg) * G) ++lg;
    if (CG == 1) l.args.split = 1 << lg;
    attr[0].val.clusterDim.x = 1u << lg;
    cfg.numAttrs = lg > 0 ? 1 : 0;
    const int n = fit[lg];
    const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(max_groups, n));
    cfg.gridDim = dim3(groups * CG * l.args.split, 1, 1);
    e = cudaLaunchKernelEx(&cfg, kern, l.x, l.w, l.sx, l.sw, l.out, l.args);
    if (e != cudaSuccess) return fail(BSQ_ERR_CUDA, "%s: launch failed (%s)", fn, cudaGetErrorString(e));
    return check_launch(fn);
}

template <int CG, bool RAW>
static bsq_status launch_kind(int kind, Launch& l, int64_t max_groups, const char* fn) {
    if (kind == MMA_NVFP4) return launch<MMA_NVFP4, CG, RAW>(l, max_groups, fn);
    if (kind == MMA_MXFP4) return launch<MMA_MXFP4, CG, RAW>(l, max_groups, fn);
    return launch<MMA_MX8, CG, RAW>(l, max_groups, fn);
}

}  // namespace smm
}  // namespace bsq

using namespace bsq;

BSQ_API bsq_status bsq_grouped_mm_scaled(bsq_format a_fmt, bsq_format w_fmt, const uint8_t* a_codes,
                                         const uint8_t* a_scales, const float* a_row_scale, const uint8_t* w_codes,
                                         const uint8_t* w_scales, const float* w_row_scale, const int32_t* offs, int E,
                                         int64_t T, int64_t N, int64_t K, void* out, uint32_t* err,
                                         bsq_stream_t stream) {
    const char* fn = "bsq_grouped_mm_scaled";
    const bool wide_w = a_fmt == BSQ_MXFP8 && w_fmt == BSQ_MXFP4;  // e2m1 weights in 8-bit containers
    int kind;
    if (a_fmt == BSQ_NVFP4 && w_fmt == BSQ_NVFP4) kind = MMA_NVFP4;
    else if (a_fmt == BSQ_MXFP4 && w_fmt == BSQ_MXFP4) kind = MMA_MXFP4;
    else if (a_fmt == BSQ_MXFP8 && (w_fmt == BSQ_MXFP8 || wide_w)) kind = MMA_MX8;
    else
        return fail(BSQ_ERR_UNSUPPORTED, "%s: formats must be NVFP4, MXFP4 or MXFP8 for both operands, or MXFP8 x MXFP4",
                    fn);
    if (E < 1 || T < 0 || N <= 0 || K <= 0) return fail(BSQ_ERR_INVALID_ARG, "%s: bad sizes", fn);
    if (!offs && E != 1) return fail(BSQ_ERR_INVALID_ARG, "%s: several experts need offs", fn);
    if (E > smm::kMaxExperts) return fail(BSQ_ERR_UNSUPPORTED, "%s: at most %d experts", fn, smm::kMaxExperts);
    if (T > (int64_t(1) << 30) || N > (int64_t(1) << 30) || K > (int64_t(1) << 30) || (int64_t)E * N > (int64_t(1) << 31))
        return fail(BSQ_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    const int kmul = wide_w ? 128 : 32;
    if (K % kmul != 0 || N % 8 != 0)
        return fail(BSQ_ERR_UNSUPPORTED, "%s: needs K %% %d == 0 and N %% 8 == 0", fn, kmul);
    if (!err) return fail(BSQ_ERR_INVALID_ARG, "%s: null error word", fn);
    if (T == 0) return BSQ_OK;
    if (!a_codes || !a_scales || !w_codes || !w_scales || !out ||
        (kind == MMA_NVFP4 && (!a_row_scale || !w_row_scale)))
        return fail(BSQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (((uintptr_t)a_codes % 16) || ((uintptr_t)w_codes % (wide_w ? 32 : 16)) || ((uintptr_t)out % 16) ||
        ((uintptr_t)a_row_scale % 4) || ((uintptr_t)w_row_scale % 4) || ((uintptr_t)offs % 4) || ((uintptr_t)err % 4))
        return fail(BSQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);

    const int64_t row_bytes = (kind == MMA_MX8) ? K : K / 2;  // of an activation row
    const int64_t row_scales = K / (kind == MMA_NVFP4 ? 16 : 32);
    const int64_t w_row_bytes = wide_w ? K / 2 : row_bytes, w_rows = (int64_t)E * N;
    const bool nv = kind == MMA_NVFP4;
    const Span outs[] = {{out, (size_t)(T * N) * 2}, {err, 4}};
    const Span read[] = {{a_codes, (size_t)(T * row_bytes)}, {a_scales, (size_t)(T * row_scales)},
                         {nv ? a_row_scale : nullptr, (size_t)T * 4}, {w_codes, (size_t)(w_rows * w_row_bytes)},
                         {w_scales, (size_t)(w_rows * row_scales)}, {nv ? w_row_scale : nullptr, (size_t)w_rows * 4},
                         {offs, (size_t)E * 4}};
    if (any_overlap(outs, read)) return fail(BSQ_ERR_INVALID_ARG, "%s: an output overlaps an input or the error word", fn);

    bsq_status st;
    EncodeTiledFn encode = encode_fn(&st, fn);
    if (!encode) return st;
    smm::Launch l;
    // The most tiles there can be; ragged experts end in partial ones.
    auto tiles = [&](int features, int tokens) {
        const int64_t f = (N + features - 1) / features;
        return (offs ? T / tokens + std::min<int64_t>(E, T) : (T + tokens - 1) / tokens) * f;
    };
    // Single CTAs where one 32-token tile mostly holds an expert's tokens, or
    // where all their tiles run at once; else pairs.  NVFP4, us, singles and
    // pairs: dense K = 7168, N = 2048: 256 tokens 14.4 and 18.5, 512 tokens
    // 22.6 and 18.5; N = 16384: 17 tokens 18.5 and 25.3, 33 tokens 27.2 and
    // 22.6; 32 experts of N = 2048, 64 tokens 49 and 63 (MXFP8 x MXFP4), 512
    // tokens 57.6 and 57.8, 1024 tokens 65.3 and 58.5.
    const bool pairs = !(offs ? T <= 16 * (int64_t)E : T <= 32) && tiles(smm::WM, 32) > sm_count();
    const int tn = pairs ? 256 : 32;
    // Scale rows by TMA where it can read them: a multiple of 16 bytes, aligned
    const bool raw = row_scales % 16 == 0 && (uintptr_t)a_scales % 16 == 0 && (uintptr_t)w_scales % 16 == 0;
    // [slabs, rows, bytes] of one code or scale per byte, or of e2m1 codes
    // widened to 8-bit containers (16 codes: 8 bytes and 8 bytes of padding);
    // weights have a slab per expert, so rows past N read as zero and never
    // as the next expert's
    CUresult r = CUDA_SUCCESS;
    auto map = [&](CUtensorMap* m, const uint8_t* p, int64_t bytes, int64_t rows, int64_t slabs, int box_bytes,
                   int box_rows, bool wide, bool swizzle) {
        const cuuint64_t dims[3] = {(cuuint64_t)(wide ? 2 * bytes : bytes), (cuuint64_t)rows, (cuuint64_t)slabs};
        const cuuint64_t strides[2] = {(cuuint64_t)bytes, (cuuint64_t)(bytes * rows)};
        const cuuint32_t box[3] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows, 1}, estr[3] = {1, 1, 1};
        if (r == CUDA_SUCCESS)
            r = encode(m, wide ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, slabs ? 3 : 2,
                       const_cast<uint8_t*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    map(&l.x, a_codes, row_bytes, T, 0, smm::BKB, pairs ? tn / 2 : tn, false, true);
    map(&l.w, w_codes, w_row_bytes, N, E, smm::BKB, smm::WM, wide_w, true);
    if (raw) {
        const int chunk = smm::raw_row_bytes(kind);
        map(&l.sx, a_scales, row_scales, T, 0, chunk, tn, false, false);
        map(&l.sw, w_scales, row_scales, N, E, chunk, smm::WM, false, false);
    } else {
        l.sx = l.x;
        l.sw = l.w;
    }
    {
        const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)T}, strides[1] = {(cuuint64_t)N * 2};
        const cuuint32_t box[2] = {32, 32}, estr[2] = {1, 1};
        if (r == CUDA_SUCCESS)
            r = encode(&l.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    if (r != CUDA_SUCCESS) return fail(BSQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", fn, (int)r);
    smm::Args& a = l.args;
    a.a_scales = a_scales;
    a.a_scales_end = a_scales + (int64_t)T * row_scales;
    a.a_row = a_row_scale;
    a.w_scales = w_scales;
    a.w_scales_end = w_scales + (int64_t)E * N * row_scales;
    a.w_row = w_row_scale;
    a.offs = offs;
    a.out = (uint16_t*)out;
    a.err = err;
    // BSQ_GMM_WAIT_NS (a positive integer, in ns) shortens the limit of each
    // pipeline wait; tests use it to make the waits run out on purpose
    a.wait_ns = smm::kWaitNs;
    if (const char* w = getenv("BSQ_GMM_WAIT_NS")) {
        char* end = nullptr;
        const unsigned long long v = strtoull(w, &end, 10);
        if (end != w && *end == '\0' && v > 0) a.wait_ns = v;
    }
    a.E = E;
    a.T = (int)T;
    a.N = (int)N;
    a.k_steps = (int)((row_bytes + smm::BKB - 1) / smm::BKB);
    a.row_scales = (int)row_scales;
    a.w_tx = wide_w ? smm::kWBytes / 2 : smm::kWBytes;  // widening: the codes count, their padding does not
    const uint32_t wf = kind == MMA_MX8 ? (wide_w ? 5u : 0u) : 1u, xf = kind == MMA_MX8 ? 0u : 1u;
    a.idesc = idesc_scaled(0, 0, wf, xf, kind == MMA_NVFP4 ? 0u : 1u);
    l.stream = (cudaStream_t)stream;
    const int64_t max_groups = tiles(pairs ? 2 * smm::WM : smm::WM, tn);
    if (pairs)
        return raw ? smm::launch_kind<2, true>(kind, l, max_groups, fn) : smm::launch_kind<2, false>(kind, l, max_groups, fn);
    return raw ? smm::launch_kind<1, true>(kind, l, max_groups, fn) : smm::launch_kind<1, false>(kind, l, max_groups, fn);
}

#ifdef BSQ_DEBUG
cudaError_t bsq_dbg_take_smm(uint32_t* count, uint32_t* first) { return bsq::dbg_take(count, first); }
#endif
