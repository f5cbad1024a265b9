// tma_encode.h -- the CUDA driver's tensor-map encoder, found once per process.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "host_util.h"

namespace bsq {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// NULL, with the reason in *st, where the CUDA driver has none.
static inline EncodeTiledFn encode_fn(bsq_status* st, const char* caller) {
    static std::mutex mu;
    static EncodeTiledFn fn = nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !p) {
            *st = fail(BSQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable (%s)", caller, cudaGetErrorString(e));
            return nullptr;
        }
        fn = (EncodeTiledFn)p;
    }
    *st = BSQ_OK;
    return fn;
}

}  // namespace bsq
