// api_util.h -- host-side argument checks shared by the C entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssm.h"

namespace ssm {

// SSM_OK, or SSM_ERR_CUDA with the error kept for ssm_last_cuda_error().
ssm_status cuda_status(cudaError_t e);
int32_t last_cuda_error();

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t esize(int32_t dtype) { return dtype == SSM_BF16 ? 2 : 4; }
inline bool dtype_ok(int32_t d) { return d == SSM_F32 || d == SSM_BF16; }

// A token-major activation: row width w elements, strides in elements.
inline ssm_status check_act(const void *p, int64_t bs, int64_t ts, int64_t w, int64_t batch, int64_t seqlen,
                            size_t es, bool required) {
    if (!p) return required ? SSM_ERR_INVALID_ARG : SSM_OK;
    if (!aligned(p, es)) return SSM_ERR_ALIGNMENT;
    if (ts < 0 || bs < 0) return SSM_ERR_INVALID_ARG;
    if (seqlen > 1 && ts < w) return SSM_ERR_INVALID_ARG;          // token rows may not overlap
    if (batch > 1 && bs < ts * (seqlen - 1) + w) return SSM_ERR_INVALID_ARG;
    return SSM_OK;
}

}  // namespace ssm

#define SSM_TRY(expr)                      \
    do {                                   \
        ssm_status st_ = (expr);           \
        if (st_ != SSM_OK) return st_;     \
    } while (0)
