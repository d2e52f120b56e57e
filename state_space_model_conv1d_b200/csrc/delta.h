// delta.h -- host-side launchers of the gated delta rule (internal to libssm).
#pragma once

#include "common.cuh"
#include "launch.h"

namespace ssm {

// Log decays at or below this are a reset: exp() rounds to zero in fp32 from
// -103.98 down.  Clamping there keeps g = -infinity out of the prefix sums,
// where it would give NaN; decay_of() is then exactly zero, not whatever
// expf() makes of the bottom of the subnormal range.
constexpr float kMinLogDecay = -104.f;
__device__ __forceinline__ float log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }   // (a NaN stays one)

__device__ __forceinline__ bool resets(float g) { return g <= kMinLogDecay; }
__device__ __forceinline__ float decay_of(float g) { return resets(g) ? 0.f : expf(g); }

// dg and dbeta of gate i: fp32 or the activations' type T.
template <typename T>
__device__ __forceinline__ void store_gates(const ssm_delta_bwd_args &b, int64_t i, float dg, float dbeta) {
    if (b.fwd.gates_f32) {
        static_cast<float *>(b.dg)[i] = dg;
        static_cast<float *>(b.dbeta)[i] = dbeta;
    } else {
        Elem<T>::st(static_cast<T *>(b.dg) + i, dg);
        Elem<T>::st(static_cast<T *>(b.dbeta) + i, dbeta);
    }
}

// Token-by-token path (any dtype and sizes).  `ckpt` (may be null) receives
// the state before every kDeltaCkpt-th token of each sequence.
constexpr int kDeltaCkpt = 32;
// Rows of checkpoints: sequence s starts at row cu[s] / kDeltaCkpt + s, a
// bound that holds without a prefix sum of rounded-up lengths.
inline int64_t delta_ckpt_rows(const ssm_delta_args &a) {
    return a.cu_seqlens ? a.seqlen / kDeltaCkpt + a.nseqs + 1
                        : a.batch * ((a.seqlen + kDeltaCkpt - 1) / kDeltaCkpt);
}
cudaError_t launch_delta_simt(const ssm_delta_args &a, const SeqView &sv, float *ckpt, cudaStream_t st);
size_t delta_simt_bwd_workspace_bytes(const ssm_delta_bwd_args &b);
cudaError_t launch_delta_simt_bwd(const ssm_delta_bwd_args &b, const SeqView &sv, void *ws, cudaStream_t st);

// Tensor-core path in blocks of 64 tokens: the shapes it takes (they decide the
// workspace), the pointers and strides it needs besides, and its launcher.
bool delta_tc_shape(const ssm_delta_args &a);
bool delta_tc_ok(const ssm_delta_args &a);
size_t delta_tc_workspace_bytes(const ssm_delta_args &a);
cudaError_t launch_delta_tc(const ssm_delta_args &a, const SeqView &sv, void *ws, cudaStream_t st);
bool delta_tc_bwd_ok(const ssm_delta_bwd_args &b);
size_t delta_tc_bwd_workspace_bytes(const ssm_delta_bwd_args &b);
cudaError_t launch_delta_tc_bwd(const ssm_delta_bwd_args &b, const SeqView &sv, void *ws, cudaStream_t st);

cudaError_t launch_delta_update(const ssm_delta_update_args &a, cudaStream_t st);

}  // namespace ssm
