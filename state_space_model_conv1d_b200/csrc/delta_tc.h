// delta_tc.h -- launchers shared by the tensor-core kernels of the gated delta rule.
#pragma once

#include "delta_tc.cuh"

namespace ssm {

// q, k as [n][group][token][row] maps, v (or dy) as a [channel][token][row] map.
struct DeltaMaps {
    CUtensorMap q, k, v;
};
bool delta_maps(const ssm_delta_args &a, DeltaMaps *m);

size_t delta_prep_bytes(const ssm_delta_args &a, bool bwd);
cudaError_t launch_delta_prep(const ssm_delta_args &a, const SeqView &sv, const DeltaMaps &m, void *out, bool bwd,
                              cudaStream_t st);
// The forward chain; with `rec` the states' pass of the backward.
cudaError_t launch_delta_chain(const ssm_delta_args &a, const SeqView &sv, const DeltaMaps &m, const void *prep,
                               const dtc::Rec *rec, cudaStream_t st);

}  // namespace ssm
