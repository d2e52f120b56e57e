// norm.h -- host-side launchers of group norm (internal to libssm).
#pragma once

#include "launch.h"

namespace ssm {

constexpr int64_t kMaxGroupWidth = 16384;   // channels of one group: 512 threads x 32 registers

cudaError_t launch_group_norm(const ssm_norm_args &a, cudaStream_t st);
// Shares of dweight / dbias, one per unit of a group.
size_t group_norm_bwd_workspace_bytes(const ssm_norm_bwd_args &b);
cudaError_t launch_group_norm_bwd(const ssm_norm_bwd_args &b, void *ws, cudaStream_t st);

}  // namespace ssm
