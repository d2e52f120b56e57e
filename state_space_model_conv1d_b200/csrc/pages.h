// pages.h -- host-side launchers of the state pages (internal to libssm).
#pragma once

#include "launch.h"

namespace ssm {

constexpr int64_t kMaxPages = 1 << 20;
constexpr int64_t kMaxPageEntries = 1 << 20;

enum class PageOp { kCopy, kFork, kFree, kCompact };
size_t pages_workspace_bytes(const ssm_pages_args &a);
// `ws` starts with the error word.
cudaError_t launch_pages(PageOp op, const ssm_pages_args &a, void *ws, cudaStream_t st);

}  // namespace ssm
