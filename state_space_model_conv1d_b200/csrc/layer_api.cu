// layer_api.cu -- C entry points of the operators beside the scan: the gated
// delta rule, group norm and the state pages.  Validation on the host, then
// the launch on the caller's stream; nothing allocates or synchronizes.
#include <cuda_runtime.h>

#include "../../include/ssm.h"
#include "api_util.h"
#include "delta.h"
#include "norm.h"
#include "pages.h"

namespace {

using ssm::aligned;
using ssm::check_act;
using ssm::cuda_status;
using ssm::dtype_ok;
using ssm::esize;

constexpr int64_t kMaxDim = 1 << 20;      // heads, headdim, groups, channels: products stay in 64 bits

ssm_status validate_delta(const ssm_delta_args *a) {
    if (!a) return SSM_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->batch < 0 || a->seqlen < 0) return SSM_ERR_INVALID_ARG;
    if (a->nheads < 1 || a->headdim < 1 || a->ngroups < 1 || a->dstate < 1 || a->nheads % a->ngroups != 0)
        return SSM_ERR_INVALID_ARG;
    if (a->dstate > ssm::kMaxDstateM2 || a->nheads > kMaxDim || a->headdim > kMaxDim ||
        a->nheads * ((a->headdim + 31) / 32) > INT32_MAX || a->seqlen > INT32_MAX || a->batch > 65535)
        return SSM_ERR_UNSUPPORTED;
    if (a->cu_seqlens &&
        (a->batch != 1 || a->nseqs < 0 || a->nseqs > 65535 || (a->nseqs == 0 && a->seqlen > 0)))
        return SSM_ERR_INVALID_ARG;
    const size_t es = esize(a->dtype);
    const bool work = a->batch > 0 && a->seqlen > 0;
    const int64_t gn = a->ngroups * a->dstate, hp = a->nheads * a->headdim, b = a->batch, t = a->seqlen;
    SSM_TRY(check_act(a->q, a->q_batch_stride, a->q_token_stride, gn, b, t, es, work));
    SSM_TRY(check_act(a->k, a->k_batch_stride, a->k_token_stride, gn, b, t, es, work));
    SSM_TRY(check_act(a->v, a->v_batch_stride, a->v_token_stride, hp, b, t, es, work));
    SSM_TRY(check_act(a->g, a->g_batch_stride, a->g_token_stride, a->nheads, b, t, 4, work));
    SSM_TRY(check_act(a->beta, a->beta_batch_stride, a->beta_token_stride, a->nheads, b, t, 4, work));
    SSM_TRY(check_act(a->y, a->y_batch_stride, a->y_token_stride, hp, b, t, es, work));
    if (!aligned(a->h0, 4) || !aligned(a->h_final, 4) || !aligned(a->cu_seqlens, 4)) return SSM_ERR_ALIGNMENT;
    return SSM_OK;
}

size_t delta_prefix(const ssm_delta_args &a) {
    return ssm::kWsOrderOffset + (a.cu_seqlens ? ssm::order_bytes(a.nseqs) : 0);
}

// Error word, cu_seqlens check and schedule, as in ssm_scan_fwd.
ssm_status delta_plan(const ssm_delta_args &a, char *ws, cudaStream_t st, ssm::SeqView *sv) {
    *sv = ssm::SeqView{nullptr, nullptr, reinterpret_cast<int32_t *>(ws + ssm::kWsErrorOffset), (int)a.batch};
    if (a.cu_seqlens) {
        sv->cu = a.cu_seqlens;
        sv->order = reinterpret_cast<int32_t *>(ws + ssm::kWsOrderOffset);
        sv->nseqs = a.nseqs;
        return cuda_status(ssm::launch_varlen_plan(a.cu_seqlens, a.nseqs, a.seqlen, sv->err,
                                                   const_cast<int32_t *>(sv->order), st));
    }
    return cuda_status(cudaMemsetAsync(sv->err, 0, sizeof(int32_t), st));
}

bool sizes_ok(const ssm_delta_args &a) {
    ssm_delta_args f = a;        // shapes alone: the workspace size does not depend on pointers
    return f.batch >= 0 && f.seqlen >= 0 && f.nseqs >= 0 && f.nheads >= 1 && f.headdim >= 1 && f.ngroups >= 1 &&
           f.dstate >= 1 && f.dstate <= ssm::kMaxDstateM2 && f.nheads <= kMaxDim && f.headdim <= kMaxDim;
}

ssm_status validate_delta_bwd(const ssm_delta_bwd_args *b) {
    if (!b) return SSM_ERR_INVALID_ARG;
    ssm_delta_args f = b->fwd;
    f.y = const_cast<void *>(b->dy);
    f.y_batch_stride = b->dy_batch_stride;
    f.y_token_stride = b->dy_token_stride;
    SSM_TRY(validate_delta(&f));
    if (f.gates_f32 != 0 && f.gates_f32 != 1) return SSM_ERR_INVALID_ARG;
    if (f.batch > 0 && f.seqlen > 0 && (!b->dq || !b->dk || !b->dv || !b->dg || !b->dbeta)) return SSM_ERR_INVALID_ARG;
    const size_t es = esize(f.dtype);
    for (const void *o : {b->dq, b->dk, b->dv})
        if (!aligned(o, es)) return SSM_ERR_ALIGNMENT;
    for (const void *o : {b->dg, b->dbeta})
        if (!aligned(o, f.gates_f32 ? 4 : es)) return SSM_ERR_ALIGNMENT;
    if (!aligned(b->dh_final, 4) || !aligned(b->dh0, 4)) return SSM_ERR_ALIGNMENT;
    return SSM_OK;
}

ssm_status validate_norm(const ssm_norm_args *a, const void *y, int64_t y_bs, int64_t y_ts) {
    if (!a) return SSM_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->mode < SSM_NORM_PLAIN || a->mode > SSM_NORM_GATE_FIRST) return SSM_ERR_INVALID_ARG;
    if ((a->subtract_mean != 0 && a->subtract_mean != 1) || !(a->eps >= 0.f)) return SSM_ERR_INVALID_ARG;
    if (a->batch < 0 || a->seqlen < 0 || a->channels < 1 || a->groups < 1 || a->channels % a->groups != 0)
        return SSM_ERR_INVALID_ARG;
    const bool gate = a->mode == SSM_NORM_GATE || a->mode == SSM_NORM_GATE_FIRST;
    const bool work = a->batch > 0 && a->seqlen > 0;
    if (work && gate != (a->z != nullptr)) return SSM_ERR_INVALID_ARG;
    if (a->channels / a->groups > ssm::kMaxGroupWidth || a->channels > INT32_MAX || a->seqlen > INT32_MAX ||
        a->batch > INT32_MAX || a->batch * a->seqlen > INT32_MAX)
        return SSM_ERR_UNSUPPORTED;
    const size_t es = esize(a->dtype);
    SSM_TRY(check_act(a->x, a->x_batch_stride, a->x_token_stride, a->channels, a->batch, a->seqlen, es, work));
    SSM_TRY(check_act(a->z, a->z_batch_stride, a->z_token_stride, a->channels, a->batch, a->seqlen, es, work && gate));
    SSM_TRY(check_act(y, y_bs, y_ts, a->channels, a->batch, a->seqlen, es, work));
    if (!aligned(a->weight, 4) || !aligned(a->bias, 4)) return SSM_ERR_ALIGNMENT;
    return SSM_OK;
}

ssm_status pages_call(ssm::PageOp op, const ssm_pages_args *a, void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return SSM_ERR_INVALID_ARG;
    if (a->nslots < 0 || a->n < 0 || a->npools < 0) return SSM_ERR_INVALID_ARG;
    if (a->nslots > ssm::kMaxPages || a->n > ssm::kMaxPageEntries || a->npools > SSM_MAX_POOLS)
        return SSM_ERR_UNSUPPORTED;
    const bool refs = op != ssm::PageOp::kCopy, src = op == ssm::PageOp::kCopy || op == ssm::PageOp::kFork;
    if ((refs && a->nslots > 0 && !a->refs) || (a->n > 0 && (!a->pages || (src && !a->src)))) return SSM_ERR_INVALID_ARG;
    if (!aligned(a->refs, 4) || !aligned(a->src, 4) || !aligned(a->pages, 4)) return SSM_ERR_ALIGNMENT;
    for (int k = 0; k < a->npools; ++k) {
        if (a->pools[k].page_bytes < 1 || (a->nslots > 0 && !a->pools[k].base)) return SSM_ERR_INVALID_ARG;
        if (a->pools[k].page_bytes > INT64_MAX / ssm::kMaxPages) return SSM_ERR_UNSUPPORTED;
    }
    if (!workspace || ws_bytes < ssm::pages_workspace_bytes(*a) || !aligned(workspace, 256)) return SSM_ERR_WORKSPACE;
    return cuda_status(ssm::launch_pages(op, *a, workspace, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

size_t ssm_delta_workspace_size(const ssm_delta_args *args) {
    if (!args || !sizes_ok(*args)) return 0;
    return delta_prefix(*args) + (ssm::delta_tc_shape(*args) ? ssm::delta_tc_workspace_bytes(*args) : 0);
}

ssm_status ssm_delta_fwd(const ssm_delta_args *args, void *workspace, size_t ws_bytes, void *stream) {
    SSM_TRY(validate_delta(args));
    const cudaStream_t st = (cudaStream_t)stream;
    if (!workspace || ws_bytes < ssm_delta_workspace_size(args) || !aligned(workspace, 256)) return SSM_ERR_WORKSPACE;
    ssm::SeqView sv;
    char *ws = static_cast<char *>(workspace);
    SSM_TRY(delta_plan(*args, ws, st, &sv));
    if (ssm::delta_tc_ok(*args)) return cuda_status(ssm::launch_delta_tc(*args, sv, ws + delta_prefix(*args), st));
    return cuda_status(ssm::launch_delta_simt(*args, sv, nullptr, st));
}

size_t ssm_delta_bwd_workspace_size(const ssm_delta_bwd_args *args) {
    if (!args || !sizes_ok(args->fwd)) return 0;
    return delta_prefix(args->fwd) + (ssm::delta_tc_bwd_ok(*args) ? ssm::delta_tc_bwd_workspace_bytes(*args)
                                                                  : ssm::delta_simt_bwd_workspace_bytes(*args));
}

ssm_status ssm_delta_bwd(const ssm_delta_bwd_args *args, void *workspace, size_t ws_bytes, void *stream) {
    SSM_TRY(validate_delta_bwd(args));
    const cudaStream_t st = (cudaStream_t)stream;
    if (!workspace || ws_bytes < ssm_delta_bwd_workspace_size(args) || !aligned(workspace, 256))
        return SSM_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    ssm::SeqView sv;
    SSM_TRY(delta_plan(args->fwd, ws, st, &sv));
    ws += delta_prefix(args->fwd);
    if (ssm::delta_tc_bwd_ok(*args)) return cuda_status(ssm::launch_delta_tc_bwd(*args, sv, ws, st));
    return cuda_status(ssm::launch_delta_simt_bwd(*args, sv, ws, st));
}

ssm_status ssm_delta_update(const ssm_delta_update_args *a, void *stream) {
    if (!a) return SSM_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->batch < 0 || a->nslots < 0) return SSM_ERR_INVALID_ARG;
    if (a->nheads < 1 || a->headdim < 1 || a->ngroups < 1 || a->dstate < 1 || a->nheads % a->ngroups != 0)
        return SSM_ERR_INVALID_ARG;
    if (a->dstate > ssm::kMaxDstateM2 || a->batch > 65535 || a->nheads > kMaxDim || a->headdim > kMaxDim ||
        a->nheads * ((a->headdim + 15) / 16) > INT32_MAX)
        return SSM_ERR_UNSUPPORTED;
    if (a->batch == 0) return SSM_OK;
    if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->y || (a->nslots > 0 && !a->state)) return SSM_ERR_INVALID_ARG;
    if (!a->state_batch_indices && a->nslots < a->batch) return SSM_ERR_INVALID_ARG;
    const int64_t gn = a->ngroups * a->dstate, hp = a->nheads * a->headdim;
    if (a->batch > 1 && (a->q_batch_stride < gn || a->k_batch_stride < gn || a->v_batch_stride < hp ||
                         a->y_batch_stride < hp || a->g_batch_stride < a->nheads || a->beta_batch_stride < a->nheads))
        return SSM_ERR_INVALID_ARG;
    const size_t es = esize(a->dtype);
    for (const void *p : {a->q, a->k, a->v, (const void *)a->y})
        if (!aligned(p, es)) return SSM_ERR_ALIGNMENT;
    if (!aligned(a->state, a->dstate % 4 == 0 ? 16 : 4) || !aligned(a->g, 4) || !aligned(a->beta, 4) ||
        !aligned(a->state_batch_indices, 4))
        return SSM_ERR_ALIGNMENT;
    return cuda_status(ssm::launch_delta_update(*a, (cudaStream_t)stream));
}

ssm_status ssm_group_norm_fwd(const ssm_norm_args *a, void *stream) {
    if (!a) return SSM_ERR_INVALID_ARG;
    SSM_TRY(validate_norm(a, a->y, a->y_batch_stride, a->y_token_stride));
    return cuda_status(ssm::launch_group_norm(*a, (cudaStream_t)stream));
}

size_t ssm_group_norm_bwd_workspace_size(const ssm_norm_bwd_args *b) {
    if (!b) return 0;
    const ssm_norm_args &a = b->fwd;
    if (a.batch < 0 || a.seqlen < 0 || a.channels < 1 || a.groups < 1 || a.channels % a.groups != 0) return 0;
    return ssm::group_norm_bwd_workspace_bytes(*b);
}

ssm_status ssm_group_norm_bwd(const ssm_norm_bwd_args *b, void *workspace, size_t ws_bytes, void *stream) {
    if (!b) return SSM_ERR_INVALID_ARG;
    SSM_TRY(validate_norm(&b->fwd, b->dy, b->dy_batch_stride, b->dy_token_stride));
    const ssm_norm_args &a = b->fwd;
    if (a.batch > 0 && a.seqlen > 0 && (!b->dx || (a.z && !b->dz))) return SSM_ERR_INVALID_ARG;
    const size_t es = esize(a.dtype);
    if (!aligned(b->dx, es) || !aligned(b->dz, es) || !aligned(b->dweight, 4) || !aligned(b->dbias, 4))
        return SSM_ERR_ALIGNMENT;
    const size_t need = ssm_group_norm_bwd_workspace_size(b);
    if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 256))) return SSM_ERR_WORKSPACE;
    return cuda_status(ssm::launch_group_norm_bwd(*b, workspace, (cudaStream_t)stream));
}

size_t ssm_pages_workspace_size(const ssm_pages_args *a) {
    if (!a || a->nslots < 0 || a->n < 0 || a->nslots > ssm::kMaxPages || a->n > ssm::kMaxPageEntries) return 0;
    return ssm::pages_workspace_bytes(*a);
}
ssm_status ssm_pages_copy(const ssm_pages_args *a, void *ws, size_t ws_bytes, void *stream) {
    return pages_call(ssm::PageOp::kCopy, a, ws, ws_bytes, stream);
}
ssm_status ssm_pages_fork(const ssm_pages_args *a, void *ws, size_t ws_bytes, void *stream) {
    return pages_call(ssm::PageOp::kFork, a, ws, ws_bytes, stream);
}
ssm_status ssm_pages_free(const ssm_pages_args *a, void *ws, size_t ws_bytes, void *stream) {
    return pages_call(ssm::PageOp::kFree, a, ws, ws_bytes, stream);
}
ssm_status ssm_pages_compact(const ssm_pages_args *a, void *ws, size_t ws_bytes, void *stream) {
    return pages_call(ssm::PageOp::kCompact, a, ws, ws_bytes, stream);
}

}  // extern "C"
