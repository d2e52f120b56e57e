"""Binding of the operators beside the scan: the gated delta rule, group norm
and the pages of a recurrent-state cache (same entry-point names as the C ABI).

Argument marshalling only, as in ``ops.py``: shapes and strides are read from
the tensors, outputs and workspaces come from PyTorch's allocator when the
caller does not pass them, and the call is enqueued on ``stream`` (the current
stream of the tensors' device when None), which need not be the current device.

Gated delta rule: q, k ``[b, T, G, N]``; v, y ``[b, T, H, P]``; g (log decay),
beta ``[b, T, H]`` fp32; h0 / h_final ``[nseq, H, P, N]`` fp32.  Packed varlen:
b = 1 and ``cu_seqlens`` int32 ``[nseq + 1]`` on the device.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _abi
from .ops import _dtype_code

_f32, _i32 = torch.float32, torch.int32


def _p(t):
    return None if t is None else t.data_ptr()


def _run(t, stream, body, *args):
    """``body(*args, stream handle)`` with t's device current and allocations made on the stream the call runs on.
    The common case (current device, current stream) enters no context: at one token a call is host-bound."""
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    idx = t.device.index
    if stream is None and idx == torch._C._cuda_getDevice():
        return body(*args, torch._C._cuda_getCurrentRawStream(idx))
    with torch.cuda.device(idx):
        s = torch.cuda.current_stream() if stream is None else stream
        if s.device != t.device:
            raise ValueError(f"stream is on {s.device}, the tensors on {t.device}")
        with torch.cuda.stream(s):
            return body(*args, s.cuda_stream)


def _act(t, name, like, shape, dtype=None):
    """Checks device, dtype and shape of a tensor (None passes)."""
    if t is None:
        return
    if t.device != like.device:
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}")
    if t.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must be {like.dtype if dtype is None else dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _strides(t, lead, name):
    """The ``lead`` leading strides of a tensor whose other dimensions are contiguous."""
    st, sh = t.stride(), t.shape
    exp = 1
    for d in range(len(sh) - 1, lead - 1, -1):
        if sh[d] != 1 and st[d] != exp:
            raise ValueError(f"{name}: the channel dimensions must be contiguous")
        exp *= sh[d]
    return st[:lead]


def _dense(t, name, like, shape, dtype):
    _act(t, name, like, shape, dtype)
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(workspace, need, like):
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=like.device)
    if workspace.device != like.device or workspace.dtype != torch.uint8 or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {like.device}")
    return workspace


# ------------------------------------------------------------ gated delta rule
def _delta_args(q, k, v, g, beta, y, y_name, scale, h0, h_final, cu_seqlens):
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k are [b, T, G, N] and v is [b, T, H, P]")
    a = _abi.DeltaArgs()
    b, T, H, P = v.shape
    G, N = q.shape[2], q.shape[3]
    _act(q, "q", v, (b, T, G, N))
    _act(k, "k", v, (b, T, G, N))
    _act(g, "g", v, (b, T, H), _f32)
    _act(beta, "beta", v, (b, T, H), _f32)
    _act(y, y_name, v, v.shape)
    nseq = b
    if cu_seqlens is not None:
        _dense(cu_seqlens, "cu_seqlens", v, (cu_seqlens.numel(),), _i32)
        nseq = cu_seqlens.numel() - 1
        a.nseqs, a.cu_seqlens = nseq, cu_seqlens.data_ptr()
    a.dtype = _dtype_code(v)
    a.batch, a.seqlen, a.nheads, a.headdim, a.ngroups, a.dstate = b, T, H, P, G, N
    a.q, (a.q_batch_stride, a.q_token_stride) = q.data_ptr(), _strides(q, 2, "q")
    a.k, (a.k_batch_stride, a.k_token_stride) = k.data_ptr(), _strides(k, 2, "k")
    a.v, (a.v_batch_stride, a.v_token_stride) = v.data_ptr(), _strides(v, 2, "v")
    a.g, (a.g_batch_stride, a.g_token_stride) = g.data_ptr(), _strides(g, 2, "g")
    a.beta, (a.beta_batch_stride, a.beta_token_stride) = beta.data_ptr(), _strides(beta, 2, "beta")
    a.y, (a.y_batch_stride, a.y_token_stride) = y.data_ptr(), _strides(y, 2, y_name)
    for t, n in ((h0, "h0"), (h_final, "h_final")):
        if t is not None:
            _dense(t, n, v, (nseq, H, P, N), _f32)
            setattr(a, n, t.data_ptr())
    a.scale = N ** -0.5 if scale is None else scale
    return a, nseq


def delta_fwd(q, k, v, g, beta, *, scale=None, h0=None, cu_seqlens=None, y=None, h_final=None,
              return_final_state=True, workspace=None, stream=None):
    """Gated delta rule over whole sequences: ``(y, h_final)``.

    Per head, ``h_t = a_t h_{t-1} + u_t k_t^T`` with ``a_t = exp(g_t)`` and
    ``u_t = beta_t (v_t - a_t h_{t-1} k_t)``; ``y_t = scale * h_t q_t`` (scale
    defaults to ``N ** -0.5``).  ``h_final`` is None when not requested.
    """
    def call(s):
        nonlocal y, h_final, workspace
        if y is None:
            y = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        if h_final is None and return_final_state:
            nseq = v.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            h_final = torch.empty((nseq, v.shape[2], v.shape[3], q.shape[3]), dtype=_f32, device=v.device)
        a, _ = _delta_args(q, k, v, g, beta, y, "y", scale, h0, h_final, cu_seqlens)
        l = _abi.lib()
        workspace = _workspace(workspace, int(l.ssm_delta_workspace_size(C.byref(a))), v)
        _abi.check(l.ssm_delta_fwd(C.byref(a), _p(workspace), workspace.numel(), s), "ssm_delta_fwd")
        return y, h_final

    return _run(v, stream, call)


def delta_bwd(q, k, v, g, beta, dy, *, scale=None, h0=None, cu_seqlens=None, dh_final=None, out=None,
              workspace=None, stream=None):
    """Gradients of ``sum(dy * y) + sum(dh_final * h_final)`` of :func:`delta_fwd`.

    Returns a dict of contiguous tensors: ``dq, dk, dv, dg, dbeta`` in v's dtype
    and ``dh0`` fp32 (always, also for ``h0=None``).  ``out`` (such a dict) is
    filled instead of allocating.
    """
    def call(s):
        nonlocal out, workspace
        b = _abi.DeltaBwdArgs()
        b.fwd, nseq = _delta_args(q, k, v, g, beta, dy, "dy", scale, h0, None, cu_seqlens)
        hshape = (nseq, v.shape[2], v.shape[3], q.shape[3])
        if out is None:
            new = lambda t: torch.empty(t.shape, dtype=v.dtype, device=v.device)
            out = dict(dq=new(q), dk=new(k), dv=new(v), dg=new(g), dbeta=new(beta),
                       dh0=torch.empty(hshape, dtype=_f32, device=v.device))
        b.dy, b.dy_batch_stride, b.dy_token_stride = _p(dy), b.fwd.y_batch_stride, b.fwd.y_token_stride
        _dense(dh_final, "dh_final", v, hshape, _f32)
        b.dh_final = _p(dh_final)
        for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
            _dense(out[n], n, v, t.shape, v.dtype)
            setattr(b, n, _p(out[n]))
        _dense(out.get("dh0"), "dh0", v, hshape, _f32)
        b.dh0 = _p(out.get("dh0"))
        l = _abi.lib()
        workspace = _workspace(workspace, int(l.ssm_delta_bwd_workspace_size(C.byref(b))), v)
        _abi.check(l.ssm_delta_bwd(C.byref(b), _p(workspace), workspace.numel(), s), "ssm_delta_bwd")
        return out

    return _run(v, stream, call)


def delta_update(state, q, k, v, g, beta, *, scale=None, state_batch_indices=None, y=None, stream=None):
    """One token of the gated delta rule per row, ``state [slots, H, P, N]`` fp32 updated in place; returns y.

    q, k ``[b, G, N]``; v, y ``[b, H, P]``; g, beta ``[b, H]`` fp32.  Row r
    uses slot ``state_batch_indices[r]`` (int32, distinct; r when None); a
    negative slot, or one past the pool, marks a padding row, whose y is 0.
    """
    def call(s):
        nonlocal y
        if v.dim() != 3 or q.dim() != 3 or state.dim() != 4:
            raise ValueError("q, k are [b, G, N], v is [b, H, P] and state is [slots, H, P, N]")
        if y is None:
            y = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        b, H, P = v.shape
        G, N = q.shape[1], q.shape[2]
        a = _abi.DeltaUpdateArgs()
        a.dtype = _dtype_code(v)
        a.scale = float(N ** -0.5 if scale is None else scale)
        a.batch, a.nheads, a.headdim, a.ngroups, a.dstate = b, H, P, G, N
        _dense(state, "state", v, (state.shape[0], H, P, N), _f32)
        a.state, a.nslots = _p(state), state.shape[0]
        _act(q, "q", v, (b, G, N))
        _act(k, "k", v, (b, G, N))
        _act(y, "y", v, (b, H, P))
        _act(g, "g", v, (b, H), _f32)
        _act(beta, "beta", v, (b, H), _f32)
        a.q, (a.q_batch_stride,) = q.data_ptr(), _strides(q, 1, "q")
        a.k, (a.k_batch_stride,) = k.data_ptr(), _strides(k, 1, "k")
        a.v, (a.v_batch_stride,) = v.data_ptr(), _strides(v, 1, "v")
        a.g, (a.g_batch_stride,) = g.data_ptr(), _strides(g, 1, "g")
        a.beta, (a.beta_batch_stride,) = beta.data_ptr(), _strides(beta, 1, "beta")
        a.y, (a.y_batch_stride,) = y.data_ptr(), _strides(y, 1, "y")
        if state_batch_indices is not None:
            _dense(state_batch_indices, "state_batch_indices", v, (b,), _i32)
        a.state_batch_indices = _p(state_batch_indices)
        _abi.check(_abi.lib().ssm_delta_update(C.byref(a), s), "ssm_delta_update")
        return y

    return _run(v, stream, call)


# ------------------------------------------------------------------ group norm
def _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y, y_name):
    if x.dim() not in (2, 3):
        raise ValueError("x is [tokens, C] or [b, T, C]")
    if z is not None and activation:
        raise ValueError("activation is for calls without a gate z")
    if z is None and gate_first:
        raise ValueError("gate_first needs a gate z")
    a = _abi.NormArgs()
    Cn = x.shape[-1]
    a.dtype = _dtype_code(x)
    a.mode = (_abi.SSM_NORM_SILU if activation else _abi.SSM_NORM_PLAIN) if z is None else \
        (_abi.SSM_NORM_GATE_FIRST if gate_first else _abi.SSM_NORM_GATE)
    a.subtract_mean, a.eps = int(bool(subtract_mean)), float(eps)
    a.batch, a.seqlen, a.channels, a.groups = (1 if x.dim() == 2 else x.shape[0]), x.shape[-2], Cn, int(groups)
    lead = x.dim() - 1
    a.x, (*bs, a.x_token_stride) = x.data_ptr(), _strides(x, lead, "x")
    if z is not None:
        _act(z, "z", x, x.shape)
        a.z, (*zs, a.z_token_stride) = z.data_ptr(), _strides(z, lead, "z")
    _act(y, y_name, x, x.shape)
    a.y, (*ys, a.y_token_stride) = y.data_ptr(), _strides(y, lead, y_name)
    if bs:
        a.x_batch_stride, a.y_batch_stride = bs[0], ys[0]
        if z is not None:
            a.z_batch_stride = zs[0]
    for t, n in ((weight, "weight"), (bias, "bias")):
        _dense(t, n, x, (Cn,), _f32)
        setattr(a, n, _p(t))
    return a


def group_norm_fwd(x, groups, *, weight=None, bias=None, z=None, subtract_mean=False, eps=1e-5, gate_first=False,
                   activation=False, y=None, stream=None):
    """Group norm of channels-last rows ``x [tokens, C]`` or ``[b, T, C]``, every token by itself.

    ``n`` is x normalised per group (root mean square, or mean and variance
    with ``subtract_mean``), ``t = n * weight + bias`` (fp32 ``[C]``).  Returns
    ``t``, ``silu(t)`` with ``activation``, ``t * silu(z)`` with a gate, or with
    ``gate_first`` the norm of ``x * silu(z)``.  ``y`` may be ``x``.
    """
    def call(s):
        nonlocal y
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        a = _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y, "y")
        _abi.check(_abi.lib().ssm_group_norm_fwd(C.byref(a), s), "ssm_group_norm_fwd")
        return y

    return _run(x, stream, call)


def group_norm_bwd(x, groups, dy, *, weight=None, bias=None, z=None, subtract_mean=False, eps=1e-5,
                   gate_first=False, activation=False, out=None, workspace=None, stream=None):
    """Gradients of ``sum(dy * y)`` of :func:`group_norm_fwd`: a dict with ``dx``,
    ``dz`` (None without a gate) in x's dtype and ``dweight``, ``dbias`` fp32 ``[C]``
    (also for weight / bias None, where they are 1 and 0).  ``out`` (such a dict) is
    filled instead of allocating; a None or missing dweight / dbias is not computed."""
    def call(s):
        nonlocal out, workspace
        b = _abi.NormBwdArgs()
        b.fwd = _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, dy, "dy")
        b.dy, b.dy_batch_stride, b.dy_token_stride = b.fwd.y, b.fwd.y_batch_stride, b.fwd.y_token_stride
        b.fwd.y = None
        Cn = x.shape[-1]
        if out is None:
            new = lambda: torch.empty(x.shape, dtype=x.dtype, device=x.device)
            par = lambda: torch.empty(Cn, dtype=_f32, device=x.device)
            out = dict(dx=new(), dz=None if z is None else new(), dweight=par(), dbias=par())
        for n, shape, dt in (("dx", x.shape, x.dtype), ("dz", x.shape, x.dtype), ("dweight", (Cn,), _f32),
                             ("dbias", (Cn,), _f32)):
            _dense(out.get(n), n, x, shape, dt)
            setattr(b, n, _p(out.get(n)))
        l = _abi.lib()
        workspace = _workspace(workspace, int(l.ssm_group_norm_bwd_workspace_size(C.byref(b))), x)
        _abi.check(l.ssm_group_norm_bwd(C.byref(b), _p(workspace), workspace.numel(), s), "ssm_group_norm_bwd")
        return out

    return _run(x, stream, call)


# ----------------------------------------------------------------- state pages
def _pages(pools, refs, src, pages, like, nslots):
    a = _abi.PagesArgs()
    a.nslots, a.n, a.npools = nslots, pages.numel(), len(pools)
    if len(pools) > _abi.SSM_MAX_POOLS:
        raise ValueError(f"at most {_abi.SSM_MAX_POOLS} pools")
    k = 0
    for i, p in enumerate(pools):
        if p.device != like.device or not p.is_contiguous() or p.dim() < 1 or p.shape[0] != nslots:
            raise ValueError(f"pool {i} must be a contiguous tensor of {nslots} pages on {like.device}")
        if p.numel() == 0:                        # pages without contents
            continue
        a.pools[k].base = _p(p)
        a.pools[k].page_bytes = p.numel() // nslots * p.element_size()
        k += 1
    a.npools = k
    for t, n in ((refs, "refs"), (src, "src"), (pages, "pages")):
        if t is None:
            continue
        _dense(t, n, like, (nslots,) if n == "refs" else (pages.numel(),), _i32)
        setattr(a, n, _p(t))
    return a


def _run_pages(what, pools, refs, src, pages, like, nslots, workspace, s):
    a = _pages(pools, refs, src, pages, like, nslots)
    l = _abi.lib()
    workspace = _workspace(workspace, int(l.ssm_pages_workspace_size(C.byref(a))), like)
    _abi.check(getattr(l, what)(C.byref(a), _p(workspace), workspace.numel(), s), what)


def _pool_rows(pools):
    if not pools:
        raise ValueError("at least one pool is needed")
    return pools[0].shape[0]


def state_pages_copy(pools, src, dst, *, workspace=None, stream=None):
    """Row ``src[i]`` of every pool to row ``dst[i]`` (int32; zeros for src -1, nothing for a negative dst).

    Entries whose dst an earlier entry writes or another entry reads are skipped
    and reported (``workspace_error(workspace)``)."""
    def call(s):
        _run_pages("ssm_pages_copy", pools, None, src, dst, dst, _pool_rows(pools), workspace, s)

    return _run(dst, stream, call)


def state_pages_fork(pools, refs, src, *, pages=None, workspace=None, stream=None):
    """A free page for every entry of ``src`` (int32), the lowest first, holding a copy of page ``src[i]``
    (zeros for -1): the page numbers, int32, -1 where none was left or the parent is not live.
    ``refs`` (int32 ``[slots]``, 0 = free) is updated."""
    def call(s):
        nonlocal pages
        if pages is None:
            pages = torch.empty(src.shape, dtype=_i32, device=src.device)
        _run_pages("ssm_pages_fork", pools, refs, src, pages, refs, refs.numel(), workspace, s)
        return pages

    return _run(refs, stream, call)


def state_pages_free(refs, pages, *, workspace=None, stream=None):
    """Give up one hold on each of ``pages`` (int32; negative entries are passed over)."""
    def call(s):
        _run_pages("ssm_pages_free", [], refs, None, pages, refs, refs.numel(), workspace, s)

    return _run(refs, stream, call)


def state_pages_compact(pools, refs, table, *, workspace=None, stream=None):
    """Move the live pages to the front of the pools (the i-th live page at or behind the live count to the
    i-th free page before it) and renumber ``refs`` and ``table`` (int32 page numbers) in place."""
    def call(s):
        _run_pages("ssm_pages_compact", pools, refs, None, table, refs, refs.numel(), workspace, s)


    return _run(refs, stream, call)