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

import contextlib
import ctypes as C

import torch

from . import _abi
from .ops import _dtype_code, _p, _rows


@contextlib.contextmanager
def _on(t, stream):
    """Device of ``t`` current, allocations on the stream the call runs on; yields the stream handle."""
    with torch.cuda.device(t.device):
        s = torch.cuda.current_stream() if stream is None else stream
        if s.device != t.device:
            raise ValueError(f"stream is on {s.device}, the tensors on {t.device}")
        with torch.cuda.stream(s):
            yield C.c_void_p(s.cuda_stream)


def _act(t, name, like, shape, dtype=None):
    """Checks device, dtype and shape of a tensor (None passes)."""
    if t is None:
        return
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}")
    if t.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must be {like.dtype if dtype is None else dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _dense(t, name, like, shape, dtype):
    _act(t, name, like, shape, dtype)
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(workspace, need, like):
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=like.device)
    if not workspace.is_cuda or workspace.device != like.device or workspace.dtype != torch.uint8 or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {like.device}")
    return workspace


# ------------------------------------------------------------ gated delta rule
def _delta_args(q, k, v, g, beta, y, y_name, scale, h0, h_final, cu_seqlens):
    if not v.is_cuda:
        raise ValueError("v must be a CUDA tensor")
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k are [b, T, G, N] and v is [b, T, H, P]")
    a = _abi.DeltaArgs()
    b, T, H, P = v.shape
    G, N = q.shape[2], q.shape[3]
    for t, n in ((q, "q"), (k, "k")):
        _act(t, n, v, (b, T, G, N))
    for t, n in ((g, "g"), (beta, "beta")):
        _act(t, n, v, (b, T, H), torch.float32)
    _act(y, y_name, v, v.shape)
    nseq = b
    if cu_seqlens is not None:
        _dense(cu_seqlens, "cu_seqlens", v, (cu_seqlens.numel(),), torch.int32)
        nseq = cu_seqlens.numel() - 1
    a.dtype, a.nseqs = _dtype_code(v), 0 if cu_seqlens is None else nseq
    a.batch, a.seqlen, a.nheads, a.headdim, a.ngroups, a.dstate = b, T, H, P, G, N
    for t, n, inner in ((q, "q", 2), (k, "k", 2), (v, "v", 2), (g, "g", 1), (beta, "beta", 1)):
        setattr(a, n, _p(t))
        bs, ts = _rows(t, inner, n)
        setattr(a, n + "_batch_stride", bs)
        setattr(a, n + "_token_stride", ts)
    a.y = _p(y)
    a.y_batch_stride, a.y_token_stride = _rows(y, 2, y_name)
    for t, n in ((h0, "h0"), (h_final, "h_final")):
        _dense(t, n, v, (nseq, H, P, N), torch.float32)
        setattr(a, n, _p(t))
    a.cu_seqlens = _p(cu_seqlens)
    a.scale = float(N ** -0.5 if scale is None else scale)
    return a, nseq


def delta_fwd(q, k, v, g, beta, *, scale=None, h0=None, cu_seqlens=None, y=None, h_final=None,
              return_final_state=True, workspace=None, stream=None):
    """Gated delta rule over whole sequences: ``(y, h_final)``.

    Per head, ``h_t = a_t h_{t-1} + u_t k_t^T`` with ``a_t = exp(g_t)`` and
    ``u_t = beta_t (v_t - a_t h_{t-1} k_t)``; ``y_t = scale * h_t q_t`` (scale
    defaults to ``N ** -0.5``).  ``h_final`` is None when not requested.
    """
    with _on(v, stream) as s:
        if y is None:
            y = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        if h_final is None and return_final_state:
            nseq = v.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            h_final = torch.empty((nseq, v.shape[2], v.shape[3], q.shape[3]), dtype=torch.float32, device=v.device)
        a, _ = _delta_args(q, k, v, g, beta, y, "y", scale, h0, h_final, cu_seqlens)
        l = _abi.lib()
        workspace = _workspace(workspace, int(l.ssm_delta_workspace_size(C.byref(a))), v)
        _abi.check(l.ssm_delta_fwd(C.byref(a), _p(workspace), workspace.numel(), s), "ssm_delta_fwd")
    return y, h_final


def delta_bwd(q, k, v, g, beta, dy, *, scale=None, h0=None, cu_seqlens=None, dh_final=None, out=None,
              workspace=None, stream=None):
    """Gradients of ``sum(dy * y) + sum(dh_final * h_final)`` of :func:`delta_fwd`.

    Returns a dict of contiguous tensors: ``dq, dk, dv, dg, dbeta`` in v's dtype
    and ``dh0`` fp32 (always, also for ``h0=None``).  ``out`` (such a dict) is
    filled instead of allocating.
    """
    with _on(v, stream) as s:
        b = _abi.DeltaBwdArgs()
        b.fwd, nseq = _delta_args(q, k, v, g, beta, dy, "dy", scale, h0, None, cu_seqlens)
        hshape = (nseq, v.shape[2], v.shape[3], q.shape[3])
        if out is None:
            new = lambda t: torch.empty(t.shape, dtype=v.dtype, device=v.device)
            out = dict(dq=new(q), dk=new(k), dv=new(v), dg=new(g), dbeta=new(beta),
                       dh0=torch.empty(hshape, dtype=torch.float32, device=v.device))
        b.dy, b.dy_batch_stride, b.dy_token_stride = _p(dy), b.fwd.y_batch_stride, b.fwd.y_token_stride
        _dense(dh_final, "dh_final", v, hshape, torch.float32)
        b.dh_final = _p(dh_final)
        for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
            _dense(out[n], n, v, t.shape, v.dtype)
            setattr(b, n, _p(out[n]))
        _dense(out.get("dh0"), "dh0", v, hshape, torch.float32)
        b.dh0 = _p(out.get("dh0"))
        l = _abi.lib()
        workspace = _workspace(workspace, int(l.ssm_delta_bwd_workspace_size(C.byref(b))), v)
        _abi.check(l.ssm_delta_bwd(C.byref(b), _p(workspace), workspace.numel(), s), "ssm_delta_bwd")
    return out


def delta_update(state, q, k, v, g, beta, *, scale=None, state_batch_indices=None, y=None, stream=None):
    """One token of the gated delta rule per row, ``state [slots, H, P, N]`` fp32 updated in place; returns y.

    q, k ``[b, G, N]``; v, y ``[b, H, P]``; g, beta ``[b, H]`` fp32.  Row r
    uses slot ``state_batch_indices[r]`` (int32, distinct; r when None); a
    negative slot, or one past the pool, marks a padding row, whose y is 0.
    """
    with _on(v, stream) as s:
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
        _dense(state, "state", v, (state.shape[0], H, P, N), torch.float32)
        a.state, a.nslots = _p(state), state.shape[0]
        for t, n, shape, dt in ((q, "q", (b, G, N), None), (k, "k", (b, G, N), None), (v, "v", (b, H, P), None),
                                (y, "y", (b, H, P), None), (g, "g", (b, H), torch.float32),
                                (beta, "beta", (b, H), torch.float32)):
            _act(t, n, v, shape, dt)
            setattr(a, n, _p(t))
            setattr(a, n + "_batch_stride", _rows(t.unsqueeze(1), len(shape) - 1, n)[0])
        if state_batch_indices is not None:
            _dense(state_batch_indices, "state_batch_indices", v, (b,), torch.int32)
        a.state_batch_indices = _p(state_batch_indices)
        _abi.check(_abi.lib().ssm_delta_update(C.byref(a), s), "ssm_delta_update")
    return y


# ------------------------------------------------------------------ group norm
def _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y, y_name):
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
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
    for t, n, f in ((x, "x", "x"), (z, "z", "z"), (y, y_name, "y")):
        _act(t, n, x, x.shape)
        if t is None:
            continue
        setattr(a, f, _p(t))
        bs, ts = _rows(t.unsqueeze(0) if t.dim() == 2 else t, 1, n)
        setattr(a, f + "_batch_stride", 0 if t.dim() == 2 else bs)
        setattr(a, f + "_token_stride", ts)
    for t, n in ((weight, "weight"), (bias, "bias")):
        _dense(t, n, x, (Cn,), torch.float32)
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
    with _on(x, stream) as s:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        a = _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y, "y")
        _abi.check(_abi.lib().ssm_group_norm_fwd(C.byref(a), s), "ssm_group_norm_fwd")
    return y


def group_norm_bwd(x, groups, dy, *, weight=None, bias=None, z=None, subtract_mean=False, eps=1e-5,
                   gate_first=False, activation=False, out=None, workspace=None, stream=None):
    """Gradients of ``sum(dy * y)`` of :func:`group_norm_fwd`: a dict with ``dx``,
    ``dz`` (None without a gate) in x's dtype and ``dweight``, ``dbias`` fp32 ``[C]``
    (also for weight / bias None, where they are 1 and 0).  ``out`` (such a dict) is
    filled instead of allocating; a None or missing dweight / dbias is not computed."""
    with _on(x, stream) as s:
        b = _abi.NormBwdArgs()
        b.fwd = _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, dy, "dy")
        b.dy, b.dy_batch_stride, b.dy_token_stride = b.fwd.y, b.fwd.y_batch_stride, b.fwd.y_token_stride
        b.fwd.y = None
        Cn = x.shape[-1]
        if out is None:
            new = lambda: torch.empty(x.shape, dtype=x.dtype, device=x.device)
            par = lambda: torch.empty(Cn, dtype=torch.float32, device=x.device)
            out = dict(dx=new(), dz=None if z is None else new(), dweight=par(), dbias=par())
        for n, shape, dt in (("dx", x.shape, x.dtype), ("dz", x.shape, x.dtype), ("dweight", (Cn,), torch.float32),
                             ("dbias", (Cn,), torch.float32)):
            _dense(out.get(n), n, x, shape, dt)
            setattr(b, n, _p(out.get(n)))
        l = _abi.lib()
        workspace = _workspace(workspace, int(l.ssm_group_norm_bwd_workspace_size(C.byref(b))), x)
        _abi.check(l.ssm_group_norm_bwd(C.byref(b), _p(workspace), workspace.numel(), s), "ssm_group_norm_bwd")
    return out


# ----------------------------------------------------------------- state pages
def _pages(pools, refs, src, pages, like, nslots):
    a = _abi.PagesArgs()
    a.nslots, a.n, a.npools = nslots, pages.numel(), len(pools)
    if len(pools) > _abi.SSM_MAX_POOLS:
        raise ValueError(f"at most {_abi.SSM_MAX_POOLS} pools")
    k = 0
    for i, p in enumerate(pools):
        if not p.is_cuda or p.device != like.device or not p.is_contiguous() or p.dim() < 1 or p.shape[0] != nslots:
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
        _dense(t, n, like, (nslots,) if n == "refs" else (pages.numel(),), torch.int32)
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
    with _on(dst, stream) as s:
        _run_pages("ssm_pages_copy", pools, None, src, dst, dst, _pool_rows(pools), workspace, s)


def state_pages_fork(pools, refs, src, *, pages=None, workspace=None, stream=None):
    """A free page for every entry of ``src`` (int32), the lowest first, holding a copy of page ``src[i]``
    (zeros for -1): the page numbers, int32, -1 where none was left or the parent is not live.
    ``refs`` (int32 ``[slots]``, 0 = free) is updated."""
    with _on(refs, stream) as s:
        if pages is None:
            pages = torch.empty(src.shape, dtype=torch.int32, device=src.device)
        _run_pages("ssm_pages_fork", pools, refs, src, pages, refs, refs.numel(), workspace, s)
    return pages


def state_pages_free(refs, pages, *, workspace=None, stream=None):
    """Give up one hold on each of ``pages`` (int32; negative entries are passed over)."""
    with _on(refs, stream) as s:
        _run_pages("ssm_pages_free", [], refs, None, pages, refs, refs.numel(), workspace, s)


def state_pages_compact(pools, refs, table, *, workspace=None, stream=None):
    """Move the live pages to the front of the pools (the i-th live page at or behind the live count to the
    i-th free page before it) and renumber ``refs`` and ``table`` (int32 page numbers) in place."""
    with _on(refs, stream) as s:
        _run_pages("ssm_pages_compact", pools, refs, None, table, refs, refs.numel(), workspace, s)
