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
import struct

import torch

from . import _abi
from .ops import _dtype_code

_f32, _i32 = torch.float32, torch.int32
# torch's own quick forms of current_device and current_stream, where this torch has them (a CPU-only one does not)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)
_cur_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _packer(struct_type):
    """``pack(*values)`` of a ctypes structure's fields in order (0 for a NULL pointer): at one token a call is
    host-bound, and packing costs a fraction of assigning the fields one by one."""
    code = {C.c_int32: "i", C.c_int64: "q", C.c_void_p: "Q", C.c_float: "f"}

    def fmt(t):
        return "".join(code[f] if f in code else fmt(f) for _, f in t._fields_)

    st = struct.Struct("@" + fmt(struct_type) + "0q")
    if st.size != C.sizeof(struct_type):
        raise RuntimeError(f"{struct_type.__name__}: packed size differs")
    return st.pack


_pack_delta = _packer(_abi.DeltaArgs)
_pack_delta_bwd = _packer(_abi.DeltaBwdArgs)
_pack_update = _packer(_abi.DeltaUpdateArgs)
_pack_norm = _packer(_abi.NormArgs)
_pack_norm_bwd = _packer(_abi.NormBwdArgs)
_pack_pages = struct.Struct("@qqii" + "Qq" * _abi.SSM_MAX_POOLS + "QQQ0q").pack


def _run(t, stream, body, *args):
    """``body(*args, stream handle)`` with t's device current and allocations made on the stream the call runs on.
    The common case (current device, current stream) enters no context."""
    idx = t.get_device()
    if idx < 0:
        raise ValueError("expected a CUDA tensor")
    if stream is None and _cur_device and _cur_stream and idx == _cur_device():
        return body(*args, _cur_stream(idx))
    with torch.cuda.device(idx):
        s = torch.cuda.current_stream() if stream is None else stream
        if s.device != t.device:
            raise ValueError(f"stream is on {s.device}, the tensors on {t.device}")
        with torch.cuda.stream(s):
            return body(*args, s.cuda_stream)


def _act(t, name, idx, shape, dtype):
    """Checks device, dtype and shape of a tensor and gives its address (0 for None)."""
    if t is None:
        return 0
    if t.get_device() != idx:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{idx}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _dense(t, name, idx, shape, dtype):
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _act(t, name, idx, shape, dtype)


def _strides(t, lead, name):
    """The ``lead`` leading strides of a tensor whose other dimensions are contiguous."""
    st = t.stride()
    if not t.is_contiguous():
        sh, exp = t.shape, 1
        for d in range(len(sh) - 1, lead - 1, -1):
            if sh[d] != 1 and st[d] != exp:
                raise ValueError(f"{name}: the channel dimensions must be contiguous")
            exp *= sh[d]
    return st[:lead]


def _new(t, shape=None, dtype=None):
    """A dense tensor on t's device: t's shape and dtype unless given."""
    if shape is None and dtype is None and t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(t.shape if shape is None else shape, dtype=t.dtype if dtype is None else dtype, device=t.device)


def _workspace(workspace, need, like, idx):
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=like.device)
    if workspace.get_device() != idx or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{idx}")
    return workspace


# ------------------------------------------------------------ gated delta rule
def _check_dims(q, v):
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k are [b, T, G, N] and v is [b, T, H, P]")


def _delta_args(q, k, v, g, beta, y, y_name, scale, h0, h_final, cu_seqlens, gates_f32=0):
    """The fields of ``ssm_delta_args`` in order, and the number of sequences."""
    idx, dt = v.get_device(), v.dtype
    b, T, H, P = v.shape
    G, N = q.shape[2], q.shape[3]
    qk, gates = (b, T, G, N), (b, T, H)
    nseq, nseqs, cu = b, 0, 0
    if cu_seqlens is not None:
        nseq = nseqs = cu_seqlens.numel() - 1
        cu = _dense(cu_seqlens, "cu_seqlens", idx, (nseq + 1,), _i32)
    hshape = (nseq, H, P, N)
    return (_dtype_code(v), nseqs, b, T, H, P, G, N,
            _act(q, "q", idx, qk, dt), *_strides(q, 2, "q"), _act(k, "k", idx, qk, dt), *_strides(k, 2, "k"),
            v.data_ptr(), *_strides(v, 2, "v"),
            _act(g, "g", idx, gates, _f32), *_strides(g, 2, "g"),
            _act(beta, "beta", idx, gates, _f32), *_strides(beta, 2, "beta"),
            _act(y, y_name, idx, v.shape, dt), *_strides(y, 2, y_name),
            _dense(h0, "h0", idx, hshape, _f32), _dense(h_final, "h_final", idx, hshape, _f32), cu,
            N ** -0.5 if scale is None else scale, gates_f32), nseq


def delta_fwd(q, k, v, g, beta, *, scale=None, h0=None, cu_seqlens=None, y=None, h_final=None,
              return_final_state=True, workspace=None, stream=None):
    """Gated delta rule over whole sequences: ``(y, h_final)``.

    Per head, ``h_t = a_t h_{t-1} + u_t k_t^T`` with ``a_t = exp(g_t)`` and
    ``u_t = beta_t (v_t - a_t h_{t-1} k_t)``; ``y_t = scale * h_t q_t`` (scale
    defaults to ``N ** -0.5``).  ``h_final`` is None when not requested.
    """
    return _run(v, stream, _delta_fwd, q, k, v, g, beta, scale, h0, cu_seqlens, y, h_final, return_final_state,
                workspace)


def _delta_fwd(q, k, v, g, beta, scale, h0, cu_seqlens, y, h_final, return_final_state, workspace, s):
    _check_dims(q, v)
    if y is None:
        y = _new(v)
    if h_final is None and return_final_state:
        nseq = v.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        h_final = _new(v, (nseq, v.shape[2], v.shape[3], q.shape[3]), _f32)
    a = _pack_delta(*_delta_args(q, k, v, g, beta, y, "y", scale, h0, h_final, cu_seqlens)[0])
    l = _abi.lib()
    workspace = _workspace(workspace, l.ssm_delta_workspace_size(a), v, v.get_device())
    _abi.check(l.ssm_delta_fwd(a, workspace.data_ptr(), workspace.numel(), s), "ssm_delta_fwd")
    return y, h_final


def delta_bwd(q, k, v, g, beta, dy, *, scale=None, h0=None, cu_seqlens=None, dh_final=None, out=None,
              gate_dtype=None, workspace=None, stream=None):
    """Gradients of ``sum(dy * y) + sum(dh_final * h_final)`` of :func:`delta_fwd`.

    Returns a dict of contiguous tensors: ``dq, dk, dv, dg, dbeta`` in v's dtype
    and ``dh0`` fp32 (always, also for ``h0=None``).  ``gate_dtype=torch.float32``
    gives ``dg`` and ``dbeta`` in fp32, as the gates themselves are: for gradients
    that are added over the tokens.  ``out`` (such a dict) is filled instead of
    allocating.
    """
    return _run(v, stream, _delta_bwd, q, k, v, g, beta, dy, scale, h0, cu_seqlens, dh_final, out, gate_dtype, workspace)


def _delta_bwd(q, k, v, g, beta, dy, scale, h0, cu_seqlens, dh_final, out, gate_dtype, workspace, s):
    _check_dims(q, v)
    idx, dt = v.get_device(), v.dtype
    gdt = dt if gate_dtype is None else gate_dtype
    if gdt not in (dt, _f32):
        raise TypeError(f"gate_dtype must be {dt} or torch.float32, got {gdt}")
    fwd, nseq = _delta_args(q, k, v, g, beta, dy, "dy", scale, h0, None, cu_seqlens, 1 if gdt == _f32 else 0)
    hshape = (nseq, v.shape[2], v.shape[3], q.shape[3])
    if out is None:
        out = dict(dq=_new(v, q.shape), dk=_new(v, k.shape), dv=_new(v), dg=_new(v, g.shape, gdt),
                   dbeta=_new(v, beta.shape, gdt), dh0=_new(v, hshape, _f32))
    a = _pack_delta_bwd(*fwd, dy.data_ptr(), *_strides(dy, 2, "dy"), _dense(dh_final, "dh_final", idx, hshape, _f32),
                        _dense(out["dq"], "dq", idx, q.shape, dt), _dense(out["dk"], "dk", idx, k.shape, dt),
                        _dense(out["dv"], "dv", idx, v.shape, dt), _dense(out["dg"], "dg", idx, g.shape, gdt),
                        _dense(out["dbeta"], "dbeta", idx, beta.shape, gdt),
                        _dense(out.get("dh0"), "dh0", idx, hshape, _f32))
    l = _abi.lib()
    workspace = _workspace(workspace, l.ssm_delta_bwd_workspace_size(a), v, idx)
    _abi.check(l.ssm_delta_bwd(a, workspace.data_ptr(), workspace.numel(), s), "ssm_delta_bwd")
    return out


def delta_update(state, q, k, v, g, beta, *, scale=None, state_batch_indices=None, y=None, stream=None):
    """One token of the gated delta rule per row, ``state [slots, H, P, N]`` fp32 updated in place; returns y.

    q, k ``[b, G, N]``; v, y ``[b, H, P]``; g, beta ``[b, H]`` fp32.  Row r
    uses slot ``state_batch_indices[r]`` (int32, distinct; r when None); a
    negative slot, or one past the pool, marks a padding row, whose y is 0.
    """
    return _run(v, stream, _delta_update, state, q, k, v, g, beta, scale, state_batch_indices, y)


def _delta_update(state, q, k, v, g, beta, scale, state_batch_indices, y, s):
    if v.dim() != 3 or q.dim() != 3 or state.dim() != 4:
        raise ValueError("q, k are [b, G, N], v is [b, H, P] and state is [slots, H, P, N]")
    if y is None:
        y = _new(v)
    idx, dt = v.get_device(), v.dtype
    b, H, P = v.shape
    G, N = q.shape[1], q.shape[2]
    slots = state.shape[0]
    a = _pack_update(_dtype_code(v), 0, N ** -0.5 if scale is None else scale, 0, b, H, P, G, N,
                     _dense(state, "state", idx, (slots, H, P, N), _f32),
                     _act(q, "q", idx, (b, G, N), dt), *_strides(q, 1, "q"),
                     _act(k, "k", idx, (b, G, N), dt), *_strides(k, 1, "k"),
                     v.data_ptr(), *_strides(v, 1, "v"),
                     _act(g, "g", idx, (b, H), _f32), *_strides(g, 1, "g"),
                     _act(beta, "beta", idx, (b, H), _f32), *_strides(beta, 1, "beta"),
                     _act(y, "y", idx, v.shape, dt), *_strides(y, 1, "y"),
                     _dense(state_batch_indices, "state_batch_indices", idx, (b,), _i32), slots)
    _abi.check(_abi.lib().ssm_delta_update(a, s), "ssm_delta_update")
    return y


# ------------------------------------------------------------------ group norm
def _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y, y_name):
    """The fields of ``ssm_norm_args`` in order."""
    nd = x.dim()
    if nd != 2 and nd != 3:
        raise ValueError("x is [tokens, C] or [b, T, C]")
    if z is None:
        if gate_first:
            raise ValueError("gate_first needs a gate z")
        mode = _abi.SSM_NORM_SILU if activation else _abi.SSM_NORM_PLAIN
    else:
        if activation:
            raise ValueError("activation is for calls without a gate z")
        mode = _abi.SSM_NORM_GATE_FIRST if gate_first else _abi.SSM_NORM_GATE
    idx, dt, shape = x.get_device(), x.dtype, x.shape
    Cn = shape[-1]

    def rows(t, name):                       # address, batch stride, token stride
        if t is None:
            return 0, 0, 0
        st = _strides(t, nd - 1, name)
        return (_act(t, name, idx, shape, dt), *(st if nd == 3 else (0, *st)))

    return (_dtype_code(x), mode, 1 if subtract_mean else 0, eps, 1 if nd == 2 else shape[0], shape[-2], Cn, groups,
            *rows(x, "x"), *rows(z, "z"), *rows(y, y_name),
            _dense(weight, "weight", idx, (Cn,), _f32), _dense(bias, "bias", idx, (Cn,), _f32))


def group_norm_fwd(x, groups, *, weight=None, bias=None, z=None, subtract_mean=False, eps=1e-5, gate_first=False,
                   activation=False, y=None, stream=None):
    """Group norm of channels-last rows ``x [tokens, C]`` or ``[b, T, C]``, every token by itself: statistics are
    those of one token's group, not of the group over all positions as in ``torch.nn.GroupNorm``.

    ``n`` is x normalised per group (root mean square, or mean and variance
    with ``subtract_mean``), ``t = n * weight + bias`` (fp32 ``[C]``).  Returns
    ``t``, ``silu(t)`` with ``activation``, ``t * silu(z)`` with a gate, or with
    ``gate_first`` the norm of ``x * silu(z)``.  ``y`` may be ``x``.
    """
    return _run(x, stream, _group_norm_fwd, x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y)


def _group_norm_fwd(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y, s):
    if y is None:
        y = _new(x)
    a = _pack_norm(*_norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, y, "y"))
    _abi.check(_abi.lib().ssm_group_norm_fwd(a, s), "ssm_group_norm_fwd")
    return y


def group_norm_bwd(x, groups, dy, *, weight=None, bias=None, z=None, subtract_mean=False, eps=1e-5,
                   gate_first=False, activation=False, out=None, workspace=None, stream=None):
    """Gradients of ``sum(dy * y)`` of :func:`group_norm_fwd`: a dict with ``dx``,
    ``dz`` (None without a gate) in x's dtype and ``dweight``, ``dbias`` fp32 ``[C]``
    (also for weight / bias None, where they are 1 and 0).  ``out`` (such a dict) is
    filled instead of allocating; a None or missing dweight / dbias is not computed."""
    return _run(x, stream, _group_norm_bwd, x, groups, dy, weight, bias, z, subtract_mean, eps, gate_first, activation,
                out, workspace)


def _group_norm_bwd(x, groups, dy, weight, bias, z, subtract_mean, eps, gate_first, activation, out, workspace, s):
    fwd = _norm_args(x, groups, weight, bias, z, subtract_mean, eps, gate_first, activation, dy, "dy")
    idx, Cn = x.get_device(), x.shape[-1]
    if out is None:
        out = dict(dx=_new(x), dz=None if z is None else _new(x), dweight=_new(x, (Cn,), _f32),
                   dbias=_new(x, (Cn,), _f32))
    # fwd ends with y's address and strides (dy's here), weight, bias
    a = _pack_norm_bwd(*fwd, *fwd[-5:-2], _dense(out["dx"], "dx", idx, x.shape, x.dtype),
                       _dense(out.get("dz"), "dz", idx, x.shape, x.dtype),
                       _dense(out.get("dweight"), "dweight", idx, (Cn,), _f32),
                       _dense(out.get("dbias"), "dbias", idx, (Cn,), _f32))
    l = _abi.lib()
    workspace = _workspace(workspace, l.ssm_group_norm_bwd_workspace_size(a), x, idx)
    _abi.check(l.ssm_group_norm_bwd(a, workspace.data_ptr(), workspace.numel(), s), "ssm_group_norm_bwd")
    return out


# ----------------------------------------------------------------- state pages
def _pages(what, pools, refs, src, pages, like, nslots, workspace, s):
    idx, n = like.get_device(), pages.numel()
    if len(pools) > _abi.SSM_MAX_POOLS:
        raise ValueError(f"at most {_abi.SSM_MAX_POOLS} pools")
    rows = []
    for i, p in enumerate(pools):
        if p.get_device() != idx or not p.is_contiguous() or p.dim() < 1 or p.shape[0] != nslots:
            raise ValueError(f"pool {i} must be a contiguous tensor of {nslots} pages on cuda:{idx}")
        if p.numel():                             # (pages without contents need no copying)
            rows += (p.data_ptr(), p.nbytes // nslots)
    k = len(rows) // 2
    rows += (0,) * (2 * (_abi.SSM_MAX_POOLS - k))
    a = _pack_pages(nslots, n, k, 0, *rows, _dense(refs, "refs", idx, (nslots,), _i32),
                    _dense(src, "src", idx, (n,), _i32), _dense(pages, "pages", idx, (n,), _i32))
    l = _abi.lib()
    workspace = _workspace(workspace, l.ssm_pages_workspace_size(a), like, idx)
    _abi.check(getattr(l, what)(a, workspace.data_ptr(), workspace.numel(), s), what)
    return pages


def state_pages_copy(pools, src, dst, *, workspace=None, stream=None):
    """Row ``src[i]`` of every pool to row ``dst[i]`` (int32; zeros for src -1, nothing for a negative dst).

    Entries whose dst an earlier entry writes or another entry reads are skipped
    and reported (``workspace_error(workspace)``)."""
    if not pools:
        raise ValueError("at least one pool is needed")
    _run(dst, stream, _pages, "ssm_pages_copy", pools, None, src, dst, dst, pools[0].shape[0], workspace)


def state_pages_fork(pools, refs, src, *, pages=None, workspace=None, stream=None):
    """A free page for every entry of ``src`` (int32), the lowest first, holding a copy of page ``src[i]``
    (zeros for -1): the page numbers, int32, -1 where none was left or the parent is not live.
    ``refs`` (int32 ``[slots]``, 0 = free) is updated."""
    return _run(refs, stream, _fork, pools, refs, src, pages, workspace)


def _fork(pools, refs, src, pages, workspace, s):
    if pages is None:
        pages = _new(src, src.shape, _i32)
    return _pages("ssm_pages_fork", pools, refs, src, pages, refs, refs.numel(), workspace, s)


def state_pages_free(refs, pages, *, workspace=None, stream=None):
    """Give up one hold on each of ``pages`` (int32; negative entries are passed over)."""
    _run(refs, stream, _pages, "ssm_pages_free", (), refs, None, pages, refs, refs.numel(), workspace)


def state_pages_compact(pools, refs, table, *, workspace=None, stream=None):
    """Move the live pages to the front of the pools (the i-th live page at or behind the live count to the
    i-th free page before it) and renumber ``refs`` and ``table`` (int32 page numbers) in place."""
    _run(refs, stream, _pages, "ssm_pages_compact", pools, refs, None, table, refs, refs.numel(), workspace)
