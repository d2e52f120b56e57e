"""The operators beside the scan on the host: structure layouts, workspace sizes
and every refusal that needs no GPU (nothing here is launched)."""
import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

import state_space_model_conv1d_b200 as ssm
from state_space_model_conv1d_b200 import _abi, layer_ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000000  # never dereferenced: every call below is rejected on the host, or has no work
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (_abi.SSM_ERR_INVALID_ARG, _abi.SSM_ERR_UNSUPPORTED, _abi.SSM_ERR_ALIGNMENT,
                                              _abi.SSM_ERR_WORKSPACE)
STRUCTS = (("ssm_delta_args", _abi.DeltaArgs), ("ssm_delta_bwd_args", _abi.DeltaBwdArgs),
           ("ssm_delta_update_args", _abi.DeltaUpdateArgs), ("ssm_norm_args", _abi.NormArgs),
           ("ssm_norm_bwd_args", _abi.NormBwdArgs), ("ssm_page_pool", _abi.PagePool), ("ssm_pages_args", _abi.PagesArgs))


def test_struct_layouts_match_header(tmp_path):
    lines = "".join(f'printf("{c} sizeof %zu\\n", sizeof({c}));' +
                    "".join(f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_) for c, py in STRUCTS)
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "ssm.h"\nint main(void){{{lines}return 0;}}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {(c, f): int(v) for c, f, v in (l.split() for l in out.splitlines())}
    for c, py in STRUCTS:
        assert got[c, "sizeof"] == C.sizeof(py), c
        for f, _ in py._fields_:
            assert got[c, f] == getattr(py, f).offset, (c, f)


def test_import_without_torchs_private_cuda_names():
    # a torch without CUDA lacks them; importing the package looks nothing up
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import state_space_model_conv1d_b200 as ssm\n"
            "assert callable(ssm.delta_fwd) and callable(ssm.scan_fwd)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _fill(a, values, at=0):
    for name, t in a._fields_:
        if hasattr(t, "_fields_"):
            at = _fill(getattr(a, name), values, at)
        else:
            setattr(a, name, values[at])
            at += 1
    return at


@pytest.mark.parametrize("pack,py", [(layer_ops._pack_delta, _abi.DeltaArgs), (layer_ops._pack_delta_bwd, _abi.DeltaBwdArgs),
                                     (layer_ops._pack_update, _abi.DeltaUpdateArgs), (layer_ops._pack_norm, _abi.NormArgs),
                                     (layer_ops._pack_norm_bwd, _abi.NormBwdArgs)])
def test_packed_structures_equal_the_ctypes_ones(pack, py):
    a = py()
    n = _fill(a, range(1, 200))
    assert pack(*range(1, n + 1)) == bytes(a)


def test_packed_pages_equal_the_ctypes_ones():
    a = _abi.PagesArgs(1, 2, 3, 0)
    for i in range(_abi.SSM_MAX_POOLS):
        a.pools[i].base, a.pools[i].page_bytes = 10 + 2 * i, 11 + 2 * i
    a.refs, a.src, a.pages = 40, 41, 42
    assert layer_ops._pack_pages(1, 2, 3, 0, *range(10, 10 + 2 * _abi.SSM_MAX_POOLS), 40, 41, 42) == bytes(a)


def _set(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _delta(**kw):
    a = _abi.DeltaArgs()
    a.dtype, a.batch, a.seqlen, a.nheads, a.headdim, a.ngroups, a.dstate, a.scale = _abi.SSM_BF16, 2, 100, 4, 64, 2, 128, 1.0
    for k, w in dict(q=256, k=256, v=256, g=4, beta=4, y=256).items():
        setattr(a, k, FAKE)
        setattr(a, k + "_token_stride", w)
        setattr(a, k + "_batch_stride", w * 100)
    return _set(a, kw)


DELTA_BAD = [
    (dict(dtype=9), INVALID), (dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID),
    (dict(nheads=0), INVALID), (dict(headdim=0), INVALID), (dict(dstate=0), INVALID), (dict(ngroups=3), INVALID),
    (dict(dstate=257), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(nheads=1 << 21), UNSUPPORTED),
    (dict(headdim=1 << 21), UNSUPPORTED), (dict(seqlen=1 << 31), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
    (dict(beta=None), INVALID), (dict(y=None), INVALID),
    (dict(q=FAKE + 1), ALIGNMENT), (dict(g=FAKE + 2), ALIGNMENT), (dict(h0=FAKE + 2), ALIGNMENT),
    (dict(cu_seqlens=FAKE + 2, nseqs=1, batch=1), ALIGNMENT),
    (dict(v_token_stride=255), INVALID), (dict(beta_batch_stride=399), INVALID), (dict(k_token_stride=-256), INVALID),
    (dict(cu_seqlens=FAKE, nseqs=2), INVALID),                     # packed sequences are one row
    (dict(cu_seqlens=FAKE, nseqs=0, batch=1), INVALID), (dict(cu_seqlens=FAKE, nseqs=-1, batch=1), INVALID),
    (dict(cu_seqlens=FAKE, nseqs=65536, batch=1), INVALID),
    (dict(), WORKSPACE),
]


@pytest.mark.parametrize("kw,status", DELTA_BAD, ids=str)
def test_delta_rejects(kw, status):
    lib = _abi.lib()
    assert lib.ssm_delta_fwd(C.byref(_delta(**kw)), None, 0, None) == status
    b = _abi.DeltaBwdArgs()
    b.fwd = _delta(**kw)
    b.dy, b.dy_batch_stride, b.dy_token_stride = b.fwd.y, b.fwd.y_batch_stride, b.fwd.y_token_stride
    b.fwd.y = None                                                 # (ignored)
    b.dq = b.dk = b.dv = b.dg = b.dbeta = FAKE
    assert lib.ssm_delta_bwd(C.byref(b), None, 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID), (dict(dg=None), INVALID),
    (dict(dbeta=None), INVALID), (dict(dy=None), INVALID), (dict(dk=FAKE + 1), ALIGNMENT), (dict(dh0=FAKE + 2), ALIGNMENT),
    (dict(dh_final=FAKE + 2), ALIGNMENT), (dict(dy_token_stride=4), INVALID), (dict(dh0=None), WORKSPACE)], ids=str)
def test_delta_bwd_rejects(kw, status):
    b = _abi.DeltaBwdArgs()
    b.fwd = _delta()
    b.dy, b.dy_batch_stride, b.dy_token_stride = FAKE, 25600, 256
    b.dq = b.dk = b.dv = b.dg = b.dbeta = b.dh0 = FAKE
    assert _abi.lib().ssm_delta_bwd(C.byref(_set(b, kw)), None, 0, None) == status


@pytest.mark.parametrize("flag,dg,status", [(0, FAKE + 2, WORKSPACE), (1, FAKE + 2, ALIGNMENT), (1, FAKE + 4, WORKSPACE),
                                            (2, FAKE, INVALID), (-1, FAKE, INVALID)])
def test_delta_bwd_gates_f32(flag, dg, status):
    b = _abi.DeltaBwdArgs()
    b.fwd = _delta(gates_f32=flag)
    b.dy, b.dy_batch_stride, b.dy_token_stride = FAKE, 25600, 256
    b.dq = b.dk = b.dv = b.dh0 = FAKE
    for name in ("dg", "dbeta"):
        b.dg = b.dbeta = FAKE
        setattr(b, name, dg)
        assert _abi.lib().ssm_delta_bwd(C.byref(b), None, 0, None) == status


def test_delta_workspace():
    lib = _abi.lib()
    size = lambda **kw: lib.ssm_delta_workspace_size(C.byref(_delta(**kw)))
    # tensor cores: T in two parts and the attention weights of 2 x 2 blocks, 4 heads, behind the error word
    assert size() - size(dtype=_abi.SSM_F32) == 2 * 2 * 4 * 3 * 8192
    assert size(q=None, v=FAKE + 2) == size()                      # shapes alone
    assert size(dtype=_abi.SSM_F32, cu_seqlens=FAKE, batch=1, nseqs=1000) >= 256 + 4 * 1000
    assert size(dstate=0) == 0 and size(nheads=-1) == 0 and lib.ssm_delta_workspace_size(None) == 0
    need = size()
    a = _delta()
    assert lib.ssm_delta_fwd(C.byref(a), FAKE, need - 1, None) == WORKSPACE
    assert lib.ssm_delta_fwd(C.byref(a), FAKE + 16, need, None) == WORKSPACE
    assert lib.ssm_delta_bwd_workspace_size(None) == 0


def _update(**kw):
    a = _abi.DeltaUpdateArgs()
    a.dtype, a.scale, a.batch, a.nheads, a.headdim, a.ngroups, a.dstate, a.nslots = _abi.SSM_F32, 1.0, 3, 4, 8, 2, 16, 5
    a.state = FAKE
    for k, w in dict(q=32, k=32, v=32, g=4, beta=4, y=32).items():
        setattr(a, k, FAKE)
        setattr(a, k + "_batch_stride", w)
    return _set(a, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), INVALID), (dict(batch=-1), INVALID), (dict(nslots=-1), INVALID), (dict(ngroups=3), INVALID),
    (dict(nheads=0), INVALID), (dict(dstate=257), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
    (dict(state=None), INVALID), (dict(q=None), INVALID), (dict(y=None), INVALID), (dict(beta=None), INVALID),
    (dict(nslots=2), INVALID),                                     # rows without a slot table need a slot each
    (dict(v_batch_stride=31), INVALID), (dict(g_batch_stride=3), INVALID), (dict(k_batch_stride=-32), INVALID),
    (dict(state=FAKE + 4), ALIGNMENT), (dict(v=FAKE + 2), ALIGNMENT), (dict(state_batch_indices=FAKE + 2), ALIGNMENT),
    (dict(batch=0), _abi.SSM_OK)], ids=str)
def test_update_rejects(kw, status):
    assert _abi.lib().ssm_delta_update(C.byref(_update(**kw)), None) == status


def _norm(**kw):
    a = _abi.NormArgs()
    a.dtype, a.mode, a.eps, a.batch, a.seqlen, a.channels, a.groups = _abi.SSM_BF16, _abi.SSM_NORM_GATE, 1e-5, 2, 5, 64, 4
    for k in "xzy":
        setattr(a, k, FAKE)
        setattr(a, k + "_token_stride", 64)
        setattr(a, k + "_batch_stride", 320)
    return _set(a, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), INVALID), (dict(mode=4), INVALID), (dict(mode=-1), INVALID), (dict(subtract_mean=2), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(groups=3), INVALID), (dict(groups=0), INVALID),
    (dict(channels=0), INVALID), (dict(batch=-1), INVALID), (dict(z=None), INVALID),
    (dict(mode=_abi.SSM_NORM_SILU), INVALID),                      # a gate without a mode that uses it
    (dict(channels=16385 * 2, groups=2, x_token_stride=40000, y_token_stride=40000, z_token_stride=40000), UNSUPPORTED),
    (dict(batch=1 << 16, seqlen=1 << 16), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=FAKE + 1), ALIGNMENT), (dict(z=FAKE + 1), ALIGNMENT), (dict(weight=FAKE + 2), ALIGNMENT),
    (dict(x_token_stride=63), INVALID), (dict(z_batch_stride=319), INVALID), (dict(batch=0), _abi.SSM_OK)], ids=str)
def test_norm_rejects(kw, status):
    lib = _abi.lib()
    assert lib.ssm_group_norm_fwd(C.byref(_norm(**kw)), None) == status
    if status == _abi.SSM_OK:
        return
    b = _abi.NormBwdArgs()
    b.fwd = _norm(**kw)
    b.dy, b.dy_batch_stride, b.dy_token_stride, b.dx, b.dz = FAKE, b.fwd.y_batch_stride, b.fwd.y_token_stride, FAKE, FAKE
    assert lib.ssm_group_norm_bwd(C.byref(b), None, 0, None) == status


@pytest.mark.parametrize("kw,status", [(dict(dx=None), INVALID), (dict(dz=None), INVALID), (dict(dy=None), INVALID),
                                       (dict(dx=FAKE + 1), ALIGNMENT), (dict(dbias=FAKE + 2), ALIGNMENT),
                                       (dict(), WORKSPACE)], ids=str)
def test_norm_bwd_rejects(kw, status):
    b = _abi.NormBwdArgs()
    b.fwd = _norm()
    b.dy, b.dy_batch_stride, b.dy_token_stride, b.dx, b.dz, b.dweight, b.dbias = FAKE, 320, 64, FAKE, FAKE, FAKE, FAKE
    assert _abi.lib().ssm_group_norm_bwd(C.byref(_set(b, kw)), None, 0, None) == status


def _pages(**kw):
    a = _abi.PagesArgs(8, 3, 2, 0)
    for i in range(2):
        a.pools[i].base, a.pools[i].page_bytes = FAKE, 64
    a.refs = a.src = a.pages = FAKE
    bytes0 = kw.pop("page_bytes", None)
    if bytes0 is not None:
        a.pools[1].page_bytes = bytes0
    if kw.pop("no_base", False):
        a.pools[1].base = None
    return _set(a, kw)


CALLS = ("copy", "fork", "free", "compact")


@pytest.mark.parametrize("kw,status,calls", [
    (dict(nslots=-1), INVALID, CALLS), (dict(n=-1), INVALID, CALLS), (dict(npools=-1), INVALID, CALLS),
    (dict(npools=9), UNSUPPORTED, CALLS), (dict(nslots=(1 << 20) + 1), UNSUPPORTED, CALLS),
    (dict(refs=None), INVALID, CALLS[1:]), (dict(src=None), INVALID, CALLS[:2]), (dict(pages=None), INVALID, CALLS),
    (dict(pages=FAKE + 2), ALIGNMENT, CALLS), (dict(page_bytes=0), INVALID, CALLS), (dict(no_base=True), INVALID, CALLS),
    (dict(page_bytes=1 << 60), UNSUPPORTED, CALLS), (dict(), WORKSPACE, CALLS)], ids=str)
def test_pages_reject(kw, status, calls):
    lib = _abi.lib()
    for c in calls:
        assert getattr(lib, "ssm_pages_" + c)(C.byref(_pages(**kw)), None, 0, None) == status, c
    a = _pages()
    need = lib.ssm_pages_workspace_size(C.byref(a))
    assert need >= 256 and lib.ssm_pages_fork(C.byref(a), FAKE, need - 1, None) == WORKSPACE
    assert lib.ssm_pages_workspace_size(C.byref(_pages(n=-1))) == 0


def test_null_arguments():
    lib = _abi.lib()
    for f in ("ssm_delta_fwd", "ssm_delta_bwd", "ssm_group_norm_bwd", *("ssm_pages_" + c for c in CALLS)):
        assert getattr(lib, f)(None, None, 0, None) == INVALID, f
    assert lib.ssm_delta_update(None, None) == lib.ssm_group_norm_fwd(None, None) == INVALID
    assert lib.ssm_group_norm_bwd_workspace_size(None) == lib.ssm_pages_workspace_size(None) == 0


def test_host_tensors_are_refused():
    x = torch.zeros(1, 2, 2, 8)
    g = torch.zeros(1, 2, 2)
    r = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ssm.delta_fwd(x, x, x, g, g), lambda: ssm.delta_bwd(x, x, x, g, g, x),
                 lambda: ssm.delta_update(x, x[0], x[0], x[0], g[0], g[0]), lambda: ssm.group_norm_fwd(x[0], 1),
                 lambda: ssm.group_norm_bwd(x[0], 1, x[0]), lambda: ssm.state_pages_copy([x[0]], r, r),
                 lambda: ssm.state_pages_fork([x[0]], r, r), lambda: ssm.state_pages_free(r, r),
                 lambda: ssm.state_pages_compact([x[0]], r, r)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="pool"):
        ssm.state_pages_copy([], r, r)
