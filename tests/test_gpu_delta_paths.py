"""The gated delta rule's paths that only larger calls take, each against the 64-bit form: the token-by-token kernels
of many rows, blocks enough for both stages of the chains' ring to be filled and emptied more than once, and a
pre-pass CTA that carries several heads of a group.  What decides the path is asserted with the call, so that a
change of a threshold does not silently drop it.

Tolerances as in test_gpu_delta.py.  Beside its largest error a bf16 result is bounded by its whole: rounding the
exact result once costs rho of its norm, and independent roundings add in squares, so n more bf16 factors in front
of the product that makes it allow sqrt(1 + n) rho: y 1 (the attention weights), dv none (1.1 rho for the rest),
dq, dk and dbeta 5.  States take no single bf16 factor: five products of two-part operands, 2^-17 each.
"""
import ctypes as C

import numpy as np
import pytest
import torch

import state_space_model_conv1d_b200 as ssm
from state_space_model_conv1d_b200 import _abi

from layer_ref import delta_bwd_ref, delta_ref
from test_gpu_delta import check_bwd, check_fwd, cu_of, make

pytestmark = pytest.mark.gpu
GATES = ("q", "k", "v", "g", "beta")


def up256(n):
    return -(-n // 256) * 256


# ------------------------------------------------------ many rows, token by token
def bwd_workspace(dtype, b, T, H, P, G, N):
    a = _abi.DeltaBwdArgs()
    f = a.fwd
    f.dtype, f.batch, f.seqlen, f.nheads, f.headdim, f.ngroups, f.dstate = _abi.SSM_BF16 if dtype == "bf16" else _abi.SSM_F32, b, T, H, P, G, N
    return _abi.lib().ssm_delta_bwd_workspace_size(C.byref(a))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [31, 32, 64, 70, 96, 128, 200, 256])
def test_many_rows(dtype, N):
    b, T, H, P, G = 3, 70, 12, 33, 4
    # a CTA of 32 rows makes ceil(33 / 32) = 2 shares of every sum, the form for few rows 5 or 9
    tok = b * T * H * 2 * 4
    many = 256 + up256(b * -(-T // 32) * H * P * N * 4) + 2 * up256(tok * N) + 2 * up256(tok)
    assert bwd_workspace(dtype, b, T, H, P, G, N) == many
    check_fwd(dtype, b, T, H, P, G, N, seed=N)
    check_bwd(dtype, b, T, H, P, G, N, seed=N + 1)


@pytest.mark.parametrize("dtype,N", [("f32", 64), ("bf16", 50), ("f32", 150)])
def test_many_rows_packed(dtype, N):
    lengths = [70, 0, 1, 33, 64, 0, 97]
    H, P, G, T = 12, 37, 3, sum([70, 0, 1, 33, 64, 0, 97])
    check_fwd(dtype, 1, T, H, P, G, N, lengths, seed=50)
    check_bwd(dtype, 1, T, H, P, G, N, lengths, seed=51)
    check_fwd(dtype, 1, T, H, P, G, N, lengths, seed=52, h0=False, scale=0.7, decay=30.0, views=True)
    check_bwd(dtype, 1, T, H, P, G, N, lengths, seed=53, h0=False, dh=False, decay=30.0, views=True)


# ------------------------------------------------------------------- many blocks
@pytest.mark.parametrize("P,N", [(64, 128), (128, 128), (128, 64), (192, 64), (24, 40)])
def test_many_blocks(P, N):
    T = 9 * 64 - 5                           # nine blocks: each stage of the ring is filled five times
    check_fwd("bf16", 1, T, 2, P, 1, N, seed=60)
    check_bwd("bf16", 1, T, 2, P, 1, N, seed=61)
    lengths = [460, 3, 0, 330, 64]
    check_fwd("bf16", 1, sum(lengths), 2, P, 1, N, lengths, seed=62, views=True)
    check_bwd("bf16", 1, sum(lengths), 2, P, 1, N, lengths, seed=63, views=True)


@pytest.mark.parametrize("shape,lengths", [((2, 300, 4, 128, 2, 128), None), ((1, 520, 4, 64, 1, 128), [200, 0, 70, 250]),
                                           ((2, 400, 3, 64, 3, 64), None)], ids=str)
def test_error_of_the_whole(shape, lengths):
    b, T, H, P, G, N = shape
    cu, cud = cu_of(lengths) if lengths else (None, None)
    dev, r = make(70, "bf16", *shape, nseq=len(lengths) if lengths else None)
    x, rx = [dev[n] for n in GATES], [r[n] for n in GATES]
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"], cu_seqlens=cud)
    d = ssm.delta_bwd(*x, dev["dy"], h0=dev["h0"], dh_final=dev["dh"], cu_seqlens=cud)
    ry, rh, _ = delta_ref(*rx, N ** -0.5, r["h0"], cu)
    want = delta_bwd_ref(*rx, N ** -0.5, r["dy"], r["dh"], r["h0"], cu)
    want |= dict(y=ry, hf=rh)
    got = d | dict(y=y, hf=hf)
    bound = dict(y=2 ** 0.5, dv=1.1, dq=6 ** 0.5, dk=6 ** 0.5, dbeta=6 ** 0.5)
    for n, w in want.items():
        if n == "dg":                        # (a difference of such sums: test_gpu_delta_gates.py)
            continue
        off = np.linalg.norm(got[n].double().cpu().numpy() - w) / np.linalg.norm(w)
        if n in ("hf", "dh0"):
            assert off <= 5 ** 0.5 * 2.0 ** -17, (n, off)
        else:
            once = torch.from_numpy(w).bfloat16().double().numpy()
            assert off <= bound[n] * np.linalg.norm(once - w) / np.linalg.norm(w), (n, off)


# ------------------------------------------------ several heads in a pre-pass CTA
@pytest.mark.parametrize("R,per_cta,nseqs", [(2, 2, 2700), (3, 3, 2700), (4, 4, 2700), (5, 5, 2700), (4, 2, 1700)])
def test_heads_of_a_group_share_a_prepass(R, per_cta, nseqs):
    lengths = [1, 0, 2, 1] * (nseqs // 4)
    lengths[5], lengths[100], lengths[nseqs - 2] = 70, 129, 64
    T = sum(lengths)
    # all heads of the group, or the largest divisor of them that leaves 16 CTAs for every SM
    slots, full = T // 64 + nseqs + 1, 16 * torch.cuda.get_device_properties(0).multi_processor_count
    assert max(n for n in range(1, R + 1) if n == 1 or (R % n == 0 and slots * (R // n) >= full)) == per_cta
    check_fwd("bf16", 1, T, R, 16, 1, 24, lengths, seed=R)
    check_bwd("bf16", 1, T, R, 16, 1, 24, lengths, seed=R + 1)
    check_fwd("bf16", 1, T, 2 * R, 64, 2, 72, lengths, seed=R + 2)
