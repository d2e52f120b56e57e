"""Strong decays and resets of the gated delta rule: the gradient of each gate on the scale of its own token.

dg_t = <d, a_t h_{t-1}> (d the gradient that reaches a_t h_{t-1}), so a token that forgets has a gradient as small
as its a_t.  Bounds, per token and head:

- token by token in fp32: 2e-5 |d| |a_t h_{t-1}| (the bound of test_gpu_delta.py for gradients);
- in blocks: every term that does not cancel holds a_t and at most five factors rounded to bf16, 6 * 2^-8
  |d| |a_t h_{t-1}|, the result's own rounding among them; the others cancel between dq . q and dk . k of the tokens
  from t to the block's end up to fp32 sums: 16 random roundings of 2^-24 (products of 128 terms, their dot product
  with q or k of 128 more) of terms that are at most four times their sum, 2 |dq| + 3 |dk| a token (unit q and k),
  over the block's 64 tokens.
"""
import numpy as np
import pytest
import torch

import state_space_model_conv1d_b200 as ssm

from layer_ref import HALF, delta_bwd_ref, delta_ref
from test_gpu_delta import make

pytestmark = pytest.mark.gpu
GATES = ("q", "k", "v", "g", "beta")


def f64(t):
    return t.double().cpu().numpy()


def gate_norms(r, dy, dh, h0, scale):
    """|d| |a_t h_{t-1}| of every token and head of one row whose heads share no keys."""
    _, _, ((_, _, _, path),) = delta_ref(*[r[n] for n in GATES], scale, h0)
    d, out = dh[0].copy(), np.zeros(r["g"].shape[1:])
    for t in reversed(range(len(path))):
        w = path[t][0]
        kt = r["k"][0, t]
        d = d + scale * dy[0, t][..., None] * r["q"][0, t][:, None]
        ds = -r["beta"][0, t][:, None] * np.einsum("hpn,hn->hp", d, kt)
        d = d + ds[..., None] * kt[:, None]
        out[t] = np.sqrt((d * d).sum((1, 2)) * (w * w).sum((1, 2)))
        d = np.exp(r["g"][0, t])[:, None, None] * d
    return out


def forgetful(seed, dtype, T, P, N):
    """Keys alike, hardly any decay, but for a few tokens of each head that forget."""
    H = 2
    dev, _ = make(seed, dtype, 1, T, H, P, H, N, decay=0.01)
    k = dev["k"].float() + 1.5 * dev["k"][:, :1].float()
    dev["k"].copy_(k / k.norm(dim=-1, keepdim=True))
    dev["beta"].mul_(0.5).add_(0.5)
    for t, h, g in ((7, 0, -12.0), (20, 0, -20.0), (75, 0, -30.0), (5, 1, -20.0), (70, 1, -15.0), (100, 1, -25.0)):
        dev["g"][0, t, h] = g
    return dev, {n: f64(dev[n]) for n in (*GATES, "dy", "dh", "h0")}


@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 64, 128), ("bf16", 128, 128), ("bf16", 64, 64)])
def test_gate_gradients_of_tokens_that_forget(dtype, P, N):
    T = 150
    dev, r = forgetful(40, dtype, T, P, N)
    got = ssm.delta_bwd(*[dev[n] for n in GATES], dev["dy"], h0=dev["h0"], dh_final=dev["dh"])
    want = delta_bwd_ref(*[r[n] for n in GATES], N ** -0.5, r["dy"], r["dh"], r["h0"])
    own = gate_norms(r, r["dy"], r["dh"], r["h0"], N ** -0.5)
    tol = (2e-5 if dtype == "f32" else 6 * HALF["bf16"]) * own
    if dtype == "bf16":
        s2 = (2 * np.linalg.norm(want["dq"][0], axis=-1) + 3 * np.linalg.norm(want["dk"][0], axis=-1)) ** 2
        block = np.concatenate([np.tile(s2[i:i + 64].sum(0), (min(64, T - i), 1)) for i in range(0, T, 64)])
        tol = tol + 16 * 4 * 2.0 ** -24 * np.sqrt(block)
    err = abs(f64(got["dg"])[0] - want["dg"][0])
    worst = (err / tol).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("g", [-torch.inf, -104.0])
@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 24, 40), ("bf16", 64, 128), ("bf16", 128, 64)])
def test_a_reset_is_exact(dtype, P, N, g):
    # whatever the state holds, the tokens from the reset on do not know: bit for bit, and no gradient passes
    dev, _ = make(41, dtype, 1, 150, 2, P, 1, N)
    x, big = [dev[n] for n in GATES], 1e30 * dev["h0"]
    for t in (0, 70, 149):
        x[3].copy_(dev["g"])
        x[3][:, t] = g
        y, hf = ssm.delta_fwd(*x)
        y2, hf2 = ssm.delta_fwd(*x, h0=big)
        assert torch.equal(y[:, t:], y2[:, t:]) and torch.equal(hf, hf2), t
        d = ssm.delta_bwd(*x, dev["dy"], h0=dev["h0"], dh_final=dev["dh"])
        assert (d["dg"][:, t] == 0).all(), t
        if t == 0:
            assert (d["dh0"] == 0).all()
    tok = [v[:, 149] for v in x]
    zero = torch.zeros_like(big)
    assert torch.equal(ssm.delta_update(big, *tok), ssm.delta_update(zero, *tok)) and torch.equal(big, zero)


@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 24, 41), ("bf16", 64, 128), ("bf16", 128, 64)])
def test_gate_gradients_in_fp32(dtype, P, N):
    # the same numbers without their last rounding: rounded once they are the default's, and their sums over the
    # tokens do not carry 8-bit errors
    dev, r = make(42, dtype, 2, 200, 4, P, 2, N)
    call = lambda **kw: ssm.delta_bwd(*[dev[n] for n in GATES], dev["dy"], h0=dev["h0"], dh_final=dev["dh"], **kw)
    d, f = call(), call(gate_dtype=torch.float32)
    assert f["dg"].dtype == f["dbeta"].dtype == torch.float32
    assert all(torch.equal(d[n], f[n].to(d[n].dtype)) for n in d)
    out = {n: torch.full_like(t, torch.nan) for n, t in f.items()}
    assert call(gate_dtype=torch.float32, out=out) is out and all(torch.equal(out[n], f[n]) for n in f)
    want = delta_bwd_ref(*[r[n] for n in GATES], N ** -0.5, r["dy"], r["dh"], r["h0"])
    if N % 8 or dtype == "f32":              # token by token: fp32 throughout
        for n in ("dg", "dbeta"):
            assert abs(f64(f[n]) - want[n]).max() <= 2e-5 * abs(want[n]).max(), n


def test_gate_dtype_refusals():
    dev, _ = make(43, "bf16", 1, 20, 2, 64, 1, 64)
    x = [dev[n] for n in GATES]
    with pytest.raises(TypeError):
        ssm.delta_bwd(*x, dev["dy"], gate_dtype=torch.float16)
    with pytest.raises(TypeError):
        ssm.delta_bwd(*[t.float() for t in x], dev["dy"].float(), gate_dtype=torch.bfloat16)
    out = ssm.delta_bwd(*x, dev["dy"])
    with pytest.raises(TypeError):
        ssm.delta_bwd(*x, dev["dy"], gate_dtype=torch.float32, out=out)
    with pytest.raises(TypeError):
        ssm.delta_bwd(*x, dev["dy"], out=ssm.delta_bwd(*x, dev["dy"], gate_dtype=torch.float32))
