"""The gated delta rule on the GPU against its 64-bit form: forward, backward, one token at a time.

Tolerances, max|err| / max|ref| of an output.  fp32: the recurrence rounds a
state about 4 times a token and a unit key with beta <= 1 never amplifies, so
over T <= 400 tokens the errors grow like sqrt(T) at worst: 4 * 20 * 2^-24 =
5e-6, and sums of N <= 256 products add 16 * 2^-24; the bound is 1e-5 (gradients
pass the chain twice: 2e-5).  bf16 outputs: half a step of the output, 2^-8, and
on the tensor cores the same for each operand that is rounded to bf16 in front
of the product that makes the output: two in the forward (attention weights,
state), at most five in a gradient.  fp32 outputs of bf16 calls (states) keep
operands split in two bf16 parts: 2^-17 each, five products in a row, 5e-5.
"""
import numpy as np
import pytest
import torch

import state_space_model_conv1d_b200 as ssm
from state_space_model_conv1d_b200 import _abi

from gpu_util import rel_err
from layer_ref import HALF, delta_bwd_ref, delta_ref

pytestmark = pytest.mark.gpu
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL_Y = {"f32": 1e-5, "bf16": 3 * HALF["bf16"]}
TOL_H = {"f32": 1e-5, "bf16": 5e-5}
TOL_D = {"f32": 2e-5, "bf16": 6 * HALF["bf16"]}


def make(seed, dtype, b, T, H, P, G, N, nseq=None, decay=1.0, views=False):
    """Device tensors and the 64-bit copies of their values."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    q, k = rnd(b, T, G, N), rnd(b, T, G, N)
    d = dict(q=q / q.norm(dim=-1, keepdim=True), k=k / k.norm(dim=-1, keepdim=True), v=rnd(b, T, H, P),
             g=-decay * torch.rand(b, T, H, generator=gen, dtype=torch.float64) ** 3,
             beta=torch.rand(b, T, H, generator=gen, dtype=torch.float64),
             h0=0.3 * rnd(nseq or b, H, P, N), dy=rnd(b, T, H, P), dh=0.3 * rnd(nseq or b, H, P, N))
    dev = {n: t.to("cuda", TDT[dtype] if n in "qkvdy" else torch.float32) for n, t in d.items()}
    if views:          # q | k | v of one projection row, g and beta of another
        w = torch.empty(b, T, 2 * G * N + H * P + 8, dtype=TDT[dtype], device="cuda")
        at = 0
        for n in ("q", "k", "v"):
            m = dev[n].shape[2] * dev[n].shape[3]
            w[..., at:at + m] = dev[n].flatten(2)
            dev[n] = w[..., at:at + m].unflatten(2, dev[n].shape[2:])
            at += m
        gb = torch.empty(b, T, 2 * H + 1, device="cuda")
        gb[..., :H], gb[..., H:2 * H] = dev["g"], dev["beta"]
        dev["g"], dev["beta"] = gb[..., :H], gb[..., H:2 * H]
    ref = {n: t.double().cpu().numpy() for n, t in dev.items()}
    return dev, ref


def cu_of(lengths):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def check_fwd(dtype, b, T, H, P, G, N, lengths=None, seed=0, h0=True, scale=None, decay=1.0, views=False):
    cu, cud = cu_of(lengths) if lengths is not None else (None, None)
    dev, ref = make(seed, dtype, b, T, H, P, G, N, nseq=None if cu is None else len(lengths), decay=decay, views=views)
    y, hf = ssm.delta_fwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], scale=scale,
                          h0=dev["h0"] if h0 else None, cu_seqlens=cud)
    ry, rh, _ = delta_ref(ref["q"], ref["k"], ref["v"], ref["g"], ref["beta"], N ** -0.5 if scale is None else scale,
                          ref["h0"] if h0 else None, cu)
    assert rel_err(y.double().cpu().numpy(), ry) <= TOL_Y[dtype]
    assert rel_err(hf.double().cpu().numpy(), rh) <= TOL_H[dtype]


def check_bwd(dtype, b, T, H, P, G, N, lengths=None, seed=0, h0=True, dh=True, decay=1.0, views=False):
    cu, cud = cu_of(lengths) if lengths is not None else (None, None)
    dev, ref = make(seed, dtype, b, T, H, P, G, N, nseq=None if cu is None else len(lengths), decay=decay, views=views)
    got = ssm.delta_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dev["dy"], h0=dev["h0"] if h0 else None,
                        dh_final=dev["dh"] if dh else None, cu_seqlens=cud)
    want = delta_bwd_ref(ref["q"], ref["k"], ref["v"], ref["g"], ref["beta"], N ** -0.5, ref["dy"],
                         ref["dh"] if dh else None, ref["h0"] if h0 else None, cu)
    for n, w in want.items():
        tol = TOL_H[dtype] if n == "dh0" and dtype == "bf16" else TOL_D[dtype]
        assert rel_err(got[n].double().cpu().numpy(), w) <= tol, n
    return got


SHAPES = [  # b, T, H, P, G, N
    (1, 1, 1, 1, 1, 1), (2, 37, 3, 5, 1, 7), (1, 64, 2, 64, 1, 128), (2, 65, 4, 64, 2, 128), (1, 200, 4, 128, 2, 128),
    (1, 130, 2, 128, 1, 64), (2, 63, 2, 40, 2, 72), (1, 70, 6, 64, 2, 64), (1, 33, 2, 192, 1, 96), (1, 40, 2, 33, 1, 200),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(dtype, shape):
    check_fwd(dtype, *shape, seed=hash(shape) % 1000)


@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 24, 40), ("bf16", 64, 128), ("bf16", 128, 128)])
def test_forward_packed(dtype, P, N):
    lengths = [70, 0, 1, 64, 129, 0, 63]
    check_fwd(dtype, 1, sum(lengths), 4, P, 2, N, lengths, seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_options(dtype):
    check_fwd(dtype, 2, 100, 4, 64, 2, 128, seed=6, h0=False, scale=1.5)
    check_fwd(dtype, 2, 100, 4, 64, 2, 128, seed=7, decay=40.0)      # decays to nothing within a block
    check_fwd(dtype, 2, 100, 4, 64, 2, 128, seed=8, decay=0.0)       # no decay
    check_fwd(dtype, 2, 100, 4, 64, 2, 128, seed=9, views=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(dtype, shape):
    check_bwd(dtype, *shape, seed=hash(shape) % 1000 + 1)


@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 24, 40), ("bf16", 64, 128), ("bf16", 128, 128)])
def test_backward_packed(dtype, P, N):
    lengths = [70, 0, 1, 64, 129, 0, 63]
    check_bwd(dtype, 1, sum(lengths), 4, P, 2, N, lengths, seed=11)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_options(dtype):
    check_bwd(dtype, 2, 100, 4, 64, 2, 128, seed=12, h0=False, dh=False)
    check_bwd(dtype, 2, 100, 4, 64, 2, 128, seed=13, decay=40.0)
    check_bwd(dtype, 2, 100, 4, 64, 2, 128, seed=14, views=True)


@pytest.mark.parametrize("P,N", [(64, 128), (24, 40)])
def test_reset_by_minus_infinity(P, N):
    # g = -inf forgets everything before it: the tokens from there on equal a fresh sequence
    dev, _ = make(15, "bf16", 1, 150, 2, P, 1, N)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    x[3][:, 70] = -torch.inf
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"])
    y2, hf2 = ssm.delta_fwd(*[t[:, 70:] for t in x])
    assert torch.isfinite(y).all()
    assert rel_err(y[:, 70:].double().cpu().numpy(), y2.double().cpu().numpy()) <= 2 * TOL_Y["bf16"]
    assert rel_err(hf.cpu().numpy(), hf2.cpu().numpy()) <= TOL_H["bf16"]


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64), (24, 40)])
def test_nothing_crosses_sequences(P, N):
    # NaN and infinities in one packed sequence leave its neighbours bit for bit
    lengths = [70, 61, 80]
    cu, cud = cu_of(lengths)
    dev, _ = make(16, "bf16", 1, sum(lengths), 2, P, 1, N, nseq=3)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"], cu_seqlens=cud)
    d = ssm.delta_bwd(*x, dev["dy"], h0=dev["h0"], dh_final=dev["dh"], cu_seqlens=cud)
    bad = [t.clone() for t in x]
    for t, val in zip(bad, (torch.nan, torch.inf, torch.nan, torch.nan, torch.inf)):
        t[:, 70:131] = val
    h0, dy, dh = dev["h0"].clone(), dev["dy"].clone(), dev["dh"].clone()
    h0[1], dy[:, 70:131], dh[1] = torch.nan, torch.inf, torch.nan
    yb, hb = ssm.delta_fwd(*bad, h0=h0, cu_seqlens=cud)
    db = ssm.delta_bwd(*bad, dy, h0=h0, dh_final=dh, cu_seqlens=cud)
    keep = torch.ones(sum(lengths), dtype=torch.bool, device="cuda")
    keep[70:131] = False
    assert torch.equal(y[:, keep], yb[:, keep]) and torch.equal(hf[[0, 2]], hb[[0, 2]])
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(d[n][:, keep], db[n][:, keep]), n
    assert torch.equal(d["dh0"][[0, 2]], db["dh0"][[0, 2]])


def test_malformed_cu_seqlens_sets_the_error_word_and_writes_nothing():
    dev, _ = make(17, "bf16", 1, 100, 2, 64, 1, 128, nseq=2)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    for cu in ([0, 60, 50], [0, 40, 101], [1, 50, 100]):
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
        y = torch.full_like(x[2], 7.0)
        hf = torch.full_like(dev["h0"], 7.0)
        ssm.delta_fwd(*x, cu_seqlens=cud, y=y, h_final=hf, workspace=ws)
        assert ssm.workspace_error(ws) == _abi.SSM_DEVERR_CU_SEQLENS
        assert (y == 7).all() and (hf == 7).all()
        out = {n: torch.full_like(t, 7.0) for n, t in ssm.delta_bwd(*x, dev["dy"]).items() if n != "dh0"}
        out["dh0"] = torch.full_like(dev["h0"], 7.0)
        ssm.delta_bwd(*x, dev["dy"], cu_seqlens=cud, out=out, workspace=ws)
        assert ssm.workspace_error(ws) == _abi.SSM_DEVERR_CU_SEQLENS
        assert all((t == 7).all() for t in out.values())


def test_empty_rows_return_h0():
    dev, _ = make(18, "bf16", 2, 1, 2, 64, 1, 128)
    x = [dev[n][:, :0] for n in ("q", "k", "v", "g", "beta")]
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"])
    assert y.shape[1] == 0 and torch.equal(hf, dev["h0"])
    d = ssm.delta_bwd(*x, dev["dy"][:, :0], dh_final=dev["dh"])
    assert torch.equal(d["dh0"], dev["dh"]) and d["dq"].numel() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,H,P,G,N", [(1, 1, 1, 1, 1), (5, 4, 33, 2, 20), (3, 6, 64, 2, 128), (40, 4, 128, 4, 128),
                                       (2, 2, 17, 1, 250), (3, 2, 20, 1, 41), (2, 4, 64, 4, 64)])
def test_update(dtype, b, H, P, G, N):
    dev, ref = make(20 + b, dtype, b, 1, H, P, G, N)
    slots = b + 3
    gen = torch.Generator().manual_seed(b)
    state = torch.randn(slots, H, P, N, generator=gen).cuda()
    idx = torch.randperm(slots, generator=gen)[:b].to(torch.int32)
    before = state.double().cpu().numpy()
    y = ssm.delta_update(state, *[dev[n][:, 0] for n in ("q", "k", "v", "g", "beta")],
                         state_batch_indices=idx.cuda())
    ry, rh, _ = delta_ref(*[ref[n] for n in ("q", "k", "v", "g", "beta")], N ** -0.5, before[idx.numpy()])
    want = before.copy()
    want[idx.numpy()] = rh
    assert rel_err(y.double().cpu().numpy(), ry[:, 0]) <= (HALF["bf16"] + 1e-5 if dtype == "bf16" else 1e-5)
    assert rel_err(state.double().cpu().numpy(), want) <= 1e-6
    others = [i for i in range(slots) if i not in idx.tolist()]
    assert np.array_equal(state.double().cpu().numpy()[others], before[others])


def test_update_padding_rows():
    dev, _ = make(30, "bf16", 4, 1, 2, 64, 1, 128)
    x = [dev[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    state = torch.randn(3, 2, 64, 128, device="cuda")
    before = state.clone()
    y = ssm.delta_update(state, *x, state_batch_indices=torch.tensor([-1, 2, 3, -7], dtype=torch.int32, device="cuda"))
    assert (y[[0, 2, 3]] == 0).all() and (y[1] != 0).any()
    assert torch.equal(state[:2], before[:2]) and not torch.equal(state[2], before[2])


def test_prefill_equals_repeated_updates():
    dev, _ = make(31, "f32", 2, 30, 4, 16, 2, 24)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"])
    state = dev["h0"].clone()
    ys = torch.stack([ssm.delta_update(state, *[t[:, i] for t in x]) for i in range(30)], 1)
    assert rel_err(ys.cpu().numpy(), y.cpu().numpy()) <= 2e-5 and rel_err(state.cpu().numpy(), hf.cpu().numpy()) <= 2e-5


@pytest.mark.parametrize("dtype,P,N", [("bf16", 64, 128), ("bf16", 128, 64), ("f32", 24, 40)])
def test_repeatable_on_another_stream_and_in_a_graph(dtype, P, N):
    lengths = [70, 5, 100]
    cu, cud = cu_of(lengths)
    dev, _ = make(32, dtype, 1, 175, 4, P, 2, N, nseq=3)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]

    def both(**kw):
        return (*ssm.delta_fwd(*x, h0=dev["h0"], cu_seqlens=cud, **kw),
                *ssm.delta_bwd(*x, dev["dy"], h0=dev["h0"], dh_final=dev["dh"], cu_seqlens=cud, **kw).values())

    want = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = both(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # two captured graphs, replayed one after the other on changed inputs and back
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = both()
        graphs.append((gr, outs))
    x[2].neg_()
    graphs[0][0].replay()
    x[2].neg_()
    graphs[1][0].replay()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
