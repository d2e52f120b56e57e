"""Group norm on the GPU against its 64-bit form, forward and backward.

Tolerances, max|err| / max|ref|: half a step of the output's type, and for the
fp32 arithmetic 1e-6 in the forward (a dozen roundings of 2^-24, __expf's 2^-21
in the gate) and 4e-6 in the backward (three sums over the group and products
of rounded factors); dweight and dbias sum up to 700 rows: 5e-6.

dx = r (dn - n mean(dn n) - mean(dn)) is a difference whose terms are as large
as r dn, and each is rounded: the fp32 part of its tolerance is relative to the
larger of max|dx| and max|r dn|.  In a group of one channel n^2 = 1 - eps r^2,
so dx = r dn (1 - n^2) = r dn eps r^2: 1e-5 and less of its terms, whose
rounding (2^-24 of r dn) is then all the digits that are left.
"""
import pytest
import torch

import state_space_model_conv1d_b200 as ssm

from gpu_util import rel_err
from layer_ref import HALF, norm_bwd_ref, norm_ref

pytestmark = pytest.mark.gpu
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
MODES = ["plain", "silu", "gate", "first"]
SIZES = [((1,), 1, 1), ((3,), 24, 3), ((5,), 520, 4), ((2, 9), 1040, 5), ((700,), 256, 2), ((4,), 2051, 1), ((3, 2), 4096, 1),
         ((33,), 640, 80), ((2,), 9000, 1), ((3,), 16384, 1), ((7,), 2000, 2), ((6,), 1920, 15)]


def make(seed, dtype, lead, C):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    d = dict(x=rnd(*lead, C) + 0.5, z=rnd(*lead, C), dy=rnd(*lead, C))
    d = {n: t.to("cuda", TDT[dtype]) for n, t in d.items()}
    d |= dict(w=(1 + 0.2 * rnd(C)).cuda(), b=(0.2 * rnd(C)).cuda())
    return d, {n: t.double().cpu().numpy() for n, t in d.items()}


def kwargs(mode, mean):
    gate = mode in ("gate", "first")
    return (dict(subtract_mean=mean, gate_first=mode == "first", activation=mode == "silu"),
            dict(mean=mean, first=mode == "first", act=mode == "silu"), gate)


def check(dtype, lead, C, G, mode, mean, seed=0, params=True):
    d, r = make(seed, dtype, lead, C)
    kw, rkw, gate = kwargs(mode, mean)
    z, rz = (d["z"], r["z"]) if gate else (None, None)
    w, b, rw, rb = (d["w"], d["b"], r["w"], r["b"]) if params else (None,) * 4
    y = ssm.group_norm_fwd(d["x"], G, weight=w, bias=b, z=z, **kw)
    assert rel_err(y.double().cpu().numpy(), norm_ref(r["x"], G, rw, rb, rz, **rkw)) <= HALF[dtype] + 1e-6
    got = ssm.group_norm_bwd(d["x"], G, d["dy"], weight=w, bias=b, z=z, **kw)
    want = norm_bwd_ref(r["x"], G, r["dy"], rw, rb, rz, **rkw)
    terms = want.pop("terms")
    for n, v in want.items():
        if v is None:
            assert got[n] is None
            continue
        big = max(abs(v).max(), abs(terms.get(n, v)).max())
        tol = HALF[dtype] * abs(v).max() + 4e-6 * big if n in ("dx", "dz") else 5e-6 * big
        assert abs(got[n].double().cpu().numpy() - v).max() <= tol, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(dtype, size):
    lead, C, G = size
    # a group of one channel minus its mean is zero whatever it holds: nothing to compare
    check(dtype, lead, C, G, "gate", C // G > 1, seed=C)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [40, 63, 104, 127, 333, 504, 777, 1536, 2047, 2048, 3001, 3200, 6000, 7001, 9001])
def test_group_widths(dtype, D):
    # every unit's width, with 16-byte accesses and without; more rows than units where rows are cheap
    check(dtype, (5 if D > 2048 else 150,), 2 * D, 2, "first" if D % 2 else "gate", D % 3 != 0, seed=D)


@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("mode", MODES)
def test_modes(mode, mean):
    check("bf16", (2, 17), 384, 6, mode, mean, seed=1)
    check("f32", (9,), 363, 11, mode, mean, seed=2)
    check("f32", (9,), 2048, 1, mode, mean, seed=3, params=False)


def test_far_mean():
    # values a thousand standard deviations from zero: the variance keeps its digits
    d, _ = make(4, "f32", (20,), 512)
    x = d["x"] + 1000.0
    y = ssm.group_norm_fwd(x, 4, subtract_mean=True)
    # x itself is rounded to 2^-24 * 1000 = 6e-5, and (x - mean) once more
    assert rel_err(y.double().cpu().numpy(), norm_ref(x.double().cpu().numpy(), 4, mean=True)) <= 5e-5


def test_constant_and_extreme_rows():
    x = torch.zeros(4, 64, device="cuda")
    x[1] = 3.0
    x[2] = 1e30                       # the squares overflow fp32: rows of zeros, as the formula in fp32 says
    x[3, 5] = torch.nan
    y = ssm.group_norm_fwd(x, 2, subtract_mean=True)
    assert (y[:2] == 0).all() and torch.isnan(y[3, :32]).all() and (y[3, 32:] == 0).all()
    d = ssm.group_norm_bwd(x[:2].contiguous(), 2, torch.ones(2, 64, device="cuda"), subtract_mean=True)
    assert torch.isfinite(d["dx"]).all() and (d["dbias"] == 2).all()


def test_views_in_place_and_strides():
    d, r = make(5, "bf16", (3, 11), 256)
    wide = torch.zeros(3, 11, 700, dtype=torch.bfloat16, device="cuda")
    wide[..., 8:264], wide[..., 264:520] = d["x"], d["z"]
    x, z = wide[..., 8:264], wide[..., 264:520]
    want = ssm.group_norm_fwd(d["x"], 4, weight=d["w"], z=d["z"])
    assert torch.equal(ssm.group_norm_fwd(x, 4, weight=d["w"], z=z), want)
    odd = torch.zeros(3, 11, 701, dtype=torch.bfloat16, device="cuda")      # no 16-byte rows
    odd[..., 1:257], odd[..., 257:513] = d["x"], d["z"]
    assert rel_err(ssm.group_norm_fwd(odd[..., 1:257], 4, weight=d["w"], z=odd[..., 257:513]).double().cpu().numpy(),
                   norm_ref(r["x"], 4, r["w"], None, r["z"])) <= HALF["bf16"] + 1e-6
    tail = wide[..., 520:].clone()
    assert ssm.group_norm_fwd(x, 4, weight=d["w"], z=z, y=x).data_ptr() == x.data_ptr()
    assert torch.equal(x, want) and torch.equal(wide[..., 520:], tail) and (wide[..., :8] == 0).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    assert ssm.group_norm_fwd(x, 2).shape == (0, 64)
    d = ssm.group_norm_bwd(x, 2, x)
    assert (d["dweight"] == 0).all() and (d["dbias"] == 0).all()


def test_repeatable_on_another_stream_and_in_a_graph():
    d, _ = make(6, "bf16", (300,), 768)
    run = lambda **kw: list(ssm.group_norm_bwd(d["x"], 6, d["dy"], weight=d["w"], bias=d["b"], z=d["z"], **kw).values())
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
