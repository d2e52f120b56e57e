"""The operators beside the scan as they are used together, and the calls that
none of their own files makes: two at once, a shared page table, strides that
pass 32 bits, rows off their alignment, gates that are zero, tiny or NaN, the
bounds-checked build, and what the binding refuses.

Tolerances as in the operators' own files (test_gpu_delta.py, test_gpu_norm.py):
every operator of a run is compared with its 64-bit form on the values it got.
"""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
import state_space_model_conv1d_b200 as ssm
from state_space_model_conv1d_b200 import _abi, layer_ops

from gpu_util import TOL, rel_err
from layer_ref import HALF, compact_ref, delta_bwd_ref, delta_ref, norm_bwd_ref, norm_ref
from test_gpu_delta import TOL_D, TOL_H, TOL_Y, check_bwd, check_fwd, cu_of, make

pytestmark = pytest.mark.gpu
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------- a layer
@pytest.mark.parametrize("dtype,H,P,G,N", [("bf16", 4, 64, 2, 128), ("bf16", 2, 128, 2, 64), ("f32", 6, 24, 3, 40)])
def test_layer(dtype, H, P, G, N):
    # packed prompts through conv (q | k | v of one projection), unit keys and queries, the delta rule, the gated
    # norm, and back again
    lengths = [70, 1, 0, 129]
    cu, cud = cu_of(lengths)
    T, Cq = sum(lengths), G * N
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()
    Cc = 2 * Cq + H * P
    proj, z, dout = rnd(1, T, Cc).to(TDT[dtype]), rnd(1, T, H * P).to(TDT[dtype]), rnd(1, T, H * P).to(TDT[dtype])
    cw, cb, cs = 0.4 * rnd(Cc, 4), 0.1 * rnd(Cc), rnd(len(lengths), Cc, 3).to(TDT[dtype])
    g, beta, h0, w = -rnd(1, T, H).abs(), torch.sigmoid(rnd(1, T, H)), 0.3 * rnd(len(lengths), H, P, N), 1 + 0.1 * rnd(H * P)
    unit = torch.full((Cq,), N ** -0.5, device="cuda")           # a group of root mean square 1 times this has length 1

    x = ssm.conv1d_fwd(proj, cw, cb, state_in=cs, cu_seqlens=cud)
    qn, kn = (ssm.group_norm_fwd(x[..., i * Cq:(i + 1) * Cq], G, weight=unit, eps=1e-6) for i in (0, 1))
    q, k, v = qn.unflatten(2, (G, N)), kn.unflatten(2, (G, N)), x[..., 2 * Cq:].unflatten(2, (H, P))
    y, hf = ssm.delta_fwd(q, k, v, g, beta, h0=h0, cu_seqlens=cud)
    o = ssm.group_norm_fwd(y.flatten(2), H, weight=w, z=z)
    d = ssm.group_norm_bwd(y.flatten(2), H, dout, weight=w, z=z)
    dd = ssm.delta_bwd(q, k, v, g, beta, d["dx"].unflatten(2, (H, P)), h0=h0, cu_seqlens=cud)
    dq = ssm.group_norm_bwd(x[..., :Cq], G, dd["dq"].flatten(2), weight=unit, eps=1e-6)

    rx, _ = oracle.conv1d_fwd(f64(proj), f64(cw), b=f64(cb), state_in=f64(cs), cu_seqlens=cu)
    assert rel_err(f64(x), rx) <= TOL[dtype]
    for i, n in enumerate((qn, kn)):
        assert rel_err(f64(n), norm_ref(f64(x[..., i * Cq:(i + 1) * Cq]), G, f64(unit), eps=1e-6)) <= HALF[dtype] + 1e-6
    args = [f64(t) for t in (q, k, v, g, beta)]
    ry, rh, _ = delta_ref(*args, N ** -0.5, f64(h0), cu)
    assert rel_err(f64(y), ry) <= TOL_Y[dtype] and rel_err(f64(hf), rh) <= TOL_H[dtype]
    assert rel_err(f64(o), norm_ref(f64(y.flatten(2)), H, f64(w), None, f64(z))) <= HALF[dtype] + 1e-6
    want = norm_bwd_ref(f64(y.flatten(2)), H, f64(dout), f64(w), None, f64(z))
    assert abs(f64(d["dx"]) - want["dx"]).max() <= HALF[dtype] * abs(want["dx"]).max() + 4e-6 * abs(want["terms"]["dx"]).max()
    rd = delta_bwd_ref(*args, N ** -0.5, f64(d["dx"].unflatten(2, (H, P))), None, f64(h0), cu)
    for n, r in rd.items():
        assert rel_err(f64(dd[n]), r) <= (TOL_H[dtype] if n == "dh0" and dtype == "bf16" else TOL_D[dtype]), n
    want = norm_bwd_ref(f64(x[..., :Cq]), G, f64(dd["dq"].flatten(2)), f64(unit), eps=1e-6)
    assert abs(f64(dq["dx"]) - want["dx"]).max() <= HALF[dtype] * abs(want["dx"]).max() + 4e-6 * abs(want["terms"]["dx"]).max()


def test_serving_with_forked_pages():
    # two prompts, samples forked from them, one given back, the pool compacted between two runs of decode steps
    H, P, G, N, S = 4, 16, 2, 24, 9
    gen = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def tokens(b, T):
        q, k = rnd(b, T, G, N), rnd(b, T, G, N)
        return [q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True), rnd(b, T, H, P),
                -0.3 * rnd(b, T, H).abs(), torch.sigmoid(rnd(b, T, H))]

    state, tag = torch.full((S, H, P, N), 7.0, device="cuda"), torch.zeros(S, 5, dtype=torch.bfloat16, device="cuda")
    pools, refs = [state, tag], torch.zeros(S, dtype=torch.int32, device="cuda")
    w = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    prompts = tokens(2, 11)
    roots = ssm.state_pages_fork(pools, refs, i32([-1, -1]), workspace=w)
    assert (state[:2] == 0).all() and (state[2:] == 7).all()
    _, hf = ssm.delta_fwd(*prompts)
    state[roots.long()] = hf
    tag[roots.long()] = torch.tensor([[1.0], [2.0]], device="cuda").to(tag.dtype).expand(2, 5)
    parents = i32([0, 1, 0, 1, 0])
    pages = ssm.state_pages_fork(pools, refs, parents, pages=parents, workspace=w)       # the table is rewritten in place
    assert pages.tolist() == [2, 3, 4, 5, 6] and ssm.workspace_error(w) == 0
    root_of = [0, 1, 0, 1, 0]
    ssm.state_pages_free(refs, roots, workspace=w)                                       # the prompts go
    history = [[t[r:r + 1] for t in prompts] for r in root_of]

    def step(table, rows):
        new = tokens(len(rows), 1)
        y = ssm.delta_update(state, *[t[:, 0] for t in new], state_batch_indices=table)
        for i, r in enumerate(rows):
            history[r] = [torch.cat([a, b[i:i + 1]], 1) for a, b in zip(history[r], new)]
            ry, rh, _ = delta_ref(*[f64(t) for t in history[r]], N ** -0.5)
            assert rel_err(f64(y[i]), ry[0, -1]) <= 1e-5 and rel_err(f64(state[table[i]]), rh[0]) <= 1e-5

    rows = [0, 1, 2, 3, 4]
    for _ in range(3):
        step(pages, rows)
    ssm.state_pages_free(refs, pages[1:2], workspace=w)
    rows, table = [0, 2, 3, 4], pages[[0, 2, 3, 4]].contiguous()
    r2, t2, _ = compact_ref(refs.tolist(), table.tolist())
    ssm.state_pages_compact(pools, refs, table, workspace=w)
    assert refs.tolist() == r2 and table.tolist() == t2 and sorted(t2) == [0, 1, 2, 3] and ssm.workspace_error(w) == 0
    assert f64(tag[table.long()])[:, 0].tolist() == [1 + root_of[r] for r in rows]
    for _ in range(3):
        step(table, rows)


def test_fork_may_write_over_its_parents():
    pool, refs = torch.randn(6, 40, device="cuda"), torch.tensor([1, 1, 0, 0, 0, 1], dtype=torch.int32, device="cuda")
    want, src = pool.clone(), torch.tensor([5, 3, 1, -1], dtype=torch.int32, device="cuda")
    want[2], want[3], want[4] = want[5].clone(), want[1].clone(), 0
    w = torch.empty(1 << 12, dtype=torch.uint8, device="cuda")
    assert ssm.state_pages_fork([pool], refs, src, pages=src, workspace=w) is src
    assert src.tolist() == [2, -1, 3, 4] and torch.equal(pool, want)
    assert ssm.workspace_error(w) == _abi.SSM_DEVERR_PAGES         # page 3 was not live


# ------------------------------------------------- what no other file's call does
def test_two_calls_at_once():
    # different calls in flight on two streams, each with its own workspace, then both again
    cases = []
    for seed, dtype, P, N in ((3, "bf16", 64, 128), (4, "bf16", 128, 128), (5, "f32", 24, 40)):
        dev, _ = make(seed, dtype, 2, 200, 4, P, 2, N)
        cases.append([dev[n] for n in ("q", "k", "v", "g", "beta")] + [dev["dy"], dev["h0"], dev["dh"]])

    def run(c, **kw):
        y, hf = ssm.delta_fwd(*c[:5], h0=c[6], **kw)
        d = ssm.delta_bwd(*c[:6], h0=c[6], dh_final=c[7], **kw)
        n = ssm.group_norm_bwd(c[2].flatten(2), 2, c[5].flatten(2), z=y.flatten(2), **kw)
        return [y, hf, *d.values(), *n.values()]

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(2):
        got = [run(c, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))


@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 64, 128), ("bf16", 128, 64)])
def test_state_in_place(dtype, P, N):
    # h_final may be h0 (empty sequences keep theirs), y of the norm may be x
    lengths = [70, 0, 1, 130]
    _, cud = cu_of(lengths)
    dev, _ = make(15, dtype, 1, sum(lengths), 4, P, 2, N, nseq=len(lengths))
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"], cu_seqlens=cud)
    h = dev["h0"].clone()
    y2, hf2 = ssm.delta_fwd(*x, h0=h, h_final=h, cu_seqlens=cud)
    assert hf2 is h and torch.equal(y, y2) and torch.equal(hf, h) and torch.equal(h[1], dev["h0"][1])
    rows = dev["v"].flatten(2)[0]
    for t in (rows, torch.cat([rows] * 30, 1)):
        want, got = ssm.group_norm_fwd(t, 1, z=t, subtract_mean=True), t.clone()
        ssm.group_norm_fwd(got, 1, z=t, subtract_mean=True, y=got)
        assert torch.equal(want, got)


@pytest.mark.parametrize("off,width", [(0, 3), (1, 0), (4, 4)])
def test_rows_off_their_alignment(off, width):
    # bf16 shapes of the tensor cores in rows that do not start on 16 bytes
    b, T, H, P, G, N = 2, 70, 2, 64, 1, 128
    dev, ref = make(6, "bf16", b, T, H, P, G, N)

    def home(t):
        buf = torch.full((b, T, t.shape[2] * t.shape[3] + off + width), torch.nan, dtype=t.dtype, device="cuda")
        v = buf[..., off:off + t.shape[2] * t.shape[3]]
        v.copy_(t.flatten(2))
        return v.unflatten(2, t.shape[2:])

    x = [home(dev[n]) for n in "qkv"] + [dev["g"], dev["beta"]]
    y = home(torch.zeros_like(dev["v"]))
    _, hf = ssm.delta_fwd(*x, h0=dev["h0"], y=y)
    args = [ref[n] for n in ("q", "k", "v", "g", "beta")]
    ry, rh, _ = delta_ref(*args, N ** -0.5, ref["h0"])
    assert rel_err(f64(y), ry) <= TOL_Y["bf16"] and rel_err(f64(hf), rh) <= TOL_H["bf16"]
    if off + width:
        base = y.as_strided((b, T, y.stride(1)), (y.stride(0), y.stride(1), 1), y.storage_offset() - off)
        assert torch.isnan(base[..., :off]).all() and torch.isnan(base[..., off + H * P:]).all()
    d = ssm.delta_bwd(*x, home(dev["dy"]), h0=dev["h0"], dh_final=dev["dh"])
    for n, r in delta_bwd_ref(*args, N ** -0.5, ref["dy"], ref["dh"], ref["h0"]).items():
        assert rel_err(f64(d[n]), r) <= (TOL_H["bf16"] if n == "dh0" else TOL_D["bf16"]), n


@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 64, 128), ("bf16", 128, 64)])
def test_zero_and_tiny_gates(dtype, P, N):
    b, T, H, G = 1, 90, 4, 2
    dev, ref = make(7, dtype, b, T, H, P, G, N)
    beta = dev["beta"]
    beta[:, ::3], beta[:, 1::7], beta[:, 2::11], beta[:, 70:75] = 0.0, 1e-30, -1e-38, 1.0
    ref["beta"] = f64(beta)
    x, args = [dev[n] for n in ("q", "k", "v", "g", "beta")], [ref[n] for n in ("q", "k", "v", "g", "beta")]
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"])
    ry, rh, _ = delta_ref(*args, N ** -0.5, ref["h0"])
    assert rel_err(f64(y), ry) <= TOL_Y[dtype] and rel_err(f64(hf), rh) <= TOL_H[dtype]
    d = ssm.delta_bwd(*x, dev["dy"], h0=dev["h0"], dh_final=dev["dh"])
    for n, r in delta_bwd_ref(*args, N ** -0.5, ref["dy"], ref["dh"], ref["h0"]).items():
        assert rel_err(f64(d[n]), r) <= (TOL_H[dtype] if n == "dh0" and dtype == "bf16" else TOL_D[dtype]), n


@pytest.mark.parametrize("dtype,P,N", [("f32", 24, 40), ("bf16", 64, 128)])
def test_nan_gates_are_not_hidden(dtype, P, N):
    dev, _ = make(8, dtype, 1, 100, 2, P, 1, N)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    x[3][:, 40, 0] = torch.nan
    y, hf = ssm.delta_fwd(*x, h0=dev["h0"])
    assert torch.isnan(y[:, 40:, 0]).all() and torch.isnan(hf[:, 0]).all() and torch.isfinite(hf[:, 1]).all()
    state = dev["h0"].clone()
    ssm.delta_update(state, *[t[:, 40] for t in x])
    assert torch.isnan(state[:, 0]).all() and torch.isfinite(state[:, 1]).all()


def test_keys_alike_and_no_decay():
    # every key the same: the triangular system of a block is as full as it can be
    for dtype, P, N in (("f32", 24, 40), ("bf16", 64, 128)):
        dev, ref = make(9, dtype, 1, 130, 2, P, 1, N, decay=0.0)
        dev["k"][:] = dev["k"][:, :1].clone()
        dev["beta"].fill_(1.0)
        x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
        y, hf = ssm.delta_fwd(*x, h0=dev["h0"])
        ry, rh, _ = delta_ref(*[f64(t) for t in x], N ** -0.5, ref["h0"])
        assert rel_err(f64(y), ry) <= TOL_Y[dtype] and rel_err(f64(hf), rh) <= TOL_H[dtype]


def test_strides_past_32_bits():
    # two batch rows more than 2^31 elements apart, in and out
    far = 2 ** 31 + 4096
    T, H, P, G, N = 70, 2, 64, 1, 128
    buf = torch.empty(far + T * 1024, dtype=torch.bfloat16, device="cuda")
    dev, ref = make(10, "bf16", 2, T, H, P, G, N)

    def home(t, at):
        v = buf.as_strided(t.shape, (far, 1024, t.shape[3], 1), at)
        v.copy_(t)
        return v

    q, k, v, dy = home(dev["q"], 0), home(dev["k"], 128), home(dev["v"], 256), home(dev["dy"], 384)
    y = home(torch.zeros_like(dev["v"]), 512)
    x = (q, k, v, dev["g"], dev["beta"])
    want, hf = ssm.delta_fwd(*[dev[n] for n in ("q", "k", "v", "g", "beta")], h0=dev["h0"])
    _, hf2 = ssm.delta_fwd(*x, h0=dev["h0"], y=y)
    assert torch.equal(want, y) and torch.equal(hf, hf2)
    d = ssm.delta_bwd(*[dev[n] for n in ("q", "k", "v", "g", "beta", "dy")], h0=dev["h0"])
    d2 = ssm.delta_bwd(*x, dy, h0=dev["h0"])
    assert all(torch.equal(a, b) for a, b in zip(d.values(), d2.values()))
    o, o2 = home(torch.zeros_like(dev["v"]), 640), None
    o2 = o.flatten(2)
    assert o2.data_ptr() == o.data_ptr()
    ssm.group_norm_fwd(y.flatten(2), 2, z=v.flatten(2), y=o2)
    assert torch.equal(o2, ssm.group_norm_fwd(want.flatten(2), 2, z=dev["v"].flatten(2)))
    # fp32 rows of the token-by-token form
    buf32 = buf[:(buf.numel() // 2) * 2].view(torch.float32)
    v32 = buf32.as_strided((2, 5, 2, 12), (far // 2, 24, 12, 1), 0)
    v32.copy_(dev["v"][:, :5, :, :12])
    q32, k32 = (dev[n][:, :5, :, :20].float().contiguous() for n in "qk")
    g, beta = dev["g"][:, :5], dev["beta"][:, :5]
    assert all(torch.equal(a, b) for a, b in zip(ssm.delta_fwd(q32, k32, v32, g, beta),
                                                 ssm.delta_fwd(q32, k32, v32.contiguous(), g, beta)))


def test_state_pool_past_32_bits():
    # slots behind 2^31 elements (8 GiB) of a pool: one token, and pages copied, moved and given back
    H, P, N = 8, 128, 256
    slots = 2 ** 31 // (H * P * N) + 6
    state = torch.empty(slots, H, P, N, device="cuda")
    dev, ref = make(11, "bf16", 3, 1, H, P, 2, N)
    idx = torch.tensor([slots - 1, slots - 3, 0], dtype=torch.int32, device="cuda")
    state[idx.long()] = dev["h0"]
    y = ssm.delta_update(state, *[dev[n][:, 0] for n in ("q", "k", "v", "g", "beta")], state_batch_indices=idx)
    ry, rh, _ = delta_ref(*[ref[n] for n in ("q", "k", "v", "g", "beta")], N ** -0.5, ref["h0"])
    assert rel_err(f64(y), ry[:, 0]) <= HALF["bf16"] + 1e-5 and rel_err(f64(state[idx.long()]), rh) <= 1e-6
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kept = state[idx.long()].clone()
    ssm.state_pages_copy([state], idx[:1], i32([slots - 2]))
    assert torch.equal(state[slots - 2], kept[0])
    refs = torch.zeros(slots, dtype=torch.int32, device="cuda")
    refs[idx.long()] = 1
    ssm.state_pages_compact([state], refs, idx)
    assert sorted(idx.tolist()) == [0, 1, 2] and torch.equal(state[idx.long()], kept)


def test_without_torchs_private_cuda_names(monkeypatch):
    # the same call by way of torch's public ones
    dev, _ = make(16, "f32", 1, 20, 2, 16, 1, 24)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    want = ssm.delta_fwd(*x, h0=dev["h0"])
    monkeypatch.setattr(layer_ops, "_cur_device", None)
    monkeypatch.setattr(layer_ops, "_cur_stream", None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ssm.delta_fwd(*x, h0=dev["h0"])
    with torch.cuda.stream(side):
        there = ssm.delta_fwd(*x, h0=dev["h0"])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, there))


# ------------------------------------------------------ the bounds-checked build
def test_checked_build_runs_clean(monkeypatch):
    chk = _abi.checked_lib()
    rec = [C.c_int32(-1), C.c_int32(-1), C.c_int64(-1), C.c_int64(-1)]
    read = lambda clear: chk.ssm_bounds_record(*[C.byref(r) for r in rec], clear)
    assert read(1) == _abi.SSM_OK
    monkeypatch.setattr(_abi, "lib", lambda: chk)
    lengths = [70, 0, 1, 64, 129]
    for dtype, P, N in (("f32", 24, 40), ("bf16", 64, 128), ("bf16", 128, 64)):
        check_fwd(dtype, 1, sum(lengths), 4, P, 2, N, lengths, seed=12)
        check_bwd(dtype, 1, sum(lengths), 4, P, 2, N, lengths, seed=13)
    test_serving_with_forked_pages()
    assert read(0) == _abi.SSM_OK
    assert rec[0].value == 0, f"bounds check fired: site {rec[1].value}, index {rec[2].value}, extent {rec[3].value}"


def test_checked_build_runs_clean_beyond_one_block(monkeypatch):
    # remainders of every kind: rows, widths, slices and blocks that fill nothing, several heads in a pre-pass CTA,
    # units of several tokens
    import test_gpu_delta_paths as paths
    import test_gpu_norm_turns as turns
    from test_gpu_norm import check as check_norm
    chk = _abi.checked_lib()
    rec = [C.c_int32(-1), C.c_int32(-1), C.c_int64(-1), C.c_int64(-1)]
    assert chk.ssm_bounds_record(*[C.byref(r) for r in rec], 1) == _abi.SSM_OK
    monkeypatch.setattr(_abi, "lib", lambda: chk)
    lengths = [70, 0, 1, 64, 200]
    for dtype, H, P, G, N in (("bf16", 6, 40, 2, 72), ("bf16", 3, 192, 1, 72), ("bf16", 4, 8, 1, 8), ("f32", 12, 33, 3, 70),
                              ("bf16", 12, 35, 4, 200), ("f32", 2, 9, 1, 60), ("f32", 2, 20, 1, 200)):
        check_fwd(dtype, 1, sum(lengths), H, P, G, N, lengths, seed=17)
        check_bwd(dtype, 1, sum(lengths), H, P, G, N, lengths, seed=18)
        check_bwd(dtype, 2, 65, H, P, G, N, seed=19)
    paths.test_heads_of_a_group_share_a_prepass(3, 3, 2700)
    for dtype, D in (("bf16", 64), ("f32", 63), ("bf16", 511), ("f32", 2048), ("bf16", 7001)):
        turns.test_units_of_several_tokens(dtype, D)
    check_norm("bf16", (3, 41), 2 * 333, 2, "first", True, seed=20)
    dev, _ = make(21, "bf16", 3, 1, 4, 33, 2, 41)
    pool = torch.randn(5, 4, 33, 41, device="cuda")
    ssm.delta_update(pool, *[dev[n][:, 0] for n in ("q", "k", "v", "g", "beta")],
                     state_batch_indices=torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda"))
    ssm.state_pages_copy([pool], *[torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([4, -1, 9], [1, 2, 3])])
    assert chk.ssm_bounds_record(*[C.byref(r) for r in rec], 0) == _abi.SSM_OK
    assert rec[0].value == 0, f"bounds check fired: site {rec[1].value}, index {rec[2].value}, extent {rec[3].value}"


# ---------------------------------------------------------------------- refusals
def test_binding_refuses():
    dev, _ = make(14, "bf16", 2, 9, 4, 8, 2, 16)
    q, k, v, g, beta = (dev[n] for n in ("q", "k", "v", "g", "beta"))
    cu = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    bad = [
        (TypeError, lambda: ssm.delta_fwd(q.float(), k, v, g, beta)),
        (TypeError, lambda: ssm.delta_fwd(q, k, v, g.bfloat16(), beta)),
        (TypeError, lambda: ssm.delta_fwd(q, k, v, g, beta, h0=dev["h0"].double())),
        (TypeError, lambda: ssm.delta_fwd(q[:1], k[:1], v[:1], g[:1], beta[:1], cu_seqlens=cu.long())),
        (ValueError, lambda: ssm.delta_fwd(q, k[:, :8], v, g, beta)),
        (ValueError, lambda: ssm.delta_fwd(q, k, v, g[..., :3], beta)),
        (ValueError, lambda: ssm.delta_fwd(q, k, v.transpose(2, 3), g, beta)),
        (ValueError, lambda: ssm.delta_fwd(q, k, v[..., ::2], g, beta)),
        (ValueError, lambda: ssm.delta_fwd(q, k, v, g, beta, h0=dev["h0"][:1])),
        (ValueError, lambda: ssm.delta_fwd(q, k.cpu(), v, g, beta)),
        (ValueError, lambda: ssm.delta_fwd(q, k, v, g, beta, y=torch.empty_like(v)[:, :5])),
        (ValueError, lambda: ssm.delta_fwd(q, k, v, g, beta, workspace=torch.empty(9, device="cuda"))),
        (ValueError, lambda: ssm.delta_fwd(q[0], k[0], v[0], g[0], beta[0])),
        (_abi.SSMError, lambda: ssm.delta_fwd(q, k, v, g, beta, cu_seqlens=cu)),                # batch 2
        (_abi.SSMError, lambda: ssm.delta_fwd(q, k, v, g, beta, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))),
        (_abi.SSMError, lambda: ssm.delta_fwd(q, k, v[:, :, :3], g[..., :3], beta[..., :3])),   # 3 heads, 2 groups
        (_abi.SSMError, lambda: ssm.delta_fwd(q.expand(2, 9, 2, 16)[:1].expand(2, 9, 2, 16), k, v, g, beta)),   # rows on one another
        (ValueError, lambda: ssm.delta_bwd(q, k, v, g, beta, dev["dy"][..., :4])),
        (ValueError, lambda: ssm.delta_update(dev["h0"].transpose(2, 3), q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0])),
        (_abi.SSMError, lambda: ssm.delta_update(dev["h0"][:1], q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0])),
        (ValueError, lambda: ssm.group_norm_fwd(v, 2)),
        (ValueError, lambda: ssm.group_norm_fwd(g, 2, gate_first=True)),
        (ValueError, lambda: ssm.group_norm_fwd(g, 2, z=g, activation=True)),
        (ValueError, lambda: ssm.group_norm_fwd(g, 2, weight=g[0, 0, :3].contiguous())),
        (ValueError, lambda: ssm.group_norm_fwd(g, 2, z=g[:, :5])),
        (_abi.SSMError, lambda: ssm.group_norm_fwd(g, 3)),
        (_abi.SSMError, lambda: ssm.group_norm_fwd(g, 2, eps=-1.0)),
        (ValueError, lambda: ssm.state_pages_copy([g[:, :, 0]], cu, cu)),
        (TypeError, lambda: ssm.state_pages_copy([g], cu.long(), cu.long())),
        (ValueError, lambda: ssm.state_pages_free(cu[:1].expand(4), cu)),
        (ValueError, lambda: ssm.state_pages_fork([g] * 9, cu, cu)),
        (ValueError, lambda: ssm.state_pages_fork([g[:1]], cu, cu)),
        (TypeError, lambda: ssm.delta_fwd(q.half(), k.half(), v.half(), g, beta)),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
