"""Cases, plain forms and work counts of the recurrent-layer operators beside the scan.

Four operators, each through the package's public calls:

- the gated delta rule, ``h_t = a_t h_{t-1} + u_t k_t^T`` with ``a_t = exp(g_t)``,
  ``u_t = beta_t (v_t - a_t h_{t-1} k_t)`` and ``y_t = scale * h_t q_t``: over whole
  sequences (``delta_fwd``), its gradients (``delta_bwd``) and one decode token
  per row on slot-indexed states (``delta_update``);
- group norm of channels-last rows with SiLU or a SiLU gate (``group_norm_fwd``,
  ``group_norm_bwd``);
- pages of a recurrent-state cache: fork, copy and free (``state_pages_fork``,
  ``state_pages_copy``, ``state_pages_free``) and compaction (``state_pages_compact``).

``run`` computes the plain form in elementary torch operations, or, with ``own``,
calls the package.  ``exact`` evaluates the definitions token by token in 64 bits.
"""
import random

import torch

own = False

CHUNK = 64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a batch of prompts through one layer; value heads share keys in pairs
        dict(name="delta_fwd_b4_l4096", op="delta_fwd", dtype="bf16", b=4, T=4096, H=32, P=128, G=16, N=128, seqs=0),
        # prompts of mixed length packed in one row, the scan benchmark's head shape
        dict(name="delta_fwd_packed16", op="delta_fwd", dtype="bf16", b=1, T=28301, H=64, P=64, G=1, N=128, seqs=16),
        # full precision, sizes that fill no tile
        dict(name="delta_fwd_f32_odd", op="delta_fwd", dtype="f32", b=2, T=333, H=6, P=40, G=3, N=72, seqs=0),
        # one layer's training step
        dict(name="delta_bwd_b4_l2048", op="delta_bwd", dtype="bf16", b=4, T=2048, H=16, P=128, G=8, N=128, seqs=0),
        # full-precision gradients of packed odd sequences (gradient checks, small models)
        dict(name="delta_bwd_f32_odd", op="delta_bwd", dtype="f32", b=1, T=517, H=4, P=48, G=2, N=64, seqs=5),
        # decode of a full serving batch, one token per row
        dict(name="delta_update_b256", op="delta_update", dtype="bf16", b=256, H=64, P=64, G=8, N=128, slots=288),
        # decode of a few rows, where the launch counts
        dict(name="delta_update_b3", op="delta_update", dtype="bf16", b=3, H=32, P=128, G=16, N=128, slots=8),
        # gated norm behind the mixer of a training batch (forward, backward)
        dict(name="norm_fwd_16k", op="norm_fwd", dtype="bf16", rows=16384, C=4096, groups=8, mean=False, gate="after"),
        dict(name="norm_bwd_16k", op="norm_bwd", dtype="bf16", rows=16384, C=4096, groups=64, mean=True, gate="before"),
        # the same norm at decode: a few rows, odd group width
        dict(name="norm_fwd_decode", op="norm_fwd", dtype="f32", rows=5, C=5130, groups=27, mean=True, gate="silu"),
        # parallel samples forked from cached prefixes, then given back
        dict(name="pages_fork_96", op="pages_fork", slots=384, live=256, n=96, H=64, P=64, N=128, conv=17408),
        # live pages moved to the front of the pool after sequences ended
        dict(name="pages_compact_300", op="pages_compact", slots=300, live=150, n=150, H=8, P=64, N=128, conv=2304),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_update", "norm_fwd", "norm_bwd", "pages_fork",
                     "pages_compact"])
    if op in ("delta_fwd", "delta_bwd"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        G = rng.choice([1, 2, 4, 5])
        H = G * rng.choice([1, 2, 3, 4])
        if dtype == "bf16":
            P, N = rng.choice([(64, 128), (128, 128), (64, 64), (128, 64), (48, 128), (192, 96), (72, 104)])
            T = _log(rng, 30, 6000 if op == "delta_fwd" else 2500)
        else:
            P, N = rng.choice([(16, 16), (24, 40), (64, 64), (33, 128), (40, 20)])
            T = _log(rng, 20, 900)
        seqs = rng.choice([0, 0, rng.randint(1, 12)])
        b = 1 if seqs else rng.randint(1, 3)
        return dict(op=op, dtype=dtype, b=b, T=max(T, seqs), H=H, P=P, G=G, N=N, seqs=seqs)
    if op == "delta_update":
        b = _log(rng, 1, 200)
        G = rng.choice([1, 2, 8])
        H = G * rng.choice([1, 2, 4])
        P, N = rng.choice([(64, 128), (128, 128), (64, 64), (40, 72), (33, 20)])
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), b=b, H=H, P=P, G=G, N=N, slots=b + rng.randint(0, 40))
    if op in ("norm_fwd", "norm_bwd"):
        groups = rng.choice([1, 2, 8, 11, 40])
        C = groups * _log(rng, 16, 4096 // groups)
        rows = _log(rng, 1, max(2, 40_000_000 // C))
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=rows, C=C, groups=groups, mean=rng.random() < 0.5,
                    gate=rng.choice(["after", "before", "silu", "none"]))
    H, P, N = _log(rng, 2, 48), rng.choice([32, 64, 128]), rng.choice([16, 64, 128])
    slots = rng.randint(20, 200)
    live = rng.randint(5, slots - 8)
    n = rng.randint(1, slots - live) if op == "pages_fork" else live
    return dict(op=op, slots=slots, live=live, n=n, H=H, P=P, N=N, conv=rng.choice([0, 33, 1024, 4101]))


# ------------------------------------------------------------------ the inputs
def _lengths(case):
    """Sequence lengths of a packed case: log-uniform shares of its tokens, an empty one among four or more."""
    r = random.Random("%d %d" % (case["seqs"], case["T"]))
    n = case["seqs"]
    share = [2.0 ** (5 * r.random()) for _ in range(n)]
    if n >= 4:
        share[r.randrange(n)] = 0.0
    cuts = [0]
    for i in range(n):
        cuts.append(round(case["T"] * sum(share[:i + 1]) / sum(share)))
    return [cuts[i + 1] - cuts[i] for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    op = case["op"]
    s = dict(case)
    if op.startswith("delta"):
        dt = DT[case["dtype"]]
        H, P, G, N = case["H"], case["P"], case["G"], case["N"]
        lead = (case["b"],) if op == "delta_update" else (case["b"], case["T"])
        q, k = rnd(*lead, G, N), rnd(*lead, G, N)
        s["q"] = (q / q.norm(dim=-1, keepdim=True)).to(dt)          # unit vectors, as the rule wants its keys
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"] = rnd(*lead, H, P).to(dt)
        s["beta"] = torch.sigmoid(rnd(*lead, H))
        # log decay -exp(A) softplus(dt + bias): from about -1e-3 to a few
        rate = torch.exp(torch.rand(H, generator=gen, device="cuda") * 2.77)
        step = torch.exp(torch.rand(H, generator=gen, device="cuda") * 4.6 - 6.9)
        s["g"] = -rate * torch.nn.functional.softplus(rnd(*lead, H) + torch.log(torch.expm1(step)))
        s["scale"] = N ** -0.5
        if op == "delta_update":
            s["state"] = 0.1 * rnd(case["slots"], H, P, N)
            s["idx"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:case["b"]].to(torch.int32)
            return s
        s["lens"] = _lengths(case) if case["seqs"] else None
        s["cu"] = None
        nseq = case["b"]
        if case["seqs"]:
            nseq = case["seqs"]
            cu = [0]
            for n in s["lens"]:
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["h0"] = 0.1 * rnd(nseq, H, P, N)
        if op == "delta_bwd":
            s["dy"] = rnd(*lead, H, P).to(dt)
            s["dh"] = 0.1 * rnd(nseq, H, P, N)
        return s
    if op.startswith("norm"):
        dt = DT[case["dtype"]]
        R, Cn = case["rows"], case["C"]
        s["x"] = (rnd(R, Cn) * (0.5 + torch.rand(R, 1, generator=gen, device="cuda")) + 0.3).to(dt)
        s["z"] = rnd(R, Cn).to(dt) if case["gate"] in ("after", "before") else None
        s["w"] = 1 + 0.1 * rnd(Cn)
        s["bias"] = 0.1 * rnd(Cn)
        if op == "norm_bwd":
            s["dy"] = rnd(R, Cn).to(dt)
        return s
    slots = case["slots"]
    s["pool"] = rnd(slots, case["H"], case["P"], case["N"])
    s["cpool"] = rnd(slots, case["conv"]).to(torch.bfloat16) if case["conv"] else None
    perm = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
    s["table"] = perm[:case["live"]].contiguous()
    s["refs"] = torch.zeros(slots, dtype=torch.int32, device="cuda")
    s["refs"][s["table"].long()] = 1
    if op == "pages_fork":
        # one entry in eight asks for a fresh (zero) page; the others fork a live one, some of them the same
        at = torch.randint(0, case["live"], (case["n"],), generator=gen, device="cuda")
        s["src"] = s["table"][at].clone()
        s["src"][torch.rand(case["n"], generator=gen, device="cuda") < 0.125] = -1
    else:
        s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
    return s


# ------------------------------------------------------------------ the plain forms
def _unit_lower_inverse(m):
    """(I + m)^-1 of strictly lower triangular m, by halves: [[A, 0], [C, B]]^-1 = [[A^-1, 0], [-B^-1 C A^-1, B^-1]]."""
    n = m.shape[-1]
    if n == 1:
        return torch.ones_like(m)
    h = n // 2
    a, b = _unit_lower_inverse(torch.stack([m[..., :h, :h], m[..., h:, h:]])).unbind(0)
    low = -(b @ m[..., h:, :h] @ a)
    return torch.cat([torch.cat([a, torch.zeros_like(low)], -1), torch.cat([low, b], -1)], -2)


def _plain_delta(q, k, v, g, beta, h0, scale):
    """fp32 [B, T, ...] (T a multiple of CHUNK, rows behind a sequence's end with beta = g = 0): y, h_final."""
    B, T, H, P = v.shape
    R, Q = H // q.shape[2], CHUNK

    def chunks(t):                                           # [B, T, H, W] -> [B, H, T/Q, Q, W]
        return t.reshape(B, T // Q, Q, *t.shape[2:]).permute(0, 3, 1, 2, 4)

    q, k = (chunks(t.repeat_interleave(R, 2)) for t in (q, k))
    v, g, beta = chunks(v), chunks(g[..., None])[..., 0], chunks(beta[..., None])
    cs = g.double().cumsum(-1)
    lower = torch.ones(Q, Q, dtype=torch.bool, device=v.device).tril()
    decay = (cs[..., :, None] - cs[..., None, :]).masked_fill(~lower, -torch.inf).exp().float()
    into = cs.exp().float()[..., None]                       # from the chunk's start to token i, inclusive
    out = (cs[..., -1:] - cs).exp().float()[..., None]       # from token i to the chunk's end
    inv = _unit_lower_inverse((beta * decay * (k @ k.mT)).tril(-1))
    attn = decay * (q @ k.mT)
    h, ys = h0, []
    for c in range(T // Q):                                  # the recurrence itself, a chunk at a time
        kc = k[:, :, c]
        u = inv[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - into[:, :, c] * (kc @ h.mT)))
        ys.append(into[:, :, c] * (q[:, :, c] @ h.mT) + attn[:, :, c] @ u)
        h = into[:, :, c, -1:, :] * h + (out[:, :, c] * u).mT @ kc
    y = torch.stack(ys, 2).permute(0, 2, 3, 1, 4).reshape(B, T, H, P)
    return scale * y, h


def _pad_index(s):
    """Rows of the padded batch [nseq, Tmax]: token indices (one past the end where there is none)."""
    T = s["v"].shape[1]
    if s["cu"] is None:
        n, top = s["v"].shape[0], -(-T // CHUNK) * CHUNK
        t = torch.arange(top, device="cuda")
        first = torch.arange(n, device="cuda")[:, None] * T
        return torch.where(t[None] < T, first + t[None], n * T)
    top = -(-max(s["lens"]) // CHUNK) * CHUNK
    t = torch.arange(top, device="cuda")[None]
    first, last = s["cu"][:-1, None].long(), s["cu"][1:, None].long()
    return torch.where(first + t < last, first + t, T)


def _padded(t, idx):
    flat = t.reshape(-1, *t.shape[2:])
    return torch.cat([flat, torch.zeros_like(flat[:1])])[idx]


def _unpadded(t, idx, like):
    out = t.new_empty((like.shape[0] * like.shape[1] + 1, *t.shape[2:]))
    out[idx] = t
    return out[:-1].reshape(like.shape[0], like.shape[1], *t.shape[2:])


def _silu(z):
    return z * torch.sigmoid(z)


def _plain_norm(s, x, z, w, bias):
    R, Cn = x.shape
    if s["gate"] == "before":
        x = x * _silu(z)
    xg = x.reshape(R, s["groups"], -1)
    if s["mean"]:
        xg = xg - xg.mean(-1, keepdim=True)
    n = (xg * torch.rsqrt((xg * xg).mean(-1, keepdim=True) + 1e-5)).reshape(R, Cn) * w + bias
    return n * _silu(z) if s["gate"] == "after" else _silu(n) if s["gate"] == "silu" else n


def _plain_run(s):
    op = s["op"]
    if op in ("delta_fwd", "delta_bwd"):
        idx = _pad_index(s)
        ins = [t.float() for t in (s["q"], s["k"], s["v"], s["g"], s["beta"])] + [s["h0"]]
        if op == "delta_fwd":
            y, h = _plain_delta(*(_padded(t, idx) for t in ins[:5]), ins[5], s["scale"])
            return _unpadded(y, idx, s["v"]).to(s["v"].dtype), h
        ins = [t.detach().requires_grad_(True) for t in ins]
        with torch.enable_grad():
            y, h = _plain_delta(*(_padded(t, idx) for t in ins[:5]), ins[5], s["scale"])
            d = torch.autograd.grad([y, h], ins, [_padded(s["dy"].float(), idx), s["dh"]])
        dt = s["v"].dtype
        return dict(dq=d[0].to(dt), dk=d[1].to(dt), dv=d[2].to(dt), dg=d[3].to(dt), dbeta=d[4].to(dt), dh0=d[5])
    if op == "delta_update":
        R, at = s["H"] // s["G"], s["idx"].long()
        q, k = (s[n].float().repeat_interleave(R, 1) for n in ("q", "k"))
        w = s["state"][at] * s["g"].exp()[..., None, None]
        u = s["beta"][..., None] * (s["v"].float() - (w * k[:, :, None]).sum(-1))
        h = w + u[..., None] * k[:, :, None]
        s["state"][at] = h
        return (s["scale"] * (h * q[:, :, None]).sum(-1)).to(s["v"].dtype), s["state"]
    if op == "norm_fwd":
        z = None if s["z"] is None else s["z"].float()
        return _plain_norm(s, s["x"].float(), z, s["w"], s["bias"]).to(s["x"].dtype)
    if op == "norm_bwd":
        z = None if s["z"] is None else s["z"].float().detach().requires_grad_(True)
        x, w, bias = (t.float().detach().requires_grad_(True) for t in (s["x"], s["w"], s["bias"]))
        ins = [x, w, bias] + ([] if z is None else [z])
        with torch.enable_grad():
            d = torch.autograd.grad(_plain_norm(s, x, z, w, bias), ins, s["dy"].float())
        dt = s["x"].dtype
        return dict(dx=d[0].to(dt), dweight=d[1], dbias=d[2], dz=None if z is None else d[3].to(dt))
    pools = [s["pool"]] + ([] if s["cpool"] is None else [s["cpool"]])
    refs = s["refs"]
    if op == "pages_fork":
        pages = torch.argsort((refs != 0).to(torch.int32), stable=True)[:s["n"]].to(torch.int32)
        at, src = pages.long(), s["src"].long()
        for p in pools:
            got = p[src.clamp_min(0)]
            got[src < 0] = 0
            p[at] = got
        refs[at] = 1
        held = refs.clone()
        refs[at] -= 1                                        # given back again: the pool is as it was
        return [pages, held, refs] + pools
    s["table"].copy_(s["table0"])
    refs.copy_(s["refs0"])
    used = refs != 0
    n = used.sum()
    here = torch.arange(refs.numel(), device="cuda")
    # the i-th live page at or behind n goes to the i-th free page before it
    move = used & (here >= n)
    free = torch.argsort((used | (here >= n)).to(torch.int32), stable=True)
    new = torch.where(move, free[(move.cumsum(0) - 1).clamp_min(0)], here)
    src = torch.argsort((~move).to(torch.int32), stable=True)
    src = src[torch.minimum(here[:s["n"]], (move.sum() - 1).clamp_min(0))]  # entries past the moves repeat the last
    dst = new[src]
    for p in pools:
        p[dst] = p[src]
    s["table"].copy_(new[s["table"].long()])
    moved = refs.clone()
    moved[src] = torch.where(move[src], 0, refs[src])
    moved[torch.where(move[src], dst, src)] = torch.where(move[src], refs[src], moved[src])
    refs.copy_(moved)
    return [s["table"], refs] + pools


def _own_run(s):
    import state_space_model_conv1d_b200 as ssm
    op = s["op"]
    if op == "delta_fwd":
        return ssm.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], h0=s["h0"],
                             cu_seqlens=s["cu"])
    if op == "delta_bwd":
        return ssm.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], scale=s["scale"], h0=s["h0"],
                             cu_seqlens=s["cu"], dh_final=s["dh"])
    if op == "delta_update":
        y = ssm.delta_update(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"],
                             state_batch_indices=s["idx"])
        return y, s["state"]
    if op.startswith("norm"):
        kw = dict(weight=s["w"], bias=s["bias"], z=s["z"], subtract_mean=s["mean"], eps=1e-5,
                  gate_first=s["gate"] == "before", activation=s["gate"] == "silu")
        if op == "norm_fwd":
            return ssm.group_norm_fwd(s["x"], s["groups"], **kw)
        return ssm.group_norm_bwd(s["x"], s["groups"], s["dy"], **kw)
    pools = [s["pool"]] + ([] if s["cpool"] is None else [s["cpool"]])
    refs = s["refs"]
    if op == "pages_fork":
        pages = ssm.state_pages_fork(pools, refs, s["src"])
        held = refs.clone()
        ssm.state_pages_free(refs, pages)
        return [pages, held, refs] + pools
    s["table"].copy_(s["table0"])
    refs.copy_(s["refs0"])
    ssm.state_pages_compact(pools, refs, s["table"])
    return [s["table"], refs] + pools


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ------------------------------------------------------------------ the work
def work(case):
    op = case["op"]
    if op.startswith("delta"):
        es = 2 if case["dtype"] == "bf16" else 4
        H, P, G, N = case["H"], case["P"], case["G"], case["N"]
        t = case["b"] * case.get("T", 1)
        states = (case["seqs"] or case["b"]) if op != "delta_update" else case["b"]
        tok = es * (2 * G * N + 2 * H * P) + 8 * H           # q, k, v, y, g, beta
        if op == "delta_bwd":                                # q, k, v, dy, dq, dk, dv; g, beta, dg, dbeta
            tok = es * (4 * G * N + 3 * H * P + 2 * H) + 8 * H
        moved = 3 if op == "delta_bwd" else 2                # h0, dh_final, dh0 | h0, h_final
        # forward: h k, the update, h q; backward: those again for u and h, and seven products of the same size
        per = 18 if op == "delta_bwd" else 6
        return dict(bytes=t * tok + moved * 4 * states * H * P * N, flops=per * t * H * P * N)
    if op.startswith("norm"):
        es = 2 if case["dtype"] == "bf16" else 4
        z = case["gate"] in ("after", "before")
        n = case["rows"] * case["C"]
        if op == "norm_fwd":
            return dict(bytes=n * es * (3 if z else 2) + 8 * case["C"], flops=10 * n)
        return dict(bytes=n * es * (5 if z else 3) + 16 * case["C"], flops=25 * n)
    page = 4 * case["H"] * case["P"] * case["N"] + 2 * case["conv"]
    if op == "pages_fork":                                   # every fork writes a page, seven of eight read one
        return dict(bytes=1.875 * case["n"] * page, flops=0)
    # of live pages spread over the slots, the share behind the live count moves
    return dict(bytes=2 * page * case["live"] * (1 - case["live"] / case["slots"]), flops=0)


# ------------------------------------------------------------------ 64 bits
def _exact_seqs(s):
    """Inputs as a padded batch in 64 bits [nseq, Tmax, ...], the token mask, and the way back."""
    b, T = s["v"].shape[:2]
    rows = [(i, 0, T) for i in range(b)]
    if s["lens"] is not None:
        rows, at = [], 0
        for n in s["lens"]:
            rows.append((0, at, at + n))
            at += n
    top = max(e - f for _, f, e in rows)

    def pad(t):
        out = torch.zeros(len(rows), top, *t.shape[2:], dtype=torch.float64, device="cuda")
        for i, (r, f, e) in enumerate(rows):
            out[i, :e - f] = t[r, f:e].double()
        return out

    def back(t):
        out = torch.empty(b, T, *t.shape[2:], dtype=torch.float64, device="cuda")
        for i, (r, f, e) in enumerate(rows):
            out[r, f:e] = t[i, :e - f]
        return out

    R = s["H"] // s["G"]
    q, k = (pad(s[n]).repeat_interleave(R, 2) for n in ("q", "k"))
    # behind a sequence's end beta = g = 0: the state stays
    return q, k, pad(s["v"]), pad(s["g"]), pad(s["beta"]), pad, back


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("delta_fwd", "delta_bwd"):
        q, k, v, g, beta, pad, back = _exact_seqs(s)
        n, T, H, P = v.shape
        a, c = g.exp(), s["scale"]
        if op == "delta_bwd" and 8 * T * n * H * P * s["N"] > 60e9:
            return None
        h, y, path, us = s["h0"].double(), torch.empty_like(v), [], []
        for t in range(T):
            w = a[:, t, :, None, None] * h
            u = beta[:, t, :, None] * (v[:, t] - torch.einsum("shpn,shn->shp", w, k[:, t]))
            if op == "delta_bwd":
                path.append(h)
                us.append(u)
            h = w + u[..., None] * k[:, t, :, None]
            y[:, t] = c * torch.einsum("shpn,shn->shp", h, q[:, t])
        if op == "delta_fwd":
            return back(y), h
        dy, d = pad(s["dy"]), s["dh"].double()
        dq, dk = torch.zeros_like(q), torch.zeros_like(k)
        dv, dg, db = torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(beta)
        for t in reversed(range(T)):
            w = a[:, t, :, None, None] * path[t]
            kt, u, bt = k[:, t], us[t], beta[:, t, :, None]
            dq[:, t] = c * torch.einsum("shpn,shp->shn", w + u[..., None] * kt[:, :, None], dy[:, t])
            d = d + c * dy[:, t, ..., None] * q[:, t, :, None]
            du = torch.einsum("shpn,shn->shp", d, kt)
            ds = -bt * du
            dv[:, t] = bt * du
            db[:, t] = (du * (v[:, t] - torch.einsum("shpn,shn->shp", w, kt))).sum(-1)
            dk[:, t] = torch.einsum("shpn,shp->shn", d, u) + torch.einsum("shpn,shp->shn", w, ds)
            d = d + ds[..., None] * kt[:, :, None]
            dg[:, t] = (d * w).sum((-1, -2))
            d = a[:, t, :, None, None] * d
        dq, dk = (t.reshape(n, T, s["G"], -1, s["N"]).sum(3) for t in (dq, dk))
        return dict(dq=back(dq), dk=back(dk), dv=back(dv), dg=back(dg), dbeta=back(db), dh0=d)
    if op == "delta_update":
        state = s["state"].double()
        R = s["H"] // s["G"]
        q, k = (s[n].double().repeat_interleave(R, 1) for n in ("q", "k"))
        at = s["idx"].long()
        w = state[at] * s["g"].double().exp()[..., None, None]
        u = s["beta"].double()[..., None] * (s["v"].double() - torch.einsum("bhpn,bhn->bhp", w, k))
        h = w + torch.einsum("bhp,bhn->bhpn", u, k)
        state[at] = h
        return s["scale"] * torch.einsum("bhpn,bhn->bhp", h, q), state
    if op.startswith("norm"):
        x, w, bias = s["x"].double(), s["w"].double(), s["bias"].double()
        R, Cn = x.shape
        groups, gate = s["groups"], s["gate"]
        z = s["z"].double() if s["z"] is not None else None
        sg = None if z is None else torch.sigmoid(z)
        xin = x * z * sg if gate == "before" else x

        def split(t):
            return t.reshape(R, groups, Cn // groups)

        xc = split(xin) - split(xin).mean(-1, keepdim=True) if s["mean"] else split(xin)
        r = 1 / torch.sqrt(xc.square().mean(-1, keepdim=True) + 1e-5)
        n = (xc * r).reshape(R, Cn)
        t = n * w + bias
        st = torch.sigmoid(t)
        if op == "norm_fwd":
            return t * z * sg if gate == "after" else t * st if gate == "silu" else t
        dy, dz = s["dy"].double(), None
        if gate == "after":
            dz = dy * t * (sg + z * sg * (1 - sg))
            dt = dy * z * sg
        else:
            dt = dy * (st + t * st * (1 - st)) if gate == "silu" else dy
        dn = split(dt * w)
        dx = dn - split(n) * (dn * split(n)).mean(-1, keepdim=True)
        if s["mean"]:
            dx = dx - dn.mean(-1, keepdim=True)
        dx = (dx * r).reshape(R, Cn)
        if gate == "before":
            dz = dx * x * (sg + z * sg * (1 - sg))
            dx = dx * z * sg
        return dict(dx=dx, dweight=(dt * n).sum(0), dbias=dt.sum(0), dz=dz)
    pools = [s["pool"]] + ([] if s["cpool"] is None else [s["cpool"]])
    refs = s["refs"].tolist()
    if op == "pages_fork":
        pages = [i for i, n in enumerate(refs) if n == 0][:s["n"]]
        for p in pools:
            for to, src in zip(pages, s["src"].tolist()):
                p[to] = p[src] if src >= 0 else 0
        held = [1 if i in set(pages) else n for i, n in enumerate(refs)]
        return [torch.tensor(pages, dtype=torch.int32), torch.tensor(held, dtype=torch.int32), s["refs"]] + \
            [p.double() for p in pools]
    n = sum(r != 0 for r in refs)
    free = [i for i in range(n) if refs[i] == 0]
    src = [i for i in range(n, len(refs)) if refs[i] != 0]
    to = dict(zip(src, free))
    for p in pools:
        for f, t in to.items():
            p[t] = p[f]
    for f, t in to.items():
        refs[t], refs[f] = refs[f], 0
    table = [to.get(i, i) for i in s["table"].tolist()]
    return [torch.tensor(table, dtype=torch.int32), torch.tensor(refs, dtype=torch.int32)] + \
        [p.double() for p in pools]
