"""Plain 64-bit forms of the operators beside the scan (numpy, token by token),
the oracle of their tests, and the tolerances."""
import numpy as np

# Largest rounding error of one value relative to it: half a step.
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def delta_ref(q, k, v, g, beta, scale, h0=None, cu=None):
    """y, h_final and the trajectory [(w, u)] per sequence; q, k [b,T,G,N], v [b,T,H,P], g, beta [b,T,H]."""
    b, T, H, P = v.shape
    G, N = q.shape[2:]
    R = H // G
    seqs = [(i, 0, T) for i in range(b)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    y, hf, traj = np.zeros(v.shape), np.zeros((len(seqs), H, P, N)), []
    for s, (r, lo, hi) in enumerate(seqs):
        h = np.zeros((H, P, N)) if h0 is None else h0[s].copy()
        path = []
        for t in range(lo, hi):
            kk, qq = (np.repeat(x[r, t], R, 0) for x in (k, q))
            w = np.exp(g[r, t])[:, None, None] * h
            u = beta[r, t][:, None] * (v[r, t] - np.einsum("hpn,hn->hp", w, kk))
            h = w + u[..., None] * kk[:, None]
            y[r, t] = scale * np.einsum("hpn,hn->hp", h, qq)
            path.append((w, u, h))
        hf[s] = h
        traj.append((r, lo, hi, path))
    return y, hf, traj


def delta_bwd_ref(q, k, v, g, beta, scale, dy, dh_final=None, h0=None, cu=None):
    H, G = v.shape[2], q.shape[2]
    R = H // G
    _, hf, traj = delta_ref(q, k, v, g, beta, scale, h0, cu)
    out = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    out["dh0"] = np.zeros(hf.shape)
    for s, (r, lo, hi, path) in enumerate(traj):
        d = np.zeros(hf.shape[1:]) if dh_final is None else dh_final[s].copy()
        for t in range(hi - 1, lo - 1, -1):
            w, u, h = path[t - lo]
            kk, qq = (np.repeat(x[r, t], R, 0) for x in (k, q))
            dyt, bt = scale * dy[r, t], beta[r, t][:, None]
            out["dq"][r, t] = np.einsum("hpn,hp->hn", h, dyt).reshape(G, R, -1).sum(1)
            d = d + dyt[..., None] * qq[:, None]
            du = np.einsum("hpn,hn->hp", d, kk)
            ds = -bt * du
            out["dv"][r, t] = bt * du
            out["dbeta"][r, t] = (du * (v[r, t] - np.einsum("hpn,hn->hp", w, kk))).sum(-1)
            dk = np.einsum("hpn,hp->hn", d, u) + np.einsum("hpn,hp->hn", w, ds)
            out["dk"][r, t] = dk.reshape(G, R, -1).sum(1)
            d = d + ds[..., None] * kk[:, None]
            out["dg"][r, t] = (d * w).sum((1, 2))
            d = np.exp(g[r, t])[:, None, None] * d
        out["dh0"][s] = d
    return out


def norm_ref(x, groups, w=None, b=None, z=None, mean=False, eps=1e-5, first=False, act=False):
    silu = lambda a: a / (1 + np.exp(-a))
    s = x * silu(z) if first else x
    sg = s.reshape(*s.shape[:-1], groups, -1)
    if mean:
        sg = sg - sg.mean(-1, keepdims=True)
    n = (sg / np.sqrt((sg * sg).mean(-1, keepdims=True) + eps)).reshape(s.shape)
    t = n * (1 if w is None else w) + (0 if b is None else b)
    return silu(t) if act else t * silu(z) if z is not None and not first else t


def norm_bwd_ref(x, groups, dy, w=None, b=None, z=None, mean=False, eps=1e-5, first=False, act=False):
    sig = lambda a: 1 / (1 + np.exp(-a))
    C = x.shape[-1]
    w = np.ones(C) if w is None else w
    b = np.zeros(C) if b is None else b
    sp = lambda a: a.reshape(*a.shape[:-1], groups, -1)
    s = x * z * sig(z) if first else x
    c = sp(s) - sp(s).mean(-1, keepdims=True) if mean else sp(s)
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = (c * r).reshape(x.shape)
    t, dt, dz = n * w + b, dy, None
    if act:
        dt = dy * (sig(t) + t * sig(t) * (1 - sig(t)))
    elif z is not None and not first:
        dz = dy * t * (sig(z) + z * sig(z) * (1 - sig(z)))
        dt = dy * z * sig(z)
    dn = sp(dt * w)
    dx = dn - sp(n) * (dn * sp(n)).mean(-1, keepdims=True) - (dn.mean(-1, keepdims=True) if mean else 0)
    dx, term = (dx * r).reshape(x.shape), (dn * r).reshape(x.shape)
    out = dict(dx=dx, dz=dz, dweight=(dt * n).sum(lead := tuple(range(x.ndim - 1))), dbias=dt.sum(lead))
    out["terms"] = dict(dx=term)
    if first:
        into = dict(dx=z * sig(z), dz=x * (sig(z) + z * sig(z) * (1 - sig(z))))
        for name, f in into.items():
            out[name], out["terms"][name] = dx * f, term * f
    return out


def compact_ref(refs, table):
    """New refs, table and {from: to} of a compaction."""
    refs, n = list(refs), sum(r > 0 for r in refs)
    free = [i for i in range(n) if refs[i] <= 0]
    src = [i for i in range(n, len(refs)) if refs[i] > 0]
    live = {i for i, r in enumerate(refs) if r > 0}
    to = dict(zip(src, free))
    for f, t in to.items():
        refs[t], refs[f] = refs[f], 0
    return refs, [p if p < 0 else to.get(p, p) if p in live else -1 for p in table], to
