"""Pins of the 64-bit forms in layer_ref.py: closed forms and central differences (no GPU)."""
import numpy as np
import pytest

from layer_ref import compact_ref, delta_bwd_ref, delta_ref, norm_bwd_ref, norm_ref


def _inputs(rng, b, T, H, P, G, N):
    k = rng.standard_normal((b, T, G, N))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return [rng.standard_normal((b, T, G, N)), k, rng.standard_normal((b, T, H, P)), -rng.random((b, T, H)),
            rng.random((b, T, H))]


def test_delta_beta_one_unit_key_reads_back_the_value():
    # beta = 1 and |k| = 1 write exactly v at k: h_t k_t = v_t, whatever was there
    q, k, v, g, beta = _inputs(np.random.default_rng(0), 1, 9, 2, 3, 1, 5)
    y, hf, _ = delta_ref(k, k, v, g, np.ones_like(beta), 1.0)
    assert np.allclose(y, v, atol=1e-12)


def test_delta_orthogonal_keys_is_the_plain_sum():
    # keys that never meet again: no correction, h = sum of decayed outer products
    T, N, P = 4, 6, 3
    rng = np.random.default_rng(1)
    k = np.eye(N)[None, :T, None]
    v, g, beta = rng.standard_normal((1, T, 1, P)), -rng.random((1, T, 1)), rng.random((1, T, 1))
    _, hf, _ = delta_ref(k, k, v, g, beta, 1.0)
    want = sum(np.exp(g[0, t + 1:, 0].sum()) * beta[0, t, 0] * np.outer(v[0, t, 0], k[0, t, 0]) for t in range(T))
    assert np.allclose(hf[0, 0], want, atol=1e-12)


def test_delta_split_and_packed():
    rng = np.random.default_rng(2)
    x = _inputs(rng, 1, 11, 4, 3, 2, 5)
    h0 = rng.standard_normal((2, 4, 3, 5))
    y, hf, _ = delta_ref(*x, 0.7, h0, [0, 4, 11])
    ya, ha, _ = delta_ref(*[t[:, :4] for t in x], 0.7, h0[:1])
    yb, hb, _ = delta_ref(*[t[:, 4:] for t in x], 0.7, h0[1:])
    assert np.allclose(y, np.concatenate([ya, yb], 1)) and np.allclose(hf, np.concatenate([ha, hb]))


def _differences(f, args, grads, rng, eps=1e-6):
    for i, gname in grads:
        for _ in range(6):
            at = tuple(int(rng.integers(n)) for n in args[i].shape)
            hi, lo = ([a.copy() for a in args] for _ in range(2))
            hi[i][at] += eps
            lo[i][at] -= eps
            num = (f(*hi) - f(*lo)) / (2 * eps)
            assert abs(num - gname[at]) <= 1e-6 * max(1, abs(num)), (i, at, num, gname[at])


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_delta_backward_against_differences(cu):
    rng = np.random.default_rng(3)
    x = _inputs(rng, 1, 7, 4, 3, 2, 5)
    h0 = rng.standard_normal((1 if cu is None else 3, 4, 3, 5))
    dy, dh = rng.standard_normal(x[2].shape), rng.standard_normal(h0.shape)

    def f(*a):
        y, hf, _ = delta_ref(*a[:5], 0.7, a[5], cu)
        return (y * dy).sum() + (hf * dh).sum()

    d = delta_bwd_ref(*x, 0.7, dy, dh, h0, cu)
    _differences(f, [*x, h0], [(i, d[n]) for i, n in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0"))], rng)


@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("mode", ["plain", "silu", "gate", "first"])
def test_norm_backward_against_differences(mode, mean):
    rng = np.random.default_rng(4)
    x, z, w, b, dy = (rng.standard_normal(s) for s in ((3, 12), (3, 12), (12,), (12,), (3, 12)))
    kw = dict(mean=mean, first=mode == "first", act=mode == "silu")
    gate = mode in ("gate", "first")

    def f(x, w, b, z):
        return (dy * norm_ref(x, 3, w, b, z if gate else None, **kw)).sum()

    d = norm_bwd_ref(x, 3, dy, w, b, z if gate else None, **kw)
    _differences(f, [x, w, b, z], [(0, d["dx"]), (1, d["dweight"]), (2, d["dbias"])] + ([(3, d["dz"])] if gate else []), rng)


def test_norm_closed_form():
    assert np.allclose(norm_ref(np.array([[3.0, 4.0, 0.0, 2.0]]), 2, eps=0.0),
                       [[3 / np.sqrt(12.5), 4 / np.sqrt(12.5), 0, np.sqrt(2)]])
    assert np.allclose(norm_ref(np.array([[1.0, 3.0]]), 1, mean=True, eps=0.0), [[-1, 1]])


def test_compact():
    refs, table, to = compact_ref([0, 2, 0, 1, 1], [4, -1, 3, 1, 2])
    assert to == {3: 0, 4: 2} and refs == [1, 2, 1, 0, 0] and table == [2, -1, 0, 1, -1]
