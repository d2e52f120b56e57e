"""Pages of a state cache on the GPU: copy, fork, free, compact (whole values, so equality throughout)."""
import pytest
import torch

import state_space_model_conv1d_b200 as ssm
from state_space_model_conv1d_b200 import _abi

from layer_ref import compact_ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def ws():
    return torch.empty(1 << 22, dtype=torch.uint8, device="cuda")


def pools(n, seed=0, conv=33):
    gen = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(n, 3, 8, 24, generator=gen, device="cuda"),
            torch.randn(n, conv, 1, generator=gen, device="cuda").to(torch.bfloat16),
            torch.randint(0, 255, (n, 7), generator=gen, device="cuda", dtype=torch.uint8)]


def test_copy():
    p = pools(9)
    want = [t.clone() for t in p]
    for t in want:
        t[4], t[7], t[2] = t[1].clone(), t[1].clone(), 0
    w = ws()
    ssm.state_pages_copy(p, i32([1, 1, -1, 3, 5]), i32([4, 7, 2, -1, 5]), workspace=w)
    assert ssm.workspace_error(w) == 0
    assert all(torch.equal(a, b) for a, b in zip(p, want))


def test_copy_skips_what_conflicts():
    # entry 0 writes page 2, which entry 1 reads; entry 3 writes page 5 like entry 2; 4 and 5 lie outside
    p = pools(8)
    want = [t.clone() for t in p]
    for t in want:
        t[5], t[6] = t[0].clone(), t[2].clone()
    w = ws()
    ssm.state_pages_copy(p, i32([1, 2, 0, 4, 8, 0, -2]), i32([2, 6, 5, 5, 1, 8, 3]), workspace=w)
    assert ssm.workspace_error(w) == _abi.SSM_DEVERR_PAGES
    assert all(torch.equal(a, b) for a, b in zip(p, want))


def test_fork_takes_the_lowest_pages_in_order():
    p, refs = pools(8), i32([1, 0, 2, 0, 0, 1, 0, 0])
    want = [t.clone() for t in p]
    for t in want:
        t[1], t[3], t[4] = t[2].clone(), 0, t[2].clone()
    w = ws()
    pages = ssm.state_pages_fork(p, refs, i32([2, -1, 2]), workspace=w)
    assert ssm.workspace_error(w) == 0
    assert pages.tolist() == [1, 3, 4] and refs.tolist() == [1, 1, 2, 1, 1, 1, 0, 0]
    assert all(torch.equal(a, b) for a, b in zip(p, want))


def test_fork_of_dead_pages_and_a_full_pool():
    p, refs = pools(4), i32([1, 0, 1, 0])
    w = ws()
    # page 1 is free, 9 and -3 are no pages: no page is spent on them; the last fork finds none left
    pages = ssm.state_pages_fork(p, refs, i32([1, 0, 9, -3, 2, 0]), workspace=w)
    assert ssm.workspace_error(w) == _abi.SSM_DEVERR_PAGES
    assert pages.tolist() == [-1, 1, -1, -1, 3, -1] and refs.tolist() == [1, 1, 1, 1]
    assert torch.equal(p[0][1], p[0][0]) and torch.equal(p[1][3], p[1][2])


def test_free():
    refs = i32([1, 0, 3, 1])
    w = ws()
    ssm.state_pages_free(refs, i32([0, 2, -1, 2]), workspace=w)
    assert ssm.workspace_error(w) == 0 and refs.tolist() == [0, 0, 1, 1]
    ssm.state_pages_free(refs, i32([1, 3, 3, 4]), workspace=w)
    assert ssm.workspace_error(w) == _abi.SSM_DEVERR_PAGES and refs.tolist() == [0, 0, 1, 0]


@pytest.mark.parametrize("n,share", [(1, 1.0), (7, 0.5), (64, 0.0), (64, 1.0), (1500, 0.3), (5000, 0.7)])
def test_compact(n, share):
    gen = torch.Generator().manual_seed(n)
    refs = (torch.rand(n, generator=gen) < share).int() * torch.randint(1, 4, (n,), generator=gen)
    table = torch.randint(-1, n, (40,), generator=gen).int()
    p = pools(n, conv=5)
    want = [t.clone() for t in p]
    rrefs, rtable, to = compact_ref(refs.tolist(), table.tolist())
    for t in want:
        for f, d in to.items():
            t[d] = t[f].clone()
    r, tb, w = refs.int().cuda(), table.cuda(), ws()
    ssm.state_pages_compact(p, r, tb, workspace=w)
    assert r.tolist() == rrefs and tb.tolist() == rtable
    assert ssm.workspace_error(w) == (_abi.SSM_DEVERR_PAGES if any(a >= 0 > b for a, b in zip(table.tolist(), rtable)) else 0)
    assert all(torch.equal(a, b) for a, b in zip(p, want))


def test_large_pages_and_many_entries():
    n = 40
    p = [torch.randn(n, 300_001, device="cuda"), torch.randn(n, 5, device="cuda", dtype=torch.float64)]
    refs = i32([1] * 7 + [0] * (n - 7))
    pages = ssm.state_pages_fork(p, refs, i32([6, 2, -1] * 11))
    assert pages.tolist() == list(range(7, n))
    assert torch.equal(p[0][7:n:3], p[0][6].expand(11, -1)) and (p[0][9:n:3] == 0).all()
    many = torch.arange(3000, dtype=torch.int32, device="cuda") % n
    q = [torch.arange(6000, device="cuda", dtype=torch.int32).reshape(6000, 1)]
    ssm.state_pages_copy(q, many, torch.arange(3000, 6000, dtype=torch.int32, device="cuda"))
    assert torch.equal(q[0][3000:, 0], many)


def test_no_entries_and_empty_pools():
    refs = i32([1, 0])
    assert ssm.state_pages_fork([torch.zeros(2, 0, device="cuda")], refs, i32([])).numel() == 0
    assert ssm.state_pages_fork([torch.zeros(2, 0, device="cuda")], refs, i32([0])).tolist() == [1]
    ssm.state_pages_compact([torch.zeros(0, 4, device="cuda")], i32([]), i32([-1]))


def test_in_a_graph():
    p, refs = pools(12), i32([1, 1] + [0] * 10)
    src = i32([0, 1, -1])
    pages = i32([0, 0, 0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssm.state_pages_fork(p, refs, src, pages=pages)
    for first in (2, 5, 8):
        g.replay()
        torch.cuda.synchronize()
        assert pages.tolist() == [first, first + 1, first + 2]
        assert torch.equal(p[0][first], p[0][0]) and (p[0][first + 2] == 0).all()
