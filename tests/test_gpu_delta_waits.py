"""Waits of the delta rule's tensor-core kernels that run out: the kernel reports it and leaves, with nothing of its
own in flight, and the next call is as good as any.

The bounds-checked build takes the limit of a wait from a variable.  With limits from nothing up to what a whole
chain needs, the pre-pass, the chains and the blocks' gradients give up in different places; a call either reports
the time-out or is complete.  Nothing here waits for something that does not come: every copy and product that a
kernel has started ends by itself, and the kernel waits for it before it leaves.
"""
import pytest
import torch

import state_space_model_conv1d_b200 as ssm
from state_space_model_conv1d_b200 import _abi

from test_gpu_delta import cu_of, make

pytestmark = pytest.mark.gpu
DEFAULT = 2_000_000_000


@pytest.fixture
def limit(monkeypatch):
    chk = _abi.checked_lib()
    monkeypatch.setattr(_abi, "lib", lambda: chk)

    def set_limit(ns):
        assert chk.ssm_delta_wait_limit(ns) == _abi.SSM_OK

    yield set_limit
    set_limit(DEFAULT)


@pytest.mark.parametrize("P,N,H,G,lengths", [(128, 128, 4, 2, None), (64, 128, 4, 1, None), (64, 64, 3, 3, [200, 0, 70, 330]),
                                             (192, 104, 2, 1, [65, 400])], ids=str)
def test_waits_that_run_out(limit, P, N, H, G, lengths):
    T = sum(lengths) if lengths else 600
    cu, cud = cu_of(lengths) if lengths else (None, None)
    dev, _ = make(80, "bf16", 1, T, H, P, G, N, nseq=len(lengths) if lengths else 1)
    x = [dev[n] for n in ("q", "k", "v", "g", "beta")]
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def fwd():
        return ssm.delta_fwd(*x, h0=dev["h0"], cu_seqlens=cud, workspace=ws)

    def bwd():
        return tuple(ssm.delta_bwd(*x, dev["dy"], h0=dev["h0"], dh_final=dev["dh"], cu_seqlens=cud, workspace=ws).values())

    for call in (fwd, bwd):
        want = call()
        assert ssm.workspace_error(ws) == 0
        seen = []
        for ns in (0, 500, 1000, 1500, 2000, 3000, 4000, 5000, 6000, 8000, 10000, 15000, 30000, 100000):
            for _ in range(3):
                limit(ns)
                got = call()
                seen.append(ssm.workspace_error(ws))
                assert seen[-1] in (0, _abi.SSM_DEVERR_TIMEOUT)
                if seen[-1] == 0:
                    assert all(torch.equal(a, b) for a, b in zip(want, got))
                limit(DEFAULT)
                again = call()
                assert ssm.workspace_error(ws) == 0 and all(torch.equal(a, b) for a, b in zip(want, again)), ns
        assert seen[0] == _abi.SSM_DEVERR_TIMEOUT, seen


def test_the_limit_is_the_checked_builds():
    lib = _abi.lib()
    assert lib.ssm_delta_wait_limit(5) == _abi.SSM_ERR_UNSUPPORTED
    assert _abi.checked_lib().ssm_delta_wait_limit(-1) == lib.ssm_delta_wait_limit(-1) == _abi.SSM_ERR_INVALID_ARG
