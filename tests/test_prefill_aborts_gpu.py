"""Calls of dsa_mla_prefill that give up at many places, by limits from none to longer than any wait: each
ends soon, records what happened, and leaves the next call alone."""
import time

import pytest
import torch

import test_prefill_gpu as prefill

pytestmark = pytest.mark.gpu
TIMEOUT = 7


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()
    return api


@pytest.mark.parametrize("base,new,heads,bs", [
    ([100] * 200, [8] * 200, 64, 64),    # units of one tile, many a cluster
    ([300] * 80, [9] * 80, 64, 100),     # of three, pages without boxes
    ([5000, 0], [40, 300], 64, 64), ([20000], [2], 64, 64)])
def test_calls_that_give_up(api, base, new, heads, bs):
    c = prefill.Case(base, new, heads, bs)
    a, ws = c.device(), api.alloc_prefill_workspace(len(base), c.q.shape[0], heads)
    out = torch.full(c.q.shape, prefill.UNTOUCHED, dtype=torch.bfloat16, device="cuda")
    want = c.run(api, workspace=ws)
    ended = set()
    for limit in (1, 500, 600, 800, 1000, 1500, 2000, 3000, 5000, 10000, 20000, 100000):
        for _ in range(3):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            with api.wait_limit(limit):
                api.prefill(*a, out=out, workspace=ws)
            status = api.read_device_status(ws)
            assert time.perf_counter() - t0 < 0.9  # a wait for what does not come takes 1 s
            assert status in (0, TIMEOUT) and api.step_device_status() == status
            ended.add(status)
            if status == 0:
                assert torch.equal(out, want), limit
            out.fill_(prefill.UNTOUCHED)
            assert torch.equal(api.prefill(*a, out=out, workspace=ws), want), limit
            assert api.read_device_status(ws) == 0
    assert TIMEOUT in ended
