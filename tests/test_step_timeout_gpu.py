"""The bounded waits of the pooled scores and the whole-cache decode: with a limit of 1 ns a wait
gives up at once; the call records DSA_ERR_TIMEOUT, drains and exits, and the next one is right."""
import pytest
import torch

import test_decode_full_gpu as full
import test_pool_scores_gpu as scores

pytestmark = pytest.mark.gpu
TIMEOUT = 7


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    return api


@pytest.mark.parametrize("n,rps,heads,q_pos,bs,kpool", [
    (2, 1, 64, [9000, 5000], 64, 4), (3, 4, 64, [30000], 64, 4), (1, 1, 64, [9000], 100, 4),  # boxes of both widths, copies
    (40, 1, 16, [7000, 1], 64, 8), (2, 1, 128, [60000, 70000], 48, 3)])                      # many units, long ranges
def test_pool_scores(api, n, rps, heads, q_pos, bs, kpool):
    c = scores.Case(n, rps, heads, q_pos, bs, kpool)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with api.wait_limit(1):
        c.run(api, status=status)
        torch.cuda.synchronize()
    assert status.item() == TIMEOUT
    c.check(api)


@pytest.mark.parametrize("n,rps,heads,lens,bs,two", [
    (2, 1, 64, [5000, 300], 64, False), (1, 1, 64, [40000], 100, False), (3, 2, 40, [0, 900, 1, 20000, 64, 7], 64, True),
    (200, 1, 64, [700], 32, False)])
def test_decode_full(api, n, rps, heads, lens, bs, two):
    c = full.Case(n, rps, heads, lens, bs, two=two)
    ws = api.alloc_full_workspace(n, rps, heads)
    with api.wait_limit(1):
        c.run(api, workspace=ws)
        torch.cuda.synchronize()
    assert api.read_device_status(ws) == TIMEOUT
    got = c.run(api, workspace=ws)
    assert api.read_device_status(ws) == 0
    c.check(api)
    assert torch.equal(got, c.run(api))


def test_limits_nest_and_belong_to_a_thread(api):
    import threading
    c = full.Case(1, 1, 64, [3000])
    ws = api.alloc_full_workspace(1, 1, 64)
    seen = []

    def other():
        c.run(api, workspace=ws)
        seen.append(api.read_device_status(ws))

    with api.wait_limit(10 ** 9):
        with api.wait_limit(1):
            t = threading.Thread(target=other)
            t.start()
            t.join()
        c.run(api, workspace=ws)
        seen.append(api.read_device_status(ws))
    assert seen == [0, 0]
    with pytest.raises(ValueError):
        with api.wait_limit(-1):
            pass
