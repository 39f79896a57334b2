"""dsa_step_device_status: what pooled scores without a status word and whole-cache decodes without
a kept workspace record is not lost."""
import pytest
import torch

import test_decode_full_gpu as full
import test_pool_scores_gpu as scores

pytestmark = pytest.mark.gpu
BOUNDS, TIMEOUT = 6, 7


@pytest.fixture
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()  # what other tests left
    return api


def bad_scores(bs):
    c = scores.Case(2, 1, 64, [639, 639], bs=bs)
    c.tables[1, 1] = -1
    return c


def bad_full(bs):
    c = full.Case(2, 1, 64, [639, 300], bs=bs)
    c.tables[0, 1] = -1
    return c


@pytest.mark.parametrize("bs", [64, 100])
def test_bad_pages(api, bs):
    scores.Case(2, 1, 64, [639, 639], bs=bs).run(api)
    full.Case(2, 1, 64, [639, 300], bs=bs).run(api)
    assert api.step_device_status() == 0
    for c in (bad_scores(bs), bad_full(bs)):
        c.run(api)
        assert api.step_device_status() == BOUNDS
        assert api.step_device_status() == 0


def test_lengths_past_the_table(api):
    c = full.Case(2, 1, 64, [639, 300])
    a = c.device()
    a[3], a[4] = a[3][:, :5].contiguous(), 5
    api.decode_full(*a)
    assert api.step_device_status() == BOUNDS


def test_kept_words(api):
    """A status word of the caller's takes the scores' status, a workspace shares the decode's."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad_scores(64).run(api, status=status)
    assert status.item() == BOUNDS and api.step_device_status() == 0
    ws = api.alloc_full_workspace(2, 1, 64)
    bad_full(64).run(api, workspace=ws)
    assert api.read_device_status(ws) == BOUNDS and api.step_device_status() == BOUNDS
    full.Case(2, 1, 64, [639, 300]).run(api, workspace=ws)
    assert api.read_device_status(ws) == 0 and api.step_device_status() == 0


def test_first_of_a_step(api):
    """The first status stays until it is read, whatever runs after it."""
    with api.wait_limit(1):
        full.Case(2, 1, 64, [6000, 300]).run(api)
    bad_scores(64).run(api)
    full.Case(2, 1, 64, [639, 300]).run(api)
    assert api.step_device_status() == TIMEOUT
    assert api.step_device_status() == 0


def test_captured_and_on_another_stream(api):
    c = bad_full(64)
    a, ws = c.device(), api.alloc_full_workspace(2, 1, 64)
    out = api.decode_full(*a, workspace=ws)
    assert api.step_device_status() == BOUNDS
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.decode_full(*a, out=out, workspace=ws)
    assert api.step_device_status() == 0
    for _ in range(2):
        graph.replay()
        assert api.step_device_status() == BOUNDS
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bad = bad_scores(64)
    bad.run(api, stream=side)
    assert api.step_device_status(stream=side) == BOUNDS


def test_refusal(api):
    assert api._lib.load().dsa_step_device_status(None, None) == 1
