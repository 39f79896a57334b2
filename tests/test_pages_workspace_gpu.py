"""One workspace for pools of several sizes in turn: each call finds it as it needs it."""
import numpy as np
import pytest
import torch

import test_pages_gpu as pages
from test_pages_gpu import cu

pytestmark = pytest.mark.gpu
LARGE, SMALL = 100000, 1000


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()
    return api


def small_fork(api, ws, forks):
    """Many forks of one request with a partly filled page: three lists of `forks` entries."""
    tables = np.full((1 + forks, 3), -1, np.int32)
    tables[0] = [5, 6, 7]
    lens = np.array([40] + [0] * forks, np.int32)
    dev = torch.zeros(SMALL, 16, dtype=torch.uint8, device="cuda")
    t, shares = cu(tables), torch.zeros(SMALL, dtype=torch.int32, device="cuda")
    free = torch.arange(100, SMALL, dtype=torch.int32, device="cuda")
    info = api.fork_pages([dev], cu(np.zeros(forks, np.int32)), cu(np.arange(1, 1 + forks, dtype=np.int32)), cu(lens), 16, t, free, shares,
                          workspace=ws)
    assert info.tolist() == [forks, forks, 0, 0]
    assert t[1:, 2].tolist() == list(range(100, 100 + forks)) and shares[5:7].tolist() == [forks, forks]


def small_compact(api, ws, g):
    tables = g.permutation(SMALL)[:400].reshape(8, 50).astype(np.int32)
    info = pages.run_compact(api, pages.pools_of(g, SMALL, (16, 32)), tables, np.full(8, 800, np.int32), 16,
                             g.integers(0, 3, SMALL).astype(np.int32), workspace=ws)
    assert info[1] > 100


def large_release(api, ws, g):
    tables = g.permutation(LARGE)[:50000].reshape(10, 5000).astype(np.int32)
    lens, keeps = np.full(10, 80000), g.integers(0, 80000, 10)
    free = np.full(LARGE, -1, np.int32)
    free[:10] = np.setdiff1d(np.arange(LARGE), tables.reshape(-1))[:10]
    info = pages.run_release(api, tables, lens, keeps, 16, np.zeros(LARGE, np.int32), free, 10, 4, workspace=ws)
    assert info[2] == 0


def large_compact(api, ws, g):
    tables = g.permutation(LARGE)[:30000].reshape(10, 3000).astype(np.int32)
    info = pages.run_compact(api, pages.pools_of(g, LARGE, (16, 16), (1, 1)), tables, np.full(10, 48000, np.int32), 16,
                             g.integers(0, 3, LARGE).astype(np.int32), workspace=ws)
    assert info[1] > 10000


@pytest.mark.parametrize("order", [("small_fork", "large_release"), ("small_fork", "large_compact"), ("small_compact", "large_release"),
                                   ("small_compact", "large_compact"), ("large_compact", "small_compact", "small_fork", "large_release"),
                                   ("large_release", "small_fork", "large_compact", "small_compact", "large_compact")])
def test_pools_take_turns(api, order):
    g = np.random.default_rng(len(order))
    ws = api.alloc_pages_workspace(LARGE)
    for what in order:
        if what == "small_fork":
            small_fork(api, ws, 800)
        else:
            globals()[what](api, ws, g)
