"""Tiles of the pooled scores whose pages are missing: all of a tile's, all of a row's, and tiles
that have some between tiles that have all."""
import numpy as np
import pytest
import torch

import step_ref as ref
from test_pool_scores_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    return api


@pytest.mark.parametrize("bs,kpool", [(64, 4), (16, 4), (8, 2), (32, 3), (128, 1), (100, 4)])
@pytest.mark.parametrize("which", ["all", "runs", "every third"])
def test_tiles_without_pages(api, bs, kpool, which):
    """Their pools score -inf whatever the ring held before, the others what they do with all pages."""
    def case():
        return Case(2, 1, 64, [40000, 39000], bs=bs, kpool=kpool)

    ok = case().run(api).cpu().numpy()
    c = case()
    i = np.arange(c.tables.shape[1])
    tiles = max(1, 128 // bs)  # entries of a tile or more
    gone = {"all": i >= 0, "runs": (i // (3 * tiles)) % 2 == 0, "every third": i % 3 == 0}[which]
    c.tables[1, gone] = -1 - (i[gone] % 5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.run(api, status=status).cpu().numpy()
    assert status.item() == ref.DEVICE_BOUNDS
    assert np.array_equal(got[0], ok[0])
    pos = np.arange(c.n_pools * kpool)
    lost = gone[np.minimum(pos // bs, len(gone) - 1)].reshape(-1, kpool)
    assert np.isneginf(got[1][lost.all(1)]).all()
    whole = ~lost.any(1)
    assert np.array_equal(got[1][whole], ok[1][whole])
    some = ~lost.all(1) & lost.any(1)  # the score of the positions that have a page
    assert (got[1][some] <= ok[1][some]).all()
