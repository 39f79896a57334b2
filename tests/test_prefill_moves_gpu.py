"""References that move on every tile in one CTA of a pair, in the other, or in both (dsa_mla_prefill): a move
that the products miss leaves what came before far too heavy."""
import numpy as np
import pytest
import torch

import step_ref as ref
import test_prefill_gpu as prefill
from parity import assert_parity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()
    return api


def rising(tiles, rows_up, new=2, heads=64, requests=1):
    """Scores that rise by 8 octaves or more a tile for the rows in rows_up (of each unit's two), and not
    for the others: dim 0 of the keys rises over the tiles, and only those rows' queries look at it."""
    c = prefill.Case([128 * tiles - new] * requests, [new] * requests, heads, two=True, seed=tiles)
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    steps = np.argsort(np.where(np.isfinite(codes) & (codes >= 2.0), codes, np.inf))[:tiles]  # ascending codes of 2.0 and more
    assert np.isfinite(codes[steps]).all() and (np.diff(codes[steps]) >= 0.25).all()
    for s in range(requests):
        for b in range(c.blocks):
            at = int(c.tables[s, b]) * c.stride
            for i in range(c.bs):
                c.k[at + i * 512] = steps[(b * c.bs + i) // 128]
    q = c.q.float()
    q[:, :, 0] = 0.0
    for t in range(q.shape[0]):
        if t % 2 in rows_up:  # two rows of 64 heads a unit: one for each CTA
            q[t] = 0.0  # beside an element this large the others would be off (a query is two 8-bit terms)
            q[t, :, 0] = 8.0 / (0.25 * c.scales[0] * c.scales[2] * np.log2(np.e))
    c.q = q.to(torch.bfloat16)
    return c


@pytest.mark.parametrize("rows_up", [(0,), (1,), (0, 1)])
@pytest.mark.parametrize("tiles,requests", [(2, 1), (40, 1), (9, 100)])
def test_moves_on_every_tile(api, rows_up, tiles, requests):
    c = rising(tiles, rows_up, requests=requests)
    got = c.run(api)
    assert api.step_device_status() == 0
    assert_parity(got[:6], c.want(set(range(6)))[:6])
    for _ in range(5):
        assert torch.equal(c.run(api), got)
