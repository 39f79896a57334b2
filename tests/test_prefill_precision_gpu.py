"""What the prompt chunks' 8-bit terms lose (dsa_mla_prefill): the mass of flat backgrounds and moderate
peaks far below a row's first position, with the bound that the whole-cache decode has (the same
account, the same terms: test_lost_mass_gpu.py derives it); and heads with one query element far
above the others, whose small elements are what the two terms make of them, no less."""
import numpy as np
import pytest
import torch

import step_ref as ref
import test_prefill_gpu as prefill
from parity import assert_parity
from test_lost_mass_gpu import FRACTIONS, FULL_BOUND, Rows
from test_prefill_query_cpu import split

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


@pytest.mark.parametrize("n,length,bs", [(1, 16384, 64), (10, 16347, 64), (76, 16384, 64), (304, 2000, 48), (152, 4096, 100)])
def test_flat_backgrounds(api, n, length, bs):
    """Rows as requests of one new token over one cache, whole and in pieces, by boxes and by copies."""
    new = torch.ones(n, dtype=torch.int32, device="cuda")
    for peak in FRACTIONS:
        r = Rows(n, length, peak, bs=bs)
        for values in (r.k, r.ones):
            got = api.prefill(r.q, r.k, values, r.tables, 0, new * (length - 1), new, 64, bs, bs * 512, 1.0, 1.0, r.sm)
            r.check(got, FULL_BOUND, ones=values is r.ones)


@pytest.mark.parametrize("factor", [100, 300, 1000, 3000, 1e6])
def test_one_large_query_element(api, factor):
    """Keys are the same in that dim, so the others alone tell them apart."""
    c = prefill.Case([700, 0], [20, 150], 24)
    c.k.reshape(-1, 512)[:, 200] = 0x30  # 0.5
    q = c.q.float()
    q[:, :, 200] = q.abs().amax(2) * factor
    c.q = q.to(torch.bfloat16)
    got = c.run(api)
    c.q = split(c.q)
    want = c.want()
    assert_parity(got, want)
    assert np.linalg.norm(ref.f64(got) - want) <= 3e-3 * np.linalg.norm(want)
