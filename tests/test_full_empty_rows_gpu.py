"""Rows of length 0 beside live ones in the whole-cache decode: a captured step's padding rows,
whose queries hold anything. Their outputs are zeros and the live rows' what they are alone."""
import numpy as np
import pytest
import torch

import step_ref as ref
from parity import assert_parity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    return api


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("n,rps,heads,lens,bs", [
    (1, 4, 16, [300, 0, 128, 0], 64),       # one unit, whole rows
    (2, 4, 16, [0, 5000, 0, 4097], 64),     # split over blocks
    (1, 2, 96, [0, 700], 100),              # units with both rows' heads, by copies
    (3, 2, 24, [0, 0, 64, 0, 0, 1], 64),    # a unit without a token among live ones
    (1, 3, 16, [0, -7, 20000], 128)])       # split in many, a negative length
def test_broken_queries_of_empty_rows(api, n, rps, heads, lens, bs, fill):
    g = np.random.default_rng(heads + len(lens))
    lens = np.resize(np.asarray(lens, np.int32), n * rps)
    blocks = -(-int(lens.max()) // bs)
    tables = g.permutation(n * blocks).reshape(n, blocks).astype(np.int32)
    cache = torch.from_numpy(np.clip(g.normal(size=n * blocks * bs * 512) * 20, -448, 448).astype(np.float32)).to(
        torch.float8_e4m3fn).view(torch.uint8)
    q = ref.bf16(g.normal(size=(n * rps, heads, 512)))
    want = ref.full(ref.f64(q), cache.numpy(), cache.numpy(), tables, lens, rps, bs, bs * 512, 0.05, 0.05, 512 ** -0.5)
    dev = [cache.cuda(), cache.cuda(), torch.from_numpy(tables).cuda(), blocks, torch.from_numpy(lens).cuda(), n, rps, heads, bs,
           bs * 512, 0.05, 0.05, 512 ** -0.5]
    clean = api.decode_full(q.cuda(), *dev)
    assert_parity(clean, want)
    empty = torch.from_numpy(lens <= 0)
    q[empty] = fill
    got = api.decode_full(q.cuda(), *dev)
    assert (got[empty.cuda()] == 0).all()
    assert torch.equal(got, clean)
    one = q.clone()
    one[empty] = 1.0
    one[int(empty.nonzero()[0]), heads - 1, 511] = fill                    # a single broken element
    assert torch.equal(api.decode_full(one.cuda(), *dev), clean)
