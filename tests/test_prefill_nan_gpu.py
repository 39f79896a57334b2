"""NaN codes in the cache of a prompt chunk (dsa_mla_prefill), element by element: what a row gets does not
depend on the unit it lies in. A NaN in a visible value makes its own dim NaN, one in a visible key the
row (its scores are NaN), and every other element is what it is without them."""
import numpy as np
import pytest
import torch

import test_prefill_gpu as prefill

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


def place(c, pool, s, pos, dim, code):
    pool[int(c.tables[s, pos // c.bs]) * c.stride + pos % c.bs * 512 + dim] = code


def spots(c, seed):
    """Request, position, dims and code: before all rows, at new tokens (each unit has some of its rows
    before them), at the last one, and behind it in its page."""
    g = np.random.default_rng(seed)
    out = []
    for s, (b, k) in enumerate(zip(c.base.tolist(), c.new.tolist())):
        at = {b - 1, b, b + k - 1, b + k, *g.integers(b, b + k + 1, 6).tolist()} if k else {b}
        for pos in sorted(at):
            if 0 <= pos < c.blocks * c.bs:
                out.append((s, pos, g.choice(512, int(g.integers(1, 4)), replace=False), (0x7F, 0xFF)[int(g.integers(2))]))
    return out


CASES = [([100, 30], [41, 5], 16, 64), ([100, 30], [41, 5], 64, 64), ([0], [300], 1, 64), ([200, 0, 3], [40, 130, 1], 20, 100),
         ([500], [9], 128, 24), ([700, 1], [6, 200], 40, 32), ([5982], [18], 64, 64), ([6000, 900], [2, 1], 64, 48), ([5990], [10], 20, 64),
         ([100] * 100, [7] * 100, 24, 64)]


@pytest.mark.parametrize("base,new,heads,bs", CASES)
def test_values(api, base, new, heads, bs):
    c = prefill.Case(base, new, heads, bs, two=True, extra=2)
    clean = c.run(api)
    assert torch.isfinite(clean.float()).all()
    todo = spots(c, heads)
    for s, pos, dims, code in todo:
        for d in dims:
            place(c, c.v, s, pos, int(d), code)
    want = clean.clone()
    for t, (s, n) in enumerate(c.lens()):
        for s2, pos, dims, _ in todo:
            if s == s2 and pos < n:
                want[t, :, torch.from_numpy(dims).cuda()] = float("nan")
    assert torch.isnan(want).any() and not torch.isnan(want).all(dim=2).any()
    got = c.run(api)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert api.step_device_status() == 0


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("base,new,heads,bs", CASES[:8])
def test_keys(api, base, new, heads, bs, two):
    """In a pool that is both, a code that breaks the values breaks the keys too."""
    c = prefill.Case(base, new, heads, bs, two=two, extra=2)
    clean = c.run(api)
    s, k = max(enumerate(new), key=lambda x: x[1])
    pos = base[s] + k // 2
    place(c, c.k, s, pos, 77, 0x7F)
    want = clean.clone()
    for t, (s2, n) in enumerate(c.lens()):
        if s2 == s and pos < n:
            want[t] = float("nan")
    got = c.run(api)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
