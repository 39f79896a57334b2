"""The step plan (dsa_plan_step) against a token-by-token plan on the CPU: all outputs are
integers and must be equal, table entries that no new token needs included."""
import numpy as np
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    return api


def check(api, base, new, bs, rps, rows=None, width=None, spare=3, tables=None, seed=0):
    g = np.random.default_rng(seed)
    base, new = np.asarray(base, np.int32), np.asarray(new, np.int32)
    n = len(base)
    if width is None:
        width = max([1] + [-(-(max(0, int(b)) + max(0, int(k))) // bs) for b, k in zip(base, new)])
    if tables is None:
        tables = g.permutation(max(1, n) * width)[:n * width].reshape(n, width).astype(np.int32)
    need = sum(-(-(max(0, int(b)) + max(0, int(k))) // bs) - -(-max(0, int(b)) // bs) for b, k in zip(base, new))
    free = (100000 + g.permutation(max(0, need + spare))).astype(np.int32)
    if rows is None:
        rows = n * rps if rps else int(np.maximum(new, 0).sum()) + 5
    want = ref.plan(base, new, free, bs, tables, rps, rows)
    dev = torch.from_numpy(tables.copy()).cuda()
    got = api.plan_step(torch.from_numpy(base).cuda(), torch.from_numpy(new).cuda(), torch.from_numpy(free).cuda(), bs, dev,
                        rows_per_seq=rps, max_rows=rows)
    again = api.plan_step(torch.from_numpy(base).cuda(), torch.from_numpy(new).cuda(), torch.from_numpy(free).cuda(), bs, dev,
                          rows_per_seq=rps, max_rows=rows)
    for name, a, b, w in zip(("slots", "positions", "row_lens", "row_seqs", "info"), got, again, want):
        assert np.array_equal(a.cpu().numpy(), w), name
        assert np.array_equal(b.cpu().numpy(), w), f"{name}, run again"
    assert np.array_equal(dev.cpu().numpy(), want[5]), "block tables"
    return want


@pytest.mark.parametrize("bs", [1, 7, 16, 64, 100])
@pytest.mark.parametrize("rps", [0, 1, 4])
@pytest.mark.parametrize("n", [1, 2, 31, 257])
def test_plan(api, n, rps, bs):
    g = np.random.default_rng(n * 10 + rps)
    want = check(api, g.integers(0, 900, n), g.integers(0, (rps or 200) + 1, n), bs, rps)
    assert want[4][2] == 0


def test_no_requests_and_no_new_tokens(api):
    check(api, [], [], 64, 0, width=4)
    check(api, [], [], 64, 3, width=4)
    check(api, [5, 0, 64], [0, 0, 0], 64, 0)
    check(api, [5, 0, 64], [0, 0, 0], 64, 2, width=3)


def test_page_borders(api):
    for rps in (0, 70):
        check(api, [0, 63, 64, 65, 127, 128], [64, 1, 64, 63, 2, 0], 64, rps)


@pytest.mark.parametrize("n", [1000, 16384])
def test_many_requests(api, n):
    g = np.random.default_rng(n)
    check(api, g.integers(0, 300, n), g.integers(0, 5, n), 16, 0)
    check(api, g.integers(0, 300, n), g.integers(0, 3, n), 16, 2)


def test_long_prompt_and_dropped_rows(api):
    check(api, [0, 40000], [70001, 3], 64, 0)
    want = check(api, [0, 40, 9], [500, 30, 8], 16, 0, rows=300)      # rows past the capacity
    assert want[4][2] == 6 and want[4][0] == 300


def test_reported_problems(api):
    assert check(api, [10, 20], [50, 60], 16, 0, spare=-3)[4][2] == 6            # free pages run out
    assert check(api, [10, 20], [50, 60], 16, 0, spare=-100)[4][1] == 0          # none at all
    assert check(api, [-5, 20], [3, -1], 16, 0)[4][2] == 6                       # negative lengths
    assert check(api, [10, 20], [5, 2], 16, 3)[4][2] == 6                        # more tokens than rows
    assert check(api, [10, 100, 60], [5, 20, 9], 16, 0, width=4)[4][2] == 6      # past the table
    assert check(api, [10, 100, 60], [5, 20, 9], 16, 20, width=4)[4][2] == 6
    tables = np.arange(8, dtype=np.int32).reshape(2, 4)
    tables[1, 1] = -1                                                            # a cached token's page is missing
    assert check(api, [5, 20], [2, 3], 16, 0, width=4, tables=tables)[4][2] == 6
    tables[1, 1], tables[0, 0] = 5, -1                                           # not a page this step needs
    assert check(api, [16, 20], [2, 3], 16, 0, width=4, tables=tables)[4][2] == 0


def test_large_page_ids(api):
    """A slot past 2^31 (page ids are 32 bits, slots 64)."""
    t = torch.tensor([[2_000_000_000, 0]], dtype=torch.int32, device="cuda")
    one = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")  # noqa: E731
    p = api.plan_step(one(3), one(70), one(2_100_000_000), 64, t, rows_per_seq=70)
    assert p.slots[0].item() == 2_000_000_000 * 64 + 3 and p.slots[69].item() == 2_100_000_000 * 64 + 8


def test_kept_buffers_in_a_captured_step(api):
    """One captured plan follows the lengths that its input buffers hold at each replay."""
    n, bs, rps = 5, 16, 2
    base, new = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    free = torch.arange(1000, 1040, dtype=torch.int32, device="cuda")
    tables = torch.full((n, 8), -7, dtype=torch.int32, device="cuda")
    out = api.alloc_step_plan(n * rps)
    call = lambda: api.plan_step(base, new, free, bs, tables, rows_per_seq=rps, out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(3):
        g = np.random.default_rng(seed)
        b, k = g.integers(0, 100, n).astype(np.int32), g.integers(0, rps + 1, n).astype(np.int32)
        t = g.permutation(n * 8).reshape(n, 8).astype(np.int32)
        base.copy_(torch.from_numpy(b))
        new.copy_(torch.from_numpy(k))
        tables.copy_(torch.from_numpy(t))
        graph.replay()
        want = ref.plan(b, k, free.cpu().numpy(), bs, t, rps, n * rps)
        for a, w in zip(tuple(out) + (tables,), want):
            assert np.array_equal(a.cpu().numpy(), w)


def test_refusals(api):
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        api.plan_step(i(1, 2), i(1, 2), i(5), 64, t)                    # packed without max_rows
    with pytest.raises(ValueError):
        api.plan_step(i(1, 2), i(1), i(5), 64, t, rows_per_seq=1)
    with pytest.raises(ValueError):
        api.plan_step(i(1, 2), i(1, 2), i(5), 64, t.t().contiguous(), rows_per_seq=1)
    with pytest.raises(ValueError):
        api.plan_step(i(1, 2), i(1, 2), i(5), 64, t, rows_per_seq=2, max_rows=5)
    with pytest.raises(ValueError):
        api.plan_step(i(1, 2).long(), i(1, 2), i(5), 64, t, rows_per_seq=2)
    with pytest.raises(ValueError):
        api.plan_step(i(1, 2), i(1, 2), i(5), 64, t, max_rows=2**32 + 2)
    with pytest.raises(api.DsaError) as e:
        api.plan_step(i(1, 2), i(1, 2), i(5), 0, t, rows_per_seq=2)
    assert e.value.status == 1
