"""The pooled index scores (dsa_pool_scores) against float64; the bound of each score is worked
out in step_ref.pool_scores. With small whole numbers every sum is exact and the scores, and
the selection made from them, must be equal."""
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


class Case:
    def __init__(self, n, rps, heads, q_pos, bs=64, kpool=4, pad=0, shared=False, whole=False, spare=0, seed=0):
        g = np.random.default_rng(seed + n * 100 + rps * 10 + heads)
        self.n, self.rps, self.heads, self.bs, self.kpool = n, rps, heads, bs, kpool
        R = n * rps
        self.q_pos = np.resize(np.asarray(q_pos, np.int32), R)
        self.n_pools = max(1, (int(self.q_pos.max()) + 1 + kpool - 1) // kpool) + spare
        blocks = max(1, -(-(int(self.q_pos.max()) + 1) // bs))
        self.blocks = 0 if shared else blocks
        self.stride = (bs * 132 + 15) // 16 * 16 + pad
        tables = 1 if shared else n
        pages = tables * blocks + 2
        self.tables = g.permutation(pages)[:tables * blocks].reshape(tables, blocks).astype(np.int32)
        self.cache = np.zeros(pages * self.stride, np.uint8)
        for p in range(pages):
            codes, scales = ref.index_page(self.cache, p, bs, self.stride)
            if whole:  # whole numbers 0..8 and scales 1 or 2
                codes[:] = np.array([0, 56, 64, 68, 72, 74, 76, 78, 80], np.uint8)[g.integers(0, 9, (bs, 128))] | \
                    (g.integers(0, 2, (bs, 128)).astype(np.uint8) << 7)
                scales[:] = g.integers(1, 3, bs)
            else:
                codes[:] = g.integers(0, 256, (bs, 128))
                codes[codes & 127 == 127] = 0
                scales[:] = g.uniform(0.001, 0.02, bs)
        if whole:
            self.q = ref.bf16(g.integers(-3, 4, (R, heads, 128)))
            self.w = torch.from_numpy(g.integers(-2, 4, (R, heads)).astype(np.float32))
        else:
            self.q = ref.bf16(g.normal(size=(R, heads, 128)) * np.exp(g.normal(size=(R, heads, 1)) * 2))
            self.w = torch.from_numpy(g.normal(size=(R, heads)).astype(np.float32))

    def run(self, api, out=None, status=None, stream=None):
        return api.pool_scores(self.q.cuda(), self.w.cuda(), torch.from_numpy(self.cache).cuda(),
                               torch.from_numpy(self.tables).cuda(), self.blocks, torch.from_numpy(self.q_pos).cuda(), self.n,
                               self.rps, self.heads, self.bs, self.stride, self.kpool, self.n_pools, out=out,
                               device_status=status, stream=stream)

    def want(self):
        return ref.pool_scores(ref.f64(self.q), ref.f64(self.w), self.cache, self.tables, self.q_pos, self.rps, self.bs,
                               self.stride, self.kpool, self.n_pools)

    def check(self, api, exact=False):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = self.run(api, status=status).cpu().numpy().astype(np.float64)
        want, tol = self.want()
        assert status.item() == 0
        hidden = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), hidden)
        err = np.abs(got[~hidden] - want[~hidden])
        assert (err <= (0 if exact else tol[~hidden])).all(), f"max err {err.max():.3g}, bound {tol[~hidden][err.argmax()]:.3g}"
        return got


@pytest.mark.parametrize("n,rps,heads,q_pos,bs,kpool", [
    (1, 1, 64, [0], 64, 1), (1, 1, 64, [3], 64, 4), (1, 1, 64, [2], 64, 4), (2, 1, 64, [-1, 255], 64, 4),
    (3, 1, 64, [126, 127, 128], 64, 4), (1, 1, 1, [700], 64, 4), (2, 2, 8, [500, 3, -1, 900], 16, 2),
    (2, 4, 32, list(range(992, 1000)), 64, 4), (1, 3, 20, [5000, 4999, 17], 48, 3), (2, 1, 128, [1023, 300], 64, 8),
    (2, 3, 128, [300], 100, 5), (1, 7, 40, [900, 0, 5, 127, 128, 130, 890], 128, 16), (1, 1, 64, [2000], 1, 4),
    (1, 2, 64, [2000, 1999], 7, 7), (2, 1, 48, [640, 1300], 32, 128), (1, 1, 64, [900], 64, 127), (1, 1, 64, [900], 64, 65),
    (1, 300, 16, list(range(300)), 64, 4), (2, 1, 64, [900, 1300], 256, 4), (1, 2, 64, [2000, 5], 16, 4), (1, 1, 32, [1500], 384, 2), (1, 130, 64, list(range(200, 330)), 64, 4), (40, 1, 64, [100, 2000], 64, 4)])
def test_scores(api, n, rps, heads, q_pos, bs, kpool):
    Case(n, rps, heads, q_pos, bs, kpool).check(api)


@pytest.mark.parametrize("n,rps,heads,q_pos,bs,kpool", [
    (3, 1, 64, [299999, 150001, 200000], 64, 4), (1, 2, 64, [400000, 399999], 128, 4), (1, 3, 24, [200001], 32, 2),
    (1, 1, 128, [260000], 64, 1), (2, 1, 32, [150000, 300001], 48, 3), (1, 2, 100, [260000, 80000], 64, 5),
    (40, 1, 16, [30000, 7000, 1], 64, 8)])
def test_long_rows(api, n, rps, heads, q_pos, bs, kpool):
    """Rows long enough that every block runs many tiles through its ring, over several units."""
    Case(n, rps, heads, q_pos, bs, kpool).check(api)


@pytest.mark.parametrize("heads,kpool", [(64, 4), (20, 3), (128, 1)])
def test_whole_numbers_are_exact(api, heads, kpool):
    Case(3, 2, heads, [700, 701, 10, 11, 1500, 1501], kpool=kpool, whole=True).check(api, exact=True)


def test_padded_pages_shared_table_and_hidden_pools(api):
    Case(2, 2, 64, [500, 501, 800, 801], pad=48).check(api)
    Case(3, 1, 64, [500, 20, 800], shared=True).check(api)
    got = Case(2, 1, 64, [100, 333], spare=77).check(api)
    assert np.isneginf(got[:, -77:]).all()


def test_rows_with_different_positions_share_keys(api):
    """What one row sees does not change with the rows beside it."""
    both = Case(1, 2, 64, [1500, 40])
    got = both.run(api).cpu()
    for r in range(2):
        one = Case(1, 2, 64, [1500, 40])
        one.q_pos[1 - r] = -1
        alone = one.run(api).cpu()
        assert torch.equal(alone[r], got[r]) and torch.isneginf(alone[1 - r]).all()


def test_broken_keys_reach_their_pool_alone(api):
    c = Case(1, 2, 64, [1000, 500])
    page = c.tables[0, 700 // 64]
    codes, scales = ref.index_page(c.cache, int(page), 64, c.stride)
    codes[700 % 64, 5] = 0x7F
    c2 = Case(1, 2, 64, [1000, 500])
    got, clean = c.run(api).cpu(), c2.run(api).cpu()
    assert torch.isnan(got[0, 700 // 4]) and torch.isneginf(got[1, 700 // 4])
    got[0, 700 // 4] = clean[0, 700 // 4]
    assert torch.equal(got, clean)
    # past every row's position nothing is read into a score
    page = c2.tables[0, 1004 // 64]
    codes, scales = ref.index_page(c2.cache, int(page), 64, c2.stride)
    codes[1001 % 64:] = 0x7F
    scales[1001 % 64:] = np.nan
    assert torch.equal(c2.run(api).cpu(), clean)


def test_broken_queries_reach_their_row_alone(api):
    clean = Case(2, 2, 64, [300])
    want = clean.run(api).cpu()
    for value in (float("nan"), float("inf")):
        c = Case(2, 2, 64, [300])
        c.q[1, 3, 7] = value
        got = c.run(api).cpu()
        assert torch.equal(got[[0, 2, 3]], want[[0, 2, 3]])
        seen = ~torch.isneginf(want[1])
        assert torch.isnan(got[1][seen]).all() and torch.isneginf(got[1][~seen]).all()
    c = Case(2, 2, 64, [300])
    c.w[2, 1] = float("nan")
    got = c.run(api).cpu()
    assert torch.equal(got[[0, 1, 3]], want[[0, 1, 3]]) and torch.isnan(got[2][~torch.isneginf(want[2])]).all()
    # a head without a weight, queries of zeros, and very large ones
    c = Case(1, 1, 64, [300])
    c.q[0, 0], c.w[0, 1] = 0, 0
    c.check(api)
    c.q[0, 2, 0] = 1e30
    c.w[0, 2] = 1e-30
    c.check(api)


def test_bad_pages_are_reported(api):
    for entry, blocks in ((-1, None), (None, 5)):
        c = Case(2, 1, 64, [639, 639])
        if entry is not None:
            c.tables[1, 3] = entry
        if blocks is not None:
            c.tables = np.ascontiguousarray(c.tables[:, :blocks])
            c.blocks = blocks
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.run(api, status=status).cpu().numpy()
        assert status.item() == 6
        ok = Case(2, 1, 64, [639, 639]).run(api).cpu().numpy()
        lost = np.zeros_like(ok, bool)
        if entry is not None:
            lost[1, 48:64] = True
        else:
            lost[:, 80:] = True
        assert np.isneginf(got[lost]).all() and np.array_equal(got[~lost], ok[~lost])
        c.run(api)                                                       # no status word: nothing to report to


def test_far_pages(api):
    """Page offsets past 2^32 bytes."""
    bs, stride, pages = 64, 1 << 20, 4200
    cache = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
    c = Case(1, 1, 64, [127], bs=bs)
    near = c.run(api)
    far = torch.tensor([[4198, 4100]], dtype=torch.int32, device="cuda")
    for i in range(2):
        at = int(c.tables[0, i]) * c.stride
        cache[int(far[0, i]) * stride:][:bs * 132] = torch.from_numpy(c.cache[at:at + bs * 132]).cuda()
    got = api.pool_scores(c.q.cuda(), c.w.cuda(), cache, far, 2, torch.from_numpy(c.q_pos).cuda(), 1, 1, 64, bs, stride, 4,
                          c.n_pools)
    assert torch.equal(got, near)


@pytest.mark.parametrize("kpool", [4, 3])
@pytest.mark.parametrize("bs", [8, 12, 24, 40, 48, 56, 80, 96, 112, 160, 192])
def test_page_sizes(api, bs, kpool):
    """Pages that end inside a tile, with boxes of 8, 16, 32 and 64 rows or none."""
    Case(3, 2, 32, [900, 1000, 2 * bs, 2 * bs + 1, bs - 1, -1], bs=bs, kpool=kpool).check(api)
    Case(1, 1, 64, [200000], bs=bs, kpool=kpool, pad=16).check(api)


@pytest.mark.parametrize("bs,kpool", [(32, 24), (64, 20), (16, 6), (64, 48), (24, 56), (128, 40), (64, 100), (16, 9), (8, 64), (64, 112)])
def test_tiles_of_whole_pools(api, bs, kpool):
    """Tiles of 72 to 128 tokens, by boxes and by copies, pools over several warps' lanes."""
    Case(3, 2, 32, [900, 1000, 2 * kpool - 1, 2 * kpool, kpool - 2, -1], bs=bs, kpool=kpool).check(api)
    Case(1, 1, 128, [3000], bs=bs, kpool=kpool).check(api)
    Case(2, 1, 64, [150000, 90001], bs=bs, kpool=kpool).check(api)


def test_streams_graphs_and_repeats(api):
    c = Case(3, 2, 64, [1200, 1201, 60, 61, 700, 701])
    want = c.run(api)
    q, w, cache, t, pos = (c.q.cuda(), c.w.cuda(), torch.from_numpy(c.cache).cuda(), torch.from_numpy(c.tables).cuda(),
                           torch.from_numpy(c.q_pos).cuda())
    call = lambda **k: api.pool_scores(q, w, cache, t, c.blocks, pos, c.n, c.rps, c.heads, c.bs, c.stride, c.kpool,  # noqa: E731
                                       c.n_pools, **k)
    for _ in range(3):
        assert torch.equal(call(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    other = call()
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out)
    q2 = q.flip(0).contiguous()
    expect = api.pool_scores(q2, w, cache, t, c.blocks, pos, c.n, c.rps, c.heads, c.bs, c.stride, c.kpool, c.n_pools)
    q.copy_(q2)
    graph.replay()
    assert torch.equal(out, expect)


def test_refusals(api):
    c = Case(1, 1, 64, [100])
    a = [c.q.cuda(), c.w.cuda(), torch.from_numpy(c.cache).cuda(), torch.from_numpy(c.tables).cuda(), c.blocks,
         torch.from_numpy(c.q_pos).cuda(), 1, 1, 64, 64, c.stride, 4, c.n_pools]
    for i, v, code in ((9, 0, 1), (10, c.stride - 16, 1), (11, 0, 1), (11, 129, 2)):
        with pytest.raises(api.DsaError) as e:
            api.pool_scores(*[v if k == i else x for k, x in enumerate(a)])
        assert e.value.status == code
    for i, v in ((0, a[0].float()), (0, a[0][:, :32].contiguous()), (1, a[1][:, :9].contiguous()), (3, a[3].long()),
                 (3, a[3][:, :1].contiguous()), (5, a[5].cpu()), (6, 2), (9, 2**32 + 64), (12, 2**32 + c.n_pools)):
        with pytest.raises(ValueError):
            api.pool_scores(*[v if k == i else x for k, x in enumerate(a)])
    with pytest.raises(ValueError):
        api.pool_scores(*a, out=torch.empty((1, 3), device="cuda"))
