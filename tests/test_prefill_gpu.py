"""Attention of packed prompt chunks (dsa_mla_prefill) against float64: rows of ragged requests,
padding rows, masks inside a tile, pages of many sizes, broken codes and queries, tables and lengths
that do not fit, graphs and streams."""
import numpy as np
import pytest
import torch

import step_ref as ref
from parity import assert_parity

pytestmark = pytest.mark.gpu
UNTOUCHED = 0.03125


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()
    return api


class Case:
    def __init__(self, base, new, heads, bs=64, two=False, pad=0, shared=False, q_scale=1.0, extra=0, seed=0):
        g = np.random.default_rng(seed + heads + bs + sum(base))
        self.base, self.new = np.asarray(base, np.int32), np.asarray(new, np.int32)
        self.heads, self.bs, self.shared = heads, bs, shared
        n = len(base)
        self.blocks = max(1, max(-(-(max(0, b) + max(0, k)) // bs) for b, k in zip(base, new)))
        self.stride = bs * 512 + pad
        pages = (1 if shared else n) * self.blocks + 1
        order = g.permutation(pages)[:pages - 1].astype(np.int32)
        self.tables = order.reshape(1 if shared else n, self.blocks)
        codes = lambda: (torch.from_numpy(g.normal(size=pages * self.stride).astype(np.float32) * 20).clamp_(-448, 448)  # noqa: E731
                         .to(torch.float8_e4m3fn).view(torch.uint8).numpy())
        self.k = codes()
        self.v = codes() if two else self.k
        self.rows = int(np.maximum(self.new, 0).sum()) + extra
        self.q = ref.bf16(g.normal(size=(max(1, self.rows), heads, 512)) * q_scale)
        self.scales = (0.05, 0.05, 512 ** -0.5)

    def lens(self):
        """Request and visible length of each row."""
        at = [(s, max(0, int(b)) + i + 1) for s, (b, k) in enumerate(zip(self.base, self.new)) for i in range(max(0, int(k)))]
        return at[:self.q.shape[0]]

    def device(self):
        k = torch.from_numpy(self.k).cuda()
        v = k if self.v is self.k else torch.from_numpy(self.v).cuda()
        return [self.q.cuda(), k, v, torch.from_numpy(self.tables).cuda(), 0 if self.shared else self.blocks,
                torch.from_numpy(self.base).cuda(), torch.from_numpy(self.new).cuda(), self.heads, self.bs, self.stride, *self.scales]

    def run(self, api, **kw):
        out = torch.full(self.q.shape, UNTOUCHED, dtype=torch.bfloat16, device="cuda")
        return api.prefill(*self.device(), out=out, **kw)

    def want(self, rows=None):
        """float64, for the given rows (all of them)."""
        out = np.full(self.q.shape, UNTOUCHED)
        q, room = ref.f64(self.q), self.blocks * self.bs
        for t, (s, n) in enumerate(self.lens()):
            if rows is None or t in rows:
                table = self.tables[:1] if self.shared else self.tables[s:s + 1]
                out[t] = ref.full(q[t:t + 1], self.k, self.v, table, [min(n, room)], 1, self.bs, self.stride, *self.scales)[0]
        return out

    def check(self, api, rows=None):
        ws = api.alloc_prefill_workspace(len(self.base), self.q.shape[0], self.heads)
        got = self.run(api, workspace=ws)
        assert api.read_device_status(ws) == 0 and api.step_device_status() == 0
        want = self.want(rows)
        pick = sorted(rows) if rows is not None else list(range(len(want)))
        assert_parity(got[pick], want[pick])
        norm = np.linalg.norm(want[pick])
        assert np.linalg.norm(got[pick].double().cpu().numpy() - want[pick]) <= 3e-3 * norm
        assert (got[len(self.lens()):] == UNTOUCHED).all()
        return got


@pytest.mark.parametrize("base,new,heads,bs", [
    ([0], [1], 16, 64), ([0], [1], 64, 64), ([62], [1], 64, 64), ([63], [1], 64, 64), ([127], [3], 64, 64), ([0], [130], 64, 64),
    ([300], [5], 16, 64), ([0], [9], 1, 64), ([100], [200], 1, 64), ([700], [3], 128, 64), ([10], [4], 200, 16), ([500], [37], 20, 48),
    ([0, 5, 300], [7, 0, 1], 64, 64), ([0, 0, 0], [0, 0, 3], 64, 64), ([0, 64, 128, 1], [64, 64, 1, 127], 24, 64),
    ([5, 900, 0, 31, 400], [100, 1, 33, 0, 64], 16, 100), ([200, 0, 129], [40, 41, 1], 8, 1), ([1000], [70], 40, 7),
    ([128], [128], 96, 128), ([3, 2, 1], [1, 2, 3], 65, 32)])
def test_prefill(api, base, new, heads, bs):
    Case(base, new, heads, bs, extra=3).check(api)


def test_many_requests(api):
    g = np.random.default_rng(1)
    Case(g.integers(0, 200, 300).tolist(), g.integers(0, 3, 300).tolist(), 8, 32).check(api)
    Case(g.integers(0, 700, 80).tolist(), [1] * 80, 64, 64).check(api)


@pytest.mark.parametrize("base,new,heads,bs,two", [
    ([40000], [300], 64, 64, False), ([0], [2000], 64, 64, False), ([9000, 0, 20000], [130, 700, 1], 32, 48, False),
    ([30000], [100], 128, 32, True), ([0, 12000], [900, 500], 20, 100, True)])
def test_long_chunks(api, base, new, heads, bs, two):
    """Work enough that every CTA runs many tiles through its ring, over several units."""
    c = Case(base, new, heads, bs, two=two)
    rows = {0, 1, c.rows - 1, c.rows - 2} | set(np.random.default_rng(2).integers(0, c.rows, 24).tolist())
    c.check(api, rows)


@pytest.mark.parametrize("new", [2, 8, 10, 13, 18])
def test_units_in_many_pieces(api, new):
    """One to nine units over the same 47 tiles: pieces by the dozen, or few, on either side of the
    choice of a join."""
    Case([6000 - new], [new], 64).check(api)


def test_buffers_and_tables(api):
    Case([500, 3], [9, 40], 64, two=True).check(api)
    Case([500, 3], [9, 40], 24, two=True, pad=48).check(api)
    Case([500, 3], [9, 40], 64, 16, pad=16 * 5).check(api)
    Case([500, 3], [9, 40], 64, 256, two=True, pad=32).check(api)
    Case([500, 3], [9, 40], 24, 20, two=True).check(api)
    Case([500, 20, 0], [3, 70, 130], 64, shared=True).check(api)


@pytest.mark.parametrize("bs", [8, 12, 24, 40, 48, 56, 80, 96, 112, 160, 192])
def test_page_sizes(api, bs):
    """Pages that end inside a tile, with boxes of several sizes or none."""
    Case([900, 2 * bs, bs - 1, 0], [70, 1, 2, bs + 3], 40, bs, two=bs == 56).check(api)


def test_any_score_scale(api):
    for sm in (-(512 ** -0.5), 0.0, 0.3):
        c = Case([300, 0], [20, 40], 24)
        c.scales = (0.05, 0.05, sm)
        c.check(api)


@pytest.mark.parametrize("q_scale", [0.0, 2.0, 4.0, 12.0, 1e-30])
def test_sharp_and_flat_scores(api, q_scale):
    Case([900, 1500], [40, 9], 64, q_scale=q_scale).check(api)


@pytest.mark.parametrize("at", [0, 1700, 2995])
def test_flat_tails(api, at):
    """One dominant position, all others alike from 1/3 to 21 octaves below it, by head."""
    c = Case([2995], [5], 64, two=True)
    one, half = torch.tensor([1.0, 0.5]).to(torch.float8_e4m3fn).view(torch.uint8).tolist()
    c.k[:] = half
    row = int(c.tables[0, at // 64]) * c.stride + at % 64 * 512
    c.k[row:row + 512] = one
    octaves = np.arange(1, 65) / 3
    c.q = ref.bf16(np.broadcast_to((octaves / (512 * 0.5 * c.scales[0] * c.scales[2] * np.log2(np.e)))[None, :, None], (5, 64, 512)).copy())
    assert_parity(c.run(api), c.want())


def test_agrees_with_the_full_decode(api):
    """The rows of one request as verify rows."""
    c = Case([900], [6], 64)
    a = c.device()
    got = c.run(api)
    full = api.decode_full(a[0], a[1], a[2], a[3], c.blocks, a[5], 1, 6, 64, c.bs, c.stride, *c.scales, verify_rows=1)
    assert (got.float() - full.float()).abs().max() <= 2 ** -7 * full.float().abs().max()


@pytest.mark.parametrize("heads,two", [(16, False), (64, False), (64, True)])
def test_nothing_hidden_reaches_a_row(api, heads, two):
    """NaN codes behind a request's tokens in its last page, and in tokens that only later rows see."""
    c = Case([100, 30], [41, 5], heads, two=two)
    clean = c.run(api)
    for s, pos, dim in ((0, 141, 7), (0, 190, 300), (0, 120, 511), (0, 133, 2), (1, 36, 260), (1, 63, 0)):
        c.v[int(c.tables[s, pos // 64]) * c.stride + (pos % 64) * 512 + dim] = 0x7F
    got = c.run(api)
    for t, (s, n) in enumerate(c.lens()):
        if s == 0 and n > 120:
            assert torch.isnan(got[t, :, 511]).all(), t
        else:
            assert torch.equal(got[t], clean[t]), t


def test_broken_queries(api):
    c = Case([100, 300], [3, 4], 40)
    clean = c.run(api)
    for value in (float("nan"), float("inf"), -float("inf")):
        c.q[4, 3, 9] = value
        got = c.run(api)
        keep = [h for h in range(40) if h != 3]
        assert torch.equal(got[4, keep], clean[4, keep]) and torch.isnan(got[4, 3]).all()
        rows = [t for t in range(7) if t != 4]
        assert torch.equal(got[rows], clean[rows])


def test_far_pages(api):
    """Cache offsets past 2^32 and 2^36 bytes / 16."""
    c = Case([180], [10], 64)
    near = c.run(api)
    stride, pages = 1 << 24, 300
    cache = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
    far = torch.tensor([[299, 256, 260]], dtype=torch.int32, device="cuda")
    for i in range(3):
        at = int(c.tables[0, i]) * c.stride
        cache[int(far[0, i]) * stride:][:64 * 512] = torch.from_numpy(c.k[at:at + 64 * 512]).cuda()
    a = c.device()
    assert torch.equal(api.prefill(a[0], cache, cache, far, 3, *a[5:9], stride, *c.scales), near)


def test_bad_tables_are_reported(api):
    c = Case([600, 290], [39, 10], 64)
    ok = c.run(api)
    c.tables[0, 4] = -1
    ws = api.alloc_prefill_workspace(2, 49, 64)
    got = c.run(api, workspace=ws)
    assert api.read_device_status(ws) == 6 and api.step_device_status() == 6
    assert torch.equal(got[39:], ok[39:]) and torch.isfinite(got.float()).all()
    spare = next(i for i in range(c.k.size // c.stride) if i not in c.tables)
    c.k[spare * c.stride:(spare + 1) * c.stride] = 0                   # its positions: keys and values of zeros
    c.tables[0, 4] = spare
    assert_parity(got, c.want())
    c.tables[0, 4] = 0
    assert torch.isfinite(c.run(api, workspace=ws).float()).all() and api.read_device_status(ws) == 0
    a = c.device()
    a[3], a[4] = a[3][:, :9].contiguous(), 9                            # the table ends inside request 0
    got = api.prefill(*a, workspace=ws)
    assert api.read_device_status(ws) == 6 and torch.equal(got[39:], ok[39:])
    c.blocks = 9
    assert_parity(got, c.want())
    api.step_device_status()


def test_bad_lengths_are_reported(api):
    c = Case([-5, 100], [3, 4], 64)
    ws = api.alloc_prefill_workspace(2, 7, 64)
    got = c.run(api, workspace=ws)
    assert api.read_device_status(ws) == 6
    assert_parity(got, c.want())
    c = Case([50, 100], [-3, 4], 64, extra=1)
    ws = api.alloc_prefill_workspace(2, 5, 64)
    got = c.run(api, workspace=ws)
    assert api.read_device_status(ws) == 6
    assert_parity(got, c.want())
    c = Case([50, 100, 7], [3, 4, 2], 64)                               # more tokens than rows
    c.q = c.q[:5].contiguous()
    ws = api.alloc_prefill_workspace(3, 5, 64)
    got = c.run(api, workspace=ws)
    assert api.read_device_status(ws) == 6
    assert_parity(got, c.want())
    c = Case([50, 100], [0, 0], 64, extra=4)                            # no new token at all
    ws = api.alloc_prefill_workspace(2, 4, 64)
    assert (c.run(api, workspace=ws) == UNTOUCHED).all() and api.read_device_status(ws) == 0
    api.step_device_status()


def test_streams_graphs_and_repeats(api):
    c = Case([1200, 0, 60, 700], [30, 200, 0, 1], 24, extra=5)
    a = c.device()
    ws = api.alloc_prefill_workspace(4, c.q.shape[0], 24)
    want = c.run(api, workspace=ws)
    for _ in range(3):
        assert torch.equal(c.run(api, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.prefill(*a, stream=side)
    other = api.prefill(*a)
    side.synchronize()
    assert torch.equal(got[:231], want[:231]) and torch.equal(other[:231], want[:231])
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.prefill(*a, out=out, workspace=ws)
    for base, new in (([3, 128, 0, 650], [90, 0, 128, 18]), ([0, 0, 0, 0], [0, 0, 0, 0]), ([1200, 0, 60, 700], [30, 200, 0, 1])):
        c.base, c.new = np.array(base, np.int32), np.array(new, np.int32)
        a[5].copy_(torch.from_numpy(c.base)), a[6].copy_(torch.from_numpy(c.new))
        for _ in range(2):
            out.fill_(UNTOUCHED)
            graph.replay()
            assert torch.equal(out, c.run(api))
        assert_parity(out, c.want())


def test_prompts_through_the_plan(api):
    """A mixed step as a serving loop runs it: plan, cache writer, attention, in one captured graph that
    is replayed with other requests; against float64 over the caches as written."""
    g = np.random.default_rng(5)
    n, rows, bs, blocks, heads = 5, 160, 64, 6, 16
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    tables, base, new = z(n, blocks), z(n), z(n)
    free = torch.arange(n * blocks, dtype=torch.int32, device="cuda").flip(0).contiguous()
    cache, kv_a, q = z(n * blocks * bs * 512, dtype=torch.uint8), z(rows, 512, dtype=torch.bfloat16), z(rows, heads, 512, dtype=torch.bfloat16)
    norm, out = torch.ones(512, dtype=torch.bfloat16, device="cuda"), z(rows, heads, 512, dtype=torch.bfloat16)
    plan, ws = api.alloc_step_plan(rows), api.alloc_prefill_workspace(n, rows, heads)

    def step():
        api.plan_step(base, new, free, bs, tables, max_rows=rows, out=plan)
        api.latent_write(kv_a, norm, plan.slots, 1e-6, 0.05, bs, bs * 512, cache)
        api.prefill(q, cache, cache, tables, blocks, base, new, heads, bs, bs * 512, 0.05, 0.05, 512 ** -0.5, out=out, workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    now = np.zeros(n, np.int32)
    for grow in ([70, 1, 0, 64, 20], [1, 60, 90, 1, 0], [100, 2, 3, 1, 50]):
        grow = np.array(grow, np.int32)
        base.copy_(torch.from_numpy(now)), new.copy_(torch.from_numpy(grow))
        kv_a.copy_(ref.bf16(g.normal(size=(rows, 512))))
        q.copy_(ref.bf16(g.normal(size=(rows, heads, 512))))
        out.fill_(UNTOUCHED)
        graph.replay()
        torch.cuda.synchronize()
        taken = int(plan.info[1])
        assert plan.info[2].item() == 0 and api.read_device_status(ws) == 0
        free.copy_(torch.cat([free[taken:], free[:taken]]))
        held, t = cache.cpu().numpy(), tables.cpu().numpy()
        lens, seqs = plan.row_lens.cpu().numpy(), plan.row_seqs.cpu().numpy()
        want = np.full((rows, heads, 512), UNTOUCHED)
        for r in range(rows):
            if seqs[r] >= 0:
                want[r] = ref.full(ref.f64(q[r:r + 1]), held, held, t[seqs[r]:seqs[r] + 1], lens[r:r + 1], 1, bs, bs * 512, 0.05, 0.05,
                                   512 ** -0.5)[0]
        assert_parity(out, want)
        now += grow


def test_refusals(api):
    c = Case([100], [4], 64)
    a = c.device()
    with pytest.raises(api.DsaError) as e:
        api.prefill(*a, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")[:0])
    assert e.value.status in (1, 3)
    for i, v, code in ((8, 0, 1), (9, c.stride - 16, 1), (4, -1, 1)):
        with pytest.raises(api.DsaError) as e:
            api.prefill(*[v if k == i else x for k, x in enumerate(a)])
        assert e.value.status == code
    for i, v in ((0, a[0].float()), (0, a[0][:, :, :32].contiguous()), (3, a[3].long()), (3, a[3][:, :1].contiguous()), (5, a[5].cpu()),
                 (6, a[6][:0].contiguous()), (7, 0), (7, 48), (8, 2**32 + c.bs)):
        with pytest.raises(ValueError):
            api.prefill(*[v if k == i else x for k, x in enumerate(a)])
    with pytest.raises(ValueError):
        api.prefill(*a, out=a[0][:, :32].contiguous())
