"""The full-cache decode (dsa_mla_decode_full) against float64.

Per element the library's decode tolerance, |err| <= 1e-2 + 1e-2*|ref| (parity.py), and over
a whole output a relative 2-norm of 3e-3: the bf16 rounding of an output is uniform over half
a step either way, 2^-8/sqrt(3) of the binade's lower end at most and 1.7e-3 in the mean over
a binade; probabilities are carried to half of 2^-8 relative, independent errors of
2^-9/sqrt(3) = 1.1e-3 rms; partial results in float16 add 2^-11/sqrt(3) = 0.3e-3. Together
2.1e-3.
"""
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


class Case:
    def __init__(self, n, rps, heads, lens, bs=64, pad=0, shared=False, two=False, verify=False, q_scale=1.0, seed=0):
        g = np.random.default_rng(seed + n * 100 + rps * 10 + heads)
        self.n, self.rps, self.heads, self.bs, self.verify = n, rps, heads, bs, verify
        R = n * rps
        self.given = np.resize(np.asarray(lens, np.int32), n if verify else R)
        self.lens = (self.given[:, None] + np.arange(rps) + 1).reshape(-1) if verify else self.given
        blocks = max(1, -(-int(self.lens.max()) // bs))
        self.blocks = 0 if shared else blocks
        self.stride = bs * 512 + pad
        tables = 1 if shared else n
        pages = tables * blocks + 2
        self.tables = g.permutation(pages)[:tables * blocks].reshape(tables, blocks).astype(np.int32)
        codes = lambda: torch.from_numpy(np.clip(g.normal(size=pages * self.stride) * 20, -448, 448).astype(np.float32)).to(  # noqa: E731
            torch.float8_e4m3fn).view(torch.uint8).numpy()
        self.k = codes()
        self.v = codes() if two else self.k
        self.q = ref.bf16(g.normal(size=(R, heads, 512)) * q_scale)
        self.scales = (0.05, 0.04 if two else 0.05, 512 ** -0.5)

    def device(self):
        k = torch.from_numpy(self.k).cuda()
        return [self.q.cuda(), k, k if self.v is self.k else torch.from_numpy(self.v).cuda(),
                torch.from_numpy(self.tables).cuda(), self.blocks, torch.from_numpy(self.given).cuda(), self.n, self.rps,
                self.heads, self.bs, self.stride, *self.scales]

    def run(self, api, **kw):
        return api.decode_full(*self.device(), verify_rows=int(self.verify), **kw)

    def want(self):
        return ref.full(ref.f64(self.q), self.k, self.v, self.tables, self.lens, self.rps, self.bs, self.stride, *self.scales)

    def check(self, api):
        ws = api.alloc_full_workspace(self.n, self.rps, self.heads)
        got = self.run(api, workspace=ws)
        assert api.read_device_status(ws) == 0
        want = self.want()
        assert_parity(got, want)
        norm = np.linalg.norm(want)
        if norm:
            assert np.linalg.norm(got.double().cpu().numpy() - want) <= 3e-3 * norm
        empty = self.lens <= 0
        assert (got[torch.from_numpy(empty).cuda()] == 0).all()
        return got


@pytest.mark.parametrize("n,rps,heads,lens,bs", [
    (1, 1, 16, [1], 64), (1, 1, 64, [63], 64), (1, 1, 64, [64], 64), (1, 1, 64, [65], 64), (3, 1, 64, [127, 128, 129], 64),
    (4, 1, 64, [0, 1, 0, 300], 64), (2, 1, 1, [700, 0], 64), (1, 1, 128, [1000], 64), (2, 1, 96, [333, 2000], 48),
    (1, 1, 200, [150], 16), (5, 2, 24, [0, 5, 100, 7, 300, 301, 64, 0, 513, 1], 100), (2, 4, 16, [700, 3, 0, 129, 1, 128, 900, 64], 64),
    (1, 3, 40, [1, 2, 3], 1), (1, 9, 8, [80 * i for i in range(9)], 128), (70, 1, 64, [100, 260, 33], 64),
    (300, 1, 8, [40, 0, 129], 32), (1, 1, 64, [6000], 64), (2, 1, 64, [900, 257], 256), (2, 2, 16, [900, 257, 1, 384], 384), (2, 1, 64, [3000, 4500], 7)])
def test_full(api, n, rps, heads, lens, bs):
    Case(n, rps, heads, lens, bs).check(api)


@pytest.mark.parametrize("n,rps,heads,lens,bs,two", [
    (2, 1, 64, [130001, 90000], 64, False), (1, 1, 128, [120000], 128, False), (40, 1, 16, [9000, 300, 5000, 1, 0], 64, False),
    (1, 2, 8, [150000, 149000], 48, False), (3, 1, 40, [20000, 40000, 127], 32, True)])
def test_long_rows(api, n, rps, heads, lens, bs, two):
    """Rows long enough that every CTA runs many tiles through its ring, over several units."""
    Case(n, rps, heads, lens, bs, two=two).check(api)


@pytest.mark.parametrize("n,rps,heads,base,bs", [
    (2, 4, 16, [700, 126], 64), (3, 4, 64, [0, 63, 500], 64), (1, 2, 128, [255], 64), (2, 3, 20, [1000, 62], 48), (4, 5, 8, [0], 64)])
def test_verify_rows(api, n, rps, heads, base, bs):
    Case(n, rps, heads, base, bs, verify=True).check(api)


def test_buffers_and_tables(api):
    Case(2, 1, 64, [500, 801], two=True).check(api)
    Case(2, 2, 24, [500, 801, 3, 64], two=True, pad=48).check(api)
    Case(2, 1, 64, [500, 801], pad=16 * 5, bs=16).check(api)
    Case(2, 1, 64, [500, 801], two=True, bs=256, pad=32).check(api)
    Case(1, 3, 24, [500, 801, 0], two=True, bs=20).check(api)
    Case(3, 1, 64, [500, 20, 801], shared=True).check(api)


def test_any_score_scale(api):
    """Negative and zero scales, and ones that make scores large."""
    for sm in (-(512 ** -0.5), 0.0, 0.3):
        c = Case(2, 2, 24, [700, 300, 128, 0])
        c.scales = (0.05, 0.05, sm)
        c.check(api)


def test_sharp_and_flat_scores(api):
    Case(2, 1, 64, [1500, 900], q_scale=12.0).check(api)
    Case(2, 1, 64, [1500, 900], q_scale=0.0).check(api)


def test_agrees_with_the_selected_decode(api):
    """With every position selected the selected decode computes the same."""
    c = Case(2, 1, 64, [900, 350])
    q, k, v, t, blocks, lens, n, rps, h, bs, stride, ks, vs, sm = c.device()
    sel = torch.arange(1024, dtype=torch.int32, device="cuda").repeat(2, 1)
    a = api.decode(q, k, v, t, blocks, lens, sel, n, rps, h, bs, stride, ks, vs, sm)
    b = c.run(api)
    assert (a.float() - b.float()).abs().max() <= 2 ** -7 * b.float().abs().max()


def test_nothing_hidden_reaches_a_row(api):
    """NaN codes past a row's length, in its last page and in pages that other rows see."""
    for heads in (16, 64):
        c = Case(1, 3, heads, [100, 300, 40])
        clean = c.run(api)
        for pos in (301, 319, 200, 120):
            at = int(c.tables[0, pos // 64]) * c.stride + (pos % 64) * 512
            c.k[at + 7] = 0x7F
        got = c.run(api)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
        assert torch.isnan(got[1]).all()


def test_broken_queries(api):
    c = Case(2, 1, 64, [100, 300])
    clean = c.run(api)
    for value in (float("nan"), float("inf")):
        c.q[1, 3, 9] = value
        got = c.run(api)
        assert torch.equal(got[0], clean[0])
        keep = [h for h in range(64) if h != 3]
        assert torch.equal(got[1, keep], clean[1, keep]) and torch.isnan(got[1, 3]).all()


def test_far_pages(api):
    """Cache offsets past 2^32 and 2^36 bytes / 16."""
    c = Case(1, 1, 64, [190])
    near = c.run(api)
    stride, pages = 1 << 24, 300
    cache = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
    far = torch.tensor([[299, 256, 260]], dtype=torch.int32, device="cuda")
    for i in range(3):
        at = int(c.tables[0, i]) * c.stride
        cache[int(far[0, i]) * stride:][:64 * 512] = torch.from_numpy(c.k[at:at + 64 * 512]).cuda()
    a = c.device()
    got = api.decode_full(a[0], cache, cache, far, 3, *a[5:10], stride, *c.scales)
    assert torch.equal(got, near)


def test_bad_tables_are_reported(api):
    c = Case(2, 1, 64, [639, 300])
    ok = c.run(api)
    c.tables[0, 4] = -1
    ws = api.alloc_full_workspace(2, 1, 64)
    got = c.run(api, workspace=ws)
    assert api.read_device_status(ws) == 6 and torch.equal(got[1], ok[1]) and torch.isfinite(got[0].float()).all()
    spare = next(i for i in range(c.k.size // c.stride) if i not in c.tables)
    c.k[spare * c.stride:(spare + 1) * c.stride] = 0                   # its positions: keys and values of zeros
    c.tables[0, 4] = spare
    assert_parity(got, c.want())
    c.tables[0, 4] = 0
    assert torch.isfinite(c.run(api, workspace=ws).float()).all() and api.read_device_status(ws) == 0
    a = c.device()
    a[3], a[4] = a[3][:, :5].contiguous(), 5                            # the table ends inside row 0
    got = api.decode_full(*a, workspace=ws)
    assert api.read_device_status(ws) == 6 and torch.equal(got[1], ok[1]) and torch.isfinite(got[0].float()).all()
    a[5] = torch.tensor([-3, 300], dtype=torch.int32, device="cuda")   # a negative length sees nothing
    got = api.decode_full(*a, workspace=ws)
    assert api.read_device_status(ws) == 0 and torch.equal(got[1], ok[1]) and (got[0] == 0).all()


@pytest.mark.parametrize("at", [0, 1700, 2999])
def test_flat_tails(api, at):
    """One dominant position, all others alike from 1/3 to 21 octaves below it, by head."""
    c = Case(1, 1, 64, [3000], two=True)
    one, half = torch.tensor([1.0, 0.5]).to(torch.float8_e4m3fn).view(torch.uint8).tolist()
    c.k[:] = half
    row = int(c.tables[0, at // 64]) * c.stride + at % 64 * 512
    c.k[row:row + 512] = one
    octaves = np.arange(1, 65) / 3
    c.q = ref.bf16(np.broadcast_to((octaves / (512 * 0.5 * c.scales[0] * c.scales[2] * np.log2(np.e)))[None, :, None], (1, 64, 512)))
    assert_parity(c.run(api), c.want())


@pytest.mark.parametrize("bs", [8, 12, 24, 40, 48, 56, 80, 96, 112, 160, 192])
def test_page_sizes(api, bs):
    """Pages that end inside a tile, with boxes of 8, 16 and 32 rows or none."""
    Case(3, 2, 40, [900, 1000, 2 * bs, 2 * bs + 1, bs - 1, 0], bs=bs).check(api)
    Case(1, 1, 64, [60000], bs=bs, pad=16).check(api)


def test_streams_graphs_and_repeats(api):
    c = Case(3, 2, 24, [1200, 1201, 60, 0, 700, 701])
    a = c.device()
    ws = api.alloc_full_workspace(3, 2, 24)
    want = api.decode_full(*a, workspace=ws)
    for _ in range(3):
        assert torch.equal(api.decode_full(*a, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.decode_full(*a, stream=side)
    other = api.decode_full(*a)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.decode_full(*a, out=out, workspace=ws)
    shorter = torch.tensor([3, 1201, 128, 127, 0, 650], dtype=torch.int32, device="cuda")
    expect = api.decode_full(*a[:5], shorter, *a[6:])
    a[5].copy_(shorter)
    for _ in range(2):
        out.fill_(7)
        graph.replay()
        assert torch.equal(out, expect)


def test_refusals(api):
    c = Case(1, 1, 64, [100])
    a = c.device()
    with pytest.raises(api.DsaError) as e:
        api.decode_full(*a, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")[:0])
    assert e.value.status in (1, 3)
    for i, v, code in ((9, 0, 1), (10, c.stride - 16, 1), (4, -1, 1)):
        with pytest.raises(api.DsaError) as e:
            api.decode_full(*[v if k == i else x for k, x in enumerate(a)])
        assert e.value.status == code
    for i, v in ((0, a[0].float()), (0, a[0][:, :32].contiguous()), (3, a[3].long()), (3, a[3][:, :1].contiguous()),
                 (5, a[5].cpu()), (6, 2), (9, 2**32 + c.bs)):
        with pytest.raises(ValueError):
            api.decode_full(*[v if k == i else x for k, x in enumerate(a)])
    with pytest.raises(ValueError):
        api.decode_full(*a, out=a[0][:, :32].contiguous())
