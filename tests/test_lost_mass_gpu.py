"""Rows whose probability lies in a first position, one moderate peak in 128 and a flat background
far below both: what the kernels' E4M3 terms lose of it, against float64.

A key with n dims of 1 (the others 0) scores n/512 of its head's F octaves, so every level is
exact. Keys are values too, 0 or 1 times v_scale = 1, so dim 0 of the output is the mass of
the first position and the peaks, dim 511 that of the first, and with the values in a buffer of
their own, all ones, every output is 1.

Bounds, on outputs of magnitude 1 at most: the whole-cache decode loses 2^-8 of a row and 1.22 *
2^-9 of each term (test_lost_mass_cpu.py), rounds a split row's parts to float16 (2^-12 each) and
the output to bf16 (2^-9): 8.6e-3 with the exponentials' 2^-18. The selected decode: 2^-8 and one tile's
128 * 1.5 * 2^-10 of a row's 2^6, 2^-9 of each term, then the same.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
FULL_BOUND = 2.0 ** -8 + 1.22 * 2.0 ** -9 + 2.0 ** -12 + 2.0 ** -9 + 2.0 ** -18
SELECTED_BOUND = 2.0 ** -8 + 128 * 1.5 * 2.0 ** -16 + 2.0 ** -9 + 2.0 ** -12 + 2.0 ** -9 + 2.0 ** -18
ONE = 0x38  # 1.0
FRACTIONS = [0, 150, 200, 240, 256, 290, 320, 333, 350, 384, 420, 460, 500]  # of 512: the peaks' level


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    return api


class Rows:
    """`n` rows of 64 heads over one cache of `length` positions; row r's head h has its first
    position F = 4 + h/4 + 4 (r % 2) octaves above the background."""

    def __init__(self, n, length, peak, at=5, bs=64):
        self.n, self.length, self.bs = n, length, bs
        pages = -(-length // bs)
        k = torch.zeros(pages * bs, 512, dtype=torch.uint8)
        k[at::128, :peak] = ONE
        k[0] = ONE
        self.k = k.view(-1).cuda()
        self.ones = torch.full_like(self.k, ONE)
        g = torch.Generator().manual_seed(peak)
        self.tables = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
        perm = torch.randperm(pages, generator=g).cuda()
        shuffled = torch.empty_like(self.k).view(pages, -1)
        shuffled[perm] = self.k.view(pages, -1)
        self.k, self.tables = shuffled.view(-1), perm.to(torch.int32).view(1, -1).contiguous()
        f = 4 + torch.arange(64) / 4 + 4 * (torch.arange(n) % 2)[:, None]
        self.q = f[:, :, None].expand(n, 64, 512).to(torch.bfloat16).contiguous().cuda()
        self.sm = 1 / (512 * np.log2(np.e))
        # mass of the first position and of the peaks, in float64
        f = f.double().numpy()
        peaks = len(range(at, length, 128))
        low = np.exp2(-f)
        first, peak_mass = np.ones_like(f), peaks * np.exp2(-f * (1 - peak / 512))
        total = first + peak_mass + (length - 1 - peaks) * low
        self.first, self.peaks = first / total, peak_mass / total
        if peak == 0:
            self.peaks = np.zeros_like(f)

    def check(self, got, bound, ones=False):
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all()
        if ones:
            assert np.abs(got - 1).max() <= bound
            return
        assert np.abs(got[:, :, 511] - self.first).max() <= bound
        assert np.abs(got[:, :, 0] - self.first - self.peaks).max() <= bound


@pytest.mark.parametrize("n,length,bs", [(1, 16384, 64), (10, 16347, 64), (76, 16384, 64), (304, 16384, 64), (304, 2000, 48),
                                         (152, 4096, 100)])
def test_whole_cache(api, n, length, bs):
    """Rows in one block, in two and in many, by boxes and by copies, keys as values and apart."""
    for peak in FRACTIONS:
        r = Rows(n, length, peak, bs=bs)
        lens = torch.full((n,), length, dtype=torch.int32, device="cuda")
        for values in (r.k, r.ones):
            got = api.decode_full(r.q, r.k, values, r.tables, 0, lens, n, 1, 64, bs, bs * 512, 1.0, 1.0, r.sm)
            r.check(got, FULL_BOUND, ones=values is r.ones)


def test_whole_cache_peaks_anywhere(api):
    """Peaks in the tokens of each thread of a pair."""
    for at in (1, 31, 32, 63, 64, 100, 127):
        r = Rows(152, 8192, 320, at=at)
        lens = torch.full((152,), 8192, dtype=torch.int32, device="cuda")
        for values in (r.k, r.ones):
            got = api.decode_full(r.q, r.k, values, r.tables, 0, lens, 152, 1, 64, 64, 64 * 512, 1.0, 1.0, r.sm)
            r.check(got, FULL_BOUND, ones=values is r.ones)


@pytest.mark.parametrize("tile", [64, 128])
@pytest.mark.parametrize("width,ctas", [(1024, 1), (2048, 1), (2048, 2), (2048, 3), (2048, 0), (8192, 1), (8192, 2), (8191, 7)])
def test_selected(api, width, ctas, tile):
    """Every position selected, in order; one row on one block, two, three and many."""
    n = 1 if ctas else 40
    ws = api.alloc_workspace(n, 1, 64, width, num_ctas=ctas)
    sel = torch.arange(width, dtype=torch.int32, device="cuda").repeat(n, 1)
    lens = torch.full((n,), width, dtype=torch.int32, device="cuda")
    for peak in FRACTIONS:
        r = Rows(n, width, peak)
        for values in (r.k, r.ones):
            got = api.decode_ws(r.q, r.k, values, r.tables, 0, lens, sel, n, 1, 64, 64, 64 * 512, 1.0, 1.0, r.sm,
                                torch.empty_like(r.q), ws, num_ctas=ctas, tile_tokens=tile)
            r.check(got, SELECTED_BOUND, ones=values is r.ones)
        assert api.read_device_status(ws) == 0
