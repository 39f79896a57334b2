"""The index-key writer (dsa_index_write) against float64.

Scales: float32 sums of 128 terms (11 roundings deep), a square root, two divisions and the
weight: under 64 roundings of 2^-24 relative to the largest |y| while the mean is not far
above the spread, so 2^-18. Codes: equal to the float64 result's unless that lies within a
relative 2^-17 of a rounding midpoint (y and the scale each within 2^-18), where either
neighbour is correct.
"""
import numpy as np
import pytest
import torch

import oracle
import step_ref as ref

pytestmark = pytest.mark.gpu
TIE = 2.0 ** -17


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    oracle.build()
    import sparse_mla_paged_gb300.api as api
    return api


def check(api, x, w, b, slots, bs, pad=0, eps=1e-6, stream=None):
    stride = api.index_page_stride(bs) + pad
    pages = int(max(slots.max(initial=0), 0)) // bs + 2
    start = np.random.default_rng(5).integers(0, 256, pages * stride, dtype=np.uint8)
    cache = torch.from_numpy(start.copy()).cuda()
    put = lambda t: None if t is None else t.cuda()  # noqa: E731
    api.index_write(x.cuda(), torch.from_numpy(slots).cuda(), bs, stride, cache, norm_weight=put(w), norm_bias=put(b),
                    eps=eps)
    got = cache.cpu().numpy()
    vals, scales = ref.index_keys(ref.f64(x), None if w is None else ref.f64(w), None if b is None else ref.f64(b), eps)
    left = np.ones(got.size, bool)
    for r, slot in enumerate(slots):
        if slot < 0:
            continue
        at, off = int(slot // bs) * stride, int(slot % bs)
        codes, sc = ref.index_page(got, int(slot // bs), bs, stride)
        left[at + off * 128:at + (off + 1) * 128] = False
        left[at + bs * 128 + 4 * off:at + bs * 128 + 4 * off + 4] = False
        assert abs(sc[off] - scales[r]) <= 2.0 ** -18 * scales[r], f"row {r}: scale"
        want = oracle.e4m3_encode(vals[r])
        bad = np.nonzero(codes[off] != want)[0]
        lo, hi = oracle.e4m3_encode(vals[r, bad] * (1 - TIE)), oracle.e4m3_encode(vals[r, bad] * (1 + TIE))
        # a zero keeps no sign that matters
        zero = (codes[off][bad] & 127 == 0) & (want[bad] & 127 == 0)
        assert (zero | ((lo != hi) & ((codes[off][bad] == lo) | (codes[off][bad] == hi)))).all(), f"row {r}: codes"
    assert np.array_equal(got[left], start[left]), "bytes outside the written rows changed"


@pytest.mark.parametrize("rows,bs,pad,scale,norm", [
    (1, 64, 0, 1.0, 2), (2, 1, 12, 1.0, 1), (37, 64, 0, 30.0, 2), (200, 16, 80, 1e-3, 0), (129, 100, 0, 1.0, 2),
    (1000, 48, 0, 5.0, 1), (333, 128, 16, 1e-30, 0)])
def test_writer(api, rows, bs, pad, scale, norm):
    g = np.random.default_rng(rows)
    x = ref.bf16((g.normal(size=(rows, 128)) + 0.3) * scale)
    w, b = ref.bf16(g.uniform(0.5, 1.5, 128)), ref.bf16(g.normal(size=128) * 0.1)
    slots = g.permutation(rows + 3 * bs)[:rows].astype(np.int64)
    if rows > 2:
        slots[rows // 2] = -1
    if bs == 1:
        pad = 12  # 132 bytes a page round up to 144
    check(api, x, w if norm else None, b if norm == 2 else None, slots, bs, pad - pad % 16)


def test_midpoints_between_codes(api):
    """Keys that lie exactly between two codes round to the even one, also where 1 / s is inexact."""
    rows = np.zeros((48, 128))
    for i in range(48):
        step = (3, 5, 7)[i % 3] * 2.0 ** (i - 24)                           # s; the largest key is 448 of it
        rows[i] = np.tile((np.arange(8, 16) + 0.5) * 2.0 ** (i % 4), 16) * step * np.where(np.arange(128) % 3, 1, -1)
        rows[i, 5] = 448 * step
    x = ref.bf16(rows)
    assert np.array_equal(ref.f64(x), rows)
    stride = api.index_page_stride(48)
    cache = torch.zeros(stride, dtype=torch.uint8, device="cuda")
    api.index_write(x.cuda(), torch.arange(48, device="cuda"), 48, stride, cache)
    codes, scales = ref.index_page(cache.cpu().numpy(), 0, 48, stride)
    vals, s = ref.index_keys(rows, None, None, 0.0)
    assert np.array_equal(scales, s.astype(np.float32)) and np.array_equal(scales.astype(np.float64), s)
    assert np.array_equal(codes, oracle.e4m3_encode(vals))


def test_extreme_values(api):
    rows = np.zeros((6, 128))
    rows[1] = 3.0                                  # constant: nothing left after the mean
    rows[2, 5] = 1e-38                             # below the scale's floor
    rows[3] = np.linspace(-3e38, 3e38, 128)        # no norm: the scale carries the range
    rows[4, ::2], rows[4, 1::2] = 1.0, -1.0
    rows[5, 7] = -448.0
    check(api, ref.bf16(rows), None, None, np.arange(6, dtype=np.int64), 4)
    w = ref.bf16(np.ones(128))
    check(api, ref.bf16(rows[[0, 1, 2, 4, 5]]), w, None, np.arange(5, dtype=np.int64), 4)


def test_broken_rows_stay_their_own(api):
    x = np.random.default_rng(1).normal(size=(4, 128))
    x[1, 3], x[2, 9] = np.nan, np.inf
    cache = torch.zeros(2 * 4 * 132, dtype=torch.uint8, device="cuda")
    w = ref.bf16(np.ones(128)).cuda()
    for norm in (None, w):
        cache.zero_()
        api.index_write(ref.bf16(x).cuda(), torch.arange(4, device="cuda"), 4, 4 * 132, cache, norm_weight=norm)
        codes, scales = ref.index_page(cache.cpu().numpy(), 0, 4, 4 * 132)
        held = ref.E4M3[codes] * scales[:, None]
        assert np.isfinite(held[[0, 3]]).all()
        for r in (1, 2):
            assert np.isnan(held[r]).any() or np.isinf(scales[r])


def test_no_rows_and_refusals(api):
    cache = torch.full((4 * 132,), 7, dtype=torch.uint8, device="cuda")
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(2, dtype=torch.int64, device="cuda")
    api.index_write(x[:0], s[:0], 4, 4 * 132, cache)
    assert (cache == 7).all()
    for kw in (dict(page_stride_bytes=4 * 132 - 16), dict(block_size=0), dict(eps=-1.0), dict(norm_bias=x[0])):
        a = dict(block_size=4, page_stride_bytes=4 * 132) | kw
        with pytest.raises(api.DsaError) as e:
            api.index_write(x, s, index_cache=cache, **a)
        assert e.value.status == 1
    with pytest.raises(ValueError):
        api.index_write(x, s[:1], 4, 4 * 132, cache)
    with pytest.raises(ValueError):
        api.index_write(x.float(), s, 4, 4 * 132, cache)
    with pytest.raises(ValueError):
        api.index_write(x, s, 4, 4 * 132, cache, norm_weight=x)
    with pytest.raises(ValueError):
        api.index_write(x, s, 2**32 + 4, 4 * 132, cache)
    assert (cache == 7).all()
