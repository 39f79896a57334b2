"""The two E4M3 terms of a BF16 query, hi = its top 4 significant bits and lo = the rest, for every
BF16 value: what is exact and how far the others are off, relative to their head's largest. The
whole-cache decode scales a head's largest to [2^7, 2^8), the pooled scores to [240, 480)."""
import numpy as np
import pytest
import torch


def _e4m3(x):
    return torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy().astype(np.float64)


@pytest.mark.parametrize("least,limit,exact_from,off", [(128.0, 256.0, 2.0 ** -9, 2.0 ** -16), (240.0, 480.0, 2.0 ** -9.9, 2.0 ** -16.9)])
def test_every_bf16(least, limit, exact_from, off):
    v = (np.arange(1, 0x7F80, dtype=np.uint32) << 16).view(np.float32)
    v = v[(v > 2.0 ** -60) & (v < limit)]
    hi = (v.view(np.uint32) & np.uint32(0xFFF00000)).view(np.float32)
    err = np.abs(_e4m3(hi) + _e4m3(v - hi) - v)
    assert err[v >= exact_from * least].max() == 0
    assert 0 < err.max() <= off * least
    assert err[v < exact_from * least].max() > 0 and v[err > 0].max() > 0.9 * exact_from * least
