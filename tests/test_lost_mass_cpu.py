"""How much of a row's probability the two E4M3 terms of P' may lose, emulated on the CPU from
the kernels' constants (csrc/common.cuh, full.cu): the account that every (row, head) pair keeps,
the reference that moves when it runs out, and the rounding itself.

The whole-cache decode: a term of P' = 2^(x - m + kPBias) is off by at most 2^-10 (by itself when
below) or 1.22 * 2^-9 of it (float16, then two E4M3 terms). A pair's account holds kLostShare of
its P' less the former, 2^-10 for each of a thread's 32 tokens and at most their sum; it stays
above zero, so the former are kLostShare of the row at most. With values of magnitude 1 an output
is off by kLostShare + 1.22 * 2^-9 in all.

The selected decode: a term is off by at most 1.5 * 2^-10 or 2^-9 of it (test_split_bounds_cpu.py). Its
account is looked at two tiles later, with the most that these may lose kept back, but not
before a row's third tile: it may be overdrawn by one tile's most, 128 * 1.5 * 2^-10 of a row
whose sum is 2^6 at least: another 0.0030 of it.
"""
import os
import re

import numpy as np
import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_mla_paged_gb300", "csrc")


def _const(name, file="common.cuh"):
    m = re.search(rf"constexpr float {name} = (0x1p-?[0-9]+|[0-9.]+)f;", open(os.path.join(CSRC, file)).read())
    assert m, name
    return float.fromhex(m.group(1)) if m.group(1).startswith("0x") else float(m.group(1))


BIAS, MARGIN, DROP, FLOOR = (_const("k" + n) for n in ("PBias", "RescaleMargin", "RescaleDrop", "RescaleFloor"))
SHARE = _const("kLostShare")
LOW = _const("kRescaleSlack")


def _e4m3(x):
    return x.to(torch.float8_e4m3fn).float()


def _split_full(p):
    f = p.half().float()
    h = _e4m3(f)
    return h + _e4m3((f - h).half().float())


def full(x, vs, account=True, tile=128):
    """Output of each row of x (log2 scores) for each of the value rows vs, as full.cu forms it."""
    slack, lost = _const("kSlack", "full.cu"), tile / 4 * 2.0 ** -10
    n = x.shape[0]
    m = torch.full((n,), -np.inf)
    top, l, credit = m.clone(), torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    out = [torch.zeros(n, dtype=torch.float64) for _ in vs]

    def form(m):
        p = torch.exp2(x[:, t0:t0 + tile] - m[:, None] + BIAS)
        q = p.double().view(n, 4, -1).sum(2)  # by the pair's four threads
        return p, (q * SHARE - q.clamp(max=lost)).sum(1)

    for t0 in range(0, x.shape[1], tile):
        tm = x[:, t0:t0 + tile].max(1).values
        first = m == -np.inf
        after = credit + form(torch.where(first, tm + slack, m))[1]
        rise, free = tm > m + MARGIN, m > top - FLOOR
        low = free & ((tm < m - DROP) | ((after < 0) & (tm < m - slack) & account))
        m_new = torch.where(rise, tm + slack, torch.where(low, torch.maximum(tm + LOW, top - FLOOR), m))
        a = torch.where(first, 0.0, torch.exp2((m - m_new).double()))
        m, top = m_new, torch.maximum(top, m_new)
        p, earned = form(m)
        l = l * a + p.double().sum(1)
        credit = torch.where(first, 0.0, credit * a) + earned
        r = _split_full(p).double()
        out = [o * a + (r * v[:, t0:t0 + tile]).sum(1) for o, v in zip(out, vs)]
    return [o / l for o in out]


def _split_selected(p):
    h = ((p.view(torch.int32) + 0x80000) & ~0xFFFFF).view(torch.float32)
    return _e4m3(h) + _e4m3(p - h)


def selected(x, vs, account=True, tile=128):
    """The same as decode.cu forms it."""
    lost = tile / 4 * 1.5 * 2.0 ** -10
    n = x.shape[0]
    m = torch.full((n,), -np.inf)
    top, l, credit = m.clone(), torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    out = [torch.zeros(n, dtype=torch.float64) for _ in vs]
    poor = torch.zeros(n, dtype=torch.bool)
    for t0 in range(0, x.shape[1], tile):
        tm = x[:, t0:t0 + tile].max(1).values
        first, rise, free = m == -np.inf, tm > m + MARGIN, m > top - FLOOR
        over = poor & (tm < m - LOW) & account
        change = rise | (free & ((tm < m - DROP) | over))
        m_new = torch.where(change, torch.maximum(torch.where(over, tm, tm + LOW), top - FLOOR), m)
        a = torch.where(first, 0.0, torch.exp2((m - m_new).double()))
        poor = (credit * a < 8 * lost) & (t0 > 0)
        m, top = m_new, torch.maximum(top, m_new)
        p = torch.exp2(x[:, t0:t0 + tile] - m[:, None] + BIAS)
        q = p.double().view(n, 4, -1).sum(2)
        credit = torch.where(first, 0.0, credit * a) + (q * SHARE - q.clamp(max=lost)).sum(1)
        l = l * a + p.double().sum(1)
        r = _split_selected(p).double()
        out = [o * a + (r * v[:, t0:t0 + tile]).sum(1) for o, v in zip(out, vs)]
    return [o / l for o in out]


SELECTED_BOUND = SHARE + 128 * 1.5 * 2.0 ** -10 / 64 + 2.0 ** -9


def rows(n, first, peak):
    """log2 scores: the first position and every 128th above a background of zeros."""
    x = torch.zeros(len(first), n)
    x[:, 5::128] = torch.tensor(peak)[:, None]
    x[:, 0] = torch.tensor(first)
    return x


def values(n):
    """Ones, and background, peaks and the first position apart."""
    v = [torch.ones(1, n, dtype=torch.float64), torch.zeros(1, n, dtype=torch.float64), torch.ones(1, n, dtype=torch.float64)]
    v[1][0, 5::128] = 1
    v[2][0, 5::128] = -1
    v[2][0, 0] = 0
    return v


FAMILY = [(f, b) for f in np.arange(4, 24.1, 0.25) for b in np.arange(0, f + 0.1, 0.25)]


def worst(emulate, x, **kw):
    vs = values(x.shape[1])
    w = torch.exp2((x - x.max(1, keepdim=True).values).double())
    return max((got - (w * v).sum(1) / w.sum(1)).abs().max().item()
               for got, v in zip(emulate(x, vs, **kw), vs))


@pytest.mark.parametrize("n", [1024, 16384])
def test_full_sinks_and_peaks(n):
    """A sink, one moderate peak a tile and a flat background, by quarter octaves."""
    x = rows(n, *zip(*FAMILY)).float()
    assert worst(full, x) <= SHARE + 1.22 * 2.0 ** -9


def test_full_loses_more_without_the_account():
    """The family tells: with the reference following tile maxima alone a seventh is lost."""
    assert worst(full, rows(16384, *zip(*FAMILY)).float(), account=False) > 0.1


@pytest.mark.parametrize("deviation", [0.5, 1.0, 2.0, 4.0, 8.0])
def test_full_normal_scores(deviation):
    g = torch.Generator().manual_seed(int(deviation * 10))
    x = torch.randn(64, 8192, generator=g) * deviation * 1.4427
    assert worst(full, x) <= SHARE + 1.22 * 2.0 ** -9
    x[:, 0] = 4 * deviation + 12
    assert worst(full, x) <= SHARE + 1.22 * 2.0 ** -9


def test_full_tails_that_fall_tile_by_tile():
    """Scores that decay so slowly that no tile alone is far below the one before."""
    n = 16384
    for step in (0.25, 1.0, 3.0, 7.5):
        x = -step * torch.arange(n).div(128, rounding_mode="floor").float().repeat(8, 1)
        x[:, 0] += torch.linspace(0, 14, 8)
        assert worst(full, x) <= SHARE + 1.22 * 2.0 ** -9


@pytest.mark.parametrize("tile", [64, 128])
@pytest.mark.parametrize("n", [1024, 2048, 8192])
def test_selected_sinks_and_peaks(n, tile):
    x = rows(n, *zip(*FAMILY)).float()
    assert worst(selected, x, tile=tile) <= SELECTED_BOUND


def test_selected_loses_more_without_the_account():
    x = rows(8192, *zip(*FAMILY)).float()
    assert worst(selected, x, account=False) > 0.05
    assert worst(selected, x[:, :2048], account=False) > 0.025


@pytest.mark.parametrize("tile", [64, 128])
def test_selected_other_scores(tile):
    """Normal ones of several deviations, with and without a sink; tails that fall tile by tile."""
    g = torch.Generator().manual_seed(5)
    for deviation in (0.5, 1.0, 2.0, 4.0, 8.0):
        x = torch.randn(64, 4096, generator=g) * deviation * 1.4427
        x[:32, 0] = 4 * deviation + 12
        assert worst(selected, x, tile=tile) <= SELECTED_BOUND
    for step in (0.25, 1.0, 3.0, 7.5):
        x = -step * torch.arange(8192).div(tile, rounding_mode="floor").float().repeat(8, 1)
        x[:, 0] += torch.linspace(0, 14, 8)
        assert worst(selected, x, tile=tile) <= SELECTED_BOUND
