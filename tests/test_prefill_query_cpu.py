"""The two E4M3 terms of a BF16 query as the prompt chunks form them (csrc/prefill.cu, make_operand): through
FP16, hi = the top 4 significant bits and lo = the rest, each rounded to E4M3."""
import numpy as np
import torch


def _e4m3(x):
    return x.to(torch.float8_e4m3fn).double()


def terms(x):
    """hi + lo of scaled values below 256 (float64)."""
    half = x.to(torch.float16)
    hi = (half.view(torch.int16) & -128).view(torch.float16)
    return _e4m3(hi.float()) + _e4m3((half - hi).float())


def split(q):
    """What a head's query is in the kernel: scaled by a power of two so that its largest lies in [128, 256)."""
    q = q.double()
    scale = torch.exp2(7 - torch.floor(torch.log2(q.abs().amax(-1, keepdim=True))))
    return terms(q * scale) / scale


def test_every_bf16():
    """Exact from 2^-9 of the least largest element on, off by 2^-16 of it below."""
    v = (np.arange(1, 0x7F80, dtype=np.uint32) << 16).view(np.float32)
    v = torch.from_numpy(v[(v > 2.0 ** -60) & (v < 256.0)])
    for x in (v, -v):
        err = (terms(x) - x.double()).abs()
        assert err[v >= 2.0 ** -2].max() == 0
        assert 0 < err.max() <= 2.0 ** -9


def test_heads():
    q = torch.randn(7, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    top = q.double().abs().amax(1, keepdim=True)
    err = (split(q) - q.double()).abs()
    assert bool((err <= 2.0 ** -16 * top).all()) and bool((err[q.double().abs() >= 2.0 ** -8 * top] == 0).all())
