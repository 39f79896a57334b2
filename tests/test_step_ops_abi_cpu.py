"""Host-side refusals of the step plan, the index-key writer, the pool scores and the
full-cache decode: each bad argument is answered before any CUDA call, with no GPU."""
import pytest

from sparse_mla_paged_gb300 import _lib


@pytest.fixture(scope="module")
def lib():
    from sparse_mla_paged_gb300 import build
    build.build()
    return _lib.load()


PLAN = dict(base=0x10000, new=0x20000, n=4, rps=0, rows=100, free=0x30000, nfree=10, bs=64, bt=0x40000, mbps=8,
            slots=0x50000, pos=0x60000, lens=0x70000, seqs=0x80000, info=0x90000)


@pytest.mark.parametrize("over,code", [
    (dict(base=0), 1), (dict(new=0), 1), (dict(n=-1), 1), (dict(rps=-1), 1), (dict(rows=-1), 1), (dict(free=0), 1),
    (dict(nfree=-1), 1), (dict(bs=0), 1), (dict(bt=0), 1), (dict(mbps=0), 1), (dict(slots=0), 1), (dict(pos=0), 1),
    (dict(lens=0), 1), (dict(seqs=0), 1), (dict(info=0), 1), (dict(slots=0x50004), 1), (dict(pos=0x60002), 1),
    (dict(bt=0x40001), 1), (dict(info=0x90002), 1), (dict(rps=2), 1), (dict(rps=25, rows=101), 1),
    (dict(n=16385), 2), (dict(mbps=1 << 25), 2)])
def test_plan_rejects_on_host(lib, over, code):
    assert lib.dsa_plan_step(*dict(PLAN, **over).values(), None) == code


WRITE = dict(x=0x10000, w=0x20000, b=0x30000, slots=0x40000, rows=4, eps=1e-6, bs=64, stride=64 * 132, cache=0x50000)


@pytest.mark.parametrize("over,code", [
    (dict(x=0), 1), (dict(slots=0), 1), (dict(cache=0), 1), (dict(w=0), 1), (dict(rows=-1), 1), (dict(bs=0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(stride=64 * 132 - 16), 1),
    (dict(stride=64 * 132 + 8), 1), (dict(x=0x10008), 1), (dict(w=0x20008), 1), (dict(b=0x30008), 1),
    (dict(slots=0x40004), 1), (dict(cache=0x50008), 1), (dict(rows=0), 0), (dict(rows=0, x=0, slots=0), 0)])
def test_index_write_rejects_on_host(lib, over, code):
    assert lib.dsa_index_write(*dict(WRITE, **over).values(), None) == code


SCORES = dict(q=0x10000, w=0x20000, cache=0x30000, bt=0x40000, mbps=8, pos=0x50000, n=2, rps=2, heads=16, bs=64,
              stride=64 * 132, kpool=4, pools=100, out=0x60000, status=0x70000)


@pytest.mark.parametrize("over,code", [
    (dict(q=0), 1), (dict(w=0), 1), (dict(cache=0), 1), (dict(bt=0), 1), (dict(mbps=-1), 1), (dict(pos=0), 1),
    (dict(n=0), 1), (dict(rps=0), 1), (dict(heads=0), 1), (dict(bs=0), 1), (dict(stride=64 * 132 - 16), 1),
    (dict(stride=64 * 132 + 4), 1), (dict(kpool=0), 1), (dict(pools=-1), 1), (dict(out=0), 1), (dict(q=0x10008), 1),
    (dict(w=0x20002), 1), (dict(cache=0x30008), 1), (dict(bt=0x40002), 1), (dict(pos=0x50002), 1),
    (dict(out=0x60002), 1), (dict(status=0x70002), 1), (dict(heads=129), 2), (dict(kpool=129), 2),
    (dict(pools=1 << 30), 2), (dict(n=1 << 20, rps=1 << 10), 2), (dict(pools=0), 0), (dict(pools=0, out=0), 0)])
def test_pool_scores_rejects_on_host(lib, over, code):
    assert lib.dsa_pool_scores(*dict(SCORES, **over).values(), None) == code


FULL = dict(q=0x10000, k=0x20000, v=0x20000, bt=0x30000, mbps=8, lens=0x40000, n=2, rps=2, heads=16, bs=64,
            stride=64 * 512, ks=0.05, vs=0.05, sm=0.04, out=0x50000, verify=0, ws=0x60000, wsb=1 << 40)


@pytest.mark.parametrize("over,code", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(bt=0), 1), (dict(mbps=-1), 1), (dict(lens=0), 1), (dict(n=0), 1),
    (dict(rps=0), 1), (dict(heads=0), 1), (dict(bs=0), 1), (dict(stride=64 * 512 - 16), 1), (dict(stride=64 * 512 + 8), 1),
    (dict(out=0), 1), (dict(verify=2), 1), (dict(verify=-1), 1), (dict(ws=0), 1), (dict(ws=0x60010), 1), (dict(q=0x10008), 1),
    (dict(k=0x20008), 1), (dict(v=0x20008), 1), (dict(bt=0x30002), 1), (dict(lens=0x40002), 1), (dict(out=0x50008), 1),
    (dict(n=1 << 12, rps=1 << 6, heads=17), 2), (dict(n=1 << 30, rps=1 << 30), 2)])
def test_full_rejects_on_host(lib, over, code):
    assert lib.dsa_mla_decode_full(*dict(FULL, **over).values(), None) == code


def test_full_workspace_of_bad_shapes_is_zero(lib):
    f = lib.dsa_mla_decode_full_workspace_bytes
    assert f(0, 1, 1) == 0 and f(1, 0, 1) == 0 and f(1, 1, 0) == 0 and f(1 << 12, 1 << 6, 17) == 0
