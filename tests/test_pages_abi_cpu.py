"""Host-side refusals of the page operators and the prompt-chunk attention: each bad argument is answered before any CUDA call."""
import ctypes

import pytest

from sparse_mla_paged_gb300 import _lib


@pytest.fixture(scope="module")
def lib():
    from sparse_mla_paged_gb300 import build
    build.build()
    return _lib.load()


POOL = dict(base=0x10000, page_stride_bytes=1024, layer_stride_bytes=1 << 20, page_bytes=1024, layers=2, reserved=0)
BAD_POOLS = [(dict(base=0), 1), (dict(base=0x10008), 1), (dict(page_stride_bytes=1008), 1), (dict(page_stride_bytes=1032), 1),
             (dict(page_bytes=0), 1), (dict(page_bytes=1000), 1), (dict(layers=0), 1), (dict(layers=-1), 1), (dict(reserved=1), 1),
             (dict(layer_stride_bytes=1008), 1), (dict(layer_stride_bytes=1 << 20 | 8), 1), (dict(layer_stride_bytes=-1024), 1),
             (dict(page_stride_bytes=-1024), 1), (dict(layers=2**31 - 1), 2),
             (dict(page_bytes=1 << 36, page_stride_bytes=1 << 36, layers=1), 2)]


def pools(n=1, **over):
    return (_lib.PagePool * n)(*[_lib.PagePool(**dict(POOL, **over)) for _ in range(n)])


COPY = dict(pools=None, n=1, src=0x20000, dst=0x30000, count=3, pages=100)
FORK = dict(pools=None, n=1, parents=0x20000, children=0x30000, forks=3, lens=0x40000, seqs=8, bs=64, bt=0x50000, mbps=8, free=0x60000,
            nfree=5, shares=0x70000, pages=100, info=0x80000, ws=0x90000, wsb=1 << 40)
RELEASE = dict(bt=0x50000, mbps=8, lens=0x40000, keeps=0x30000, seqs=8, bs=64, shares=0x70000, pages=100, free=0x60000, nfree=0x61000,
               taken=0x62000, info=0x80000, ws=0x90000, wsb=1 << 40)
COMPACT = dict(pools=None, n=1, bt=0x50000, mbps=8, lens=0x40000, seqs=8, bs=64, shares=0x70000, pages=100, free=0x60000, nfree=0x61000,
               info=0x80000, ws=0x90000, wsb=1 << 40)


def call(fn, args, over, **pool):
    a = dict(args, **over)
    if "pools" in a and a["pools"] is None:
        a["pools"] = pools(max(1, min(a["n"], 20)), **pool)
    return fn(*a.values(), None)


@pytest.mark.parametrize("over,code", BAD_POOLS)
def test_bad_pools(lib, over, code):
    for fn, args in ((lib.dsa_copy_pages, COPY), (lib.dsa_fork_pages, FORK), (lib.dsa_compact_pages, COMPACT)):
        assert call(fn, args, {}, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(pools=ctypes.POINTER(_lib.PagePool)()), 1), (dict(n=0), 1), (dict(n=17), 2), (dict(src=0), 1), (dict(dst=0), 1),
    (dict(src=0x20002), 1), (dict(dst=0x30002), 1), (dict(count=-1), 1), (dict(pages=0), 1), (dict(count=2**31 - 1), 2),
    (dict(count=0), 0), (dict(count=0, src=0, dst=0), 0)])
def test_copy_rejects_on_host(lib, over, code):
    # a page of 2 layers: 2^31 - 1 pages are just below 2^32 pieces, three layers pass it
    assert call(lib.dsa_copy_pages, COPY, over, **(dict(layers=3) if over.get("count", 0) > 100 else {})) == code


TABLES = [(dict(bt=0), 1), (dict(bt=0x50002), 1), (dict(mbps=0), 1), (dict(lens=0), 1), (dict(lens=0x40002), 1), (dict(seqs=-1), 1),
          (dict(bs=0), 1), (dict(pages=0), 1), (dict(info=0), 1), (dict(info=0x80002), 1), (dict(shares=0), 1), (dict(shares=0x70002), 1),
          (dict(ws=0), 1), (dict(ws=0x90010), 1), (dict(wsb=1000), 3), (dict(seqs=16385), 2), (dict(pages=(1 << 30) + 1), 2),
          (dict(mbps=1 << 25), 2), (dict(seqs=16384, bs=1, mbps=1 << 25), 2)]


@pytest.mark.parametrize("over,code", TABLES + [
    (dict(parents=0), 1), (dict(children=0), 1), (dict(parents=0x20002), 1), (dict(forks=-1), 1), (dict(nfree=-1), 1), (dict(free=0), 1),
    (dict(free=0x60002), 1), (dict(forks=16385), 2), (dict(n=0), 1), (dict(n=17), 2)])
def test_fork_rejects_on_host(lib, over, code):
    assert call(lib.dsa_fork_pages, FORK, over) == code


@pytest.mark.parametrize("over,code", TABLES + [
    (dict(keeps=0), 1), (dict(keeps=0x30002), 1), (dict(free=0), 1), (dict(free=0x60002), 1), (dict(nfree=0), 1), (dict(nfree=0x61002), 1),
    (dict(taken=0x62002), 1)])
def test_release_rejects_on_host(lib, over, code):
    assert call(lib.dsa_release_pages, RELEASE, over) == code


@pytest.mark.parametrize("over,code", TABLES + [
    (dict(free=0), 1), (dict(free=0x60002), 1), (dict(nfree=0), 1), (dict(nfree=0x61002), 1), (dict(n=0), 1), (dict(n=17), 2)])
def test_compact_rejects_on_host(lib, over, code):
    assert call(lib.dsa_compact_pages, COMPACT, over) == code


def test_workspace_of_bad_sizes_is_zero(lib):
    f = lib.dsa_pages_workspace_bytes
    assert f(0) == 0 and f(-1) == 0 and f((1 << 30) + 1) == 0 and f(1) > 0


def test_pool_struct_layout():
    assert ctypes.sizeof(_lib.PagePool) == 40 and _lib.PagePool.layers.offset == 32


PREFILL = dict(q=0x10000, k=0x20000, v=0x20000, bt=0x30000, mbps=8, base=0x40000, new=0x48000, n=2, rows=20, heads=16, bs=64,
               stride=64 * 512, ks=0.05, vs=0.05, sm=0.04, out=0x50000, ws=0x60000, wsb=1 << 40)


@pytest.mark.parametrize("over,code", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(bt=0), 1), (dict(mbps=-1), 1), (dict(base=0), 1), (dict(new=0), 1), (dict(n=0), 1),
    (dict(rows=0), 1), (dict(heads=0), 1), (dict(bs=0), 1), (dict(stride=64 * 512 - 16), 1), (dict(stride=64 * 512 + 8), 1),
    (dict(out=0), 1), (dict(ws=0), 1), (dict(ws=0x60010), 1), (dict(q=0x10008), 1), (dict(k=0x20008), 1), (dict(v=0x20008), 1),
    (dict(bt=0x30002), 1), (dict(base=0x40002), 1), (dict(new=0x48002), 1), (dict(out=0x50008), 1), (dict(n=16385), 2),
    (dict(rows=1 << 20, heads=33), 2), (dict(rows=2**31 - 1, heads=2**31 - 1), 2)])
def test_prefill_rejects_on_host(lib, over, code):
    assert lib.dsa_mla_prefill(*dict(PREFILL, **over).values(), None) == code


def test_prefill_workspace_of_bad_shapes_is_zero(lib):
    f = lib.dsa_mla_prefill_workspace_bytes
    assert f(0, 1, 1) == 0 and f(1, 0, 1) == 0 and f(1, 1, 0) == 0 and f(16385, 1, 1) == 0 and f(1, 1 << 20, 33) == 0
