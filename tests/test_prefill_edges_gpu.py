"""What a serving process may do with dsa_mla_prefill beside plain calls: waits that run out, a first
call inside a capture, calls of several threads and streams, more than 2^31 query elements, and the
whole loop of prompts, forks and compacted pages."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import step_ref as ref
import test_prefill_gpu as prefill
from parity import assert_parity

pytestmark = pytest.mark.gpu
TIMEOUT = 7


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()
    return api


@pytest.mark.parametrize("base,new,heads,bs,two", [
    ([5000, 0], [3, 40], 64, 64, False), ([900], [1], 16, 64, False), ([20000], [30], 64, 100, False),
    ([0, 900, 1, 3000], [200, 1, 64, 7], 40, 48, True), ([100] * 60, [9] * 60, 64, 32, False)])
def test_waits_that_run_out(api, base, new, heads, bs, two):
    """With a limit of 1 ns a wait gives up at once; the call records it, ends, and the next is right."""
    c = prefill.Case(base, new, heads, bs, two=two)
    ws = api.alloc_prefill_workspace(len(base), c.q.shape[0], heads)
    with api.wait_limit(1):
        c.run(api, workspace=ws)
        torch.cuda.synchronize()
    assert api.read_device_status(ws) == TIMEOUT and api.step_device_status() == TIMEOUT
    got = c.run(api, workspace=ws)
    assert api.read_device_status(ws) == 0
    assert torch.equal(got, c.check(api))


FIRST = """
import torch
import sparse_mla_paged_gb300.api as api
q = torch.zeros(6, 16, 512, dtype=torch.bfloat16, device="cuda")
cache = torch.zeros(8 * 64 * 512, dtype=torch.uint8, device="cuda")
tables = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
base = torch.tensor([100, 0], dtype=torch.int32, device="cuda")
new = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
out = torch.ones_like(q)
ws = api.alloc_prefill_workspace(2, 6, 16)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    api.prefill(q, cache, cache, tables, 4, base, new, 16, 64, 64 * 512, 1.0, 1.0, 0.1, out=out, workspace=ws)
graph.replay()
torch.cuda.synchronize()
assert (out == 0).all()
"""


def test_first_call_of_a_process_is_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST], cwd=root, check=True, timeout=300)


def test_threads(api):
    """Four host threads, a stream each, the same inputs: every result is the one alone."""
    c = prefill.Case([900, 1, 0, 2000], [40, 3, 130, 1], 40)
    want = c.run(api)
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = c.run(api)
                stream.synchronize()
                if not torch.equal(got, want):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert api.step_device_status() == 0


def test_more_than_31_bits_of_queries(api):
    """16384 requests of five or six new tokens: 2.7 thousand million query elements, the most requests."""
    n, heads, bs = 16384, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    base = torch.randint(0, 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    new = torch.randint(5, 7, (n,), generator=g, device="cuda", dtype=torch.int32)
    rows = int(new.sum())
    assert rows * heads * 512 > 2 ** 31
    tables = torch.randperm(2 * n, generator=g, device="cuda").to(torch.int32).view(n, 2)
    cache = (torch.randn(2 * n, bs * 512, generator=g, device="cuda") * 20).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(rows, heads, 512, generator=g, device="cuda", dtype=torch.bfloat16)
    got = api.prefill(q, cache, cache, tables, 2, base, new, heads, bs, bs * 512, 0.05, 0.05, 512 ** -0.5)
    assert api.step_device_status() == 0
    ends = torch.cumsum(new, 0).tolist()
    held, t, b, k = cache.view(-1).cpu().numpy(), tables.cpu().numpy(), base.tolist(), new.tolist()
    for s in (0, 1, 777, 8191, 16000, 16382, 16383):
        for i in range(k[s]):
            row = ends[s] - k[s] + i
            want = ref.full(ref.f64(q[row:row + 1]), held, held, t[s:s + 1], [b[s] + i + 1], 1, bs, bs * 512, 0.05, 0.05, 512 ** -0.5)
            assert_parity(got[row:row + 1], want)


def test_prompts_forks_and_compacted_pages(api):
    """A serving loop over both caches: prompts are planned, written and attended; samples fork from them and
    go on token by token; some end and the pool is compacted. Each step's attention against float64 over
    the tokens that each request has been given, wherever their pages have gone."""
    g = np.random.default_rng(8)
    n, rows, bs, blocks, heads, pages = 7, 96, 16, 10, 16, 80
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    tables, shares, free, count = torch.full((n, blocks), -1, dtype=torch.int32, device="cuda"), z(pages), z(pages), z(1)
    free.copy_(torch.from_numpy(g.permutation(pages).astype(np.int32)))
    count.fill_(pages)
    latent, index = z(pages, bs * 512, dtype=torch.uint8), z(pages, api.index_page_stride(bs), dtype=torch.uint8)
    norm = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    ws, pages_ws = api.alloc_prefill_workspace(n, rows, heads), api.alloc_pages_workspace(pages)
    has = [np.zeros((0, 512), np.uint8) for _ in range(n)]  # each request's codes

    def ints(v):
        return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")

    def step(new):
        base = [len(h) for h in has]
        plan = api.plan_step(ints(base), ints(new), free, bs, tables, max_rows=rows)
        api.release_pages(tables, ints(base), ints(base), bs, shares, free, count, taken=plan.info[1:2], workspace=pages_ws)
        assert plan.info[2].item() == 0
        kv_a, keys = ref.bf16(g.normal(size=(rows, 512))).cuda(), ref.bf16(g.normal(size=(rows, 128))).cuda()
        api.latent_write(kv_a, norm, plan.slots, 1e-6, 0.05, bs, bs * 512, latent)
        api.index_write(keys, plan.slots, bs, index.shape[1], index)
        q = ref.bf16(g.normal(size=(rows, heads, 512))).cuda()
        out = api.prefill(q, latent, latent, tables, blocks, ints(base), ints(new), heads, bs, bs * 512, 0.05, 0.05, 512 ** -0.5, workspace=ws)
        assert api.read_device_status(ws) == 0
        slots, held = plan.slots.cpu().numpy(), latent.cpu().numpy().reshape(-1, 512)
        row = 0
        for s in range(n):
            has[s] = np.concatenate([has[s], held[slots[row:row + new[s]]]])
            codes = np.ascontiguousarray(has[s]).reshape(-1)
            for i in range(new[s]):
                want = ref.full(ref.f64(q[row:row + 1]), codes, codes, np.zeros((1, 1), np.int32), [base[s] + i + 1], 1, 1 << 20, 0, 0.05, 0.05,
                                512 ** -0.5)
                assert_parity(out[row:row + 1], want)
                row += 1

    def fork(parent, children):
        lens = ints(len(h) for h in has)
        info = api.fork_pages([latent, index], ints([parent] * len(children)), ints(children), lens, bs, tables, free, shares, workspace=pages_ws)
        assert info[2].item() == 0 and info[0].item() == len(children)
        for c in children:
            has[c] = has[parent].copy()
        lens = ints(len(h) for h in has)
        api.release_pages(tables, lens, lens, bs, shares, free, count, taken=info[1:2], workspace=pages_ws)

    def end(requests):
        lens = [len(h) for h in has]
        for r in requests:
            has[r] = has[r][:0]
        info = api.release_pages(tables, ints(lens), ints(len(h) for h in has), bs, shares, free, count, workspace=pages_ws)
        assert info[2].item() == 0

    step([50, 37, 0, 0, 0, 0, 0])
    fork(0, [2, 3, 4])
    fork(1, [5])
    step([1, 3, 1, 20, 1, 1, 16])
    end([0, 3])
    info = api.compact_pages([latent, index], tables, ints(len(h) for h in has), bs, shares, free, count, workspace=pages_ws)
    assert info[2].item() == 0 and info[1].item() > 0
    step([5, 1, 30, 40, 1, 1, 1])
    fork(6, [])
    end([1, 2, 3, 4, 5, 6, 0])
    assert count.item() == pages and not bool(shares.any()) and sorted(free.tolist()) == list(range(pages))
