"""Calls that the interface allows at its edges: many rows a sequence in the whole-cache decode
(prompt chunks), the first call of a process inside a capture, calls of several threads at once."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import test_decode_full_gpu as full
import test_pool_scores_gpu as scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    return api


@pytest.mark.parametrize("n,rps,heads,lens,bs,verify", [
    (1, 130, 16, [900], 64, True), (2, 257, 8, [0, 1000], 64, True), (1, 1000, 1, list(range(0, 2000, 2)), 100, False),
    (1, 70, 128, [300], 32, True), (2, 100, 24, [0, 700, 3, 128, 129, 64, 0], 64, False), (3, 64, 64, [63], 48, True)])
def test_many_rows(api, n, rps, heads, lens, bs, verify):
    full.Case(n, rps, heads, lens, bs, verify=verify).check(api)


FIRST = """
import sys
import torch
from sparse_mla_paged_gb300 import api
which, bs = sys.argv[1], 64
cuda = dict(device="cuda")
q = torch.randn(2, 16, 512, **cuda).bfloat16()
cache = torch.zeros(8 * bs * 512, dtype=torch.uint8, **cuda)
tables = torch.arange(8, dtype=torch.int32, **cuda).view(2, 4)
lens = torch.tensor([100, 200], dtype=torch.int32, **cuda)
new = torch.ones(2, dtype=torch.int32, **cuda)
out, ws = torch.empty_like(q), torch.zeros(1 << 27, dtype=torch.uint8, **cuda)
stride = api.index_page_stride(bs)
index = torch.zeros(8 * stride, dtype=torch.uint8, **cuda)
iq, w = torch.randn(2, 16, 128, **cuda).bfloat16(), torch.randn(2, 16, **cuda)
at, scores, plan = lens - 1, torch.full((2, 60), 7.0, **cuda), api.alloc_step_plan(2)
slots = torch.tensor([5, 70], **cuda)
keys = torch.randn(2, 128, **cuda).bfloat16()
calls = {
    "full": lambda: api.decode_full(q, cache, cache, tables, 4, lens, 2, 1, 16, bs, bs * 512, 1.0, 1.0, 0.05, out=out, workspace=ws),
    "scores": lambda: api.pool_scores(iq, w, index, tables, 4, at, 2, 1, 16, bs, stride, 4, 60, out=scores),
    "plan": lambda: api.plan_step(lens, new, tables[0].contiguous(), bs, tables, rows_per_seq=1, out=plan),
    "write": lambda: api.index_write(keys, slots, bs, stride, index),
}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls[which]()
graph.replay()
torch.cuda.synchronize()
ok = {"full": lambda: (out == 0).all(), "scores": lambda: (scores[0, :25] == 0).all() and torch.isneginf(scores[0, 25:]).all(),
      "plan": lambda: plan.positions.tolist() == [100, 200], "write": lambda: index.any()}
assert ok[which]()
"""


@pytest.mark.parametrize("which", ["full", "scores", "plan", "write"])
def test_first_call_of_a_process_is_captured(api, which):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST, which], cwd=root, check=True, timeout=300)


def test_threads(api):
    """Four host threads, a stream each, the same inputs: every result is the one alone."""
    c, s = full.Case(3, 2, 40, [900, 1, 0, 2000, 64, 333]), scores.Case(2, 2, 64, [5000, 300, 20, 4000])
    api.step_device_status()  # what other tests left
    want = c.run(api), s.run(api)
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = c.run(api), s.run(api)
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert api.step_device_status() == 0
