"""A serving step end to end: plan_step's pages and slots, both cache writers, pool_scores,
select_pools, and the selected and full decodes, eager and as one captured graph that serves a
changing batch. Index queries, keys and weights are small whole numbers and the index keys
are written without a norm from rows whose largest magnitude is 448/2^k, so that scores are
exact and the selection has to be equal to the float64 one."""
import numpy as np
import pytest
import torch

import oracle
import step_ref as ref
from parity import assert_parity

pytestmark = pytest.mark.gpu
BS, KPOOL, TOPK, HEADS, IHEADS, WIDTH = 64, 4, 24, 64, 16, 12
SCALES = (0.05, 0.05, 512 ** -0.5)


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    oracle.build()
    import sparse_mla_paged_gb300.api as api
    return api


def index_keys(g, rows):
    """Rows of whole numbers whose largest magnitude is 7 (scale 1/64): codes 64*y are exact."""
    y = g.integers(-6, 7, (rows, 128)).astype(np.float32)
    y[y == 5] = 6
    y[y == -5] = -6
    y[:, 0] = 7
    return ref.bf16(y)


class Serving:
    def __init__(self, api, n, rps):
        self.api, self.n, self.rps = api, n, rps
        z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        pages = n * WIDTH
        self.tables, self.base, self.new = z(n, WIDTH), z(n), z(n)
        self.free = z(pages)
        self.latent, self.index = z(pages * BS * 512, dtype=torch.uint8), z(pages * BS * 132, dtype=torch.uint8)
        R = n * rps
        self.kv_a, self.keys = z(R, 512, dtype=torch.bfloat16), z(R, 128, dtype=torch.bfloat16)
        self.q, self.iq = z(R, HEADS, 512, dtype=torch.bfloat16), z(R, IHEADS, 128, dtype=torch.bfloat16)
        self.iw = z(R, IHEADS, dtype=torch.float32)
        self.norm = torch.ones(512, dtype=torch.bfloat16, device="cuda")
        self.plan = api.alloc_step_plan(R)
        self.scores = z(R, WIDTH * BS // KPOOL, dtype=torch.float32)
        self.sel, self.out, self.full = z(R, TOPK * KPOOL), torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.ws = api.alloc_workspace(n, rps, HEADS, TOPK * KPOOL)
        self.full_ws = api.alloc_full_workspace(n, rps, HEADS)
        self.status = z(1)

    def step(self):
        a, p = self.api, self.plan
        a.plan_step(self.base, self.new, self.free, BS, self.tables, rows_per_seq=self.rps, out=p)
        a.latent_write(self.kv_a, self.norm, p.slots, 1e-6, SCALES[0], BS, BS * 512, self.latent)
        a.index_write(self.keys, p.slots, BS, BS * 132, self.index)
        a.pool_scores(self.iq, self.iw, self.index, self.tables, WIDTH, p.positions, self.n, self.rps, IHEADS, BS, BS * 132,
                      KPOOL, self.scores.shape[1], out=self.scores, device_status=self.status)
        a.select_pools(self.scores, p.positions, KPOOL, TOPK, out=self.sel)
        a.decode_ws(self.q, self.latent, self.latent, self.tables, WIDTH, p.row_lens, self.sel, self.n, self.rps, HEADS, BS,
                    BS * 512, *SCALES, self.out, self.ws)
        a.decode_full(self.q, self.latent, self.latent, self.tables, WIDTH, p.row_lens, self.n, self.rps, HEADS, BS, BS * 512,
                      *SCALES, out=self.full, workspace=self.full_ws)


@pytest.mark.parametrize("n,rps", [(4, 1), (3, 3)])
def test_step(api, n, rps):
    g = np.random.default_rng(n)
    s = Serving(api, n, rps)
    # caches as earlier steps left them: every page holds rows
    old = n * WIDTH
    slots = torch.arange(old * BS, device="cuda")
    api.latent_write(ref.bf16(g.normal(size=(old * BS, 512))).cuda(), s.norm, slots, 1e-6, SCALES[0], BS, BS * 512, s.latent)
    api.index_write(index_keys(g, old * BS).cuda(), slots, BS, BS * 132, s.index)
    order = g.permutation(old).astype(np.int32)
    base = np.array([0, 63, 500, 700][:n], np.int32)
    have = [-(-int(b) // BS) for b in base]
    t = np.full((n, WIDTH), -1, np.int32)
    used = 0
    for i in range(n):
        t[i, :have[i]] = order[used:used + have[i]]
        used += have[i]
    free = order[used:]
    graph = None
    s.step()  # loads the kernels, with no request at all
    for turn in range(4):
        new = g.integers(0, rps + 1, n).astype(np.int32) if turn else np.full(n, rps, np.int32)
        R = n * rps
        s.base.copy_(torch.from_numpy(base))
        s.new.copy_(torch.from_numpy(new))
        s.tables.copy_(torch.from_numpy(t))
        s.free.zero_()
        s.free[:len(free)] = torch.from_numpy(free).cuda()
        s.kv_a.copy_(ref.bf16(g.normal(size=(R, 512))))
        s.keys.copy_(index_keys(g, R))
        s.q.copy_(ref.bf16(g.normal(size=(R, HEADS, 512))))
        s.iq.copy_(ref.bf16(g.integers(-2, 3, (R, IHEADS, 128))))
        s.iw.copy_(torch.from_numpy(g.integers(-1, 3, (R, IHEADS)).astype(np.float32)))
        if turn < 2:
            s.step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    s.step()
            graph.replay()
        torch.cuda.synchronize()
        assert s.status.item() == 0 and api.read_device_status(s.ws) == 0 and api.read_device_status(s.full_ws) == 0
        slots, pos, lens, seqs, info, t2 = ref.plan(base, new, s.free.cpu().numpy(), BS, t, rps, R)
        for got, want in zip(tuple(s.plan) + (s.tables,), (slots, pos, lens, seqs, info, t2)):
            assert np.array_equal(got.cpu().numpy(), want)
        index, latent = s.index.cpu().numpy(), s.latent.cpu().numpy()
        live = slots >= 0
        for r in np.nonzero(live)[0]:
            codes, scale = ref.index_page(index, int(slots[r]) // BS, BS, BS * 132)
            held = ref.E4M3[codes[slots[r] % BS]] * scale[slots[r] % BS]
            assert np.array_equal(held, ref.f64(s.keys)[r])
        want, _ = ref.pool_scores(ref.f64(s.iq), ref.f64(s.iw), index, t2, pos, rps, BS, BS * 132, KPOOL, s.scores.shape[1])
        assert np.array_equal(s.scores.cpu().numpy().astype(np.float64), want)
        sel = s.sel.cpu().numpy()
        for r in range(R):
            order_r = sorted(range(int(np.isfinite(want[r]).sum())), key=lambda p: (-want[r, p], p))[:TOPK]
            ids = [p * KPOOL + c for p in sorted(order_r) for c in range(KPOOL)]
            assert sel[r].tolist() == ids + [-1] * (TOPK * KPOOL - len(ids))
        full = ref.full(ref.f64(s.q), latent, latent, t2, lens, rps, BS, BS * 512, *SCALES)
        assert_parity(s.full, full, "full decode")
        sparse = np.zeros_like(full)
        for r in range(R):
            ids = sel[r][sel[r] >= 0]
            if len(ids):
                one = np.concatenate([latent[int(t2[r // rps, j // BS]) * BS * 512 + (j % BS) * 512:][:512] for j in ids])
                sparse[r] = ref.full(ref.f64(s.q)[r:r + 1], one, one, np.zeros((1, 1), np.int32), [len(ids)], 1, len(ids),
                                     len(ids) * 512, *SCALES)[0]
        assert_parity(s.out, sparse, "selected decode")
        taken = int(info[1])
        free, base, t = free[taken:], base + new, t2
