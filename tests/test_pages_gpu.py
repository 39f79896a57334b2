"""Copying, forking, releasing and compacting pages against page-by-page forms on the CPU: books
and copied bytes are whole numbers and must be equal."""
import numpy as np
import pytest
import torch

import page_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mla_paged_gb300 import build
    build.build()
    import sparse_mla_paged_gb300.api as api
    api.step_device_status()
    return api


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def pools_of(g, pages, widths=(1056, 512), layers=(1, 3)):
    return [g.integers(0, 256, (n, pages, w)).astype(np.uint8) for n, w in zip(layers, widths)]


def on_gpu(pools):
    return [cu(p[0] if p.shape[0] == 1 else p) for p in pools]


def same(got, want, what):
    assert np.array_equal(got.cpu().numpy().reshape(want.shape), want), what


def same_pools(got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        same(a, b, f"pool {i}")


# ---------------------------------------------------------------------------------------------
# copy
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("width", [16, 1056, 16384, 16400, 33000 // 16 * 16])
@pytest.mark.parametrize("count", [0, 1, 7, 400])
def test_copy(api, count, width):
    g = np.random.default_rng(count)
    pools = pools_of(g, 2 * count + 3, (width, 48))
    order = g.permutation(2 * count + 3).astype(np.int32)
    src, dst = order[:count].copy(), order[count:2 * count].copy()
    src[1::5] = -1
    dst[2::7] = -1
    dev = on_gpu(pools)
    api.copy_pages(dev, cu(src), cu(dst))
    same_pools(dev, ref.copy(pools, src, dst))
    assert api.step_device_status() == 0


def test_copy_strides_and_neighbours(api):
    """Pages inside wider rows, layers inside pages: nothing beside the pages' own bytes changes."""
    g = np.random.default_rng(1)
    whole = g.integers(0, 256, (9, 4, 160)).astype(np.uint8)  # [pages, layers, bytes]
    dev = cu(whole)
    view = dev.permute(1, 0, 2)[1:3, :, 32:112]
    src, dst = np.array([0, 8, 3], np.int32), np.array([5, 1, 3], np.int32)
    api.copy_pages([view], cu(src), cu(dst))
    want = whole.copy()
    for a, b in zip(src, dst):
        want[b, 1:3, 32:112] = whole[a, 1:3, 32:112]
    same(dev, want, "bytes")


def test_copy_bad_pages(api):
    g = np.random.default_rng(2)
    pools = pools_of(g, 20)
    for src, dst in (([20, 3], [4, 5]), ([2, 3], [4, 20]), ([2**31 - 1, 3], [1, 2])):
        dev = on_gpu(pools)
        api.copy_pages(dev, cu(np.array(src, np.int32)), cu(np.array(dst, np.int32)))
        same_pools(dev, ref.copy(pools, src, dst))
        assert api.step_device_status() == ref.BOUNDS and api.step_device_status() == 0


def test_copy_past_32_bits(api):
    """Pages and layers more than 4 GB from the pool's start."""
    pool = torch.zeros(2, 4700, 1 << 20, dtype=torch.uint8, device="cuda")
    pool[:, 4699] = torch.randint(0, 256, (2, 1 << 20), dtype=torch.uint8, device="cuda")
    api.copy_pages([pool], torch.tensor([4699], dtype=torch.int32, device="cuda"), torch.tensor([4500], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[:, 4500], pool[:, 4699]) and not torch.equal(pool[0, 4500], pool[1, 4500])
    assert int(pool[:, :4500].any()) == 0 and int(pool[:, 4501:4699].any()) == 0


# ---------------------------------------------------------------------------------------------
# fork
# ---------------------------------------------------------------------------------------------

def run_fork(api, pools, parents, children, lens, bs, tables, free, shares):
    dev, t, s = on_gpu(pools), cu(tables), cu(shares)
    a = np.asarray(parents, np.int32), np.asarray(children, np.int32), np.asarray(lens, np.int32)
    info = api.fork_pages(dev, cu(a[0]), cu(a[1]), cu(a[2]), bs, t, cu(np.asarray(free, np.int32)), s)
    p2, t2, s2, i2 = ref.fork(pools, *a, bs, tables, np.asarray(free, np.int32), shares)
    same(info, i2, "info")
    same(t, t2, "tables")
    same(s, s2, "shares")
    same_pools(dev, p2)
    return i2


@pytest.mark.parametrize("bs", [1, 7, 64])
@pytest.mark.parametrize("seqs,fan,blocks", [(1, 1, 1), (1, 4, 9), (5, 3, 300), (40, 31, 4)])
def test_fork(api, seqs, fan, blocks, bs):
    g = np.random.default_rng(seqs)
    forks, pages = seqs * fan, seqs * blocks + seqs * fan + 2
    order = g.permutation(pages).astype(np.int32)
    tables = np.full((seqs + forks, blocks), -7, np.int32)
    tables[:seqs] = order[:seqs * blocks].reshape(seqs, blocks)
    lens = np.concatenate([g.integers(0, blocks * bs + 1, seqs), np.full(forks, 3)])
    rows = seqs + g.permutation(forks)
    parents = np.arange(forks) // fan
    children = rows.copy()
    parents[3::11] = -1
    children[5::13] = -4
    info = run_fork(api, pools_of(g, pages), parents, children, lens, bs, tables, order[seqs * blocks:],
                    g.integers(0, 3, pages).astype(np.int32))
    assert info[2] == 0


def test_fork_of_many_blocks_of_forks(api):
    """More forks than one turn of the planning block has."""
    g = np.random.default_rng(3)
    forks, pages = 2500, 2600
    tables = np.full((2 + forks, 3), -1, np.int32)
    tables[:2] = [[5, 6, 7], [8, 9, 10]]
    lens = np.array([20, 33] + [0] * forks)
    info = run_fork(api, pools_of(g, pages, (16, 32)), np.arange(forks) % 2, 2 + g.permutation(forks), lens, 16, tables,
                    np.arange(11, pages), np.zeros(pages, np.int32))
    assert info[0] == forks and info[2] == 0


@pytest.mark.parametrize("what", ["same child", "child is a parent", "itself", "past the requests", "no page", "bad page", "bad last page",
                                  "length", "negative length", "free list"])
def test_fork_refusals(api, what):
    g = np.random.default_rng(4)
    pages, bs = 40, 8
    tables = np.full((8, 4), -1, np.int32)
    tables[:3] = g.permutation(pages)[:12].reshape(3, 4)
    lens, parents, children, free = [20, 32, 9, 0, 0, 0, 0, 0], [0, 1, 2], [3, 4, 5], [30, 31, 32, 33]
    if what == "same child":
        children = [3, 3, 5]
    if what == "child is a parent":
        children = [1, 4, 5]
    if what == "itself":
        children = [0, 4, 5]
    if what == "past the requests":
        parents, children = [0, 8, 2], [3, 4, 2**31 - 1]
    if what == "no page":
        free = [30]
    if what == "bad page":
        tables[0, 1], tables[1, 3] = -1, 40
    if what == "bad last page":
        tables[0, 2], tables[2, 1] = -5, 2**31 - 1
    if what == "length":
        lens[1] = 33
    if what == "negative length":
        lens[1] = -1
    if what == "free list":
        free = [30, 40, -1]
    info = run_fork(api, pools_of(g, pages), parents, children, lens, bs, tables, free, np.zeros(pages, np.int32))
    assert info[2] == ref.BOUNDS


def test_fork_of_nothing(api):
    g = np.random.default_rng(5)
    info = run_fork(api, pools_of(g, 4), [], [], [3], 8, np.full((1, 2), -1, np.int32), [], np.zeros(4, np.int32))
    assert info.tolist() == [0, 0, 0, 0]


# ---------------------------------------------------------------------------------------------
# release
# ---------------------------------------------------------------------------------------------

def run_release(api, tables, lens, keeps, bs, shares, free, num_free, taken, workspace=None):
    t, s, f, n = cu(tables), cu(shares), cu(free), cu(np.array([num_free], np.int32))
    a = np.asarray(lens, np.int32), np.asarray(keeps, np.int32)
    info = api.release_pages(t, cu(a[0]), cu(a[1]), bs, s, f, n, taken=None if taken is None else cu(np.array([taken], np.int32)),
                             workspace=workspace)
    t2, s2, f2, n2, i2 = ref.release(tables, *a, bs, shares, free, num_free, 0 if taken is None else taken)
    same(info, i2, "info")
    same(t, t2, "tables")
    same(s, s2, "shares")
    same(f, f2, "free list")
    assert n.item() == n2
    return i2


def batch(g, seqs, blocks, pages, group):
    """Tables over distinct pages, the first column shared by groups; shares to match; a free list."""
    order = g.permutation(pages).astype(np.int32)
    tables = order[:seqs * blocks].reshape(seqs, blocks).copy()
    tables[:, 0] = tables[np.arange(seqs) // group * group, 0]
    shares = np.zeros(pages, np.int32)
    for s in range(seqs):
        if s % group:
            shares[tables[s, 0]] += 1
    free = np.full(pages, -1, np.int32)
    free[:pages - seqs * blocks] = order[seqs * blocks:]
    return tables, shares, free, pages - seqs * blocks


@pytest.mark.parametrize("taken", [None, 0, 5, 60])
@pytest.mark.parametrize("seqs,blocks,bs", [(1, 1, 1), (3, 4, 16), (17, 130, 7), (300, 3, 64)])
def test_release(api, seqs, blocks, bs, taken):
    g = np.random.default_rng(seqs)
    tables, shares, free, count = batch(g, seqs, blocks, seqs * blocks + 70, 4)
    lens = g.integers(0, blocks * bs + 1, seqs)
    keeps = np.where(g.random(seqs) < 0.4, 0, np.maximum(0, lens - g.integers(0, 2 * bs + 1, seqs)))
    # a group's shared page is named as often as its requests have tokens
    held = np.bincount(tables[lens > 0, 0], minlength=len(shares))
    shares = np.maximum(held - 1, 0).astype(np.int32)
    info = run_release(api, tables, lens, keeps, bs, shares, free, count, taken)
    assert info[2] == 0
    assert info[0] == sum(-(-a // bs) - -(-min(a, b) // bs) for a, b in zip(lens, keeps))


@pytest.mark.parametrize("count,taken,frees", [(0, 0, 0), (0, 0, 9), (10, 10, 0), (10, 10, 3), (10, 10, 10), (10, 10, 12), (10, 9, 0),
                                               (10, 7, 2), (10, 4, 1), (100, 90, 3), (3000, 2500, 7)])
def test_free_list(api, count, taken, frees):
    """Gaps wider and narrower than what fills them, and than what is left of the list."""
    g = np.random.default_rng(count)
    pages = count + frees + 40
    order = g.permutation(pages).astype(np.int32)
    free = np.full(pages, -1, np.int32)
    free[:count] = order[:count]
    tables = order[count:count + max(frees, 1)].reshape(1, -1).copy()
    info = run_release(api, tables, [frees], [0], 1, np.zeros(pages, np.int32), free, count, taken)
    assert info.tolist() == [frees, frees, 0, count - taken + frees]


def test_release_of_many_pages(api):
    """Several listing blocks; one workspace over several calls."""
    g = np.random.default_rng(6)
    pages = 150001
    ws = api.alloc_pages_workspace(pages)
    for turn in range(3):
        tables, shares, free, count = batch(g, 100, 1400, pages, 10)
        lens = g.integers(1, 1400 * 16, 100)
        keeps = np.where(g.random(100) < 0.5, 0, lens) if turn else lens * 0
        info = run_release(api, tables, lens, keeps, 16, shares, free, count, 100 * turn, workspace=ws)
        assert info[2] == 0 and not bool(ws[:256 + 32 * 600].any())


def test_books_of_a_large_pool(api):
    """More pages than one turn of every listing block: 3 million, against sets on the GPU's own side."""
    pages, n, blocks = 3000001, 40, 4000
    order = torch.randperm(pages, device="cuda").to(torch.int32)
    tables = order[:n * blocks].view(n, blocks).clone()
    lens = torch.full((n,), blocks * 16, dtype=torch.int32, device="cuda")
    keeps = torch.where(torch.arange(n, device="cuda") % 2 == 0, lens, 0).to(torch.int32)
    shares = torch.zeros(pages, dtype=torch.int32, device="cuda")
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = api.alloc_pages_workspace(pages)
    gone, kept = tables[1::2].reshape(-1).sort().values, tables[::2].clone()
    info = api.release_pages(tables, lens, keeps, 16, shares, free, count, workspace=ws)
    assert info.tolist() == [n // 2 * blocks, n // 2 * blocks, 0, n // 2 * blocks]
    assert torch.equal(free[:len(gone)], gone) and (free[len(gone):] == -1).all() and torch.equal(tables[::2], kept)
    pool = torch.arange(pages, dtype=torch.int32, device="cuda").view(torch.uint8).view(pages, 4).repeat(1, 4)
    info = api.compact_pages([pool], tables, keeps, 16, shares, free, count, workspace=ws)
    m = n // 2 * blocks
    assert info.tolist() == [m, int((kept >= m).sum()), 0, pages - m] and count.item() == pages - m
    assert torch.equal(tables[::2].reshape(-1).sort().values, torch.arange(m, dtype=torch.int32, device="cuda"))
    held = pool.view(torch.int32)[:, 0]
    assert torch.equal(held[tables[::2].long()], kept)
    moved = kept >= m
    assert torch.equal(tables[::2][~moved], kept[~moved])
    assert torch.equal(tables[::2][moved][kept[moved].argsort()], tables[::2][moved].sort().values)  # in order
    assert torch.equal(free[:pages - m], torch.arange(m, pages, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("what", ["given back twice", "too often", "past the pages", "negative entry", "length", "negative keep",
                                  "negative count", "count", "taken", "negative taken", "full list"])
def test_release_refusals(api, what):
    g = np.random.default_rng(7)
    pages, bs = 50, 8
    tables, shares, free, count = batch(g, 4, 5, pages, 1)
    lens, keeps, taken = [40, 33, 9, 8], [0, 16, 0, 8], 2
    if what == "given back twice":
        tables[0, 1] = tables[0, 0]
    if what == "too often":
        tables[0, :4] = tables[2, 0]
        shares[tables[2, 0]] = 1
    if what == "past the pages":
        tables[0, 2], tables[1, 4] = 50, 2**31 - 1
    if what == "negative entry":
        tables[0, 2] = -3
    if what == "length":
        lens[1] = 41
    if what == "negative keep":
        keeps[0] = -1
    if what == "negative count":
        count = -1
    if what == "count":
        count = 51
    if what == "taken":
        taken = 31
    if what == "negative taken":
        taken = -1
    if what == "full list":
        free[:] = np.arange(50)
        count = 50
    info = run_release(api, tables, lens, keeps, bs, shares, free, count, taken)
    assert info[2] == (0 if what == "negative entry" else ref.BOUNDS)


def test_a_list_that_is_short(api):
    """A plan over the whole buffer of a list with two pages: tokens without a page get no slot, and the
    release that brings the list up to date reports it; what the plan did not get is left out."""
    base, new = cu(np.array([0, 0], np.int32)), cu(np.array([20, 20], np.int32))
    tables = torch.full((2, 4), 9, dtype=torch.int32, device="cuda")
    free, count = cu(np.array([7, 3] + [-1] * 6, np.int32)), cu(np.array([2], np.int32))
    plan = api.plan_step(base, new, free, 8, tables, max_rows=40)
    assert plan.info.tolist()[:2] == [40, 6]
    slots = plan.slots.tolist()
    assert slots[:16] == list(range(56, 64)) + list(range(24, 32)) and slots[16:] == [-1] * 24
    shares = torch.zeros(8, dtype=torch.int32, device="cuda")
    info = api.release_pages(tables, new, cu(np.array([8, 0], np.int32)), 8, shares, free, count, taken=plan.info[1:2])
    assert info.tolist() == [1, 1, ref.BOUNDS, 1] and free.tolist() == [3] + [-1] * 7
    assert tables.tolist() == [[7, -1, -1, 9], [-1, -1, -1, 9]]


def test_release_without_requests(api):
    free = np.arange(16, dtype=np.int32)
    run_release(api, np.zeros((0, 3), np.int32), [], [], 8, np.zeros(16, np.int32), free, 9, 4)


# ---------------------------------------------------------------------------------------------
# compact
# ---------------------------------------------------------------------------------------------

def run_compact(api, pools, tables, lens, bs, shares, workspace=None):
    dev, t, s = on_gpu(pools), cu(tables), cu(shares)
    pages = len(shares)
    f, n = torch.full((pages,), 99, dtype=torch.int32, device="cuda"), torch.full((1,), 99, dtype=torch.int32, device="cuda")
    lens = np.asarray(lens, np.int32)
    info = api.compact_pages(dev, t, cu(lens), bs, s, f, n, workspace=workspace)
    p2, t2, s2, f2, n2, i2 = ref.compact(pools, tables, lens, bs, shares)
    same(info, i2, "info")
    same(t, t2, "tables")
    same(s, s2, "shares")
    same(f, f2, "free list")
    assert n.item() == n2
    same_pools(dev, p2)
    return i2


@pytest.mark.parametrize("spare", [0, 1, 200])
@pytest.mark.parametrize("seqs,blocks,bs", [(1, 1, 1), (3, 4, 16), (17, 140, 7), (200, 3, 64)])
def test_compact(api, seqs, blocks, bs, spare):
    g = np.random.default_rng(seqs + spare)
    pages = seqs * blocks + spare
    tables, shares, _, _ = batch(g, seqs, blocks, pages, 3)
    shares = g.integers(0, 4, pages).astype(np.int32)
    info = run_compact(api, pools_of(g, pages), tables, g.integers(0, blocks * bs + 1, seqs), bs, shares)
    assert info[2] == 0


def test_compact_large_and_again(api):
    g = np.random.default_rng(8)
    pages = 70000
    ws = api.alloc_pages_workspace(pages)
    for turn in range(2):
        tables, shares, _, _ = batch(g, 64, 500, pages, 4)
        info = run_compact(api, pools_of(g, pages, (16, 32), (1, 2)), tables, g.integers(0, 8000, 64), 16, shares, workspace=ws)
        assert info[2] == 0 and info[1] > 5000 and not bool(ws[256:256 + 70000 // 8].any())


def test_compact_edges(api):
    g = np.random.default_rng(9)
    pages = 33
    pools = pools_of(g, pages)
    none = np.full((2, 4), -1, np.int32)
    assert run_compact(api, pools, none, [0, 0], 8, np.ones(pages, np.int32)).tolist() == [0, 0, 0, 33]
    assert run_compact(api, pools, np.zeros((0, 4), np.int32), [], 8, np.ones(pages, np.int32)).tolist() == [0, 0, 0, 33]
    full = g.permutation(32).astype(np.int32).reshape(4, 8)
    assert run_compact(api, pools, full, [64] * 4, 8, np.ones(pages, np.int32)).tolist() == [32, 0, 0, 1]
    full[0, 0], full[1, 1] = -1, 33
    assert run_compact(api, pools, full, [65, 64, 64, 64], 8, np.ones(pages, np.int32))[2] == ref.BOUNDS


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------

def test_life_of_a_pool(api):
    """Requests are planned, forked, roll back and end, and the pool is compacted, all captured in one
    graph that is replayed with other lengths: books as the CPU forms keep them, and every request's
    tokens where its table says."""
    g = np.random.default_rng(10)
    n, blocks, bs, pages = 6, 8, 16, 64
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.zeros(pages, bs * 16, dtype=torch.uint8, device="cuda")
    tables, shares, free, count = torch.full((n, blocks), -1, dtype=torch.int32, device="cuda"), z(pages), z(pages), z(1)
    base, new, keeps, later, parents, children = z(n), z(n), z(n), z(n), z(2), z(2)
    ws = api.alloc_pages_workspace(pages)
    plan = api.alloc_step_plan(n * 40)
    infos = [z(4), z(4), z(4)]

    def step():
        api.plan_step(base, new, free, bs, tables, rows_per_seq=40, out=plan)
        api.release_pages(tables, later, keeps, bs, shares, free, count, taken=plan.info[1:2], info=infos[0], workspace=ws)
        api.fork_pages([pool], parents, children, keeps, bs, tables, free, shares, info=infos[1], workspace=ws)
        api.release_pages(tables, z0, z0, bs, shares, free, count, taken=infos[1][1:2], info=infos[0], workspace=ws)
        api.compact_pages([pool], tables, lens, bs, shares, free, count, info=infos[2], workspace=ws)

    z0, lens = z(n), z(n)
    free.copy_(torch.arange(pages, device="cuda").flip(0))
    count.fill_(pages)
    step()  # loads the kernels: with nothing to do
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    cpu = np.zeros((n, blocks * bs), np.uint8)  # what each request's tokens hold
    now = np.zeros(n, np.int32)
    marks = 0
    for turn in range(12):
        ended = g.random(n) < 0.3
        grow = np.where(g.random(n) < 0.6, g.integers(0, 40, n), 0).astype(np.int32)
        grow = np.minimum(grow, blocks * bs - now)
        grow[5] = 0
        after = now + grow
        keep = np.where(ended, 0, np.maximum(after - g.integers(0, 20, n), 0)).astype(np.int32)
        if turn % 2 == 0:
            keep[5] = 0
        elif not ended[0]:
            keep[0] = after[0]  # back into a page that request 5 shares it may not go and write again
        fork = turn % 2 == 0
        base.copy_(cu(now)), new.copy_(cu(grow)), later.copy_(cu(after)), keeps.copy_(cu(keep))
        parents.copy_(cu(np.array([0 if fork else -1, -1], np.int32)))
        children.copy_(cu(np.array([5, -1], np.int32)))
        final = keep.copy()
        if fork:
            final[5] = keep[0]
        lens.copy_(cu(final))
        # the tokens' bytes are written after the plan: replay in two parts would split the graph, so
        # they go in beforehand through the plan of a dry run on copies
        t2 = tables.clone()
        dry = api.plan_step(base, new, free, bs, t2, rows_per_seq=40)
        slots = dry.slots.cpu().numpy().reshape(n, 40)
        for s in range(n):
            for i in range(int(grow[s])):
                marks = marks % 250 + 1
                assert slots[s, i] >= 0
                pool.view(-1, 16)[int(slots[s, i])] = marks
                cpu[s, now[s] + i] = marks
        graph.replay()
        torch.cuda.synchronize()
        if fork:
            cpu[5] = cpu[0]
        now = final
        table, held = tables.cpu().numpy(), pool.view(-1, 16).cpu().numpy()
        assert infos[0][2].item() == 0 and infos[1][2].item() == 0 and infos[2][2].item() == 0
        used = set()
        for s in range(n):
            for j in range(int(now[s])):
                page = int(table[s, j // bs])
                used.add(page)
                assert (held[page * bs + j % bs] == cpu[s, j]).all(), (turn, s, j)
        assert used == set(range(len(used))) and infos[2][0].item() == len(used)
        refs = np.bincount([p for s in range(n) for p in table[s, :-(-int(now[s]) // bs)]], minlength=pages)
        assert np.array_equal(shares.cpu().numpy(), np.maximum(refs - 1, 0)), turn
        assert count.item() == pages - len(used)
        assert np.array_equal(free.cpu().numpy()[:count.item()], np.arange(len(used), pages))


def test_other_stream(api):
    g = np.random.default_rng(11)
    pools = pools_of(g, 30)
    dev, side = on_gpu(pools), torch.cuda.Stream()
    torch.cuda.synchronize()
    src, dst = cu(np.arange(10, dtype=np.int32)), cu(np.arange(15, 25, dtype=np.int32))
    torch.cuda.synchronize()
    api.copy_pages(dev, src, dst, stream=side)
    side.synchronize()
    same_pools(dev, ref.copy(pools, range(10), range(15, 25)))


def test_tables_of_two_billion_columns(api):
    """Rows as wide as they may be, so that the turns over a row pass 31 bits when rounded up; of the
    entries only those of the lengths are looked at."""
    columns = 2**31 - 1
    if torch.cuda.mem_get_info()[0] < 24 * 2**30:
        pytest.skip("24 GB of device memory")
    tables = torch.empty(2, columns, dtype=torch.int32, device="cuda")
    tables[:, :8] = -1
    tables[0, :3] = cu(np.array([5, 2, 7], np.int32))
    pools = pools_of(np.random.default_rng(5), 9)
    dev, shares = on_gpu(pools), torch.zeros(9, dtype=torch.int32, device="cuda")
    lens = cu(np.array([3, 0], np.int32))
    free = cu(np.array([0, 1, 3, 4, 6, 8, -1, -1, -1], np.int32))
    info = api.fork_pages(dev, cu(np.array([0], np.int32)), cu(np.array([1], np.int32)), lens, 1, tables, free, shares)
    assert info.tolist() == [1, 0, 0, 0]
    assert tables[1, :8].tolist() == [5, 2, 7, -1, -1, -1, -1, -1]
    assert shares.tolist() == [0, 0, 1, 0, 0, 1, 0, 1, 0]
    lens[1] = 3
    num_free = cu(np.array([6], np.int32))
    info = api.release_pages(tables, lens, cu(np.array([0, 2], np.int32)), 1, shares, free, num_free)
    assert info.tolist() == [4, 1, 0, 7]
    assert tables[:, :4].tolist() == [[-1, -1, -1, -1], [5, 2, -1, -1]]
    assert shares.tolist() == [0] * 9 and free[:7].tolist() == [0, 1, 3, 4, 6, 8, 7]
    lens[0], lens[1] = 0, 2
    info = api.compact_pages(dev, tables, lens, 1, shares, free, num_free)
    assert info.tolist() == [2, 2, 0, 7]
    assert tables[1, :2].tolist() == [1, 0] and free.tolist() == [2, 3, 4, 5, 6, 7, 8, -1, -1]
    want = [p.copy() for p in pools]
    for p in want:
        p[:, 0], p[:, 1] = p[:, 2].copy(), p[:, 5].copy()
    same_pools([d[..., :2, :] for d in dev], [w[:, :2] for w in want])
