"""Measured calls of the operators that fill a paged cache and look after its pages: the attention of
prompt chunks over the cache, and copying, forking, releasing and compacting pages.

`run` computes each in plain torch operations, or with `own` set calls the framework. A case is a
dict of plain values; request lengths follow from the case alone, the data from the seed.
"""
import math
import random

import torch

own = False

LATENT, INDEX = 512, 128


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # The tail of one short prompt on a shard of 16 heads: latency.
        dict(name="prefill_tiny", op="prefill", seqs=1, heads=16, lo=300, hi=300, new_lo=5, new_hi=5, bs=64, one=True, pad=0),
        # A mixed step: decoding requests of one token beside prompts of some hundred, a padded batch.
        dict(name="prefill_mixed", op="prefill", seqs=48, heads=64, lo=0, hi=8192, new_lo=1, new_hi=300, bs=64, one=True, pad=9),
        # Odd sizes: heads that fill no group, pages that are no power of two, K and V in buffers of their own.
        dict(name="prefill_odd", op="prefill", seqs=5, heads=20, lo=0, hi=3001, new_lo=0, new_hi=777, bs=100, one=False, pad=3),
        # A chunk of 1024 tokens of one long prompt, 32 thousand tokens before it: arithmetic.
        dict(name="prefill_chunk_1024", op="prefill", seqs=1, heads=64, lo=32768, hi=32768, new_lo=1024, new_hi=1024, bs=64, one=True, pad=0),
        # A few pages of one layer to other places: latency.
        dict(name="copy_8", op="copy", pages=64, count=8, layers=1, bs=64, gaps=False),
        # Pages of several requests through all layers of a stage.
        dict(name="copy_1024", op="copy", pages=4096, count=1024, layers=4, bs=64, gaps=True),
        # One request goes on in four ways: latency.
        dict(name="fork_beam", op="fork", seqs=1, fan=4, lo=8000, hi=8000, layers=1, bs=64),
        # 32 prompts with eight samples each, over several layers.
        dict(name="fork_samples", op="fork", seqs=32, fan=8, lo=1024, hi=16384, layers=4, bs=64),
        # A step's rejected drafts: 64 requests give back what few pages they had taken too many.
        dict(name="release_drafts", op="release", seqs=64, group=1, lo=8192, hi=32768, keep="draft", bs=64, taken=64),
        # Half of a batch ends, prompts shared by groups of four.
        dict(name="release_finished", op="release", seqs=256, group=4, lo=16384, hi=131072, keep="some", bs=64, taken=1000),
        # A small pool with a third of it in use.
        dict(name="compact_small", op="compact", seqs=8, lo=100, hi=1000, spare=2.5, layers=1, bs=48),
        # A pool of several layers after many requests came and went.
        dict(name="compact_large", op="compact", seqs=64, lo=1024, hi=4096, spare=2.0, layers=3, bs=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "copy", "fork", "release", "compact"])
    bs = rng.choice([16, 24, 32, 48, 64, 64, 100, 128])
    if op == "prefill":
        heads = rng.choice([1, 8, 16, 20, 24, 40, 64, 64, 96, 128])
        seqs = _log_int(rng, 1, 128)
        new_hi = _log_int(rng, 1, max(2, min(2048, 8192 // seqs)))
        most = max(64, min(131072, 1024 * 32768 * 64 // (seqs * new_hi * heads) - new_hi, 2097152 // seqs))
        hi = _log_int(rng, 64, most)
        return dict(op=op, seqs=seqs, heads=heads, lo=rng.choice([0, 0, hi // 2, hi]), hi=hi, new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi,
                    bs=bs, one=rng.random() < 0.8, pad=rng.choice([0, 0, 1, 17]))
    layers = _log_int(rng, 1, 6)
    room = 16384 * 64 // (bs * layers)  # pages that the largest pools hold
    if op == "copy":
        pages = _log_int(rng, 8, min(16384, room))
        return dict(op=op, pages=pages, count=_log_int(rng, 1, pages // 2), layers=layers, bs=bs, gaps=rng.random() < 0.5)
    if op == "fork":
        fan = rng.choice([1, 2, 4, 8, 16])
        seqs = _log_int(rng, 1, 256 // fan)
        hi = _log_int(rng, 1, max(2, min(32768, room * bs // (2 * seqs))))
        return dict(op=op, seqs=seqs, fan=fan, lo=rng.randint(0, hi), hi=hi, layers=layers, bs=bs)
    if op == "release":
        seqs = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, 131072)
        return dict(op=op, seqs=seqs, group=rng.choice([1, 1, 2, 5]), lo=rng.randint(0, hi), hi=hi,
                    keep=rng.choice(["all", "some", "draft"]), bs=max(bs, 32), taken=rng.choice([0, 3, seqs, 500]))
    seqs = _log_int(rng, 1, 128)
    hi = _log_int(rng, 1, max(2, min(8192, room * bs // (4 * seqs))))
    return dict(op=op, seqs=seqs, lo=rng.randint(0, hi), hi=hi, spare=rng.choice([1.0, 1.5, 2.0, 3.0]), layers=layers, bs=bs)


def _spread(n, lo, hi, salt):
    r = random.Random("%d %d %d %s" % (n, lo, hi, salt))
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    return _spread(case["seqs"], case["lo"], case["hi"], "len")


def _news(case):
    """New tokens per request; of a batch's requests every third one decodes a single token."""
    new = _spread(case["seqs"], case["new_lo"], case["new_hi"], "new")
    return [min(n, 1) if case["seqs"] > 2 and i % 3 == 2 else n for i, n in enumerate(new)]


def _keeps(case):
    lens, r = _lens(case), random.Random("keep %d" % case["seqs"])
    if case["keep"] == "all":
        return [0] * len(lens)
    if case["keep"] == "some":
        return [0 if r.random() < 0.5 else n for n in lens]
    return [max(0, n - r.randint(0, 7)) for n in lens]


def _pages_of(n, bs):
    return -(-n // bs)


def _blocks(case):
    """Pages that the longest request needs."""
    more = _news(case) if case["op"] == "prefill" else [0] * case["seqs"]
    return max(1, max(_pages_of(a + b, case["bs"]) for a, b in zip(_lens(case), more)))


def _index_stride(bs):
    return -(-bs * (INDEX + 4) // 16) * 16


def _page_bytes(case):
    """Bytes of a page in all pools: latent rows, index codes with their scales, in every layer."""
    return case["layers"] * (case["bs"] * LATENT + _index_stride(case["bs"]))


def _prefix(case):
    """Pages that each request shares with the first one of its group."""
    lens, g, bs = _lens(case), case["group"], case["bs"]
    first = [lens[i - i % g] for i in range(len(lens))]
    return [min(a, b) // 2 // bs if g > 1 else 0 for a, b in zip(lens, first)]


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pools(g, case, pages):
    """The caches of every layer, filled with codes and scales that are numbers (no byte has bit 3)."""
    out = []
    for width in (case["bs"] * LATENT, _index_stride(case["bs"])):
        t = torch.randint(0, 256, (case["layers"], pages, width), generator=g, device="cuda", dtype=torch.uint8)
        out.append(t.bitwise_and_(0xF7))
    return out


def _keep_ints(st, **parts):
    """What a call changes in the requests' books, in one buffer, and how it stood: each pass starts from there."""
    sizes = [t.numel() for t in parts.values()]
    st["saved"] = torch.cat([t.reshape(-1) for t in parts.values()])
    st["books"] = st["saved"].clone()
    at = 0
    for (name, t), n in zip(parts.items(), sizes):
        st[name] = st["books"][at:at + n].view(t.shape)
        at += n


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, bs = case["op"], case["bs"]
    perm = lambda n: torch.randperm(n, generator=g, device="cuda").to(torch.int32)  # noqa: E731
    st = {"case": case}
    if op == "prefill":
        n, h, lens, new = case["seqs"], case["heads"], _lens(case), _news(case)
        blocks = _blocks(case)
        pages, rows = n * blocks, sum(new) + case["pad"]
        st.update(tables=perm(pages).view(n, blocks), blocks=blocks, base=_ints(lens), new=_ints(new),
                  q=torch.randn(max(1, rows), h, LATENT, generator=g, device="cuda").to(torch.bfloat16),
                  out=torch.full((max(1, rows), h, LATENT), 0.03125, dtype=torch.bfloat16, device="cuda"),
                  k_scale=0.05, v_scale=0.05, sm_scale=LATENT ** -0.5)
        for name in ("k", "v"):
            if name == "v" and case["one"]:
                st["v"] = st["k"]
                continue
            st[name] = torch.empty(pages, bs * LATENT, dtype=torch.uint8, device="cuda")
            for at in range(0, pages, 1 << 14):  # in parts: the pool in 32 bits would be four times its size
                part = torch.randn(min(1 << 14, pages - at), bs * LATENT, generator=g, device="cuda").mul_(20.0)
                st[name][at:at + (1 << 14)] = part.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return st
    if op == "copy":
        order = perm(case["pages"])
        src, dst = order[:case["count"]].clone(), order[case["count"]:2 * case["count"]].clone()
        if case["gaps"]:
            src[torch.rand(case["count"], generator=g, device="cuda") < 0.05] = -1
        st.update(pools=_pools(g, case, case["pages"]), src=src, dst=dst)
        return st
    n, blocks, lens = case["seqs"], _blocks(case), _lens(case)
    if op == "fork":
        forks = n * case["fan"]
        pages = n * blocks + forks + 5
        order = perm(pages)
        tables = torch.full((n + forks, blocks), -1, dtype=torch.int32, device="cuda")
        tables[:n] = order[:n * blocks].view(n, blocks)
        _keep_ints(st, tables=tables, shares=torch.zeros(pages, dtype=torch.int32, device="cuda"))
        st.update(lens=_ints(lens + [0] * forks), parents=_ints([i // case["fan"] for i in range(forks)]),
                  children=_ints([n + i for i in range(forks)]), free=order[n * blocks:].clone(), pools=_pools(g, case, pages),
                  pages=pages)
        return st
    if op == "release":
        pages = n * blocks + case["taken"] + 999
        order = perm(pages)
        tables = order[:n * blocks].view(n, blocks).clone()
        pre = _prefix(case)
        first = torch.arange(n, device="cuda") // case["group"] * case["group"]
        shared = torch.arange(blocks, device="cuda")[None, :] < _ints(pre)[:, None]
        tables = torch.where(shared, tables[first], tables)
        shares = torch.zeros(pages, dtype=torch.int32, device="cuda")
        others = shared & (first != torch.arange(n, device="cuda"))[:, None]
        shares.index_add_(0, tables[others].long(), torch.ones_like(tables[others]))
        free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        free[:case["taken"] + 999] = order[n * blocks:]
        _keep_ints(st, tables=tables, shares=shares, free=free, num_free=_ints([case["taken"] + 999]))
        st.update(lens=_ints(lens), keeps=_ints(_keeps(case)), taken=_ints([case["taken"]]), pages=pages)
        return st
    pages = max(n * blocks, int(n * blocks * case["spare"]))
    order = perm(pages)
    shares = torch.zeros(pages, dtype=torch.int32, device="cuda")
    _keep_ints(st, tables=order[:n * blocks].view(n, blocks).clone(), shares=shares,
               free=torch.full((pages,), -1, dtype=torch.int32, device="cuda"), num_free=_ints([0]))
    st["saved"][n * blocks:n * blocks + pages] = torch.randint(0, 3, (pages,), generator=g, device="cuda", dtype=torch.int32)
    st.update(lens=_ints(lens), pools=_pools(g, case, pages), pages=pages)
    return st


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if "books" in state:
        state["books"].copy_(state["saved"])
    if own:
        return {"prefill": _own_prefill, "copy": _own_copy, "fork": _own_fork, "release": _own_release,
                "compact": _own_compact}[op](state)
    return {"prefill": _plain_prefill, "copy": _plain_copy, "fork": _plain_fork, "release": _plain_release,
            "compact": _plain_compact}[op](state)


def _values(st):
    """The pools as the values they hold: latent codes, index codes, index scales."""
    n = st["case"]["bs"] * INDEX
    latent, index = st["pools"]
    return [latent.view(torch.float8_e4m3fn), index[:, :, :n].view(torch.float8_e4m3fn),
            index[:, :, n:n + 4 * st["case"]["bs"]].view(torch.float32)]


def _workspace(st):
    from sparse_mla_paged_gb300 import api

    if "workspace" not in st:  # kept from call to call, as a serving loop does
        st["workspace"] = api.alloc_pages_workspace(st["pages"])
    return st["workspace"]


def _own_prefill(st):
    from sparse_mla_paged_gb300 import api

    c = st["case"]
    if "workspace" not in st:
        st["workspace"] = api.alloc_prefill_workspace(c["seqs"], st["q"].shape[0], c["heads"])
    return api.prefill(st["q"], st["k"], st["v"], st["tables"], st["blocks"], st["base"], st["new"], c["heads"], c["bs"],
                       c["bs"] * LATENT, st["k_scale"], st["v_scale"], st["sm_scale"], out=st["out"], workspace=st["workspace"])


def _plain_prefill(st):
    c, bs = st["case"], st["case"]["bs"]
    h, at = c["heads"], 0
    for s, (base, new) in enumerate(zip(_lens(c), _news(c))):
        if new == 0:
            continue
        n = base + new
        table = st["tables"][s, :_pages_of(n, bs)].long()
        k = st["k"][table].view(-1, LATENT)[:n].view(torch.float8_e4m3fn).float()
        v = k if c["one"] else st["v"][table].view(-1, LATENT)[:n].view(torch.float8_e4m3fn).float()
        step = max(1, (1 << 29) // (h * n))  # rows whose scores take 2 GB
        for i in range(0, new, step):
            m = min(step, new - i)
            seen = torch.arange(n, device="cuda") <= base + i + torch.arange(m, device="cuda")[:, None, None]
            x = torch.matmul(st["q"][at + i:at + i + m].float().view(m * h, LATENT), k.t()).view(m, h, n)
            x = torch.where(seen, x * (st["sm_scale"] * st["k_scale"]), -math.inf)
            p = torch.exp(x - x.amax(2, keepdim=True))
            p = p / p.sum(2, keepdim=True)
            o = torch.matmul(p.view(m * h, n), v) * st["v_scale"]
            st["out"][at + i:at + i + m] = o.view(m, h, LATENT).to(torch.bfloat16)
        at += new
    return st["out"]


def _own_copy(st):
    from sparse_mla_paged_gb300 import api

    api.copy_pages(st["pools"], st["src"], st["dst"])
    return _values(st)


def _plain_copy(st):
    live = (st["src"] >= 0) & (st["dst"] >= 0)
    src, dst = st["src"][live].long(), st["dst"][live].long()
    for pool in st["pools"]:
        pool[:, dst] = pool[:, src]
    return _values(st)


def _own_fork(st):
    from sparse_mla_paged_gb300 import api

    info = api.fork_pages(st["pools"], st["parents"], st["children"], st["lens"], st["case"]["bs"], st["tables"], st["free"],
                          st["shares"], workspace=_workspace(st))
    return [st["tables"], st["shares"], info] + _values(st)


def _plain_fork(st):
    bs, tables, shares = st["case"]["bs"], st["tables"], st["shares"]
    parents, children = st["parents"].long(), st["children"].long()
    n = st["lens"][parents].long()
    whole, part = n // bs, n % bs > 0
    col = torch.arange(tables.shape[1], device="cuda")[None, :]
    mine = tables[parents]
    common = col < whole[:, None]
    shares.index_add_(0, mine[common].long(), torch.ones_like(mine[common]))
    fresh = st["free"][(torch.cumsum(part.long(), 0) - 1).clamp(min=0)]
    last = part[:, None] & (col == whole[:, None])
    src, dst = mine[last].long(), fresh[part].long()
    tables[children] = torch.where(common, mine, torch.where(last, fresh[:, None], tables[children]))
    for pool in st["pools"]:
        pool[:, dst] = pool[:, src]
    taken = part.sum()
    info = torch.stack([taken * 0 + parents.numel(), taken, taken * 0, taken * 0]).int()
    return [tables, shares, info] + _values(st)


def _own_release(st):
    from sparse_mla_paged_gb300 import api

    info = api.release_pages(st["tables"], st["lens"], st["keeps"], st["case"]["bs"], st["shares"], st["free"], st["num_free"],
                             taken=st["taken"], workspace=_workspace(st))
    return [st["tables"], st["shares"], st["free"], st["num_free"], info]


def _plain_release(st):
    bs, tables, shares, free = st["case"]["bs"], st["tables"], st["shares"], st["free"]
    have, keep = (st["lens"] + bs - 1) // bs, (torch.minimum(st["keeps"], st["lens"]) + bs - 1) // bs
    col = torch.arange(tables.shape[1], device="cuda")[None, :]
    gone = (col >= keep[:, None]) & (col < have[:, None])
    back = torch.bincount(tables[gone].long(), minlength=st["pages"]).int()
    ends = back > shares
    freed = torch.nonzero(ends).view(-1).int()
    shares.copy_(torch.where(ends, 0, shares - back))
    tables[gone] = -1
    count, room = st["num_free"].clone(), torch.arange(st["pages"], device="cuda")
    taken = torch.minimum(st["taken"], count)
    left, f = count - taken, torch.full_like(taken, freed.numel())
    moved = torch.minimum((taken - f).clamp(min=0), left)
    # Entry i: of the pages given back, of the list's last ones, as it was, or none.
    given = torch.cat([freed, freed.new_full((1,), -1)])
    which = torch.where(room < taken, room, torch.where(room >= count, room - count + taken, st["pages"])).clamp(max=freed.numel())
    mine = given[which]
    from_end = free[(count - moved + room - f).clamp(0, st["pages"] - 1)]
    new = torch.where(mine >= 0, mine, torch.where((room >= f) & (room < f + moved), from_end, free))
    free.copy_(torch.where(room < left + f, new, -1))
    st["num_free"].copy_(left + f)
    info = torch.cat([gone.sum().view(1).int(), f, f * 0, left + f])
    return [tables, shares, free, st["num_free"], info]


def _own_compact(st):
    from sparse_mla_paged_gb300 import api

    info = api.compact_pages(st["pools"], st["tables"], st["lens"], st["case"]["bs"], st["shares"], st["free"], st["num_free"],
                             workspace=_workspace(st))
    return [st["tables"], st["shares"], st["free"], st["num_free"], info] + _values(st)


def _plain_compact(st):
    bs, tables, shares, pages = st["case"]["bs"], st["tables"], st["shares"], st["pages"]
    used = torch.arange(tables.shape[1], device="cuda")[None, :] < ((st["lens"] + bs - 1) // bs)[:, None]
    live = torch.zeros(pages, dtype=torch.bool, device="cuda")
    live[tables[used].long()] = True
    n = int(live.sum())
    src, dst = torch.nonzero(live[n:]).view(-1) + n, torch.nonzero(~live[:n]).view(-1)
    to = torch.arange(pages, dtype=torch.int32, device="cuda")
    to[src] = dst.int()
    tables.copy_(torch.where(used, to[tables.clamp(min=0).long()], tables))
    shares[dst] = shares[src]
    shares[n:] = 0
    for pool in st["pools"]:
        pool[:, dst] = pool[:, src]
    at = torch.arange(pages, dtype=torch.int32, device="cuda")
    st["free"].copy_(torch.where(at < pages - n, at + n, -1))
    st["num_free"].fill_(pages - n)
    info = _ints([n, src.numel(), 0, pages - n])
    return [tables, shares, st["free"], st["num_free"], info] + _values(st)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op, bs = case["op"], case["bs"]
    if op == "prefill":
        lens, new, h = _lens(case), _news(case), case["heads"]
        keys = sum(a + b for a, b in zip(lens, new) if b)
        seen = sum(b * a + b * (b + 1) // 2 for a, b in zip(lens, new))
        table = sum(_pages_of(a + b, bs) for a, b in zip(lens, new) if b) * 4
        return {"bytes": keys * LATENT * (1 if case["one"] else 2) + sum(new) * h * LATENT * 4 + 8 * len(lens) + table,
                "flops": 4 * LATENT * h * seen}
    if op == "copy":
        return {"bytes": 2 * case["count"] * _page_bytes(case) + 8 * case["count"], "flops": 0}
    lens = _lens(case)
    if op == "fork":
        whole, part = sum(n // bs for n in lens), sum(1 for n in lens if n % bs)
        return {"bytes": case["fan"] * (2 * part * _page_bytes(case) + 4 * whole + 16 * case["seqs"]) + 12 * whole, "flops": 0}
    if op == "release":
        gone = sum(max(0, _pages_of(a, bs) - _pages_of(min(a, b), bs)) for a, b in zip(lens, _keeps(case)))
        return {"bytes": 8 * case["seqs"] + 20 * gone, "flops": 0}
    used = sum(_pages_of(n, bs) for n in lens)
    pages = max(case["seqs"] * _blocks(case), int(case["seqs"] * _blocks(case) * case["spare"]))
    moved = used * (pages - used) // pages  # on average: pages lie anywhere
    return {"bytes": moved * (2 * _page_bytes(case) + 16) + 4 * used + 8 * (pages - used) + 4 * case["seqs"], "flops": 0}


# ---------------------------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------

def _e4m3_values():
    """The 256 values of the 8-bit code: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = math.nan if code & 127 == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def exact(case, seed):
    if case["op"] != "prefill" or work(case)["flops"] > 8e12:
        return None  # whole numbers and copied bytes only; or too long in 64 bits
    st = prepare(case, seed)
    value, bs, h = _e4m3_values(), case["bs"], case["heads"]
    out = st["out"].double()
    row = 0
    for s, (base, new) in enumerate(zip(_lens(case), _news(case))):
        pages = st["tables"][s].long()
        keys = value[st["k"][pages].view(-1, LATENT)[:base + new].int()]
        vals = keys if case["one"] else value[st["v"][pages].view(-1, LATENT)[:base + new].int()]
        i = 0
        while i < new:
            m = min(new - i, max(1, (1 << 28) // (h * (base + new))))
            q = st["q"][row:row + m].double() * (st["k_scale"] * st["sm_scale"])
            score = torch.einsum("mhd,nd->mhn", q, keys)
            for r in range(m):  # what comes after a row's own token is not there
                score[r, :, base + i + r + 1:] = -math.inf
            weight = (score - torch.logsumexp(score, 2, keepdim=True)).exp_()
            out[row:row + m] = torch.einsum("mhn,nd->mhd", weight, vals) * st["v_scale"]
            i += m
            row += m
    return out
