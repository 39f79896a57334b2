"""Measured calls of the operators around the sparse decode: the step plan (pages and slots of new
tokens), the index-key writer, the pooled index scores and the attention over a whole paged cache.

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
        # One decode step of 64 requests in a ragged batch, one new token each: only latency counts.
        dict(name="plan_decode_64", op="plan", seqs=64, rps=1, lo=8192, hi=32768, new_lo=1, new_hi=1, bs=64),
        # A large mixed prefill: packed prompts from one token to several thousand.
        dict(name="plan_prefill_256", op="plan", seqs=256, rps=0, lo=0, hi=16384, new_lo=1, new_hi=4001, bs=64),
        # The index keys of one decode step.
        dict(name="index_write_64", op="write", rows=64, bs=64, norm=True, gaps=False),
        # The index keys of a prefill chunk, padding rows among them.
        dict(name="index_write_262144", op="write", rows=262144, bs=64, norm=True, gaps=True),
        # A small odd call: a draft of three rows, few heads, a page size that is no power of two.
        dict(name="scores_odd", op="scores", seqs=3, rps=3, heads=20, lo=1200, hi=5001, bs=48, kpool=3, verify=True),
        # The ragged decode batch: one row a request, contexts of 8k to 32k.
        dict(name="scores_ragged", op="scores", seqs=64, rps=1, heads=64, lo=8192, hi=32768, bs=64, kpool=4, verify=True),
        # The 128k decode batch, the most keys that a decode step reads.
        dict(name="scores_pooled_128k", op="scores", seqs=128, rps=1, heads=64, lo=131072, hi=131072, bs=64, kpool=4, verify=True),
        # A prefill chunk of one request: 1024 rows over a 32k context, bound by arithmetic.
        dict(name="scores_prefill", op="scores", seqs=1, rps=1024, heads=64, lo=32768, hi=32768, bs=64, kpool=4, verify=True),
        # One short request on a shard of 16 heads: latency.
        dict(name="full_tiny", op="full", seqs=1, rps=1, heads=16, lo=777, hi=777, bs=64, verify=False),
        # The ragged decode batch attended without a selection.
        dict(name="full_ragged", op="full", seqs=64, rps=1, heads=64, lo=8192, hi=32768, bs=64, verify=False),
        # Four verify rows of 32 requests on a shard of 16 heads.
        dict(name="full_verify_k4", op="full", seqs=32, rps=4, heads=16, lo=16384, hi=16384, bs=64, verify=True),
        # Two very long contexts with all heads: split over the cache's length and joined.
        dict(name="full_long", op="full", seqs=2, rps=1, heads=128, lo=500001, hi=524288, bs=64, verify=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "scores", "scores", "full", "full"])
    bs = rng.choice([16, 32, 48, 64, 64, 100, 128])
    if op == "plan":
        seqs = _log_int(rng, 1, 4096)
        base = _log_int(rng, 16, 32768)
        if rng.random() < 0.5:
            rps = rng.randint(1, 8)
            return dict(op=op, seqs=seqs, rps=rps, lo=0, hi=base, new_lo=0, new_hi=rps, bs=bs)
        return dict(op=op, seqs=seqs, rps=0, lo=0, hi=base, new_lo=0, new_hi=_log_int(rng, 1, max(2, 1000000 // seqs)), bs=bs)
    if op == "write":
        return dict(op=op, rows=_log_int(rng, 1, 262144), bs=bs, norm=rng.random() < 0.7, gaps=rng.random() < 0.5)
    if op == "scores":
        heads = rng.choice([8, 20, 32, 48, 64, 64, 128])
        seqs, rps = _log_int(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4, 7, _log_int(rng, 16, 600)])
        seqs = max(1, min(seqs, 256 // rps))
        most = min(131072, (1024 * 32768 * 64) // (seqs * rps * heads), 16777216 // seqs)
        hi = _log_int(rng, min(200, most), most)
        return dict(op=op, seqs=seqs, rps=rps, heads=heads, lo=rng.randint(1, hi), hi=hi, bs=bs,
                    kpool=rng.choice([1, 2, 3, 4, 4, 4, 8, 16]), verify=rng.random() < 0.7)
    heads = rng.choice([1, 8, 16, 24, 40, 64, 64, 96, 128])
    seqs, rps = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4])
    most = min(524288, (64 * 20000 * 64) // (seqs * rps * heads), 1310720 // seqs)
    hi = _log_int(rng, min(64, most), most)
    return dict(op=op, seqs=seqs, rps=rps, heads=heads, lo=rng.randint(0, hi), hi=hi, bs=bs, verify=rng.random() < 0.5)


def _spread(n, lo, hi, salt):
    r = random.Random("%d %d %d %s" % (n, lo, hi, salt))
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    """Per sequence: tokens in the cache before the rows (verify rows) or in all."""
    return _spread(case["seqs"], case["lo"], case["hi"], "len")


def _row_lens(case):
    """Visible length of each row, row by row of each sequence."""
    lens = _lens(case)
    if case["verify"]:
        return [[n + i + 1 for i in range(case["rps"])] for n in lens]
    r = random.Random("rows %d %d" % (case["seqs"], case["hi"]))
    return [[n] + [r.randint(0, n) for _ in range(case["rps"] - 1)] for n in lens]


def _blocks(case):
    """Pages that the longest sequence needs."""
    return max(1, -(-max(max(x) for x in _row_lens(case)) // case["bs"]))


def _pools(case):
    return max(1, -(-max(max(x) for x in _row_lens(case)) // case["kpool"]))


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(g, seqs, blocks):
    """Block tables over a scattered pool: a permutation of its pages."""
    pages = seqs * blocks
    return torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(seqs, blocks), pages


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, bs = case["op"], case["bs"]
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    if op == "plan":
        n, rps = case["seqs"], case["rps"]
        base = _lens(case)
        new = _spread(n, case["new_lo"], case["new_hi"], "new")
        blocks = max(1, max(-(-(b + x) // bs) for b, x in zip(base, new)))
        tables, pages = _tables(g, n, blocks)
        need = sum(-(-(b + x) // bs) - -(-b // bs) for b, x in zip(base, new))
        st.update(base=_ints(base), new=_ints(new), tables=tables.contiguous(), blocks=blocks,
                  rows=n * rps if rps else sum(new) + 5,
                  free=(pages + torch.randperm(need + 7, generator=g, device="cuda")).to(torch.int32))
    elif op == "write":
        rows = case["rows"]
        pages = -(-rows // bs) + 3
        st.update(x=normal(rows, INDEX).to(torch.bfloat16), w=(1.0 + 0.2 * normal(INDEX)).to(torch.bfloat16),
                  b=(0.1 * normal(INDEX)).to(torch.bfloat16), stride=-(-bs * (INDEX + 4) // 16) * 16)
        slots = torch.randperm(pages * bs, generator=g, device="cuda")[:rows].contiguous()
        if case["gaps"]:
            slots[torch.rand(rows, generator=g, device="cuda") < 0.03] = -1
        st.update(slots=slots, cache=torch.zeros(pages, st["stride"], dtype=torch.uint8, device="cuda"))
    elif op == "scores":
        n, rps, h = case["seqs"], case["rps"], case["heads"]
        blocks = _blocks(case)
        tables, pages = _tables(g, n, blocks)
        stride = -(-bs * (INDEX + 4) // 16) * 16
        cache = torch.empty(pages, stride, dtype=torch.uint8, device="cuda")
        codes = normal(pages, bs * INDEX).mul_(120.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        cache[:, :bs * INDEX] = codes.view(torch.uint8)
        del codes
        scales = (0.005 + 0.01 * torch.rand(pages, bs, generator=g, device="cuda"))
        cache[:, bs * INDEX:bs * (INDEX + 4)] = scales.view(torch.uint8)
        st.update(q=normal(n * rps, h, INDEX).to(torch.bfloat16), w=normal(n * rps, h) / math.sqrt(h * INDEX), cache=cache,
                  stride=stride, tables=tables, blocks=blocks, pools=_pools(case),
                  q_pos=_ints([x - 1 for r in _row_lens(case) for x in r]))
    else:
        n, rps, h = case["seqs"], case["rps"], case["heads"]
        blocks = _blocks(case)
        tables, pages = _tables(g, n, blocks)
        cache = torch.empty(pages, bs * LATENT, dtype=torch.uint8, device="cuda")
        for at in range(0, pages, 1 << 14):  # in parts: the pool in 32 bits would be four times its size
            part = normal(min(1 << 14, pages - at), bs * LATENT).mul_(20.0).clamp_(-448.0, 448.0)
            cache[at:at + (1 << 14)] = part.to(torch.float8_e4m3fn).view(torch.uint8)
        st.update(q=normal(n * rps, h, LATENT).to(torch.bfloat16), cache=cache, tables=tables, blocks=blocks,
                  k_scale=0.05, v_scale=0.05, sm_scale=LATENT ** -0.5,
                  lens=_ints(_lens(case)) if case["verify"] else _ints([x for r in _row_lens(case) for x in r]))
    return st


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "write": _own_write, "scores": _own_scores, "full": _own_full}[op](state)
    return {"plan": _plain_plan, "write": _plain_write, "scores": _plain_scores, "full": _plain_full}[op](state)


def _cache_values(st):
    """The index cache as the values it holds: codes and scales."""
    n = st["case"]["bs"] * INDEX
    return st["cache"][:, :n].view(torch.float8_e4m3fn), st["cache"][:, n:n + 4 * st["case"]["bs"]].view(torch.float32)


def _own_plan(st):
    from sparse_mla_paged_gb300 import api

    c = st["case"]
    p = api.plan_step(st["base"], st["new"], st["free"], c["bs"], st["tables"], rows_per_seq=c["rps"], max_rows=st["rows"])
    return [p.slots, p.positions, p.row_lens, p.row_seqs, p.info, st["tables"]]


def _plain_plan(st):
    c, bs, tables, free = st["case"], st["case"]["bs"], st["tables"], st["free"]
    base, new = st["base"].long(), st["new"].long()
    have, want = (base + bs - 1) // bs, (base + new + bs - 1) // bs
    grow = want - have
    g0 = torch.cumsum(grow, 0) - grow
    col = torch.arange(st["blocks"], device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (g0[:, None] + col - have[:, None]).clamp(0, free.numel() - 1)
    tables.copy_(torch.where(fresh, free[at], tables))
    row = torch.arange(st["rows"], device="cuda")
    if c["rps"]:
        seq, i = row // c["rps"], row % c["rps"]
        live = i < new[seq]
    else:
        ends = torch.cumsum(new, 0)
        seq = torch.searchsorted(ends, row, right=True)
        live = seq < c["seqs"]
        seq = seq.clamp(max=c["seqs"] - 1)
        i = row - (ends - new)[seq]
    pos = torch.where(live, base[seq] + i, 0)
    slot = tables[seq, pos // bs].long() * bs + pos % bs
    info = torch.stack([new.sum(), grow.sum(), grow.sum() * 0, grow.sum() * 0])
    return [torch.where(live, slot, -1), torch.where(live, pos, -1).int(), torch.where(live, pos + 1, 0).int(),
            torch.where(live, seq, -1).int(), info.int(), tables]


def _own_write(st):
    from sparse_mla_paged_gb300 import api

    norm = st["case"]["norm"]
    api.index_write(st["x"], st["slots"], st["case"]["bs"], st["stride"], st["cache"],
                    norm_weight=st["w"] if norm else None, norm_bias=st["b"] if norm else None, eps=1e-6)
    return _cache_values(st)


def _plain_write(st):
    c, bs, cache = st["case"], st["case"]["bs"], st["cache"]
    y = st["x"].float()
    if c["norm"]:
        y = y - y.mean(1, keepdim=True)
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * st["w"].float() + st["b"].float()
    scale = y.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100) / 448.0
    codes = (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    live = st["slots"] >= 0
    slots = torch.where(live, st["slots"], 0)
    page, off = slots // bs, slots % bs
    at = page[:, None] * st["stride"] + off[:, None] * INDEX + torch.arange(INDEX, device="cuda")
    flat = cache.view(-1)
    flat[at[live]] = codes[live]
    at = page[:, None] * st["stride"] + bs * INDEX + 4 * off[:, None] + torch.arange(4, device="cuda")
    flat[at[live]] = scale.view(torch.uint8)[live]
    return _cache_values(st)


def _own_scores(st):
    from sparse_mla_paged_gb300 import api

    c = st["case"]
    return api.pool_scores(st["q"], st["w"], st["cache"], st["tables"], st["blocks"], st["q_pos"], c["seqs"], c["rps"],
                           c["heads"], c["bs"], st["stride"], c["kpool"], st["pools"])


def _plain_scores(st):
    c = st["case"]
    n, rps, h, bs, kpool, pools = c["seqs"], c["rps"], c["heads"], c["bs"], c["kpool"], st["pools"]
    codes, scales = _cache_values(st)
    t = st["tables"].long()
    k = codes.view(torch.uint8).view(-1, bs, INDEX)[t].view(torch.float8_e4m3fn).float().view(n, -1, INDEX)
    ks = scales[t].view(n, -1)
    dots = torch.matmul(st["q"].float().view(n, rps * h, INDEX), k.transpose(1, 2)).view(n, rps, h, -1)
    s = (dots.clamp_(min=0.0) * st["w"].view(n, rps, h, 1)).sum(2) * ks[:, None, :]
    width = pools * kpool
    full = torch.full((n, rps, max(width, s.shape[2])), -math.inf, device="cuda")
    full[:, :, :s.shape[2]] = s
    score = full[:, :, :width].view(n * rps, pools, kpool).amax(2)
    last = (torch.arange(pools, device="cuda") + 1) * kpool - 1
    return torch.where(last[None, :] <= st["q_pos"][:, None], score, -math.inf)


def _own_full(st):
    from sparse_mla_paged_gb300 import api

    c = st["case"]
    if "workspace" not in st:  # kept from call to call, as a serving loop does
        st["workspace"] = api.alloc_full_workspace(c["seqs"], c["rps"], c["heads"])
    return api.decode_full(st["q"], st["cache"], st["cache"], st["tables"], st["blocks"], st["lens"], c["seqs"], c["rps"],
                           c["heads"], c["bs"], c["bs"] * LATENT, st["k_scale"], st["v_scale"], st["sm_scale"],
                           verify_rows=int(c["verify"]), workspace=st["workspace"])


def _plain_full(st):
    c = st["case"]
    n, rps, h, bs = c["seqs"], c["rps"], c["heads"], c["bs"]
    kv = st["cache"].view(-1, bs, LATENT)[st["tables"].long()].view(torch.float8_e4m3fn).float().view(n, -1, LATENT)
    lens = st["lens"].view(n, -1)
    if c["verify"]:
        lens = lens + 1 + torch.arange(rps, device="cuda")
    seen = torch.arange(kv.shape[1], device="cuda") < lens.view(n, rps, 1, 1)
    x = torch.matmul(st["q"].float().view(n, rps * h, LATENT), kv.transpose(1, 2)).view(n, rps, h, -1)
    x = torch.where(seen, x * (st["sm_scale"] * st["k_scale"]), -math.inf)
    top = x.amax(3, keepdim=True)
    p = torch.where(seen, torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
    p = p / p.sum(3, keepdim=True).clamp(min=1e-30)
    out = torch.matmul(p.view(n, rps * h, -1), kv) * st["v_scale"]
    return out.view(n * rps, h, LATENT).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op, bs = case["op"], case["bs"]
    if op == "plan":
        n = case["seqs"]
        base, new = _lens(case), _spread(n, case["new_lo"], case["new_hi"], "new")
        fresh = sum(-(-(b + x) // bs) - -(-b // bs) for b, x in zip(base, new))
        old = sum(1 for b, x in zip(base, new) if x and b % bs)
        rows = n * case["rps"] if case["rps"] else sum(new) + 5
        return {"bytes": 8 * n + 8 * fresh + 4 * old + 20 * rows + 16, "flops": 0}
    if op == "write":
        return {"bytes": case["rows"] * (2 * INDEX + 8 + INDEX + 4) + 4 * INDEX, "flops": 12 * INDEX * case["rows"]}
    n, rps, h = case["seqs"], case["rps"], case["heads"]
    rows = _row_lens(case)
    table = sum(-(-max(r) // bs) for r in rows) * 4
    if op == "scores":
        kp = case["kpool"]
        seen = [[x // kp * kp for x in r] for r in rows]
        keys = sum(max(r) for r in seen)
        return {"bytes": keys * (INDEX + 4) + n * rps * (h * (2 * INDEX + 4) + 4 + 4 * _pools(case)) + table,
                "flops": sum(map(sum, seen)) * h * (2 * INDEX + 3)}
    return {"bytes": sum(max(r) for r in rows) * LATENT + n * rps * h * LATENT * 4 + 4 * n * rps + table,
            "flops": 4 * LATENT * h * sum(map(sum, rows))}


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
    op = case["op"]
    if op == "plan":
        return None  # whole numbers only
    st = prepare(case, seed)
    return {"write": _exact_write, "scores": _exact_scores, "full": _exact_full}[op](st)


def _exact_write(st):
    c, bs = st["case"], st["case"]["bs"]
    x = st["x"].double()
    if c["norm"]:
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        x = (x - mean) * (var + 1e-6).rsqrt() * st["w"].double() + st["b"].double()
    top = x.abs().max(1).values.clamp(min=2.0 ** -100)
    grid = _e4m3_values()[:127]
    z = (x.abs() * (448.0 / top)[:, None]).clamp(max=448.0)
    mid = (grid[1:] + grid[:-1]) / 2
    near = grid[torch.bucketize(z, mid)] * torch.sign(x)
    pages = st["cache"].shape[0]
    codes = torch.zeros(pages * bs, INDEX, dtype=torch.float64, device="cuda")
    scales = torch.zeros(pages * bs, dtype=torch.float64, device="cuda")
    live = st["slots"] >= 0
    codes[st["slots"][live]] = near[live]
    scales[st["slots"][live]] = (top / 448.0)[live]
    return codes.view(pages, bs * INDEX), scales.view(pages, bs)


def _exact_scores(st):
    c = st["case"]
    rps, h, bs, kp, pools = c["rps"], c["heads"], c["bs"], c["kpool"], st["pools"]
    value = _e4m3_values()
    out = torch.full((c["seqs"] * rps, pools), -math.inf, dtype=torch.float64, device="cuda")
    pos = st["q_pos"].tolist()
    for s in range(c["seqs"]):
        rows = st["cache"][st["tables"][s].long()]
        k = value[rows[:, :bs * INDEX].reshape(-1, INDEX).int()]
        k = k * rows[:, bs * INDEX:bs * (INDEX + 4)].contiguous().view(torch.float32).reshape(-1, 1).double()
        for r in range(s * rps, (s + 1) * rps):
            m = (pos[r] + 1) // kp
            if m < 1:
                continue
            d = k[:m * kp] @ st["q"][r].double().t()
            token = torch.relu(d) @ st["w"][r].double()
            out[r, :m] = token.view(m, kp).max(1).values
    return out


def _exact_full(st):
    c = st["case"]
    rps, h, bs = c["rps"], c["heads"], c["bs"]
    value = _e4m3_values()
    lens = [x for r in _row_lens(c) for x in r]
    out = torch.zeros(c["seqs"] * rps, h, LATENT, dtype=torch.float64, device="cuda")
    for s in range(c["seqs"]):
        kv = value[st["cache"][st["tables"][s].long()].view(-1, LATENT).int()]
        for r in range(s * rps, (s + 1) * rps):
            if lens[r] < 1:
                continue
            own_kv = kv[:lens[r]]
            x = st["q"][r].double() @ own_kv.t() * (st["k_scale"] * st["sm_scale"])
            e = torch.exp(x - x.max(1, keepdim=True).values)
            out[r] = (e @ own_kv) * st["v_scale"] / e.sum(1, keepdim=True)
    return out
