"""Page by page forms of the page operators on numpy arrays (test infrastructure; no library code)."""
import numpy as np

BOUNDS = 6


def _len(n, table, bs):
    """A length cut to the table, and whether it had to be."""
    room = table.shape[1] * bs
    return min(max(int(n), 0), room), n < 0 or n > room


def copy(pools, src, dst):
    """pools: arrays [layers, pages, bytes]; returns new ones."""
    out = [p.copy() for p in pools]
    pages = pools[0].shape[1]
    for a, b in zip(src, dst):
        if 0 <= a < pages and 0 <= b < pages:
            for p, o in zip(pools, out):
                o[:, b] = p[:, a]
    return out


def fork(pools, parents, children, lens, bs, tables, free, shares):
    tables, shares = tables.copy(), shares.copy()
    n, pages = len(lens), len(shares)
    named = [(int(a), int(c)) for a, c in zip(parents, children) if 0 <= a < n and 0 <= c < n]
    everyone, seen = {a for a, _ in named}, set()
    bad, made, wanted, src, dst = False, 0, 0, [], []
    for a, c in zip(parents, children):
        if a < 0 or c < 0:
            continue
        if a >= n or c >= n:
            bad = True
            continue
        first, _ = c not in seen, seen.add(int(c))
        if not first or c in everyone:
            bad = True
            continue
        made += 1
        m, cut = _len(lens[a], tables, bs)
        bad |= cut
        for k in range(m // bs):
            page = tables[a, k]
            good = 0 <= page < pages
            bad |= not good
            tables[c, k] = page if good else -1
            if good:
                shares[page] += 1
        if m % bs:
            page = tables[a, m // bs]
            if not 0 <= page < pages:
                tables[c, m // bs] = -1
                bad = True
                continue
            fresh = int(free[wanted]) if wanted < len(free) else -1
            wanted += 1
            if not 0 <= fresh < pages:
                fresh, bad = -1, True
            tables[c, m // bs] = fresh
            src.append(page)
            dst.append(fresh)
    info = [made, min(wanted, len(free)), BOUNDS if bad else 0, 0]
    return copy(pools, src, dst), tables, shares, np.array(info, np.int32)


def release(tables, lens, keeps, bs, shares, free, num_free, taken):
    tables, shares, free = tables.copy(), shares.copy(), free.copy()
    pages, bad, refs, left = len(shares), False, 0, {}
    for s in range(len(lens)):
        n, cut = _len(lens[s], tables, bs)
        bad |= cut or keeps[s] < 0
        for k in range(-(-min(max(int(keeps[s]), 0), n) // bs), -(-n // bs)):
            page = int(tables[s, k])
            tables[s, k] = -1
            if page >= pages:
                bad = True
            elif page >= 0:
                refs += 1
                left[page] = left.get(page, 0) + 1
    freed = []
    for page in sorted(left):
        more = left[page] - int(shares[page])
        bad |= more > 1
        if more > 0:
            freed.append(page)
        shares[page] = 0 if more > 0 else -more
    count = min(max(int(num_free), 0), pages)
    t = min(max(int(taken), 0), count)
    bad |= count != num_free or t != taken
    rest = [int(x) for x in free[t:count]]
    gap = t - len(freed)
    if gap <= 0:
        new = freed[:t] + rest + freed[t:]
    else:
        last = rest[max(0, len(rest) - gap):]
        new = freed + last + rest[:len(rest) - len(last)]
        if len(last) < gap:
            assert not rest[:len(rest) - len(last)]
    bad |= len(new) > pages
    new = new[:pages]
    free[:len(new)] = new
    free[len(new):max(count, len(new))] = -1
    return tables, shares, free, len(new), np.array([refs, len(freed), BOUNDS if bad else 0, len(new)], np.int32)


def compact(pools, tables, lens, bs, shares):
    tables, shares = tables.copy(), shares.copy()
    pages, bad, live = len(shares), False, set()
    spans = []
    for s in range(len(lens)):
        n, cut = _len(lens[s], tables, bs)
        bad |= cut
        spans.append(-(-n // bs))
        for page in tables[s, :spans[-1]]:
            bad |= page >= pages
            if 0 <= page < pages:
                live.add(int(page))
    n = len(live)
    src = sorted(p for p in live if p >= n)
    dst = [p for p in range(n) if p not in live]
    to = dict(zip(src, dst))
    old = shares.copy()
    shares[n:] = 0
    for a, b in to.items():
        shares[b] = old[a]
    for s, span in enumerate(spans):
        tables[s, :span] = [to.get(int(p), p) for p in tables[s, :span]]
    free = np.full(pages, -1, np.int32)
    free[:pages - n] = np.arange(n, pages)
    return copy(pools, src, dst), tables, shares, free, pages - n, np.array([n, len(src), BOUNDS if bad else 0, pages - n], np.int32)
