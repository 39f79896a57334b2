"""Plain float64 forms of the step plan, the index-key writer, the pool scores and the
full-cache decode, on numpy arrays (test infrastructure; no library code)."""
import math

import numpy as np
import torch

LATENT, INDEX = 512, 128
DEVICE_BOUNDS = 6


def e4m3_table() -> np.ndarray:
    """The 256 values of OCP E4M3: bias 7, subnormals m/8 * 2^-6, 0x7F and 0xFF NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if c & 127 == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if c & 128 else x
    return v


E4M3 = e4m3_table()


def bf16(a) -> torch.Tensor:
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def plan(base, new, free, bs, tables, rps, rows):
    """Token by token; returns slots, positions, row_lens, row_seqs, info and the new tables."""
    n, width = tables.shape
    tables = tables.copy()
    slots, pos = np.full(rows, -1, np.int64), np.full(rows, -1, np.int32)
    lens, seqs = np.zeros(rows, np.int32), np.full(rows, -1, np.int32)
    bad, taken, tokens = False, 0, 0
    for s in range(n):
        b, k = max(0, int(base[s])), max(0, int(new[s]))
        bad |= base[s] < 0 or new[s] < 0
        if rps and k > rps:
            bad, k = True, rps
        have, want = -(-b // bs), -(-(b + k) // bs)
        bad |= want > width
        for blk in range(min(have, width), min(want, width)):
            if taken < len(free):
                tables[s, blk] = free[taken]
            else:
                tables[s, blk] = -1
                bad = True
            taken += 1
        for i in range(k):
            row = s * rps + i if rps else tokens
            tokens += 1
            if row >= rows:
                bad = True
                continue
            blk = (b + i) // bs
            if blk >= width:
                continue
            page = int(tables[s, blk])
            bad |= page < 0
            slots[row] = page * bs + (b + i) % bs if page >= 0 else -1
            pos[row], lens[row], seqs[row] = b + i, b + i + 1, s
    info = np.array([tokens if rps else min(tokens, rows), min(taken, len(free)), DEVICE_BOUNDS if bad else 0, 0], np.int32)
    return slots, pos, lens, seqs, info, tables


def index_keys(x, w, b, eps):
    """(y / s before rounding, s) of each row."""
    y = np.asarray(x, dtype=np.float64)
    if w is not None:
        y = y - y.mean(1, keepdims=True)
        y = y / np.sqrt((y * y).mean(1, keepdims=True) + eps) * w + (0 if b is None else b)
    s = np.maximum(np.abs(y).max(1), 2.0 ** -100) / 448
    return y / s[:, None], s


def index_page(cache, page, bs, stride):
    """Codes [bs, 128] and scales [bs] of one page of an index cache (flat uint8 array)."""
    at = page * stride
    codes = cache[at:at + bs * INDEX].reshape(bs, INDEX)
    return codes, cache[at + bs * INDEX:at + bs * (INDEX + 4)].view(np.float32)


def pool_scores(q, w, cache, tables, q_pos, rps, bs, stride, kpool, n_pools):
    """(scores, bound): the float64 scores and, for every visible pool, how far a float32 result
    formed from two-term E4M3 queries may be off.

    Query split: an element at least 2^-9 of its head's largest is exact, a smaller one off by at
    most half the last E4M3 step, 2^-10 where the largest is at least 2^7: 2^-17 of it. Sums:
    256 products and then H terms in float32, each addition off by at most 2^-23 of the
    magnitudes summed so far (round toward zero allowed)."""
    R, H, _ = q.shape
    out, tol = np.full((R, n_pools), -math.inf), np.zeros((R, n_pools))
    for r in range(R):
        m = min(n_pools, max(0, int(q_pos[r]) + 1) // kpool)
        if m == 0:
            continue
        row = tables[r // rps if tables.shape[0] > 1 else 0]
        pages = [index_page(cache, int(row[i]), bs, stride) for i in range(-(-m * kpool // bs))]
        k = E4M3[np.concatenate([p[0] for p in pages])][:m * kpool]
        s = np.concatenate([p[1] for p in pages])[:m * kpool].astype(np.float64)
        with np.errstate(invalid="ignore"):
            d = k @ q[r].T
            i = s * (np.maximum(d, 0) @ w[r])
        out[r, :m] = i.reshape(m, kpool).max(1)
        mag = np.abs(k) @ np.abs(q[r]).T
        split = 2.0 ** -17 * np.abs(k).sum(1)[:, None] * np.abs(q[r]).max(1)[None, :]
        e = np.abs(s) * ((split + (256 + H + 4) * 2.0 ** -23 * mag) @ np.abs(w[r]))
        tol[r, :m] = e.reshape(m, kpool).max(1)
    return out, tol


def full(q, k_cache, v_cache, tables, lens, rps, bs, stride, k_scale, v_scale, sm_scale):
    """float64 attention of each row over its first lens[r] positions; caches flat uint8."""
    R, H, _ = q.shape
    out = np.zeros((R, H, LATENT))
    for r in range(R):
        n = int(lens[r])
        if n <= 0:
            continue
        j = np.arange(n)
        page = tables[r // rps if tables.shape[0] > 1 else 0][j // bs].astype(np.int64)
        at = (page * stride + (j % bs) * LATENT)[:, None] + np.arange(LATENT)
        k, v = E4M3[k_cache[at]], E4M3[v_cache[at]]
        x = (q[r] @ k.T) * (sm_scale * k_scale)
        p = np.exp(x - x.max(1, keepdims=True))
        out[r] = (p / p.sum(1, keepdims=True)) @ v * v_scale
    return out
