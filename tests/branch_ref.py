"""Drafted trees and branching sequences in plain Python and 64-bit numpy (test infrastructure)."""
import numpy as np

from .parity import bf16_to_f64


def parents_of(r, n, chain=False, roots=False):
    """A tree of n nodes, parents before children; several roots if asked."""
    up = [-1]
    for i in range(1, n):
        up.append(i - 1 if chain else -1 if roots and r.random() < 0.2 else int(r.integers(max(0, (i - 1) // 4), i)))
    return up[:n]


def masks_of(parents):
    """Masks as Python integers."""
    rows = []
    for i, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else 0) | 1 << i)
    return rows


def words_of(masks, words):
    return np.array([[m >> 32 * w & 0xffffffff for w in range(words)] for m in masks], np.uint32).reshape(-1, words)


def tree_attention(cache, q, starts, masks, words, scale, softcap=0.0, window=0, slopes=None, sinks=None):
    """As paged_ref.attention, for masks (Python integers) [tokens]."""
    tokens, heads, d = q.shape
    qf = bf16_to_f64(q).reshape(q.shape)
    group = heads // cache.kv_heads
    out, spread = np.zeros((tokens, heads, d)), np.zeros((tokens, heads, d))
    lse = np.full((tokens, heads), -np.inf)
    slack = np.zeros((tokens, heads))
    if sinks is not None:
        lse[:] = sinks
    for b in range(len(cache.lens)):
        full, first, last = int(cache.lens[b]), int(starts[b]), int(starts[b + 1])
        n = last - first
        if n <= 0 or full == 0:
            continue
        past = full - n
        k, v, ok = cache.rows(b)
        most = min(n, 32 * words)
        sees = np.array([[m >> i & 1 for i in range(most)] + [0] * (n - most) for m in masks[first:last]], bool)
        depth = np.maximum(sees.sum(1) - 1, 0)
        place = np.array([t if t < past else past + depth[t - past] for t in range(full)])
        far = place[None, :] - (past + depth)[:, None]
        t = np.arange(full)
        see = np.where(t < past, True, sees[:, np.clip(t - past, 0, n - 1)]) & ok
        see &= (past + np.arange(n) >= 0)[:, None]
        if window:
            see &= -far < window
        for h in range(heads):
            kk, vv = k[h // group], v[h // group]
            rows = qf[first:last, h]
            z = scale * (rows @ kk.T)
            err = 2 * d * 2.0 ** -24 * abs(scale) * (np.abs(rows) @ np.abs(kk).T)
            if softcap:
                z = softcap * np.tanh(z / softcap)
                err = np.minimum(err, 2 * softcap) + softcap * 2.0 ** -21
            if slopes is not None:
                z = z + float(slopes[h]) * far
                err = err + np.abs(z) * 2.0 ** -23
            z = np.where(see, z, -np.inf)
            top = z.max(1, initial=-np.inf)
            if sinks is not None:
                top = np.maximum(top, float(sinks[h]))
            top = np.where(np.isfinite(top), top, 0.0)
            w = np.exp(z - top[:, None])
            total = w.sum(1)
            if sinks is not None:
                total = total + np.exp(float(sinks[h]) - top)
            w = w / np.where(total > 0, total, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                lse[first:last, h] = np.log(total) + top
            out[first:last, h] = w @ vv
            spread[first:last, h] = w @ np.abs(vv)
            slack[first:last, h] = np.where(see, err, 0.0).max(1, initial=0.0)
    return out, lse, spread, slack


def accept(parents, drafts, chosen, starts, width):
    """(path, counts, next) of every sequence."""
    path, counts, nxt = [], [], []
    for b in range(len(starts) - 1):
        s, n = starts[b], starts[b + 1] - starts[b]
        way = [0] if n else []
        while way and len(way) < width:
            below = [c for c in range(way[-1] + 1, n)
                     if parents[s + c] == way[-1] and drafts[s + c] == chosen[s + way[-1]]]
            if not below:
                break
            way.append(below[0])
        path.append(way + [-1] * (width - len(way)))
        counts.append(len(way))
        nxt.append(int(chosen[s + way[-1]]) if way else -1)
    return path, counts, nxt


def lowest_free(table, pages, held=()):
    used = {int(p) for row in table for p in row if 0 <= p < pages} | set(held)
    return [p for p in range(pages) if p not in used]


def resize(table, lens, want, pages, page, held=()):
    """(table, lens, left)."""
    table = [list(map(int, row)) for row in table]
    out, holes = [], []
    for b, (row, n, w) in enumerate(zip(table, lens, want)):
        out.append(int(n) if w < 0 else min(int(n), int(w)))
        if w < 0:
            continue
        need = -(-int(w) // page)
        row[need:] = [-1] * (len(row) - len(row[:need]))
        holes += [(b, e) for e in range(-(-int(n) // page), need) if row[e] < 0 or row[e] >= pages]
    for b, e in holes:
        table[b][e] = -1
    free = lowest_free(table, pages, held)
    for (b, e), p in zip(holes, free):
        table[b][e] = p
    return table, out, len(free) - len(holes)


def fork(table, lens, come, pages, page, held=()):
    """(table, lens, left, copies [(from page, to page, rows)])."""
    old = [list(map(int, row)) for row in table]
    new, out, copies, owner = [], [], [], {b: b for b, a in enumerate(come) if a == b}
    for b, a in enumerate(come):
        n = int(lens[a]) if a >= 0 else 0
        row = [-1] * len(old[0]) if a < 0 else list(old[a])
        if a >= 0 and a != b:
            row[-(-n // page):] = [-1] * (len(row) - -(-n // page))
            if n % page and owner.setdefault(a, b) != b and 0 <= row[n // page] < pages:
                copies.append((b, n // page, row[n // page], n % page))
                row[n // page] = -1
        new.append(row)
        out.append(n)
    free = lowest_free(new, pages, held)
    done = []
    for (b, e, p, rows), to in zip(copies, free):
        new[b][e] = to
        done.append((p, to, rows))
    return new, out, len(free) - len(copies), done


def compact(table, pages, held=()):
    """(table, span, copies [(from page, to page)])."""
    used = sorted({int(p) for row in table for p in row if 0 <= p < pages} - set(held))
    slots = [p for p in range(pages) if p not in set(held)][:len(used)]
    goes, holes = [p for p in used if p not in set(slots)], [p for p in slots if p not in set(used)]
    to = dict(zip(goes, holes))
    return [[to.get(int(p), int(p)) for p in row] for row in table], slots[-1] + 1 if slots else 0, list(to.items())
