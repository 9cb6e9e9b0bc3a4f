"""fp64 definitions of the operators of a latent cache: block tables and slots
from request lengths, rows into the cache, attention over it in the absorbed
form, attention of prompt segments over expanded keys (test infrastructure)."""
from __future__ import annotations

import numpy as np

PAGE = 16

BAD_PARENT, BAD_BLOCK, CTX_OVERFLOW, BAD_ROWS, NO_PAGES = 0x1, 0x2, 0x4, 0x8, 0x100


def tree_depth(parent, j):
    d = 0
    while parent[j] >= 0:
        j, d = parent[j], d + 1
    return d


def extend(table, ref, ctx, rows, max_rows, kinds=None, parent=None):
    """Returns (table, ref, cu_rows, row_seq, position, slot, status bits); the
    inputs stay as they are."""
    table, ref = table.copy(), ref.copy()
    seqs, width = table.shape
    bad = 0
    if (ref < 0).any():
        bad |= BAD_BLOCK
    kinds = np.zeros(seqs, np.uint8) if kinds is None else kinds
    fresh = []
    for s in range(seqs):
        c, n = int(ctx[s]), int(rows[s])
        if n < 0 or (kinds[s] and n > 32):
            bad |= BAD_ROWS
        elif c < 0 or -(-(c + n) // PAGE) > width:
            bad |= CTX_OVERFLOW
        elif n:
            for e in range(c // PAGE, -(-(c + n) // PAGE)):
                page = table[s, e]
                if page == -1 and e * PAGE >= c:
                    fresh.append((s, e))
                elif not (0 <= page < ref.size and ref[page] == 1):
                    bad |= BAD_BLOCK
    total = int(np.maximum(rows, 0).sum())
    if not bad and total > max_rows:
        bad |= BAD_ROWS
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    if not bad:
        for s in range(seqs):
            for j in range(int(rows[s])):
                if kinds[s] and not -1 <= parent[cu[s] + j] < j:
                    bad |= BAD_PARENT
    free = np.flatnonzero(ref == 0)
    if not bad and len(free) < len(fresh):
        bad |= NO_PAGES
    row_seq = np.full(max_rows, -1, np.int32)
    position, slot = row_seq.copy(), np.full(max_rows, -1, np.int64)
    if bad:
        return table, ref, np.zeros(seqs + 1, np.int32), row_seq, position, slot, bad
    for (s, e), page in zip(fresh, free):
        table[s, e] = page
        ref[page] = 1
    for s in range(seqs):
        for j in range(int(rows[s])):
            r, t = cu[s] + j, int(ctx[s]) + j
            row_seq[r] = s
            depth = tree_depth(parent[cu[s]:cu[s + 1]], j) if kinds[s] else j
            position[r] = ctx[s] + depth
            slot[r] = int(table[s, t // PAGE]) * PAGE + t % PAGE
    return table, ref, cu, row_seq, position, slot, 0


def rotate(x, cos, sin, interleaved):
    """Pairs of the last dimension turned; cos, sin broadcast over pairs."""
    h = x.shape[-1] // 2
    out = np.empty_like(x)
    i, j = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, h), slice(h, None))
    out[..., i] = x[..., i] * cos - x[..., j] * sin
    out[..., j] = x[..., i] * sin + x[..., j] * cos
    return out


def append(cache, kv, position, slot, rope, weight=None, eps=1e-6, interleaved=False, q_rope=None, q=None):
    """cache [slots][latent + rope], q [rows][heads][latent + rope] or None; returns copies."""
    cache, q = cache.copy(), None if q is None else q.copy()
    d = rope.shape[1]
    latent = cache.shape[1] - d
    for r in range(len(position)):
        if not 0 <= position[r] < len(rope) or not -1 <= slot[r] < len(cache):
            continue
        cos, sin = rope[position[r], :d // 2], rope[position[r], d // 2:]
        if q is not None:
            q[r, :, latent:] = rotate(q_rope[r], cos, sin, interleaved)
        if slot[r] < 0:
            continue
        x = kv[r, :latent]
        if weight is not None:
            x = x / np.sqrt((x * x).mean() + eps) * weight
        cache[slot[r], :latent] = x
        cache[slot[r], latent:] = rotate(kv[r, latent:latent + d], cos, sin, interleaved)
    return cache, q


def attend(q, k, v, seen, scale):
    """q [rows][heads][dk], k [keys][heads or 1][dk], v [keys][heads or 1][dv],
    seen [rows][keys].  Returns o, lse, and the sums of p |v| (what roundings of
    p may move); a row that sees nothing has o 0 and lse -inf."""
    n, heads = q.shape[:2]
    o = np.zeros((n, heads, v.shape[2]))
    a, lse = o.copy(), np.full((n, heads), -np.inf)
    for h in range(heads):
        kh, vh = (x[:, h if x.shape[1] > 1 else 0] for x in (k, v))
        z = np.where(seen, q[:, h] @ kh.T * scale, -np.inf)
        some = seen.any(1)
        if not some.any():
            continue
        z = z[some]
        m = z.max(1, keepdims=True)
        w = np.exp(z - m)
        total = w.sum(1, keepdims=True)
        o[some, h], a[some, h] = (w / total) @ vh, (w / total) @ np.abs(vh)
        lse[some, h] = (m + np.log(total))[:, 0]
    return o, lse, a


def visible(n, ctx, kind, parent):
    """[n][ctx + n]: which tokens a sequence's rows see."""
    seen = np.zeros((n, ctx + n), bool)
    seen[:, :ctx] = True
    for j in range(n):
        up = int(parent[j]) if kind else j - 1
        if up >= 0:
            seen[j] = seen[up]
        seen[j, ctx + j] = True
    return seen


def latent(q, rows_of, cu, ctx, scale, latent_dim, kinds=None, parent=None):
    """Absorbed form: rows_of(s, count) gives the first count cache rows of
    sequence s.  Returns o, lse, sums of p |c|."""
    out = np.zeros((*q.shape[:2], latent_dim))
    mag, lse = out.copy(), np.zeros(q.shape[:2])
    for s in range(len(ctx)):
        a, b = int(cu[s]), int(cu[s + 1])
        k = rows_of(s, int(ctx[s]) + b - a)[:, None]
        kind = 0 if kinds is None else int(kinds[s])
        seen = visible(b - a, int(ctx[s]), kind, None if parent is None else parent[a:b])
        out[a:b], lse[a:b], mag[a:b] = attend(q[a:b], k, k[..., :latent_dim], seen, scale)
    return out, lse, mag


def prompt(q, kv, k_rope, cu, cu_kv, scale, nope, causal=True):
    """Expanded form; kv [keys][heads][nope + value].  Returns o, lse, sums of p |v|."""
    out = np.zeros((*q.shape[:2], kv.shape[2] - nope))
    mag, lse = out.copy(), np.full(q.shape[:2], -np.inf)
    for s in range(len(cu) - 1):
        a, b, x, y = int(cu[s]), int(cu[s + 1]), int(cu_kv[s]), int(cu_kv[s + 1])
        n, keys = b - a, y - x
        kr = np.broadcast_to(k_rope[x:y, None], (keys, kv.shape[1], k_rope.shape[1]))
        k = np.concatenate([kv[x:y, :, :nope], kr], 2)
        t, j = np.arange(keys)[None], np.arange(n)[:, None]
        seen = t <= keys - n + j if causal else np.ones((n, keys), bool)
        out[a:b], lse[a:b], mag[a:b] = attend(q[a:b], k, kv[x:y, :, nope:], seen, scale)
    return out, lse, mag
