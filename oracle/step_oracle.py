"""fp64 CPU oracle of the operators around a verify step: acceptance of
drafted tokens, and the pages of a paged cache.

TEST INFRASTRUCTURE ONLY, like ``verify_oracle``; it shares no code with the
library.  Plain definitions, one sequence and one step at a time.
"""
from __future__ import annotations

import numpy as np

PAGE = 16


# ---------------------------------------------------------------------------
# Acceptance.

def target(row, temperature: float):
    """The target's distribution for the token after a row, or None where
    the row has none (NaN, +inf, or nothing but -inf)."""
    z = np.asarray(row, np.float64)
    if np.isnan(z).any() or z.max() == np.inf or z.max() == -np.inf:
        return None
    if temperature == 0.0:
        p = np.zeros(len(z))
        p[int(np.argmax(z))] = 1.0  # numpy: the lowest index of the maximum
        return p
    with np.errstate(over="ignore"):
        w = np.exp((z - z.max()) / np.float64(np.float32(temperature)))
    return w / w.sum()


def accept_decisions(logits, probs, tokens, parent, u, v, temperature: float):
    """One sequence: rows of logits [n][V], drafted probabilities by parent
    row (or None), tokens, parents (parent[0] = -1), numbers u [n] and v.
    Returns (path, next token or -1, tests, draw): tests holds for each child
    that was tried its relative distance |u g - r| / max(u g, r) from the
    border, how many of its siblings were rejected before it, and the share of
    p's mass that they left; draw is the distance of v from the nearest border
    of the running sums (inf where nothing was drawn) and the share of p's mass
    that they run over."""
    n = len(tokens)
    node, path, tests = 0, [0], []
    while True:
        p = target(logits[node], temperature)
        if p is None:
            return path, -1, tests, (np.inf, 1.0)
        r = p.copy()
        taken, before, left = None, 0, 1.0
        for j in range(1, n):
            if parent[j] != node:
                continue
            x = int(tokens[j])
            if temperature == 0.0:
                if r[x] > 0:
                    taken = j
                    break
                continue
            g = np.zeros(len(p)) if probs is None else np.clip(np.nan_to_num(
                np.asarray(probs[node], np.float64)), 0.0, 1.0)
            if probs is None:
                g[x] = 1.0
            proposed, wanted = float(u[j]) * g[x], r[x]
            if max(proposed, wanted) > 0:
                tests.append((abs(proposed - wanted) / max(proposed, wanted), before, left))
            if proposed < wanted:
                taken = j
                break
            if probs is None:
                r[x] = 0.0
            else:
                r = np.maximum(r - g, 0.0)
            before, left = before + 1, left * r.sum()
            if r.sum() > 0:
                r = r / r.sum()
            else:
                r, left = p.copy(), 1.0
        if taken is None:
            break
        node = taken
        path.append(taken)
    c = np.cumsum(r)
    border = float(v) * c[-1]
    token = int(np.argmax(c > border))
    return path, token, tests, (float(np.abs(c - border).min()) if temperature else np.inf, left)


def accept_sequence(logits, probs, tokens, parent, u, v, temperature: float):
    """(path, next token or -1, margin): margin is the smallest relative
    distance of any decision from its border, so that a caller can tell a
    close call from a wrong one."""
    path, token, tests, draw = accept_decisions(logits, probs, tokens, parent, u, v, temperature)
    return path, token, min([draw[0]] + [t[0] for t in tests])


def accept(logits, probs, tokens, parent, kinds, cu_rows, u, v, temperature):
    """A launch: (accepted_len, accepted_nodes, promote_len, next_token,
    smallest margin)."""
    seqs, total = len(cu_rows) - 1, int(cu_rows[-1])
    length, token, promote = (np.zeros(seqs, np.int32) for _ in range(3))
    nodes = np.full(total, -1, np.int32)
    margins = np.full(seqs, np.inf)
    for s in range(seqs):
        a, b = int(cu_rows[s]), int(cu_rows[s + 1])
        if a == b:
            token[s] = -1
            continue
        par = [int(x) for x in parent[a:b]] if kinds[s] else list(range(-1, b - a - 1))
        path, token[s], margins[s] = accept_sequence(
            logits[a:b], None if probs is None else probs[a:b], tokens[a:b], par, u[a:b], v[s],
            float(temperature[s]))
        length[s] = len(path)
        promote[s] = len(path) if kinds[s] else 0
        nodes[a:a + len(path)] = path
    return length, nodes, promote, token, margins


# ---------------------------------------------------------------------------
# Pages.

def _in_use(ref, e):
    return 0 <= e < len(ref) and ref[e] > 0


def pages_fork(table, ref, src, dst, length, pages):
    """(table', ref', copies, reasons); any reason leaves both unchanged."""
    t, r = np.array(table), np.array(ref)
    seqs, width = t.shape
    bad = set()
    if (r < 0).any():
        bad.add("block")
    fresh = []  # (command, entry), in order
    for i, (a, b, n, m) in enumerate(zip(src, dst, length, pages)):
        if not (0 <= a < seqs and 0 <= b < seqs):
            bad.add("rows")
            continue
        if n < 0 or m < 0 or m > width or n > m * PAGE:
            bad.add("overflow")
            continue
        full, keep = n // PAGE, -(-n // PAGE)
        for c in range(m if a == b else keep):
            if t[a, c] != -1 and not _in_use(r, t[a, c]):
                bad.add("block")
        if a != b and keep > full and t[a, full] < 0:
            bad.add("block")
        if list(dst).count(b) > 1 or (a != b and a in list(dst)):
            bad.add("rows")
        fresh += [(i, c) for c in range(width)
                  if (keep <= c < m and t[a, c] < 0 if a == b else full <= c < m)]
    free = [b for b in range(len(r)) if r[b] == 0]
    if not bad and len(free) < len(fresh):
        bad.add("pages")
    if bad:
        return np.array(table), np.array(ref), [], bad
    place = dict(zip(fresh, free))
    copies = []
    for i, (a, b, n, m) in enumerate(zip(src, dst, length, pages)):
        full, keep = n // PAGE, -(-n // PAGE)
        row = []
        for c in range(width):
            if (i, c) in place:
                page = place[i, c]
                r[page] = 1
                if a != b and c == full and keep > full:
                    copies.append((int(table[a][c]), page))
            elif a == b:
                page = table[a][c]
            else:
                page = table[a][c] if c < full else -1
                if page >= 0:
                    r[page] += 1
            row.append(page)
        t[b] = row
    return t, r, copies, bad


def pages_free(table, ref, seq, first, last):
    t, r = np.array(table), np.array(ref)
    bad = set()
    for s, a, b in zip(seq, first, last):
        if not 0 <= s < t.shape[0]:
            bad.add("rows")
        elif not 0 <= a <= b <= t.shape[1]:
            bad.add("overflow")
        elif any(e != -1 and not _in_use(r, e) for e in t[s, a:b]):
            bad.add("block")
    if bad:
        return np.array(table), np.array(ref), bad
    for s, a, b in zip(seq, first, last):
        for c in range(a, b):
            if t[s, c] >= 0:
                r[t[s, c]] -= 1
                t[s, c] = -1
    return t, r, bad


def pages_compact(table, ref):
    t, r = np.array(table), np.array(ref)
    if (r < 0).any() or any(e != -1 and not _in_use(r, e) for e in t.reshape(-1)):
        return t, r, [], 0, {"block"}
    live = int((r > 0).sum())
    holes = [b for b in range(live) if r[b] == 0]
    moved = [b for b in range(live, len(r)) if r[b] > 0]
    to = dict(zip(moved, holes))
    for a, b in to.items():
        r[b], r[a] = r[a], 0
    t = np.vectorize(lambda e: to.get(int(e), int(e)))(t).astype(np.int32)
    return t, r, list(to.items()), live, set()


# ---------------------------------------------------------------------------
# Windowed verify attention.

def window_places(ctx: int, n: int, kind: int, parent_local):
    """Position of each draft row: ctx + j in a chain, ctx + depth in a tree."""
    depth = []
    for j in range(n):
        up = j - 1 if kind == 0 else int(parent_local[j])
        depth.append(0 if up < 0 else depth[up] + 1)
    return [ctx + d for d in depth]


def window_tokens(ctx: int, n: int, kind: int, parent_local, j: int, window: int, sinks: int) -> list:
    """Cache tokens (drafts as ctx + a) that row j sees."""
    place = window_places(ctx, n, kind, parent_local)
    path, a = [], j
    while a >= 0:
        path.append(a)
        a = a - 1 if kind == 0 else int(parent_local[a])
    seen = lambda pos: pos > place[j] - window or pos < sinks  # noqa: E731
    return [t for t in range(ctx) if seen(t)] + [ctx + a for a in sorted(path) if seen(place[a])]


def window_case(case, window: int, sinks: int):
    """O [rows, H, D] and LSE [rows, H] of a case object (see verify_case)."""
    from . import verify_oracle as vo
    H, KVH, D = case.num_heads, case.num_kv_heads, case.head_dim
    G, total = H // KVH, int(case.cu_rows[-1])
    scale = case.scale or 1.0 / np.sqrt(D)
    Q = vo.decode_q(np.asarray(case.q).reshape(total, H, -1), case.q_dtype)
    O, LSE = np.full((total, H, D), np.nan), np.full((total, H), np.nan)
    flat = {"k": case.k.reshape(-1, case.k.shape[-1]), "v": case.v.reshape(-1, case.v.shape[-1])}
    for s in range(len(case.ctx_len)):
        lo, hi, ctx = int(case.cu_rows[s]), int(case.cu_rows[s + 1]), int(case.ctx_len[s])
        kind = vo.seq_kind_of(s, case.seq_kind, case.mode)
        scratch = case.draft_k is not None and kind == 1
        for j in range(hi - lo):
            t = np.asarray(window_tokens(ctx, hi - lo, kind, case.parent[lo:hi], j, window, sinks), np.int64)
            for kvh in range(KVH):
                rows = {}
                for name, draft in (("k", case.draft_k), ("v", case.draft_v)):
                    cached = t[t < ctx] if scratch else t
                    got = flat[name][vo.gather_index(s, kvh, cached, page_size=case.page_size,
                                                     capacity=case.capacity, num_kv_heads=KVH,
                                                     block_table=case.block_table)]
                    if scratch:
                        got = np.concatenate([got, draft[lo + (t[t >= ctx] - ctx), kvh]])
                    rows[name] = vo.decode_rows(got, case.kv_dtype)
                for h in range(kvh * G, (kvh + 1) * G):
                    O[lo + j, h], LSE[lo + j, h], _ = vo.attend(Q[lo + j, h], rows["k"], rows["v"], scale)
    return O, LSE


def seen_tokens(case, window: int, sinks: int):
    """Per sequence, the set of cache tokens that some row sees."""
    from . import verify_oracle as vo
    out = []
    for s in range(len(case.ctx_len)):
        lo, hi, ctx = int(case.cu_rows[s]), int(case.cu_rows[s + 1]), int(case.ctx_len[s])
        kind = vo.seq_kind_of(s, case.seq_kind, case.mode)
        seen = set()
        for j in range(hi - lo):
            seen |= set(window_tokens(ctx, hi - lo, kind, case.parent[lo:hi], j, window, sinks))
        out.append(seen)
    return out
