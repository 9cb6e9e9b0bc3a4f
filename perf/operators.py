"""Measured cases of the operators around a verify step: windowed verify attention over the
cache, acceptance of drafted tokens, and the pages of a paged cache (fork, free, compact, copy).

Each case runs ONE call of an operator as a serving loop makes it.  ``run`` computes it either in
plain torch operations (``own`` false) or through the library (``own`` true); ``exact`` restates the
definition in 64 bits with numpy.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
ROW_BYTES = {"f32": 4.0, "bf16": 2.0, "q8_0": 34.0 / 32.0}  # bytes of one cache element
CODE = {"f32": 0, "bf16": 1, "q8_0": 2}
MODE = {"chain": 0, "tree": 1, "mixed": 2}


# ------------------------------------------------------------------------------------------ cases

def _window(name, kv, heads, kv_heads, dim, mode, seqs, rows, ragged, ctx, spread, window, sinks, paged,
            evicted, out, splits):
    return {"name": name, "op": "window", "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "mode": mode, "seqs": seqs, "rows": rows, "ragged": ragged, "ctx": ctx, "spread": spread,
            "window": window, "sinks": sinks, "paged": paged, "evicted": evicted, "out": out,
            "splits": splits}


def _accept(name, mode, seqs, rows, ragged, vocab, pad, logits, probs, temperature):
    return {"name": name, "op": "accept", "mode": mode, "seqs": seqs, "rows": rows, "ragged": ragged,
            "vocab": vocab, "pad": pad, "logits": logits, "probs": probs, "temperature": temperature}


def _fork(name, seqs, forks, ctx, spread, slack, pool, pools, page_bytes):
    return {"name": name, "op": "fork", "seqs": seqs, "forks": forks, "ctx": ctx, "spread": spread,
            "slack": slack, "pool": pool, "pools": pools, "page_bytes": page_bytes}


def _compact(name, seqs, pages, pool, pools, page_bytes):
    return {"name": name, "op": "compact", "seqs": seqs, "pages": pages, "pool": pool, "pools": pools,
            "page_bytes": page_bytes}


def _splits(seqs, kv_heads, tokens):
    """Chunks a caller asks for: enough CTAs to fill the GPU once, at least 256 tokens each."""
    return max(1, min(152 // max(1, seqs * kv_heads), (tokens + 255) // 256, 16))


def listed():
    return [
        # One direct (one-row) step of one request: the smallest serving call.
        _window("window one token", "bf16", 32, 8, 128, "chain", 1, 1, False, 8192, 0, 1024, 4, True,
                True, "bf16", _splits(1, 8, 1028)),
        # A full batch of direct rows; pages behind the window were given back.
        _window("window batch of one token", "bf16", 32, 8, 128, "chain", 64, 1, False, 28000, 2000,
                4096, 4, True, True, "f32", 1),
        # A 16-row verify of a Q8_0 cache, paged, the width of the framework's headline call.
        _window("window chain q8", "q8_0", 24, 4, 256, "chain", 6, 16, False, 20676, 8000, 4096, 16, True,
                True, "bf16", _splits(6, 4, 4112)),
        # Width-8 trees and direct rows of ragged contexts, some shorter than the window.
        _window("window trees ragged", "bf16", 24, 4, 256, "mixed", 9, 8, True, 333, 4001, 1500, 33, False,
                False, "f32", _splits(9, 4, 1533)),
        # The fp32 chain of the smallest shape, a prompt segment inside its own window.
        _window("window segment f32", "f32", 4, 1, 64, "chain", 2, 200, True, 256, 77, 100, 1, False,
                False, "f32", 4),
        # Greedy acceptance of a short chain.
        _accept("accept greedy chain", "chain", 1, 4, False, 32768, 0, "bf16", False, 0.0),
        # Width-8 trees of top-ranked tokens and direct rows, sampled.
        _accept("accept trees", "mixed", 8, 8, False, 131072, 0, "bf16", False, 0.8),
        # A batch of 16-row chains drawn from a drafter's probabilities.
        _accept("accept chains drawn", "chain", 32, 16, False, 131072, 0, "bf16", True, 1.0),
        # Wide trees whose children share a drafter's distribution; odd vocabulary, odd strides.
        _accept("accept trees drawn odd", "tree", 5, 32, True, 100003, 5, "f32", True, 0.7),
        # A request forked into a few continuations: one partial page each.
        _fork("fork few", 16, 3, 1016, 40, 2, 2048, 2, 17408),
        # A whole batch forked, every layer's tail pages copied.
        _fork("fork batch", 128, 60, 4097, 4000, 2, 32768, 32, 32768),
        # A fragmented pool pulled together.
        _compact("compact", 96, 100, 16384, 8, 17408),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 5e13)


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        c = _draw(rng)
        if _cost(c) <= top[c["op"]]:
            return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["window", "window", "accept", "accept", "fork", "compact"])
    if op == "window":
        kv = rng.choice(["bf16", "bf16", "q8_0", "q8_0", "f32"])
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 8])
        mode = rng.choice(["chain", "chain", "tree", "mixed"])
        small = kv == "f32"
        rows = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 200 if small else 400)]) if mode == "chain" \
            else _log(rng, 2, 32)
        seqs = _log(rng, 1, 4 if small else 64)
        window = _log(rng, 1, 600 if small else 8192)
        sinks = rng.choice([0, 1, 4, 16, rng.randint(1, 200)])
        paged = rng.random() < 0.6
        ctx = _log(rng, 1, 1000 if small else 12000) - 1
        spread = _log(rng, 1, 400 if small else 3000) - 1
        splits = max(_splits(seqs, kv_heads, window + sinks), rng.choice([1, 1, 3]))
        out = "f32" if kv == "f32" else "bf16" if kv == "q8_0" else rng.choice(["f32", "bf16"])
        c = _window("", kv, heads, kv_heads, dim, mode, seqs, rows, rng.random() < 0.5, ctx, spread, window,
                    sinks, paged, paged and rng.random() < 0.6, out, splits)
    elif op == "accept":
        mode = rng.choice(["chain", "tree", "mixed"])
        rows = _log(rng, 1, 64) if mode == "chain" else _log(rng, 1, 32)
        c = _accept("", mode, _log(rng, 1, 48), rows, rng.random() < 0.5,
                    rng.choice([_log(rng, 2, 3000), _log(rng, 1000, 200000)]), rng.choice([0, 0, 3, 64]),
                    rng.choice(["bf16", "f32"]), rng.random() < 0.6, rng.choice([0.0, 0.6, 1.0, 1.3]))
    elif op == "fork":
        seqs = _log(rng, 2, 256)
        ctx = _log(rng, 1, 4000) - 1
        spread = _log(rng, 1, 3000) - 1
        forks = rng.randint(1, max(1, seqs // 2))
        need = seqs * ((ctx + spread) // PAGE + 4)
        c = _fork("", seqs, forks, ctx, spread, rng.randint(0, 3), need + rng.randint(need // 2, 2 * need + 8),
                  rng.choice([2, 4, 8, 16, 24]), rng.choice([2048, 4352, 8704, 16384, 17408]))
    else:
        seqs = _log(rng, 1, 200)
        pages = _log(rng, 1, 120)
        pool = int(seqs * pages * rng.uniform(1.02, 3.0)) + 3
        c = _compact("", seqs, pages, pool, rng.choice([2, 4, 6, 8]), rng.choice([2048, 4352, 8704, 16384, 17408]))
    del c["name"]
    return c


# -------------------------------------------------------------------------- what a case's lengths are

def _rows_of(case):
    """Rows and kind (1: tree) of each sequence of a window or accept case."""
    n, kinds = [], []
    for i in range(case["seqs"]):
        tree = case["mode"] == "tree" or (case["mode"] == "mixed" and i % 4 != 0)
        r = 1 if case["mode"] == "mixed" and not tree else case["rows"]
        if case["ragged"] and i:
            r = 1 + (r * (7 * i + 3)) // 11 % r
        n.append(r)
        kinds.append(1 if tree else 0)
    return n, kinds


def _ctx_of(case):
    return [case["ctx"] + (977 * i) % (case["spread"] + 1) for i in range(case["seqs"])]


def _visible(ctx, n, window, sinks):
    """Cache tokens that some row of the sequence sees: [0, a) and [b, ctx + n)."""
    b = max(0, ctx - window + 1)
    return min(sinks, b), b


def work(case):
    if case["op"] == "window":
        rows, _ = _rows_of(case)
        tokens = pairs = 0
        for ctx, n in zip(_ctx_of(case), rows):
            a, b = _visible(ctx, n, case["window"], case["sinks"])
            tokens += a + ctx + n - b
            pairs += sum(a + min(case["window"], ctx + j + 1) for j in range(n))
        q = sum(rows) * case["heads"] * case["dim"]
        kv = 2 * tokens * case["kv_heads"] * case["dim"] * ROW_BYTES[case["kv"]]
        return {"bytes": kv + q * (4 if case["kv"] == "f32" else 2) + q * (4 if case["out"] == "f32" else 2)
                + sum(rows) * case["heads"] * 4, "flops": 4.0 * case["dim"] * case["heads"] * pairs}
    if case["op"] == "accept":
        # A row that can be left by one of its children has its logits read; a sequence's last row too,
        # and with drafted probabilities one row of those.  A tree keeps about half its rows as leaves.
        rows, kinds = _rows_of(case)
        read = sum((n // 2 if k else n - 1) + 1 for n, k in zip(rows, kinds))
        size = 2 if case["logits"] == "bf16" else 4
        b = read * case["vocab"] * size + (case["seqs"] * case["vocab"] * 4 if case["probs"] else 0)
        return {"bytes": float(b + 16 * sum(rows)), "flops": 4.0 * read * case["vocab"]}
    ints = 4.0 * (case["pool"] + case["seqs"] * _width(case))
    if case["op"] == "fork":
        tails = sum(1 for length in _fork_lengths(case) if length % PAGE)
        return {"bytes": 2 * ints + 2.0 * tails * case["pools"] * case["page_bytes"], "flops": 0.0}
    live = case["seqs"] * case["pages"]
    moved = live * (1 - live / case["pool"])  # the pool is filled at random
    return {"bytes": 2 * ints + 2.0 * moved * case["pools"] * case["page_bytes"], "flops": 0.0}


def _width(case):
    if case["op"] == "compact":
        return case["pages"] + 8
    return (case["ctx"] + case["spread"]) // PAGE + 1 + case["slack"] + 5


def _fork_lengths(case):
    ctx = [case["ctx"] + (977 * i) % (case["spread"] + 1) for i in range(case["seqs"])]
    return [ctx[i % (case["seqs"] - case["forks"])] for i in range(case["forks"])]


# ----------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _trees(case, seed):
    """cu_rows, parent and kinds: chains, and random trees with parent[j] < j."""
    rows, kinds = _rows_of(case)
    r = random.Random(int(seed) * 31 + 5)
    parent = []
    for n, k in zip(rows, kinds):
        parent += [(-1 if j == 0 else r.randrange(j)) if k else j - 1 for j in range(n)]
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return rows, kinds, cu, parent


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def prepare(case, seed):
    return {"window": _prepare_window, "accept": _prepare_accept, "fork": _prepare_pages,
            "compact": _prepare_pages}[case["op"]](case, seed)


def _cache(g, kind, shape, dim):
    """Cache rows of the given leading shape: normal values, or Q8_0 blocks (fp16 scale, 32 codes)."""
    if kind == "f32":
        return torch.randn(*shape, dim, generator=g, device="cuda")
    if kind == "bf16":
        return torch.randn(*shape, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    raw = torch.randint(0, 255, (*shape, dim // 32, 34), generator=g, device="cuda", dtype=torch.uint8)
    raw[..., 2:] = (raw[..., 2:].to(torch.int16) - 127).to(torch.int8).view(torch.uint8)
    scale = torch.empty((*shape, dim // 32, 1), device="cuda").uniform_(0.002, 0.02, generator=g)
    raw[..., :2] = scale.to(torch.float16).view(torch.uint8)
    return raw.reshape(*shape, dim // 32 * 34)


def _prepare_window(case, seed):
    g = _gen(seed)
    rows, kinds, cu, parent = _trees(case, seed)
    ctx = _ctx_of(case)
    kvh, dim, seqs = case["kv_heads"], case["dim"], case["seqs"]
    qd = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    q = torch.randn(cu[-1], case["heads"], dim, generator=g, device="cuda").to(qd)
    s = {"case": case, "rows": rows, "kinds": kinds, "ctx": ctx, "q": q, "cu": _int(cu), "ctx_len": _int(ctx),
         "parent": _int(parent), "kind": _int(kinds, torch.uint8), "table": None, "blocks": 0, "capacity": 0}
    if case["paged"]:
        need = [-(-(c + n) // PAGE) for c, n in zip(ctx, rows)]
        keep = []
        for c, n, pages in zip(ctx, rows, need):
            a, b = _visible(c, n, case["window"], case["sinks"])
            keep.append([p for p in range(pages)
                         if not case["evicted"] or p * PAGE < a or (p + 1) * PAGE > b])
        total = sum(len(k) for k in keep)
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(int(seed))).tolist()
        table = np.full((seqs, max(need)), -1, dtype=np.int32)
        at = 0
        for i, k in enumerate(keep):
            table[i, k] = perm[at:at + len(k)]
            at += len(k)
        s["table"], s["blocks"] = torch.from_numpy(table).cuda(), total
        shape = (total, kvh, PAGE)
    else:
        s["capacity"] = max(-(-(c + n) // PAGE) * PAGE for c, n in zip(ctx, rows))
        shape = (seqs, kvh, s["capacity"])
    s["k"], s["v"] = _cache(g, case["kv"], shape, dim), _cache(g, case["kv"], shape, dim)
    if own:
        import speculative_decoding_verify_kv_gb300 as va
        p = va.Problem(num_seqs=seqs, num_heads=case["heads"], q_dtype=va.F32 if case["kv"] == "f32" else va.BF16,
                       q=q, cu_rows=s["cu"], ctx_len=s["ctx_len"], parent=s["parent"], seq_kind=s["kind"],
                       total_rows=cu[-1], max_rows_per_seq=max(rows), num_splits=case["splits"])
        kv = va.KV(CODE[case["kv"]], kvh, dim, s["k"], s["v"], page_size=PAGE if case["paged"] else 0,
                   capacity=s["capacity"], block_table=s["table"],
                   max_blocks_per_seq=s["table"].shape[1] if case["paged"] else 0, num_blocks=s["blocks"])
        win = va.Window(case["window"], case["sinks"], CODE[case["out"]])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["call"] = va.WindowCall(p, kv, MODE[case["mode"]], win, status=s["status"])
    return s


def _prepare_accept(case, seed):
    g = _gen(seed)
    rows, kinds, cu, parent = _trees(case, seed)
    vocab, stride, total = case["vocab"], case["vocab"] + case["pad"], cu[-1]
    ld = torch.bfloat16 if case["logits"] == "bf16" else torch.float32
    logits = torch.empty(total, stride, device="cuda", dtype=ld).normal_(0.0, 2.5, generator=g)
    glob = [cu[i] + parent[cu[i] + j] if parent[cu[i] + j] >= 0 else cu[i]
            for i, n in enumerate(rows) for j in range(n)]
    up = _int(glob, torch.int64)  # each row's parent among all rows
    temp = case["temperature"] if case["temperature"] > 0 else 1.0
    tokens = torch.zeros(total, dtype=torch.int32, device="cuda")
    probs = None
    if case["probs"]:
        probs = torch.zeros(total, stride, device="cuda")
        for a in range(0, total, 64):  # the drafter's guess at the target: its logits, blurred
            x = logits[a:a + 64, :vocab].float()
            x = (x + torch.randn(x.shape, generator=g, device="cuda")) / temp
            probs[a:a + 64, :vocab] = torch.softmax(x, -1)
        for a in range(0, total, 64):  # a token drawn from its parent's distribution
            e = torch.empty(min(64, total - a), vocab, device="cuda").exponential_(generator=g)
            tokens[a:a + 64] = (probs[up[a:a + 64], :vocab] / e).argmax(-1).to(torch.int32)
    else:
        rank, seen = [], {}
        for p in glob:  # the k-th child of a row proposes the k-th ranked token
            rank.append(seen.get(p, 0))
            seen[p] = rank[-1] + 1
        rank = _int([min(r, vocab - 1) for r in rank], torch.int64)
        for a in range(0, total, 64):
            x = logits[up[a:a + 64], :vocab].float()
            x = x + 0.3 * torch.randn(x.shape, generator=g, device="cuda")
            top = x.topk(min(32, vocab), -1).indices
            tokens[a:a + 64] = top.gather(1, rank[a:a + 64, None].clamp(max=top.shape[1] - 1))[:, 0].to(torch.int32)
    s = {"case": case, "rows": rows, "cu": _int(cu), "parent": _int(parent), "kind": _int(kinds, torch.uint8),
         "logits": logits, "probs": probs, "tokens": tokens,
         "u": torch.rand(total, generator=g, device="cuda"), "v": torch.rand(case["seqs"], generator=g, device="cuda"),
         "temperature": torch.full((case["seqs"],), case["temperature"], device="cuda")}
    s["starts"], s["lens"] = _int(cu[:-1], torch.int64), _int(rows, torch.int64)
    if own:
        import speculative_decoding_verify_kv_gb300 as va
        p = va.Problem(num_seqs=case["seqs"], num_heads=1, q_dtype=va.BF16, q=None, cu_rows=s["cu"], ctx_len=None,
                       parent=s["parent"], seq_kind=s["kind"], total_rows=total, max_rows_per_seq=max(rows))
        d = va.Draft(logits=logits, vocab=vocab, logits_dtype=CODE[case["logits"]], logits_stride=stride,
                     draft_probs=probs, draft_stride=stride, tokens=tokens, accept_u=s["u"], sample_u=s["v"],
                     temperature=s["temperature"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["call"] = va.AcceptCall(p, d, MODE[case["mode"]], status=s["status"])
    return s


def _prepare_pages(case, seed):
    g = _gen(seed)
    seqs, pool, width = case["seqs"], case["pool"], _width(case)
    perm = np.asarray(torch.randperm(pool, generator=torch.Generator().manual_seed(int(seed))).tolist(), np.int32)
    table = np.full((seqs, width), -1, np.int32)
    ref = np.zeros(pool, np.int32)
    s = {"case": case}
    if case["op"] == "fork":
        parents = seqs - case["forks"]
        ctx = [case["ctx"] + (977 * i) % (case["spread"] + 1) for i in range(parents)]
        at = 0
        for i, c in enumerate(ctx):
            n = -(-c // PAGE)
            table[i, :n] = perm[at:at + n]
            at += n
        lengths = _fork_lengths(case)
        s["src"] = _int([i % parents for i in range(case["forks"])])
        s["dst"] = _int([parents + i for i in range(case["forks"])])
        s["len"] = _int(lengths)
        s["pages"] = _int([-(-n // PAGE) + case["slack"] for n in lengths])
        most = case["forks"]
    else:
        for i in range(seqs):
            table[i, :case["pages"]] = perm[i * case["pages"]:(i + 1) * case["pages"]]
        most = pool // 2
    ref[table[table >= 0]] = 1
    meta = torch.from_numpy(np.concatenate([table.reshape(-1), ref])).cuda()
    s["meta0"], s["meta"] = meta, meta.clone()
    s["table"], s["ref"] = s["meta"][:seqs * width].view(seqs, width), s["meta"][seqs * width:]
    s["copies"] = torch.full((most, 2), -1, dtype=torch.int32, device="cuda")
    s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["pools"] = [torch.randint(-2 ** 31, 2 ** 31 - 1, (pool, case["page_bytes"] // 4), generator=g, device="cuda",
                                dtype=torch.int32) for _ in range(case["pools"])]
    if own:
        import speculative_decoding_verify_kv_gb300 as va
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        pages = va.PagePool(s["table"], s["ref"])
        if case["op"] == "fork":
            s["plan"] = va.ForkCall(pages, s["src"], s["dst"], s["len"], s["pages"], copies=s["copies"],
                                    num_copies=s["count"], status=s["status"])
        else:
            s["plan"] = va.CompactCall(pages, copies=s["copies"], num_copies=s["count"], status=s["status"])
        s["copy"] = va.PageCopyCall(s["pools"], s["copies"], s["count"], status=s["status"])
    return s


# -------------------------------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if op == "window":
        return state["call"]() if own else _plain_window(state)
    if op == "accept":
        return state["call"]() if own else _plain_accept(state)
    state["meta"].copy_(state["meta0"])  # the tables that this pass starts from
    if own:
        state["plan"]()
        state["copy"]()
    elif op == "fork":
        _plain_fork(state)
    else:
        _plain_compact(state)
    return {"table": state["table"], "ref": state["ref"], "copies": state["copies"], "count": state["count"],
            "pools": state["pools"]}


def _decode(raw, kind, dim):
    if kind != "q8_0":
        return raw.float()
    b = raw.view(*raw.shape[:-1], dim // 32, 34)
    scale = b[..., :2].contiguous().view(torch.float16).float()
    return (scale * b[..., 2:].contiguous().view(torch.int8).float()).flatten(-2)


def _ancestors(parent, n):
    """[seqs, n, n] truth values: row j sees draft position a (itself or an ancestor)."""
    j = torch.arange(n, device=parent.device)
    link = (j[None, :] == j[:, None])[None] | (parent[:, :, None] == j[None, None, :])
    for _ in range(max(1, (n - 1).bit_length())):
        link = torch.matmul(link.float(), link.float()) > 0
    return link


def _plain_window(s):
    """All sequences at once, padded to the most rows and the most visible tokens of one."""
    case = s["case"]
    dim, kvh, heads, seqs = case["dim"], case["kv_heads"], case["heads"], case["seqs"]
    grp, window, sinks, n = heads // kvh, case["window"], case["sinks"], max(s["rows"])
    ctx, start = s["ctx_len"].long(), s["cu"][:-1].long()
    lens = s["cu"][1:].long() - start
    b = (ctx - window + 1).clamp(min=0)
    a = b.clamp(max=sinks)
    most = max(sum(_visible(c, r, window, sinks)[:1]) + c + r - _visible(c, r, window, sinks)[1]
               for c, r in zip(s["ctx"], s["rows"]))
    i = torch.arange(most, device="cuda")[None]
    t = torch.where(i < a[:, None], i, i - a[:, None] + b[:, None])  # [seqs, most]
    real = t < (ctx + lens)[:, None]
    t = torch.where(real, t, ctx[:, None])
    one = torch.arange(seqs, device="cuda")[:, None]
    if case["paged"]:
        blk, at = s["table"][one, t // PAGE].long(), t % PAGE
        k, v = s["k"][blk, :, at], s["v"][blk, :, at]  # [seqs, most, kvh, row]
    else:
        k, v = s["k"][one, :, t], s["v"][one, :, t]
    k, v = _decode(k, case["kv"], dim), _decode(v, case["kv"], dim)
    j = torch.arange(n, device="cuda")
    have = j[None] < lens[:, None]
    r = start[:, None] + torch.where(have, j[None], 0)
    if case["mode"] == "chain":
        see, depth = (j[:, None] >= j[None, :])[None], j[None].expand(seqs, n)
    else:
        see = _ancestors(torch.where(have, s["parent"][r].long(), -1), n)
        depth = see.sum(-1) - 1
    own_pos = ctx[:, None] + depth
    drafted = (t - ctx[:, None]).clamp(0, n - 1)
    place = torch.where(t < ctx[:, None], t, ctx[:, None] + depth.gather(1, drafted))  # a draft stands at its depth
    ok = (place[:, None] > own_pos[:, :, None] - window) | (place < sinks)[:, None]
    drafts = see.expand(seqs, n, n).gather(2, drafted[:, None].expand(seqs, n, most))
    ok &= ((t < ctx[:, None])[:, None] | drafts) & real[:, None]
    q = s["q"][r].float().view(seqs, n, kvh, grp, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kvh, grp * n, dim)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(dim))  # [seqs, kvh, grp * n, most]
    z = z.masked_fill(~ok.repeat(1, grp, 1)[:, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    w = torch.exp(z - m)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v.transpose(1, 2)) / total
    o = o.view(seqs, kvh, grp, n, dim).permute(0, 3, 1, 2, 4).reshape(seqs, n, heads, dim)
    lse = (m + torch.log(total)).view(seqs, kvh, grp, n).permute(0, 3, 1, 2).reshape(seqs, n, heads)
    return o[have].to(torch.float32 if case["out"] == "f32" else torch.bfloat16), lse[have]


def _plain_accept(s):
    """All sequences at once, one row index after another: a row is tried when its parent is the
    node reached so far.  Probabilities and residuals in 64 bits: a draw may fall next to a border."""
    case = s["case"]
    vocab, seqs, width = case["vocab"], case["seqs"], max(s["rows"])
    start, lens = s["starts"], s["lens"]
    one = torch.arange(seqs, device="cuda")
    greedy = s["temperature"] <= 0
    inv = 1.0 / torch.where(greedy, 1.0, s["temperature"]).double()

    def target(node):
        x = s["logits"][start + node, :vocab].double()
        top = x.amax(-1, keepdim=True)
        p = torch.exp((x - top) * inv[:, None])
        p = p / p.sum(-1, keepdim=True)
        first = torch.where(x == top, torch.arange(vocab, device="cuda"), vocab).amin(-1)
        hot = torch.arange(vocab, device="cuda")[None] == first[:, None]
        return torch.where(greedy[:, None], hot.double(), p)

    node = torch.zeros(seqs, dtype=torch.int64, device="cuda")
    count = torch.ones(seqs, dtype=torch.int32, device="cuda")
    path = torch.full((s["u"].shape[0],), -1, dtype=torch.int32, device="cuda")
    path[start] = 0
    rest = target(node)
    for j in range(1, width):
        live = lens > j
        r = start + torch.where(live, j, 0)
        up = s["parent"][r].long()
        live = live & (up == node)
        x = s["tokens"][r].long()
        have = rest[one, x]
        if s["probs"] is None:
            guess = torch.ones_like(have)
        else:
            guess = torch.where(greedy, 1.0, s["probs"][start + node, x].double())
        yes = live & torch.where(greedy, have > 0, s["u"][r].double() * guess < have)
        no = live & ~yes & ~greedy
        if s["probs"] is None:
            cut = rest.clone()
            cut[one, x] = 0.0
        else:
            cut = (rest - s["probs"][start + node, :vocab].double()).clamp(min=0.0)
        mass = cut.sum(-1, keepdim=True)
        cut = torch.where(mass > 0, cut / torch.where(mass > 0, mass, 1.0), target(node))
        rest = torch.where(no[:, None], cut, rest)
        node = torch.where(yes, j, node)
        path[torch.where(yes, start + count, start)] = torch.where(yes, j, 0).to(torch.int32)
        count = count + yes.to(torch.int32)
        rest = torch.where(yes[:, None], target(node), rest)
    run_sum = rest.cumsum(-1)
    over = run_sum > s["v"].double()[:, None] * run_sum[:, -1:]
    token = torch.where(over, torch.arange(vocab, device="cuda"), vocab).amin(-1).to(torch.int32)
    return {"accepted_len": count, "accepted_nodes": path, "next_token": token}


def _plain_fork(s):
    src, dst, length, pages = (s[k].long() for k in ("src", "dst", "len", "pages"))
    table, ref = s["table"], s["ref"]
    col = torch.arange(table.shape[1], device="cuda")[None]
    full, keep = (length // PAGE)[:, None], (-(-length // PAGE))[:, None]
    rows = table[src]
    fresh = (col >= full) & (col < pages[:, None])
    shared = (col < full) & (rows >= 0)
    got = torch.nonzero(ref == 0)[:, 0][:int(fresh.sum())].to(torch.int32)
    new = torch.where(shared, rows, -1)
    new[fresh] = got
    ref.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    ref[got.long()] = 1
    table[dst] = new
    tail = torch.nonzero((keep > full)[:, 0])[:, 0]
    pair = torch.stack([rows[tail, full[tail, 0]], new[tail, full[tail, 0]]], 1)
    _plain_copy(s, pair)


def _plain_compact(s):
    table, ref = s["table"], s["ref"]
    live = ref > 0
    n = int(live.sum())
    holes = torch.nonzero(~live[:n])[:, 0]
    moved = torch.nonzero(live[n:])[:, 0] + n
    to = torch.arange(ref.shape[0], device="cuda", dtype=torch.int32)
    to[moved] = holes.to(torch.int32)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    ref[holes] = ref[moved]
    ref[moved] = 0
    _plain_copy(s, torch.stack([moved, holes], 1).to(torch.int32))


def _plain_copy(s, pair):
    s["copies"][:pair.shape[0]] = pair
    s["count"].fill_(pair.shape[0])
    a, b = pair[:, 0].long(), pair[:, 1].long()
    for p in s["pools"]:
        p[b] = p[a]


# ------------------------------------------------------------------------------------------ exact

def exact(case, seed):
    """Windowed attention from its definition in 64 bits.  The other operators return whole numbers."""
    if case["op"] != "window":
        return None
    rows, _ = _rows_of(case)
    if work(case)["flops"] > 1e10 or work(case)["bytes"] > 3e8:  # over some 20 seconds
        return None
    s = _prepare_window(case, seed)
    parent = s["parent"].cpu().numpy()
    dim, kvh, grp = case["dim"], case["kv_heads"], case["heads"] // case["kv_heads"]
    q = s["q"].double().cpu().numpy()
    table = s["table"].cpu().numpy() if case["paged"] else None
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    first = 0
    for i, (n, c) in enumerate(zip(rows, s["ctx"])):
        depth, chain = [], []
        for j in range(n):
            up = int(parent[first + j]) if s["kinds"][i] else j - 1
            depth.append(0 if up < 0 else depth[up] + 1)
            chain.append((chain[up] if up >= 0 else []) + [j])
        span = sorted(set(range(min(case["sinks"], c))) | set(range(max(0, c - case["window"] + 1), c + n)))
        where = {t: at for at, t in enumerate(span)}
        t = np.asarray(span)
        if case["paged"]:
            at = torch.from_numpy(table[i, t // PAGE].astype(np.int64)).cuda(), torch.from_numpy(t % PAGE).cuda()
            raw = [x[at[0], :, at[1]].cpu().numpy() if case["kv"] != "bf16" else
                   x[at[0], :, at[1]].float().cpu().numpy() for x in (s["k"], s["v"])]
        else:
            raw = [(x[i].float() if case["kv"] == "bf16" else x[i])[:, torch.from_numpy(t).cuda()].cpu().numpy()
                   .swapaxes(0, 1) for x in (s["k"], s["v"])]
        if case["kv"] == "q8_0":
            blocks = [np.ascontiguousarray(x).reshape(len(span), kvh, dim // 32, 34) for x in raw]
            raw = [(np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
                    * np.ascontiguousarray(b[..., 2:]).view(np.int8).astype(np.float64)).reshape(len(span), kvh, dim)
                   for b in blocks]
        k, v = (x.astype(np.float64) for x in raw)
        for j in range(n):
            pos = c + depth[j]
            low = pos - case["window"] + 1
            seen = [where[x] for x in span if x < c and (x >= low or x < case["sinks"])]
            seen += [where[c + a] for a in chain[j] if c + depth[a] >= low or c + depth[a] < case["sinks"]]
            kk, vv = k[seen], v[seen]
            for h in range(kvh):
                z = q[first + j, h * grp:(h + 1) * grp] @ kk[:, h].T / math.sqrt(dim)
                m = z.max(1, keepdims=True)
                w = np.exp(z - m)
                out[first + j, h * grp:(h + 1) * grp] = (w @ vv[:, h]) / w.sum(1, keepdims=True)
                lse[first + j, h * grp:(h + 1) * grp] = m[:, 0] + np.log(w.sum(1))
        first += n
    return out, lse
