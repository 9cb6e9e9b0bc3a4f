"""Measured cases of the operators of a latent cache, whose keys and values come from one vector a
token: block tables and slots from request lengths (extend), rows normalised, rotated and written to
their slots (append), verify attention over the cache in the absorbed form (latent), and attention of
prompt segments over expanded keys and values (prompt).

Each case runs ONE call of an operator as a serving loop makes it.  ``run`` computes it either in
plain torch operations (``own`` false) or through the library (``own`` true); ``exact`` restates the
definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
ROPE = 64
MODE = {"chain": 0, "tree": 1, "mixed": 2}
FLOAT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases

def _extend(name, mode, seqs, rows, ragged, ctx, spread, pad, pool):
    return {"name": name, "op": "extend", "mode": mode, "seqs": seqs, "rows": rows, "ragged": ragged,
            "ctx": ctx, "spread": spread, "pad": pad, "pool": pool}


def _append(name, dtype, rows, heads, latent, norm, interleaved, pad, positions):
    return {"name": name, "op": "append", "dtype": dtype, "rows": rows, "heads": heads, "latent": latent,
            "norm": norm, "interleaved": interleaved, "pad": pad, "positions": positions}


def _latent(name, dtype, heads, latent, mode, seqs, rows, ragged, ctx, spread, paged):
    return {"name": name, "op": "latent", "dtype": dtype, "heads": heads, "latent": latent, "mode": mode,
            "seqs": seqs, "rows": rows, "ragged": ragged, "ctx": ctx, "spread": spread, "paged": paged}


def _prompt(name, dtype, heads, nope, value, seqs, rows, ragged, ctx, spread, causal):
    return {"name": name, "op": "prompt", "dtype": dtype, "heads": heads, "nope": nope, "value": value,
            "mode": "chain", "seqs": seqs, "rows": rows, "ragged": ragged, "ctx": ctx, "spread": spread,
            "causal": causal}


def listed():
    return [
        # A step of direct (one-row) requests, a row short of the fixed row count of its graph.
        _extend("extend direct rows", "chain", 40, 1, False, 1016, 997, 1, 8192),
        # A full batch of width-8 trees and direct rows over a large pool.
        _extend("extend mixed", "mixed", 256, 8, True, 4097, 4001, 64, 131072),
        # One new token of one request.
        _append("append one token", "bf16", 1, 16, 512, True, False, 0, 8192),
        # The rows of prompt segments, queries of all heads among them.
        _append("append prompt rows", "bf16", 4096, 128, 512, True, True, 0, 32768),
        # Odd counts, the narrow latent, fp32, rows cut out of wider ones.
        _append("append odd f32", "f32", 77, 5, 256, False, True, 12, 1000),
        # One new token of one request, few heads: the smallest attention call.
        _latent("latent one token", "bf16", 16, 512, "chain", 1, 1, False, 8192, 0, True),
        # A batch of direct rows with all heads on one GPU.
        _latent("latent batch of one token", "bf16", 128, 512, "chain", 32, 1, False, 4097, 2000, True),
        # Drafted chains at long contexts.
        _latent("latent chains", "bf16", 64, 512, "chain", 4, 16, False, 20676, 3000, True),
        # Width-8 trees and direct rows of ragged contexts, fp32, contiguous cache, odd head count.
        _latent("latent trees f32", "f32", 10, 256, "mixed", 5, 8, True, 333, 401, False),
        # One prompt segment behind a cached context.
        _prompt("prompt segment", "bf16", 32, 128, 128, 1, 256, False, 777, 0, True),
        # Long segments with all heads on one GPU.
        _prompt("prompt batch", "bf16", 128, 128, 128, 2, 2048, False, 2048, 0, True),
        # Short ragged segments, fp32, narrow heads.
        _prompt("prompt odd f32", "f32", 5, 64, 64, 3, 77, True, 45, 31, True),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / (1e15 if case.get("dtype") == "bf16" else 4e13))


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        c = _draw(rng)
        if _cost(c) <= top[c["op"]] and (c["op"] != "prompt" or _plain_scores(c) <= 3e9):
            return c


def _plain_scores(case):
    rows = _rows_of(case)[0]
    return case["seqs"] * case["heads"] * max(rows) * (max(_ctx_of(case)) + max(rows))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["extend", "append", "latent", "latent", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "extend":
        mode = rng.choice(["chain", "tree", "mixed"])
        seqs = _log(rng, 1, 300)
        rows = _log(rng, 1, 32) if mode != "chain" else rng.choice([1, _log(rng, 1, 600)])
        ctx, spread = _log(rng, 1, 6000) - 1, _log(rng, 1, 4000) - 1
        need = seqs * ((ctx + spread + rows) // PAGE + 2)
        c = _extend("", mode, seqs, rows, rng.random() < 0.5, ctx, spread, rng.choice([0, 1, 7, 100]),
                    need + rng.randint(need // 8, need + 8))
    elif op == "append":
        c = _append("", dtype, _log(rng, 1, 4000), rng.choice([0, 1, 3, 8, 16, 40, 128]), rng.choice([256, 512]),
                    rng.random() < 0.7, rng.random() < 0.5, rng.choice([0, 0, 8, 24]), _log(rng, 8, 30000))
    elif op == "latent":
        mode = rng.choice(["chain", "chain", "tree", "mixed"])
        small = dtype == "f32"
        rows = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 40 if small else 300)]) if mode == "chain" \
            else _log(rng, 2, 32)
        c = _latent("", dtype, rng.choice([1, 2, 5, 8, 16, 16, 20, 32, 64, 128]), rng.choice([256, 512, 512]), mode,
                    _log(rng, 1, 4 if small else 64), rows, rng.random() < 0.5, _log(rng, 1, 900 if small else 30000) - 1,
                    _log(rng, 1, 400 if small else 4000) - 1, rng.random() < 0.7)
    else:
        small = dtype == "f32"
        wide = rng.random() < 0.7
        c = _prompt("", dtype, _log(rng, 1, 8 if small else 128), 128 if wide else 64, 128 if wide else 64,
                    _log(rng, 1, 4 if small else 8), _log(rng, 1, 200 if small else 2500), rng.random() < 0.5,
                    _log(rng, 1, 200 if small else 4000) - 1, _log(rng, 1, 100 if small else 500) - 1,
                    rng.random() < 0.8)
    del c["name"]
    return c


# -------------------------------------------------------------------------- what a case's lengths are

def _rows_of(case):
    """Rows and kind (1: tree) of each sequence."""
    n, kinds = [], []
    for i in range(case["seqs"]):
        tree = case["mode"] == "tree" or (case["mode"] == "mixed" and i % 4 != 0)
        r = 1 if case["mode"] == "mixed" and not tree else case["rows"]
        if case["ragged"] and i:
            r = 1 + (r * (7 * i + 3)) // 11 % r
        if case["op"] == "extend" and i % 9 == 5:
            r = 0  # a request that sits this step out
        n.append(r)
        kinds.append(1 if tree else 0)
    return n, kinds


def _ctx_of(case):
    return [case["ctx"] + (977 * i) % (case["spread"] + 1) for i in range(case["seqs"])]


def _entries(case):
    """Entries of a row of the block table."""
    return (case["ctx"] + case["spread"] + max(_rows_of(case)[0])) // PAGE + 3


def work(case):
    op = case["op"]
    if op == "append":
        width = case["latent"] + ROPE
        b = 2 * SIZE[case["dtype"]] * case["rows"] * (width + case["heads"] * ROPE)
        angles = min(case["rows"], case["positions"]) * ROPE * 4
        return {"bytes": float(b + angles + 12 * case["rows"]),
                "flops": float(case["rows"] * (4 * case["latent"] + 3 * ROPE * (case["heads"] + 1)))}
    rows, _ = _rows_of(case)
    ctx = _ctx_of(case)
    if op == "extend":
        # Reference counts up to the last page taken, about one table entry per 16 rows read and written,
        # a row's four outputs.
        fresh = sum(-(-(c + n) // PAGE) - -(-c // PAGE) for c, n in zip(ctx, rows))
        return {"bytes": 4.0 * case["pool"] + 8.0 * fresh + 12.0 * case["seqs"] + 20.0 * (sum(rows) + case["pad"]),
                "flops": 0.0}
    size, heads = SIZE[case["dtype"]], case["heads"]
    if op == "latent":
        dim = case["latent"]
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, rows))
        tokens = sum(c + n for c, n in zip(ctx, rows))
        return {"bytes": float(size * (tokens * (dim + ROPE) + sum(rows) * heads * (2 * dim + ROPE))
                               + 4 * sum(rows) * heads),
                "flops": 2.0 * heads * pairs * (2 * dim + ROPE)}
    nope, value = case["nope"], case["value"]
    pairs = sum(n * c + (n * (n + 1) // 2 if case["causal"] else n * n) for c, n in zip(ctx, rows))
    keys = sum(c + n for c, n in zip(ctx, rows))
    return {"bytes": float(size * (keys * (heads * (nope + value) + ROPE) + sum(rows) * heads * (nope + ROPE + value))
                           + 4 * sum(rows) * heads),
            "flops": 2.0 * heads * pairs * (nope + ROPE + value)}


# ----------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _trees(case, seed):
    """Rows, kinds, row offsets and parents: chains, and random trees with parent[j] < j."""
    rows, kinds = _rows_of(case)
    r = random.Random(int(seed) * 37 + 11)
    parent, cu = [], [0]
    for n, k in zip(rows, kinds):
        parent += [(-1 if j == 0 else r.randrange(j)) if k else j - 1 for j in range(n)]
        cu.append(cu[-1] + n)
    return rows, kinds, cu, parent


def prepare(case, seed):
    return {"extend": _prepare_extend, "append": _prepare_append, "latent": _prepare_latent,
            "prompt": _prepare_prompt}[case["op"]](case, seed)


def _prepare_extend(case, seed):
    rows, kinds, cu, parent = _trees(case, seed)
    r = np.random.default_rng(int(seed) * 53 + 3)
    ctx, width = _ctx_of(case), _entries(case)
    held = [-(-c // PAGE) for c in ctx]
    pages = r.permutation(case["pool"])[:sum(held)].astype(np.int32)
    meta = np.zeros(case["seqs"] * width + case["pool"], dtype=np.int32)  # the table, then the counts
    table, ref = meta[:case["seqs"] * width].reshape(case["seqs"], width), meta[case["seqs"] * width:]
    table[:] = -1
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = pages[at:at + h]
        at += h
    ref[pages] = 1
    m0 = torch.from_numpy(meta).cuda()
    m = m0.clone()
    cells = case["seqs"] * width
    s = {"case": case, "meta0": m0, "meta": m, "table": m[:cells].view(case["seqs"], width), "ref": m[cells:],
         "ctx": _int(ctx), "n": _int(rows), "total": cu[-1], "most": max(rows),
         "parent": _int(parent + [-1] * case["pad"]), "kind": _int(kinds, torch.uint8)}
    if own:
        import speculative_decoding_verify_kv_gb300 as va
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["call"] = va.ExtendCall(va.PagePool(s["table"], s["ref"]), s["ctx"], s["n"], cu[-1] + case["pad"],
                                  MODE[case["mode"]], parent=s["parent"], seq_kind=s["kind"], status=s["status"])
    return s


def _prepare_append(case, seed):
    g = _gen(seed)
    dt, rows, heads, latent = FLOAT[case["dtype"]], case["rows"], case["heads"], case["latent"]
    width = latent + ROPE
    kv = torch.randn(rows, width + case["pad"], generator=g, device="cuda").mul_(2.5).to(dt)[:, :width]
    slots = rows + 64
    slot = torch.randperm(slots, generator=g, device="cuda")[:rows]
    position = torch.randint(0, case["positions"], (rows,), generator=g, device="cuda", dtype=torch.int32)
    angle = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] \
        * 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    rope = torch.cat([angle.cos(), angle.sin()], -1).float()
    weight = (1.0 + 0.1 * torch.randn(latent, generator=g, device="cuda")).to(dt) if case["norm"] else None
    q_rope = torch.randn(rows, heads, ROPE + case["pad"], generator=g, device="cuda").to(dt)[..., :ROPE]
    s = {"case": case, "kv": kv, "slot": slot, "position": position, "rope": rope, "weight": weight,
         "q_rope": q_rope, "cache": torch.randn(slots, width, generator=g, device="cuda").to(dt),
         "q": torch.randn(rows, heads, width, generator=g, device="cuda").to(dt)}
    if own:
        import speculative_decoding_verify_kv_gb300 as va
        cache = va.LatentKV(va.F32 if case["dtype"] == "f32" else va.BF16, latent, ROPE, s["cache"], capacity=slots)
        new = va.LatentRows(kv, position, slot, rope=rope, norm_weight=weight, norm_eps=EPS,
                            interleaved=case["interleaved"], q_rope=q_rope if heads else None,
                            q=s["q"] if heads else None)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["call"] = va.LatentAppendCall(cache, new, status=s["status"])
    return s


def _prepare_latent(case, seed):
    g = _gen(seed)
    rows, kinds, cu, parent = _trees(case, seed)
    ctx, dt, seqs, width = _ctx_of(case), FLOAT[case["dtype"]], case["seqs"], case["latent"] + ROPE
    s = {"case": case, "rows": rows, "kinds": kinds, "ctx": ctx, "cu": _int(cu), "ctx_len": _int(ctx),
         "parent": _int(parent), "kind": _int(kinds, torch.uint8), "table": None, "blocks": 0, "capacity": 0,
         "scale": 1.0 / math.sqrt(128 + ROPE),
         "q": torch.randn(cu[-1], case["heads"], width, generator=g, device="cuda").to(dt)}
    if case["paged"]:
        need = [-(-(c + n) // PAGE) for c, n in zip(ctx, rows)]
        order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(int(seed))).numpy()
        table = np.full((seqs, max(need)), -1, dtype=np.int32)
        at = 0
        for i, h in enumerate(need):
            table[i, :h] = order[at:at + h]
            at += h
        s["table"], s["blocks"] = torch.from_numpy(table).cuda(), sum(need)
        shape = (sum(need), PAGE, width)
    else:
        s["capacity"] = max(-(-(c + n) // PAGE) * PAGE for c, n in zip(ctx, rows))
        shape = (seqs, s["capacity"], width)
    s["cache"] = torch.randn(*shape, generator=g, device="cuda", dtype=dt)
    if own:
        import speculative_decoding_verify_kv_gb300 as va
        code = va.F32 if case["dtype"] == "f32" else va.BF16
        kv = va.LatentKV(code, case["latent"], ROPE, s["cache"], page_size=PAGE if case["paged"] else 0,
                         capacity=s["capacity"], block_table=s["table"],
                         max_blocks_per_seq=s["table"].shape[1] if case["paged"] else 0, num_blocks=s["blocks"])
        p = va.Problem(num_seqs=seqs, num_heads=case["heads"], q_dtype=code, q=s["q"], cu_rows=s["cu"],
                       ctx_len=s["ctx_len"], parent=s["parent"], seq_kind=s["kind"], total_rows=cu[-1],
                       max_rows_per_seq=max(rows), scale=s["scale"])
        p.num_splits = va.latent_splits(p, kv)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["call"] = va.LatentCall(p, kv, MODE[case["mode"]], status=s["status"])
    return s


def _prepare_prompt(case, seed):
    g = _gen(seed)
    rows, _, cu, _ = _trees(case, seed)
    ctx, dt, heads = _ctx_of(case), FLOAT[case["dtype"]], case["heads"]
    cu_kv = [0]
    for c, n in zip(ctx, rows):
        cu_kv.append(cu_kv[-1] + c + n)
    s = {"case": case, "rows": rows, "ctx": ctx, "cu": _int(cu), "cu_kv": _int(cu_kv),
         "scale": 1.0 / math.sqrt(case["nope"] + ROPE),
         "q": torch.randn(cu[-1], heads, case["nope"] + ROPE, generator=g, device="cuda").to(dt),
         "kv": torch.randn(cu_kv[-1], heads, case["nope"] + case["value"], generator=g, device="cuda").to(dt),
         # The rotated key part stands in the rows of the latent cache, behind 512 latent values.
         "k_rope": torch.randn(cu_kv[-1], 512 + ROPE, generator=g, device="cuda").to(dt)[:, 512:]}
    if own:
        import speculative_decoding_verify_kv_gb300 as va
        code = va.F32 if case["dtype"] == "f32" else va.BF16
        p = va.Problem(num_seqs=case["seqs"], num_heads=heads, q_dtype=code, q=s["q"], cu_rows=s["cu"], ctx_len=None,
                       parent=None, seq_kind=None, total_rows=cu[-1], max_rows_per_seq=max(rows), scale=s["scale"])
        kv = va.PromptKV(code, case["nope"], ROPE, case["value"], s["kv"], s["k_rope"], s["cu_kv"])
        p.num_splits = va.prompt_splits(p, kv)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["call"] = va.PromptCall(p, kv, causal=case["causal"], status=s["status"])
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if op == "extend":
        state["meta"].copy_(state["meta0"])  # the tables that this pass starts from
        out = state["call"]() if own else _plain_extend(state)
        return {"table": state["table"], "ref": state["ref"], "cu_rows": out["cu_rows"], "row_seq": out["row_seq"],
                "position": out["position"], "slot": out["slot"]}
    if op == "append":
        state["call"]() if own else _plain_append(state)
        return {"cache": state["cache"], "q": state["q"]}
    if own:
        return state["call"]()
    return _plain_latent(state) if op == "latent" else _plain_prompt(state)


def _ancestors(parent, n):
    """[seqs, n, n] truth values: row j sees draft position a (itself or an ancestor)."""
    j = torch.arange(n, device=parent.device)
    link = (j[None, :] == j[:, None])[None] | (parent[:, :, None] == j[None, None, :])
    for _ in range(max(1, (n - 1).bit_length())):
        link = torch.matmul(link.float(), link.float()) > 0
    return link


def _plain_extend(s):
    case = s["case"]
    table, ref, ctx, n = s["table"], s["ref"], s["ctx"].long(), s["n"].long()
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n.cumsum(0)])
    r = torch.arange(s["total"] + case["pad"], device="cuda")
    real = r < s["total"]
    seq = (r[:, None] >= cu[None, 1:]).sum(1).clamp(max=case["seqs"] - 1)
    j = r - cu[seq]
    depth = j
    if case["mode"] != "chain":
        k = torch.arange(min(32, s["most"]), device="cuda")
        have = k[None] < n[:, None]
        up = s["parent"][cu[:-1, None] + torch.where(have, k[None], 0)].long()
        deep = _ancestors(torch.where(have, up, -1), k.shape[0]).sum(-1) - 1
        tree = torch.ones_like(n) if case["mode"] == "tree" else s["kind"].long()
        depth = torch.where(tree[seq] != 0, deep[seq, j.clamp(0, k.shape[0] - 1)], j)
    col = torch.arange(table.shape[1], device="cuda")[None]
    need = (col >= (-(-ctx // PAGE))[:, None]) & (col < (-(-(ctx + n) // PAGE))[:, None]) & (table < 0)
    got = torch.nonzero(ref == 0)[:, 0][:int(need.sum())]
    table[need] = got.to(torch.int32)
    ref[got] = 1
    at = torch.where(real, ctx[seq] + j, 0)
    slot = table[seq, at // PAGE].long() * PAGE + at % PAGE
    return {"cu_rows": cu.to(torch.int32), "row_seq": torch.where(real, seq, -1).to(torch.int32),
            "position": torch.where(real, ctx[seq] + depth, -1).to(torch.int32), "slot": torch.where(real, slot, -1)}


def _turn(x, cos, sin, interleaved):
    """Pairs (2i, 2i + 1), or (i, i + half), turned by angle i."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_append(s):
    case = s["case"]
    latent = case["latent"]
    x = s["kv"].float()
    angle = s["rope"][s["position"].long()]
    cos, sin = angle[:, :ROPE // 2], angle[:, ROPE // 2:]
    c = x[:, :latent]
    if case["norm"]:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat([c, _turn(x[:, latent:], cos, sin, case["interleaved"])], -1)
    s["cache"][s["slot"]] = row.to(s["cache"].dtype)
    if case["heads"]:
        q = _turn(s["q_rope"].float(), cos[:, None], sin[:, None], case["interleaved"])
        s["q"][..., latent:] = q.to(s["q"].dtype)


def _plain_latent(s):
    """All sequences at once, padded to the most rows and the most tokens of one."""
    case = s["case"]
    seqs, heads, latent, n = case["seqs"], case["heads"], case["latent"], max(s["rows"])
    most = max(c + r for c, r in zip(s["ctx"], s["rows"]))
    ctx, start = s["ctx_len"].long(), s["cu"][:-1].long()
    lens = s["cu"][1:].long() - start
    t = torch.arange(most, device="cuda")[None]
    real = t < (ctx + lens)[:, None]
    t = torch.where(real, t, 0)
    one = torch.arange(seqs, device="cuda")[:, None]
    k = (s["cache"][s["table"][one, t // PAGE].long(), t % PAGE] if case["paged"] else s["cache"][one, t]).float()
    j = torch.arange(n, device="cuda")
    have = j[None] < lens[:, None]
    r = start[:, None] + torch.where(have, j[None], 0)
    if case["mode"] == "chain":
        see = (j[:, None] >= j[None, :])[None].expand(seqs, n, n)
    else:
        see = _ancestors(torch.where(have, s["parent"][r].long(), -1), n)
    drafted = (t - ctx[:, None]).clamp(0, n - 1)
    ok = (t < ctx[:, None])[:, None] | see.gather(2, drafted[:, None].expand(seqs, n, most))
    ok = ok & real[:, None]
    q = s["q"][r].float().view(seqs, n * heads, latent + ROPE)
    z = (torch.matmul(q, k.transpose(1, 2)) * s["scale"]).view(seqs, n, heads, most)
    z = z.masked_fill(~ok[:, :, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    w = torch.exp(z - m)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(seqs, n * heads, most), k[..., :latent]).view(seqs, n, heads, latent) / total
    return o[have].to(s["q"].dtype), (m + torch.log(total))[..., 0][have]


def _plain_prompt(s):
    """All sequences at once, padded to the most rows and the most keys of one."""
    case = s["case"]
    seqs, nope, n = case["seqs"], case["nope"], max(s["rows"])
    most = max(c + r for c, r in zip(s["ctx"], s["rows"]))
    start, first = s["cu"][:-1].long(), s["cu_kv"][:-1].long()
    lens, keys = s["cu"][1:].long() - start, s["cu_kv"][1:].long() - first
    t, j = torch.arange(most, device="cuda")[None], torch.arange(n, device="cuda")[None]
    have, real = j < lens[:, None], t < keys[:, None]
    at = first[:, None] + torch.where(real, t, 0)
    r = start[:, None] + torch.where(have, j, 0)
    kv, kr, q = s["kv"][at].float(), s["k_rope"][at].float(), s["q"][r].float()  # [seqs, most | n, heads, ..]
    z = torch.matmul(q[..., :nope].transpose(1, 2), kv[..., :nope].permute(0, 2, 3, 1))
    z += torch.matmul(q[..., nope:].transpose(1, 2), kr.transpose(1, 2)[:, None])
    z *= s["scale"]
    ok = real[:, None].expand(seqs, n, most)
    if case["causal"]:
        ok = ok & (t[:, None] <= (keys - lens)[:, None, None] + j[..., None])
    z = z.masked_fill_(~ok[:, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    w = torch.exp(z.sub_(m))
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, kv[..., nope:].transpose(1, 2)) / total
    lse = (m + torch.log(total))[..., 0]
    return o.transpose(1, 2)[have].to(s["q"].dtype), lse.transpose(1, 2)[have]


# ------------------------------------------------------------------------------------------ exact

def exact(case, seed):
    """From the definition in 64 bits, sequence by sequence.  Extending returns whole numbers."""
    op = case["op"]
    if op == "extend":
        return None
    if op == "append":
        return _exact_append(case, seed)
    if work(case)["flops"] > 2e12:
        return None
    return _exact_latent(case, seed) if op == "latent" else _exact_prompt(case, seed)


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    x, latent, half = s["kv"].double(), case["latent"], ROPE // 2
    angle = s["rope"].double()[s["position"].long()]
    turn = torch.complex(angle[:, :half], angle[:, half:])

    def turned(v, by):
        pairs = v.unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
        if not case["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
        return (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)

    c = x[:, :latent]
    if case["norm"]:
        c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / latent + EPS) * s["weight"].double()
    cache, q = s["cache"].double(), s["q"].double()
    cache[s["slot"], :latent] = c
    cache[s["slot"], latent:] = turned(x[:, latent:], turn)
    if case["heads"]:
        q[..., latent:] = turned(s["q_rope"].double(), turn[:, None])
    return {"cache": cache, "q": q}


def _weigh(z, v):
    """softmax(z) v and log sum exp z; z [heads, rows, keys] with -inf where nothing is seen, v [heads or 1, keys, dim]."""
    m = z.max(-1, keepdim=True).values
    w = (z - m).exp()
    total = w.sum(-1, keepdim=True)
    return (w / total) @ v, (m + total.log())[..., 0]


def _exact_latent(case, seed):
    s = _prepare_latent(case, seed)
    q, latent = s["q"].double(), case["latent"]
    parent = s["parent"].tolist()
    out, lse = torch.zeros_like(q[..., :latent]), torch.zeros_like(q[..., 0])
    first = 0
    for i, (n, c) in enumerate(zip(s["rows"], s["ctx"])):
        if case["paged"]:
            k = s["cache"][s["table"][i, :-(-(c + n) // PAGE)].long()].double().flatten(0, 1)[:c + n]
        else:
            k = s["cache"][i, :c + n].double()
        seen = np.zeros((n, c + n), dtype=bool)
        seen[:, :c] = True
        for j in range(n):
            up = parent[first + j] if s["kinds"][i] else j - 1
            if up >= 0:
                seen[j] = seen[up]
            seen[j, c + j] = True
        hide = ~torch.from_numpy(seen).cuda()
        z = torch.einsum("nhd,td->hnt", q[first:first + n], k) * s["scale"]
        o, one = _weigh(z.masked_fill_(hide, -math.inf), k[None, :, :latent])
        out[first:first + n], lse[first:first + n] = o.transpose(0, 1), one.T
        first += n
    return out, lse


def _exact_prompt(case, seed):
    s = _prepare_prompt(case, seed)
    nope, heads = case["nope"], case["heads"]
    total = s["q"].shape[0]
    out = torch.zeros(total, heads, case["value"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(total, heads, dtype=torch.float64, device="cuda")
    a = b = 0
    for n, c in zip(s["rows"], s["ctx"]):
        keys = torch.arange(c + n, device="cuda")
        hide = keys[None, :] > c + torch.arange(n, device="cuda")[:, None] if case["causal"] else None
        kr = s["k_rope"][b:b + c + n].double()
        for h in range(heads):
            kv = s["kv"][b:b + c + n, h].double()
            z = s["q"][a:a + n, h].double() @ torch.cat([kv[:, :nope], kr], 1).T * s["scale"]
            if hide is not None:
                z = z.masked_fill_(hide, -math.inf)
            o, one = _weigh(z[None], kv[None, :, nope:])
            out[a:a + n, h], lse[a:a + n, h] = o[0], one[0]
        a, b = a + n, b + c + n
    return out, lse
