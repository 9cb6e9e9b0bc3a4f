"""Edges of attention over a latent cache: queries and cached values that are no
numbers where a sequence has one tile or every tile moves a row's maximum, and
rows in the company of other sequences (GB300)."""
import ctypes

import numpy as np
import pytest

from latent_util import Latent, Prompt, check

import speculative_decoding_verify_kv_gb300 as va

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def rising(case, upto):
    """Column 0 of sequence 0's first tokens grows with the token."""
    t = torch.arange(upto, device="cuda")
    table = case.kv.block_table[0].long()
    case.kv.cache[table[t // 16], t % 16, 0] = (t.float() / 6).to(case.kv.cache.dtype)


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads,rows", [(2, 5), (16, 1), (6, 5), (32, 1), (40, 2)])
@pytest.mark.parametrize("ctx", [0, 1, 40, 59, 130])
@pytest.mark.parametrize("splits", [1, 3])
def test_nan_query_of_few_tokens(latent, heads, rows, ctx, splits):
    """One tile or a few: the row is NaN, not an empty row's outputs."""
    case = Latent("bf16", heads, latent, [ctx, 7], [rows, 1], seed=ctx + heads, splits=splits)
    want = [t.clone() for t in case.run()]
    case.q[rows - 1, 1, 7] = float("nan")
    o, lse = case.run()
    assert case.status.item() == 0
    assert o[rows - 1, 1].isnan().all() and lse[rows - 1, 1].isnan()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[rows - 1, 1] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads", [4, 20, 48])
@pytest.mark.parametrize("splits", [1, 4])
def test_nan_query_of_rising_scores(latent, heads, splits):
    """Every tile, the last one too, moves the other rows' maximum."""
    case = Latent("bf16", heads, latent, [895], [1], seed=4, splits=splits, scale=0.1)
    case.q.zero_()
    case.q[..., 0] = 8.0
    rising(case, 896)
    case.q[0, 2, 5] = float("nan")
    o, lse = case.run()
    assert o[0, 2].isnan().all() and lse[0, 2].isnan()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[0, 2] = False
    assert o[keep].isfinite().all() and lse[keep].isfinite().all()


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads", [3, 24, 40])
@pytest.mark.parametrize("token", [0, 37, 130])
def test_nan_token(latent, heads, token):
    """A cached key that every row sees and that is no number makes them NaN."""
    case = Latent("bf16", heads, latent, [140], [1], seed=heads, splits=1)
    case.kv.cache[case.kv.block_table[0, token // 16].long(), token % 16, latent + 3] = float("nan")
    o, lse = case.run()
    assert o.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads,rows", [(4, 1), (8, 1), (5, 4), (40, 1)])
@pytest.mark.parametrize("splits", [1, 3])
def test_alone_and_in_company(latent, heads, rows, splits):
    """A row's bits do not depend on the next sequence's queries, which stand behind
    its own in memory and whose scores over its tokens rise all the way."""
    both = Latent("bf16", heads, latent, [900, 30], [rows, rows], seed=latent + heads, splits=splits)
    rising(both, 900)
    both.q[:rows, :, 0] = 0
    both.q[rows:].zero_()
    both.q[rows:, :, 0] = 50.0
    o, lse = both.run()
    p = va.Problem(**{**vars(both.p), "num_seqs": 1, "q": both.q[:rows].contiguous(), "total_rows": rows,
                      "cu_rows": both.p.cu_rows[:2].contiguous(), "ctx_len": both.p.ctx_len[:1].contiguous()})
    kv = va.LatentKV(**{**vars(both.kv), "block_table": both.kv.block_table[:1].contiguous()})
    o1, lse1 = va.verify_attn_latent(p, kv, 0)
    assert torch.equal(o[:rows], o1) and torch.equal(lse[:rows], lse1)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e38])
def test_few_rows_beside_queries_of_any_value(value):
    both = Latent("bf16", 4, 512, [300, 30], [1, 1], seed=3)
    want = [t[:1].clone() for t in both.run()]
    both.q[1:] = value
    o, lse = both.run()
    assert torch.equal(o[:1], want[0]) and torch.equal(lse[:1], want[1])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("latent,heads,ctx,rows,splits", [
    (512, 24, [700, 900, 0, 300], [40, 2, 0, 30], 17), (256, 24, [700, 1500], [40, 2], 17), (512, 7, [1500, 300], [3, 1], 9),
    (512, 130, [500], [25], 60), (256, 5, [200, 800, 1000], [1, 70, 9], 12)])
def test_workspace_of_row_blocks(kind, latent, heads, ctx, rows, splits):
    """Partials of long and short sequences stand in the workspace that the library asks
    for, which holds no more than a row block a sequence and chunk; nothing behind it."""
    case = Latent(kind, heads, latent, ctx, rows, seed=heads, splits=splits)
    need = va.lib.va_latent_workspace_size(ctypes.byref(case.p.c()), ctypes.byref(case.kv.c()))
    block = 16 if kind == "f32" else 128
    assert need <= splits * min(len(ctx) * block, sum(rows) * heads) * (latent + 2) * 4 + 512
    ws = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = case.run(ws=ws)
    assert case.status.item() == 0 and (ws[need:] == 0x5A).all()
    check((o, lse), case.oracle(), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,keys,splits", [([300, 7, 200], [2100, 1900, 200], 6), ([900], [1300], 16), ([5, 0, 9], [1500, 3, 800], 5)])
def test_prompt_workspace_of_row_blocks(kind, dim, rows, keys, splits):
    case = Prompt(kind, 3, dim, rows, keys, seed=dim, splits=splits)
    need = va.lib.va_latent_prompt_workspace_size(ctypes.byref(case.p.c()), ctypes.byref(case.kv.c()))
    block = 16 if kind == "f32" else 128
    assert need <= splits * min(len(rows) * block, sum(rows)) * 3 * (dim + 2) * 4 + 512
    ws = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = case.run(ws=ws)
    assert case.status.item() == 0 and (ws[need:] == 0x5A).all()
    check((o, lse), case.oracle(), kind)


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("what,bits", [("block", va.DEV_BAD_BLOCK), ("far block", va.DEV_BAD_BLOCK), ("parent", va.DEV_BAD_PARENT),
                                       ("ctx", va.DEV_CTX_OVERFLOW), ("negative", va.DEV_CTX_OVERFLOW), ("rows", va.DEV_BAD_ROWS),
                                       ("tree", va.DEV_BAD_ROWS)])
@pytest.mark.parametrize("splits", [1, 6])
def test_findings_of_many_rows(latent, what, bits, splits):
    """More than 32 query rows (pairs of CTAs, of which both have to know, and 128-row
    blocks): a bad sequence is NaN and flagged, the others are as always."""
    heads, rows = 24, [9, 6, 3]
    case = Latent("bf16", heads, latent, [700, 300, 150], rows, "tree", True, seed=8, splits=splits)
    want = case.oracle()
    bad = slice(0, 9)
    if what == "block":
        case.kv.block_table[0, 20] = case.kv.num_blocks
    elif what == "far block":
        case.kv.block_table[0, 44] = -2       # the last page of the drafts, at the end of a ragged tile
    elif what == "parent":
        case.p.parent[2], bad = 2, slice(2, 3)
    elif what == "ctx":
        case.p.ctx_len[0] = 16 * case.kv.max_blocks_per_seq
    elif what == "negative":
        case.p.ctx_len[0] = -5
    elif what == "rows":
        case.p.max_rows_per_seq = 8
    else:
        case.p.ctx_len[0] = 0
        case.p.cu_rows[:] = torch.tensor([0, 33, 34, 37], device="cuda")
        case.p.max_rows_per_seq, case.p.total_rows = 40, 37
        q = torch.zeros(37, heads, latent + 64, dtype=case.q.dtype, device="cuda")
        q[34:] = case.q[15:]
        parent = torch.full((37,), -1, dtype=torch.int32, device="cuda")
        parent[34:] = case.p.parent[15:18]
        case.p.q, case.p.parent = q, parent
    mode = 2 if what == "tree" else case.mode_code  # (trees alone may not have a bound of more than 32 rows)
    o, lse = va.verify_attn_latent(case.p, case.kv, mode, status=case.status)
    assert case.status.item() == bits
    if what == "tree":
        assert o[:33].isnan().all() and lse[:33].isnan().all()
        check((o[34:], lse[34:]), tuple(x[15:] for x in want), "bf16")
        return
    assert lse[bad].isnan().all() and o[bad].isnan().all()
    check((o[9:], lse[9:]), tuple(x[9:] for x in want), "bf16")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [3, 20])
@pytest.mark.parametrize("splits", [1, 4])
def test_findings_of_too_many_rows(kind, heads, splits):
    """A sequence longer than the bound is NaN in all its rows; the others are as always."""
    case = Latent(kind, heads, 512, [200, 400, 100], [2, 9, 3], seed=3, splits=splits)
    want = case.oracle()
    case.p.max_rows_per_seq = 8
    o, lse = case.run()
    assert case.status.item() == va.DEV_BAD_ROWS
    assert o[2:11].isnan().all() and lse[2:11].isnan().all()
    for part in (slice(0, 2), slice(11, 14)):
        check((o[part], lse[part]), tuple(x[part] for x in want), kind)


@pytest.mark.parametrize("kind,heads,latent", [("bf16", 16, 512), ("bf16", 40, 512), ("bf16", 40, 256), ("f32", 4, 256)])
@pytest.mark.parametrize("splits", [1, 6])
def test_replayed_over_other_lengths(kind, heads, latent, splits):
    """A captured call reads lengths, offsets and tables when it runs: fewer and more
    chunks hold tokens than at capture, rows move between the sequences."""
    case = Latent(kind, heads, latent, [1500, 900], [2, 2], seed=7, splits=splits)
    ws = va.lib.va_latent_workspace_size(ctypes.byref(case.p.c()), ctypes.byref(case.kv.c()))
    call = va.LatentCall(case.p, case.kv, 0, ws=torch.empty(max(ws, 256), dtype=torch.uint8, device="cuda"), status=case.status)
    case.p.ctx_len[:] = torch.tensor([70, 200], device="cuda")
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for ctx, cu in (([70, 200], [0, 2, 4]), ([1500, 900], [0, 2, 4]), ([0, 830], [0, 2, 3]), ([1200, 0], [0, 1, 3]), ([3, 900], [0, 0, 2])):
        case.p.ctx_len[:] = torch.tensor(ctx, device="cuda")
        case.p.cu_rows[:] = torch.tensor(cu, device="cuda")
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert case.status.item() == 0
        fresh = va.LatentCall(case.p, case.kv, 0, o=torch.full_like(out[0], 7), lse=torch.full_like(out[1], 7))()
        assert all(torch.equal(a, b) for a, b in zip(out, fresh))
        case.ctx, case.cu = np.array(ctx, np.int32), np.array(cu, np.int32)
        n = cu[-1]
        case.p.total_rows = 4
        check(tuple(t[:n] for t in out), tuple(x[:n] for x in case.oracle()), kind)
        assert (out[0][n:] == 7).all() and (out[1][n:] == 7).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("splits", [1, 5])
def test_prompts_replayed_over_other_lengths(kind, splits):
    case = Prompt(kind, 3, 128, [130, 70], [900, 500], seed=7, splits=splits)
    call = va.PromptCall(case.p, case.kv, status=case.status)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for cu, cu_kv in (([0, 130, 200], [0, 900, 1400]), ([0, 70, 200], [0, 100, 1400]), ([0, 100, 130], [0, 1300, 1350]), ([0, 0, 130], [0, 0, 130])):
        case.p.cu_rows[:] = torch.tensor(cu, device="cuda")
        case.kv.cu_kv[:] = torch.tensor(cu_kv, device="cuda")
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert case.status.item() == 0
        n = cu[-1]
        case.cu, case.cu_kv = np.array(cu, np.int32), np.array(cu_kv, np.int32)
        check(tuple(t[:n] for t in out), tuple(x[:n] for x in case.oracle()), kind)
        assert (out[0][n:] == 7).all() and (out[1][n:] == 7).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads", [2, 20, 40])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_scores(kind, latent, heads, sign):
    """One token whose score is +-2^28: its value and the score come back.  (Scaled to
    log2 units the score is rounded, 2^-24 of it, by a kernel's maximum and by its
    exponent apart: a weight of 2^+-16 that its sum has too.)"""
    case = Latent(kind, heads, latent, [0], [1], seed=1, scale=1.0)
    case.q.zero_()
    case.q[..., 0] = sign * 2.0 ** 14
    row = case.kv.cache[case.kv.block_table[0, 0].long(), 0]
    row[0] = 2.0 ** 14
    o, lse = case.run()
    v = row[:latent].double()
    # Three roundings of a score, at 2^-24 each, and the last bit of the sum.
    assert ((lse.double() - sign * 2.0 ** 28).abs() <= 2.0 ** 28 * 2.0 ** -22).all()
    # bf16: the weight's rounding and o's, 2^-8 each at most; fp32: weight, sum, its inverse, product.
    step = 2.0 ** -7 if kind == "bf16" else 2.0 ** -21
    assert ((o.double() - v).abs() <= step * v.abs()).all()
