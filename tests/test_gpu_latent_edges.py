"""Edges of attention over a latent cache: queries and cached values that are no
numbers where a sequence has one tile or every tile moves a row's maximum, and
rows in the company of other sequences (GB300)."""
import ctypes

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
