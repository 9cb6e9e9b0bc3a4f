"""Attention over latent caches and of prompt segments against the fp64 oracle
(GB300)."""
import numpy as np
import pytest

from latent_util import Latent, Prompt, check

import speculative_decoding_verify_kv_gb300 as va

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def run_check(case, **kw):
    got = case.run(**kw)
    torch.cuda.synchronize()
    assert case.status.item() == 0
    return check(got, case.oracle(), case.kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads,ctx,rows,mode,paged,splits", [
    (1, [0], [1], "chain", True, 1),                          # one token, nothing before it
    (16, [1], [1], "chain", True, 4),
    (16, [1000], [1], "chain", True, 8),                      # a direct row in chunks
    (5, [15, 16, 17, 63, 64, 65, 127], [1] * 7, "chain", True, 3),
    (128, [200, 513], [1, 1], "chain", True, 2),              # all heads: one row block each
    (20, [130, 0, 77], [7, 3, 1], "chain", False, 2),         # row blocks with rows cut between heads
    (3, [40, 41, 300, 5], [32, 1, 17, 9], "mixed", True, 5),
    (8, [129, 64], [32, 31], "tree", False, 1),
    (2, [33], [200], "chain", True, 4),                       # a segment of several row blocks
    (7, [10, 0, 20], [0, 2, 0], "chain", True, 2),            # sequences without rows
    (2, [60, 200], [16, 9], "tree", True, 2),                 # few query rows: trees,
    (3, [127, 128, 1], [5, 3, 1], "mixed", True, 3),          # trees and chains,
    (1, [500], [32], "tree", False, 2),                       # one head,
    (4, [300, 130], [4, 8], "chain", True, 2),                # chains
    (1, [130, 3, 255], [16, 5, 1], "mixed", False, 1),
])
def test_latent(kind, latent, heads, ctx, rows, mode, paged, splits):
    run_check(Latent(kind, heads, latent, ctx, rows, mode, paged, seed=heads + latent, splits=splits))


@pytest.mark.parametrize("heads,ctx,rows,splits", [(16, 5000, 1, 37), (128, 3001, 2, 16), (64, 2500, 16, 64),
                                                   (33, 4100, 4, 9), (16, 2049, 2, 150)])
def test_latent_long(heads, ctx, rows, splits):
    run_check(Latent("bf16", heads, 512, [ctx, ctx // 3], [rows, rows], "chain", True, seed=ctx, splits=splits))


def test_latent_cuda_cores():
    """The CUDA-core kernel over bf16, asked for, next to the tensor cores'."""
    case = Latent("bf16", 6, 512, [190, 7], [5, 6], "mixed", True, seed=3, splits=2)
    run_check(case)
    case.p.flags = va.FLAG_CUDA_CORES
    run_check(case)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-3, 0.5])
def test_latent_flat_and_peaked(kind, scale):
    """Weights all alike, and on one token (the running maximum moves)."""
    case = Latent(kind, 12, 512, [700, 90], [3, 2], seed=9, splits=3, scale=scale)
    got = case.run()
    want = case.oracle()
    if scale < 0.1:
        check(got, want, kind)
    else:  # scores of +-50: the same relative errors are 8 times as large
        o, lse = (t.double().cpu().numpy() for t in got)
        assert np.abs(lse - want[1]).max() <= 2e-3
        assert np.linalg.norm(o - want[0]) <= 6e-3 * np.linalg.norm(want[0])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_latent_rising_scores(kind):
    """Each tile's scores are above all before: every tile moves the maximum."""
    case = Latent(kind, 4, 256, [900], [1], seed=4, splits=1, scale=0.05)
    q = torch.zeros_like(case.q)
    q[..., 0] = 8.0
    c = case.kv.cache
    ramp = torch.arange(901, device="cuda", dtype=torch.float32) / 6
    t = torch.arange(901, device="cuda")
    table = case.kv.block_table[0].long()
    c[table[t // 16], t % 16, 0] = ramp.to(c.dtype)
    case.q.copy_(q)
    case.q64, case.cache64 = q.double().cpu().numpy(), c.double().cpu().numpy()
    run_check(case)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_latent_rows_of_no_sequence(kind):
    case = Latent(kind, 9, 256, [50, 80], [2, 3], splits=2, seed=6, pad=4)
    o = torch.full((9, 9, 256), 7.0, device="cuda", dtype=case.q.dtype)
    lse = torch.full((9, 9), 7.0, device="cuda")
    case.p.total_rows = 9
    run_check_rows = case.run(o=o, lse=lse)
    assert case.status.item() == 0
    assert (o[5:] == 7).all() and (lse[5:] == 7).all()
    want = tuple(x[:5] for x in case.oracle())
    check(tuple(t[:5] for t in run_check_rows), want, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("what,bits", [("block", va.DEV_BAD_BLOCK), ("parent", va.DEV_BAD_PARENT),
                                       ("ctx", va.DEV_CTX_OVERFLOW), ("rows", va.DEV_BAD_ROWS)])
@pytest.mark.parametrize("splits", [1, 4])
def test_latent_findings(kind, what, bits, splits):
    """A bad sequence is NaN and flagged; the other one is as always."""
    case = Latent(kind, 4, 256, [400, 300], [6, 5], "tree", True, seed=8, splits=splits)
    want = case.oracle()
    first = 0
    if what == "block":
        case.kv.block_table[0, 20] = case.kv.num_blocks
    elif what == "parent":
        case.p.parent[2], first = 2, 2
    elif what == "ctx":
        case.p.ctx_len[0] = 16 * case.kv.max_blocks_per_seq
    else:
        case.p.cu_rows[:] = torch.tensor([0, 40, 11], device="cuda")
    o, lse = case.run()
    assert case.status.item() & bits
    if what == "rows":
        assert lse.isnan().any()
        return
    assert lse[first].isnan().all() and o[first].isnan().all()
    check((o[6:], lse[6:]), tuple(x[6:] for x in want), kind)


@pytest.mark.parametrize("splits", [1, 4])
def test_latent_alone_and_in_company(splits):
    """A row's result depends on its own sequence alone, and repeats."""
    both = Latent("bf16", 16, 512, [700, 300], [3, 3], seed=12, splits=splits)
    o, lse = both.run()
    again = both.run()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    one = both.kv.block_table[1:].contiguous()
    p = va.Problem(**{**vars(both.p), "num_seqs": 1, "q": both.q[3:].contiguous(), "total_rows": 3,
                      "cu_rows": torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                      "ctx_len": both.p.ctx_len[1:].contiguous()})
    kv = va.LatentKV(**{**vars(both.kv), "block_table": one})
    o1, lse1 = va.verify_attn_latent(p, kv, 0)
    assert torch.equal(o[3:], o1) and torch.equal(lse[3:], lse1)


@pytest.mark.parametrize("kind,heads,rows,latent", [("f32", 3, 5, 256), ("bf16", 3, 5, 512), ("bf16", 16, 5, 512), ("bf16", 16, 5, 256)])
@pytest.mark.parametrize("splits", [1, 3])
def test_latent_not_a_number(kind, heads, rows, latent, splits):
    """A query that is no number is its own row's matter."""
    case = Latent(kind, heads, latent, [300, 40], [rows, 2], seed=2, splits=splits)
    want = [t.clone() for t in case.run()]
    case.q[2, 1, 7] = float("nan")
    o, lse = case.run()
    assert o[2, 1].isnan().all() and lse[2, 1].isnan()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("splits", [1, 3])
def test_prompt_not_a_number(kind, splits):
    case = Prompt(kind, 2, 128, [140, 3], [400, 3], seed=2, splits=splits)
    want = [t.clone() for t in case.run()]
    case.p.q[130, 1, 7] = float("nan")
    o, lse = case.run()
    assert o[130, 1].isnan().all() and lse[130, 1].isnan()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[130, 1] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


@pytest.mark.parametrize("heads,ctx,rows,splits", [(128, 1000, 3, 1), (64, 1, 1, 1), (33, 127, 1, 2), (40, 128, 7, 6), (128, 640, 1, 5)])
def test_latent_pairs(heads, ctx, rows, splits):
    """Pairs of CTAs: second halves without rows, odd tiles, one tile."""
    run_check(Latent("bf16", heads, 512, [ctx, ctx + 63, 0, 5 * ctx], [rows, 1, rows, rows], "chain", heads % 2 == 0, seed=heads,
                     splits=splits))


def test_latent_far_pages():
    """Offsets past 2^32 bytes: pages at the end of a pool of 6 GB."""
    width, blocks = 576, 330_000
    cache = torch.zeros(blocks, 16, width, dtype=torch.bfloat16, device="cuda")
    case = Latent("bf16", 16, 512, [100], [1], seed=5, splits=2)
    need = case.table.shape[1]
    cache[-need:] = case.kv.cache[case.kv.block_table[0].long()]
    far = torch.arange(blocks - need, blocks, dtype=torch.int32, device="cuda")[None]
    kv = va.LatentKV(va.BF16, 512, 64, cache, page_size=16, block_table=far, max_blocks_per_seq=need, num_blocks=blocks)
    a, b = case.run(), va.verify_attn_latent(case.p, kv, 0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(b, case.oracle(), "bf16")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,rows,keys,causal,splits", [
    (1, [1], [1], True, 1),
    (3, [5, 1, 40], [5, 700, 41], True, 3),
    (2, [129, 64], [129, 65], True, 1),
    (4, [300], [301], True, 2),
    (2, [77, 9], [130, 500], False, 4),
    (5, [20, 3, 4], [7, 0, 4], True, 2),       # rows before the first key, a sequence of none
    (3, [6, 5], [0, 33], False, 1),
    (1, [0, 4, 0], [9, 128, 0], True, 1),
])
def test_prompt(kind, dim, heads, rows, keys, causal, splits):
    run_check(Prompt(kind, heads, dim, rows, keys, seed=heads + dim, causal=causal, splits=splits,
                     stride=64 if heads % 2 else 576))


def test_prompt_long():
    run_check(Prompt("bf16", 2, 128, [700, 1025], [1700, 1025], seed=3))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal,splits", [(True, 1), (True, 6), (False, 1), (False, 3)])
def test_prompt_many_blocks(dim, causal, splits):
    """Several row blocks to a CTA one after the other, among them some without rows
    or keys, ragged and whole tiles; the same again, whichever CTA takes a block."""
    case = Prompt("bf16", 70, dim, [300, 0, 1, 130, 128, 5], [420, 60, 1, 130, 384, 0], seed=dim, causal=causal, splits=splits)
    first = [t.clone() for t in case.run()]
    for _ in range(3):
        again = case.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    run_check(case)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("splits", [1, 2])
def test_prompt_many_sequences(kind, splits):
    """More sequences than a warp looks at at once, most far below the bound, one bad."""
    rows = [(7 * s) % 5 if s % 11 else 140 for s in range(77)]
    keys = [r + s % 3 for s, r in enumerate(rows)]
    case = Prompt(kind, 3, 64, rows, keys, seed=5, splits=splits)
    want = case.oracle()
    case.p.max_rows_per_seq = 1000
    run_check(case)
    case.p.max_rows_per_seq = 139
    o, lse = case.run()
    assert case.status.item() == va.DEV_BAD_ROWS
    ok = torch.ones(len(lse), dtype=torch.bool)
    for s in range(0, 77, 11):
        ok[case.cu[s]:case.cu[s + 1]] = False
    assert o[~ok].isnan().all() and lse[~ok].isnan().all()
    check((o[ok], lse[ok]), tuple(x[ok.numpy()] for x in want), kind)


def test_prompt_more_blocks_than_rows_have():
    """Offsets that go back and forth: more blocks than a launch of that many rows has
    otherwise, every second sequence bad and without rows."""
    case = Prompt("bf16", 2, 128, [300], [300], seed=6)
    want = case.oracle()
    p = va.Problem(**{**vars(case.p), "num_seqs": 41, "cu_rows": torch.tensor([0, 300] * 21, dtype=torch.int32, device="cuda")})
    kv = va.PromptKV(**{**vars(case.kv), "cu_kv": torch.tensor([0, 300] * 21, dtype=torch.int32, device="cuda")})
    got = va.verify_attn_latent_prompt(p, kv, status=case.status)
    assert case.status.item() == va.DEV_BAD_ROWS
    check(got, want, "bf16")


def test_prompt_many_blocks_findings():
    """A sequence with bad offsets among many blocks."""
    case = Prompt("bf16", 70, 128, [200, 140, 256], [300, 150, 600], seed=4)
    want = case.oracle()
    case.kv.cu_kv[2] = -3        # the end of the second sequence, the start of the third
    o, lse = case.run()
    assert case.status.item() == va.DEV_BAD_ROWS
    assert o[200:].isnan().all() and lse[200:].isnan().all()
    check((o[:200], lse[:200]), tuple(x[:200] for x in want), "bf16")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_prompt_parts_join(kind):
    """A context part and the segment itself, joined by their lse, are the whole."""
    whole = Prompt(kind, 3, 128, [50], [250], seed=2)
    o, lse = (t.double() for t in whole.run())
    parts = []
    for a, b, causal in ((0, 200, False), (200, 250, True)):
        kv = va.PromptKV(**{**vars(whole.kv), "kv": whole.kv.kv[a:b].contiguous(), "k_rope": whole.kv.k_rope[a:b],
                            "cu_kv": torch.tensor([0, b - a], dtype=torch.int32, device="cuda")})
        parts.append([t.double() for t in va.verify_attn_latent_prompt(whole.p, kv, causal=causal)])
    both = torch.logaddexp(parts[0][1], parts[1][1])
    sum_o = sum(t * torch.exp(w - both)[..., None] for t, w in parts)
    tol = 1e-5 if kind == "f32" else 3 * 2.0 ** -8
    assert (both - lse).abs().max() <= (1e-5 if kind == "f32" else 1e-4)
    assert (sum_o - o).norm() <= tol * o.norm()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["cu_rows", "cu_kv", "long"])
def test_prompt_findings(kind, which):
    case = Prompt(kind, 2, 64, [6, 5], [9, 9], seed=8)
    want = case.oracle()
    if which == "cu_rows":
        case.p.cu_rows[1] = 40
    elif which == "cu_kv":
        case.kv.cu_kv[1] = -3
    else:
        case.p.max_rows_per_seq = 5
    o, lse = case.run()
    assert case.status.item() == va.DEV_BAD_ROWS
    assert lse[0].isnan().all() and o[0].isnan().all()
    if which == "long":
        check((o[6:], lse[6:]), tuple(x[6:] for x in want), kind)


@pytest.mark.parametrize("make", [lambda: Latent("bf16", 16, 512, [900, 40], [2, 3], splits=6, seed=1),
                                  lambda: Latent("f32", 4, 256, [300], [9], splits=2, seed=1),
                                  lambda: Prompt("bf16", 3, 128, [70, 5], [300, 5], splits=2, seed=1)])
def test_captured_and_replayed(make):
    """A captured call, replayed over other queries and lengths of keys."""
    case = make()
    cls = va.LatentCall if isinstance(case, Latent) else va.PromptCall
    args = (case.p, case.kv, 0) if cls is va.LatentCall else (case.p, case.kv)
    call = cls(*args, status=case.status)
    eager = [t.clone() for t in call()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
        for _ in range(2):
            call()
    for t in out:
        t.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    case.p.q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    fresh = cls(*args)()
    assert all(torch.equal(a, b) for a, b in zip(out, fresh))
    assert not torch.equal(out[0], eager[0])


def test_other_stream():
    case = Latent("bf16", 16, 512, [900, 40], [2, 3], splits=6, seed=1)
    want = [t.clone() for t in case.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = case.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
