"""Windowed verify attention on the GPU against the fp64 oracle (bounds in
window_util).  Tokens that no row sees hold NaN, and the block-table entries
of pages without a visible token hold no page."""
import dataclasses

import numpy as np
import pytest

import oracle
import oracle.step_oracle as so
import synthetic as sy
from window_util import check, poison_unseen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verify_kv_gb300 as va  # noqa: E402


def run(case, window, sinks, out=va.F32, splits=1, flags=0, status=0, device="cuda"):
    p, kv, mode = va.upload(case, device, num_splits=splits, flags=flags)
    st = torch.zeros(1, dtype=torch.int32, device=device)
    o, lse = va.verify_attn_window(p, kv, mode, va.Window(window, sinks, out), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status, f"{int(st.item()):#x}"
    return o.float().cpu().numpy(), lse.cpu().numpy()


def make(kv, heads, kvh, dim, ctx, rows, kinds=None, mode="chain", paged=False, seed=0):
    return sy.make_case("window", num_heads=heads, num_kv_heads=kvh, head_dim=dim, kv_dtype=kv,
                        q_dtype="f32" if kv == "f32" else "bf16", ctx=ctx, rows=rows, kinds=kinds, mode=mode,
                        paged=paged, seed=seed, extra_blocks=3 if paged else 0)


SHAPES = [("bf16", 8, 2, 128), ("bf16", 6, 1, 256), ("bf16", 4, 4, 64), ("q8_0", 6, 1, 256), ("q8_0", 8, 2, 128),
          ("q8_0", 2, 2, 64), ("f32", 4, 1, 64), ("f32", 2, 1, 128), ("f32", 3, 3, 256)]


@pytest.mark.parametrize("kv,heads,kvh,dim", SHAPES)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("window,sinks,splits", [(1, 0, 1), (1, 3, 2), (17, 4, 1), (64, 0, 3), (100, 33, 2),
                                                 (250, 16, 4), (512, 200, 1)])
def test_chains(kv, heads, kvh, dim, paged, window, sinks, splits):
    case = make(kv, heads, kvh, dim, [0, 5, 63, 200, 777], [1, 3, 16, 1, 5], paged=paged, seed=window + dim)
    case = poison_unseen(case, window, sinks)
    ref = so.window_case(case, window, sinks)
    for out in (va.F32, va.BF16):
        check(case, *run(case, window, sinks, out, splits), ref, out == va.BF16, f"out {out}")


@pytest.mark.parametrize("kv,heads,kvh,dim", SHAPES)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("scratch", [False, True])
@pytest.mark.parametrize("window,sinks,splits", [(1, 0, 1), (2, 1, 1), (5, 200, 2), (90, 18, 3), (333, 0, 2)])
def test_trees_and_direct_rows(kv, heads, kvh, dim, paged, scratch, window, sinks, splits):
    """Trees deeper than the window, sinks that reach into the drafts."""
    case = make(kv, heads, kvh, dim, [0, 190, 401, 3, 130], [32, 8, 1, 9, 7], kinds=[1, 1, 0, 1, 0], mode="mixed",
                paged=paged, seed=window * 7 + dim)
    if scratch:
        case = sy.with_tree_scratch(case)
        keep = dataclasses.replace(case)
        case = poison_unseen(case, window, sinks)
        case = dataclasses.replace(case, draft_k=keep.draft_k, draft_v=keep.draft_v)
    else:
        case = poison_unseen(case, window, sinks)
    ref = so.window_case(case, window, sinks)
    check(case, *run(case, window, sinks, va.F32, splits), ref, False)


@pytest.mark.parametrize("kv", ["bf16", "q8_0"])
def test_deep_trees(kv):
    """Chains as trees: a window shorter than the tree."""
    n = 32
    case = make(kv, 4, 2, 128, [100, 7], [n, n], mode="tree", paged=True, seed=3)
    par = np.concatenate([np.arange(-1, n - 1)] * 2).astype(np.int32)
    case = dataclasses.replace(case, parent=par)
    for window, sinks in [(3, 0), (20, 9), (40, 103)]:
        c = poison_unseen(case, window, sinks)
        check(c, *run(c, window, sinks, splits=2), so.window_case(c, window, sinks), False)
        chain = dataclasses.replace(c, mode="chain", seq_kind=np.zeros(2, np.uint8))
        a, b = run(c, window, sinks, splits=2), run(chain, window, sinks, splits=2)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("kv,heads,kvh,dim", SHAPES)
def test_many_rows(kv, heads, kvh, dim):
    """A prompt segment of several row blocks beside a direct row."""
    case = make(kv, heads, kvh, dim, [150, 260], [150, 1], paged=True, seed=dim)
    for window, sinks, splits in [(40, 5, 1), (170, 0, 5)]:
        c = poison_unseen(case, window, sinks)
        check(c, *run(c, window, sinks, splits=splits), so.window_case(c, window, sinks), False)


@pytest.mark.parametrize("kv,heads,kvh,dim", SHAPES)
@pytest.mark.parametrize("flags", [0, va.FLAG_CUDA_CORES])
def test_a_wide_window_is_the_unwindowed_call(kv, heads, kvh, dim, flags):
    case = make(kv, heads, kvh, dim, [300, 17, 0], [8, 1, 4], kinds=[1, 0, 1], mode="mixed", paged=True, seed=4)
    O, L = oracle.verify_case(case)
    for window in (2 ** 31 - 1, 310):
        check(case, *run(case, window, 0, splits=2, flags=flags), (O, L), False)


@pytest.mark.parametrize("kv,heads,kvh,dim", SHAPES)
def test_cuda_core_kernel(kv, heads, kvh, dim):
    case = make(kv, heads, kvh, dim, [200, 90], [16, 6], kinds=[0, 1], mode="mixed", paged=True, seed=8)
    c = poison_unseen(case, 50, 20, entry=2 ** 30)
    check(c, *run(c, 50, 20, splits=2, flags=va.FLAG_CUDA_CORES), so.window_case(c, 50, 20), False)


def test_a_sequence_does_not_depend_on_the_launch():
    case = make("q8_0", 6, 1, 256, [700, 90, 333, 40], [16, 1, 8, 1], kinds=[0, 0, 1, 0], mode="mixed", paged=True,
                seed=12)
    for splits in (1, 3):
        whole = run(case, 300, 4, splits=splits)
        for s in range(4):
            p, kv, mode = va.upload(sy.subset_sequences(case, [s]), "cuda", num_splits=splits)
            p.max_rows_per_seq = 16  # the bound of the whole launch
            got = [x.cpu().numpy() for x in va.verify_attn_window(p, kv, mode, va.Window(300, 4))]
            a, b = int(case.cu_rows[s]), int(case.cu_rows[s + 1])
            assert np.array_equal(got[0], whole[0][a:b]) and np.array_equal(got[1], whole[1][a:b])


FEW = [(kv, h, k, d) for kv in ("bf16", "q8_0") for h, k, d in ((8, 1, 64), (8, 2, 128), (3, 3, 128), (5, 1, 256))]


@pytest.mark.parametrize("kv,heads,kvh,dim,rows", [("bf16", 8, 2, 64, 1), ("bf16", 8, 2, 128, 7), ("q8_0", 6, 1, 256, 2),
                                                   ("q8_0", 6, 1, 256, 16), ("bf16", 6, 1, 256, 16)])
@pytest.mark.parametrize("splits", [2, 5, 8, 12, 16])
def test_many_sequences_and_one_give_the_same_bits(kv, heads, kvh, dim, rows, splits):
    """Few clusters are joined in their kernel, many go through the merge
    kernel: a sequence's bits are the same."""
    one = make(kv, heads, kvh, dim, [2300], [rows], paged=True, seed=splits)
    many = dataclasses.replace(one, ctx_len=np.repeat(one.ctx_len, 120), block_table=np.repeat(one.block_table, 120, 0),
                               cu_rows=np.arange(121, dtype=np.int32) * rows, parent=np.tile(one.parent, 120),
                               seq_kind=np.repeat(one.seq_kind, 120), q=np.tile(one.q, (120, 1, 1)))
    a, b = run(one, 2000, 4, splits=splits), run(many, 2000, 4, splits=splits)
    for x, y in zip(a, b):
        assert np.array_equal(np.tile(x, (120,) + (1,) * (x.ndim - 1)), y)


@pytest.mark.parametrize("kv,heads,kvh,dim", FEW)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("window,sinks,splits", [(1, 0, 1), (17, 4, 1), (40, 33, 2), (700, 0, 1), (700, 20, 3),
                                                 (1300, 5, 1), (1300, 5, 7)])
def test_few_rows(kv, heads, kvh, dim, paged, window, sinks, splits):
    """At most 16 query rows per KV head: rings that go round, chunks of no
    and of one page, trees of two and three rows, both outputs."""
    n = 16 * kvh // heads
    case = make(kv, heads, kvh, dim, [0, 15, 16, 130, 1500], [n, 1, min(n, 3), n, 1], kinds=[1, 0, 1, 0, 0],
                mode="mixed", paged=paged, seed=window + dim)
    case = poison_unseen(case, window, sinks)
    ref = so.window_case(case, window, sinks)
    for out in (va.F32, va.BF16):
        check(case, *run(case, window, sinks, out, splits), ref, out == va.BF16, f"out {out}")


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("rows", [1, 16])
def test_rows_that_no_sequence_covers_stay(splits, rows):
    case = make("bf16", 4, 2, 64, [300, 20], [rows, 1], seed=3)
    p, kv, mode = va.upload(case, "cuda", num_splits=splits)
    ref = so.window_case(case, 64, 2)
    total = p.total_rows
    p.total_rows += 2
    p.q = torch.cat([p.q, p.q[:2]])
    o = torch.full((total + 2, 4, 64), 7.0, device="cuda")
    lse = torch.full((total + 2, 4), 7.0, device="cuda")
    va.verify_attn_window(p, kv, mode, va.Window(64, 2), o=o, lse=lse)
    assert (o[total:] == 7).all() and (lse[total:] == 7).all()
    check(case, o[:total].cpu().numpy(), lse[:total].cpu().numpy(), ref, False)


@pytest.mark.parametrize("kv,heads,kvh,dim", [SHAPES[0], SHAPES[3], SHAPES[6], ("bf16", 8, 2, 64), ("q8_0", 2, 1, 256)])
@pytest.mark.parametrize("splits", [1, 2])
def test_device_errors_poison_only_their_sequence(kv, heads, kvh, dim, splits):
    case = make(kv, heads, kvh, dim, [200, 90, 64], [4, 4, 4], kinds=[0, 1, 0], mode="mixed", paged=True, seed=2)
    ref = so.window_case(case, 40, 3)
    for what in ("block", "parent", "ctx", "rows"):
        c = dataclasses.replace(case, block_table=case.block_table.copy(), parent=case.parent.copy(),
                                ctx_len=case.ctx_len.copy(), cu_rows=case.cu_rows.copy())
        p, kvs, mode = va.upload(c, "cuda", num_splits=splits)
        if what == "block":      # a page inside the window; pages out of sight hold none
            kvs.block_table[1, 4] = 10 ** 6
            kvs.block_table[0, 3] = -5
        elif what == "parent":
            p.parent[5] = 3
        elif what == "ctx":
            p.ctx_len[1] = 10 ** 6
        else:
            p.cu_rows[1:3] = torch.tensor([8, 6], dtype=torch.int32)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = va.verify_attn_window(p, kvs, mode, va.Window(40, 3), status=st)
        bit = {"block": va.DEV_BAD_BLOCK, "parent": va.DEV_BAD_PARENT, "ctx": va.DEV_CTX_OVERFLOW,
               "rows": va.DEV_BAD_ROWS}[what]
        assert int(st.item()) == bit, (what, hex(int(st.item())))
        o, lse = o.cpu().numpy(), lse.cpu().numpy()
        if what == "rows":
            continue
        assert np.isnan(lse[4:8]).any(), what
        keep = np.r_[0:4, 8:12]
        sub = dataclasses.replace(case)
        check(sub, o[keep], lse[keep], (ref[0][keep], ref[1][keep]), False, what)


def test_graphs_streams_and_rows_behind_the_last_sequence():
    case = make("bf16", 8, 2, 128, [500, 90], [4, 1], paged=True, seed=6)
    p, kv, mode = va.upload(case, "cuda", num_splits=2)
    ref = so.window_case(case, 128, 4)
    calls = [va.WindowCall(p, kv, mode, va.Window(128, 4, va.BF16)) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c()
        graphs.append((g, out))
    for _, (o, lse) in graphs:
        o.zero_(), lse.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, (o, lse) in graphs:
        check(case, o.float().cpu().numpy(), lse.cpu().numpy(), ref, True)


def test_offsets_past_32_bits():
    """A contiguous bf16 cache of two times 4.8 GB: windows past 2^31 elements and 2^32 bytes."""
    cap, ctx = 9 * 2 ** 20, 9 * 2 ** 20 - 30
    k = torch.zeros(2, 1, cap, 256, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(3)
    for t in (slice(0, 4), slice(ctx - 40, ctx + 2)):
        for x in (k, v):
            x[:, :, t] = torch.randn(x[:, :, t].shape, generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.randn(4, 4, 256, generator=g, device="cuda", dtype=torch.bfloat16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    p = va.Problem(2, 4, va.BF16, q, i32(0, 2, 4), i32(ctx, ctx), i32(-1, 0, -1, 0),
                   torch.zeros(2, dtype=torch.uint8, device="cuda"), 4, 2, num_splits=1)
    o, lse = va.verify_attn_window(p, va.KV(va.BF16, 1, 256, k, v, capacity=cap), 0, va.Window(30, 4))
    for s in range(2):
        for j in range(2):
            pos = ctx + j
            t = torch.tensor(list(range(4)) + list(range(pos - 29, pos + 1)), device="cuda")
            z = q[2 * s + j].double() @ k[s, 0, t].double().T / 256 ** 0.5
            want = torch.softmax(z, -1) @ v[s, 0, t].double()
            assert (o[2 * s + j].double() - want).abs().max() < 2e-4
            assert (lse[2 * s + j].double() - torch.logsumexp(z, -1)).abs().max() < 1e-4


@pytest.mark.parametrize("kv,heads,kvh,dim,rows", [("bf16", 4, 1, 64, 2), ("bf16", 4, 1, 64, 9), ("bf16", 4, 1, 128, 4),
                                                   ("bf16", 4, 1, 128, 8), ("q8_0", 4, 1, 256, 3), ("q8_0", 4, 1, 256, 16),
                                                   ("bf16", 4, 1, 256, 9), ("f32", 4, 1, 64, 5)])
@pytest.mark.parametrize("splits", [9, 16, 20, 256])
def test_many_chunks_joined_and_merged(kv, heads, kvh, dim, rows, splits):
    """Partials through the workspace; most chunks hold two tiles, many none."""
    case = make(kv, heads, kvh, dim, [2900, 100, 1500], [rows, 1, rows], paged=True, seed=splits + rows)
    c = poison_unseen(case, 2600, 30)
    check(c, *run(c, 2600, 30, splits=splits), so.window_case(c, 2600, 30), False)


@pytest.mark.parametrize("rows", [1, 20])
def test_long_windows_in_one_chunk_stay_exact_in_fp32(rows):
    """O in fp32 over 9,000 bf16 tokens, one chunk asked for: the tensor cores'
    running sums would be off by some 2e-5 of O; within 8e-6 of the norm (P
    carries 16 bits or more: 2^-18 of each term, and 2,048 tokens of drift)."""
    case = make("bf16", 4, 1, 256, [9000], [rows], paged=True, seed=rows)
    O, L = so.window_case(case, 9000, 0)
    o, lse = run(case, 9000, 0, splits=1)
    assert np.linalg.norm(o - O) <= 8e-6 * np.linalg.norm(O)
    assert np.abs(lse - L).max() < 1e-4


def test_fp32_cache_with_bf16_queries():
    case = dataclasses.replace(make("f32", 4, 1, 64, [200, 30], [7, 1], paged=True, seed=5), q_dtype="bf16")
    case = dataclasses.replace(case, q=sy.f32_to_bf16_bits(case.q))
    check(case, *run(case, 50, 3, splits=2), so.window_case(case, 50, 3), False)


FIRST = """
import sys, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {root!r} + "/tests")
import numpy as np
import speculative_decoding_verify_kv_gb300 as va, synthetic as sy
case = sy.make_case("first", num_heads=4, num_kv_heads=1, head_dim=64, kv_dtype={kv!r}, q_dtype="bf16", ctx=[300, 9],
                    rows=[{rows}, 1], paged=True, seed=1)
p, kv, mode = va.upload(case, "cuda", num_splits=2)
call = va.WindowCall(p, kv, mode, va.Window(64, 2))
z = torch.randn(p.total_rows, 500, device="cuda")
f = lambda n: torch.rand(n, device="cuda")
d = va.Draft(z, 500, torch.zeros(p.total_rows, dtype=torch.int32, device="cuda"), f(p.total_rows), f(2), logits_dtype=va.F32)
accept = va.AcceptCall(p, d, 0)
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
table, ref = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
pool = va.PagePool(table, ref)
plan, pack = va.ForkCall(pool, i32(0), i32(0), i32(0), i32(3)), va.CompactCall(pool)
copy = va.PageCopyCall([torch.zeros(9, 64, device="cuda")], *plan._out)
free = va.FreeCall(pool, i32(0), i32(1), i32(2))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for c in (call, accept, plan, copy, free, pack):
        c()
g.replay()
torch.cuda.synchronize()
o = call._out[0].clone()
assert table.tolist() == [[0, -1, 1, -1], [-1] * 4], table
call()
assert torch.equal(o, call._out[0])
print("captured first")
"""


@pytest.mark.parametrize("kv,rows", [("bf16", 1), ("bf16", 6), ("q8_0", 6)])
def test_the_first_calls_of_a_process_may_be_captured(kv, rows):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, kv=kv, rows=rows)], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
