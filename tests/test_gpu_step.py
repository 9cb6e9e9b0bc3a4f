"""The operators around a verify step as a serving loop runs them: pages grown
and forked, windowed attention over the paged cache with tree drafts in a
scratch KV, acceptance, commit of the accepted paths, pages behind the window
and behind the context given back, the pool pulled together; every step's
attention and acceptance against the oracle on plain host copies."""
from types import SimpleNamespace

import numpy as np
import pytest

import oracle.step_oracle as so
import synthetic as sy
from window_util import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verify_kv_gb300 as va  # noqa: E402

H, KVH, PAGE, VOCAB = 4, 2, 16, 700


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


@pytest.mark.parametrize("kv,dim", [("bf16", 64), ("q8_0", 128)])
@pytest.mark.parametrize("window,sinks", [(48, 4), (20, 0), (400, 16)])
def test_serving_loop(kv, dim, window, sinks):
    g = np.random.default_rng(dim + window)
    seqs, width, blocks = 5, 24, 96
    table, ref = i32(np.full((seqs, width), -1)), i32(np.zeros(blocks))
    pool = va.PagePool(table, ref)
    relems, sdt = sy.row_elems(kv, dim), sy.storage_dtype(kv)
    rows_of = lambda n: sy._q8_values(g, (n, KVH, dim)) if kv == "q8_0" else sy._values(g, kv, (n, KVH, dim))  # noqa: E731
    raw = lambda a: torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()  # noqa: E731
    k, v = (raw(np.zeros((blocks, KVH, PAGE, relems), sdt)) for _ in range(2))
    host = {}  # sequence -> [K rows, V rows], every token of its context
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def put(s, first, kr, vr):
        """Rows of sequence s from token `first` on, into its pages."""
        t = np.arange(first, first + len(kr))
        blk = table[s].cpu().numpy()[t // PAGE]
        assert (blk >= 0).all()
        at = torch.from_numpy(blk.astype(np.int64)).cuda(), torch.from_numpy(t % PAGE).cuda()
        k[at[0], :, at[1]] = raw(kr)
        v[at[0], :, at[1]] = raw(vr)

    def grow(live, held, need):  # from the tokens that already have pages to the pages wanted
        va.verify_attn_pages_fork(pool, i32(live), i32(live), i32(held), i32(need), status=status)
        assert int(status.item()) == 0

    for s, n in enumerate((70, 33, 5)):
        host[s] = [rows_of(n), rows_of(n)]
    grow([0, 1, 2], [0, 0, 0], [-(-len(host[s][0]) // PAGE) for s in range(3)])
    for s in host:
        put(s, 0, *host[s])

    for step in range(5):
        live = sorted(host)
        kinds = [0 if s == 1 else 1 for s in live]
        n = [int(g.integers(1, 9)) for _ in live]
        ctx = [len(host[s][0]) for s in live]
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        parent = np.concatenate([sy.random_tree_parents(g, m) if t else np.arange(-1, m - 1)
                                 for m, t in zip(n, kinds)]).astype(np.int32)
        total = int(cu[-1])
        dk, dv = rows_of(total), rows_of(total)
        grow(live, ctx, [-(-(c + m) // PAGE) for c, m in zip(ctx, n)])
        for i, s in enumerate(live):
            if kinds[i] == 0:  # a chain's drafts are written to the cache
                put(s, ctx[i], dk[cu[i]:cu[i + 1]], dv[cu[i]:cu[i + 1]])
        q = sy._values(g, "bf16", (total, H, dim))
        sub = table[torch.tensor(live, device="cuda")].contiguous()  # the launch's sequences
        p = va.Problem(len(live), H, va.BF16, raw(q), i32(cu), i32(ctx), i32(parent),
                       torch.tensor(kinds, dtype=torch.uint8, device="cuda"), total, max(n), num_splits=2)
        cache = va.KV(va.DTYPE_CODES[kv], KVH, dim, k, v, page_size=PAGE, block_table=sub, max_blocks_per_seq=width,
                      num_blocks=blocks, draft_k=raw(dk), draft_v=raw(dv))
        o, lse = va.verify_attn_window(p, cache, va.MODE_MIXED, va.Window(window, sinks), status=status)
        # The same on host copies laid out contiguously.
        cap = max(c + m for c, m in zip(ctx, n))
        hk, hv = (np.zeros((len(live), KVH, cap, relems), sdt) for _ in range(2))
        for i, s in enumerate(live):
            for dst, src, draft in ((hk, host[s][0], dk), (hv, host[s][1], dv)):
                dst[i, :, :ctx[i]] = src.transpose(1, 0, 2)
                dst[i, :, ctx[i]:ctx[i] + n[i]] = draft[cu[i]:cu[i + 1]].transpose(1, 0, 2)
        case = SimpleNamespace(num_heads=H, num_kv_heads=KVH, head_dim=dim, kv_dtype=kv, q_dtype="bf16", q=q, k=hk,
                               v=hv, ctx_len=ctx, cu_rows=cu, parent=parent, seq_kind=kinds, mode="mixed", scale=0.0,
                               page_size=0, capacity=cap, block_table=None, draft_k=None, draft_v=None)
        assert int(status.item()) == 0
        check(case, o.cpu().numpy(), lse.cpu().numpy(), so.window_case(case, window, sinks), False, f"step {step}")

        # Acceptance, and the commit of the trees' paths.
        z = (g.standard_normal((total, VOCAB)) * 2).astype(np.float32)
        up = np.concatenate([[max(0, x) for x in parent[cu[i]:cu[i + 1]]] for i in range(len(live))]) + np.repeat(cu[:-1], n)
        tokens = (z[up] + g.standard_normal((total, VOCAB))).argmax(-1).astype(np.int32)
        u, w = g.random(total).astype(np.float32), g.random(len(live)).astype(np.float32)
        draft = va.Draft(torch.from_numpy(z).cuda(), VOCAB, i32(tokens), torch.from_numpy(u).cuda(),
                         torch.from_numpy(w).cuda(), logits_dtype=va.F32)
        promote = torch.zeros(len(live), dtype=torch.int32, device="cuda")
        out = va.verify_attn_accept(p, draft, va.MODE_MIXED, promote_len=promote, status=status)
        want = so.accept(z, None, tokens, parent, kinds, cu, u, w, np.ones(len(live)))
        assert (want[4] > 1e-6).all()
        for name, x in zip(("accepted_len", "accepted_nodes", "promote_len", "next_token"), want):
            assert np.array_equal(out[name].cpu().numpy(), x), name
        va.verify_attn_promote(p, cache, va.MODE_MIXED, promote, out["accepted_nodes"], status)
        assert int(status.item()) == 0
        for i, s in enumerate(live):
            path = want[1][cu[i]:cu[i] + want[0][i]] + cu[i]
            host[s] = [np.concatenate([host[s][0], dk[path]]), np.concatenate([host[s][1], dv[path]])]

        # Pages that no later row can see, and pages behind the context, go back.
        ranges = []
        for s in live:
            c = len(host[s][0])
            ranges.append((s, -(-sinks // PAGE), max(-(-sinks // PAGE), (c - window + 1) // PAGE)))
            ranges.append((s, -(-c // PAGE), width))
        va.verify_attn_pages_free(pool, *(i32(x) for x in zip(*ranges)), status=status)
        copies = None
        if step in (1, 3):  # a request is forked into a free row of the table
            src, dst = (0, 3) if step == 1 else (2, 4)
            c = len(host[src][0])
            copies = va.verify_attn_pages_fork(pool, i32([src]), i32([dst]), i32([c]), i32([-(-c // PAGE)]), status=status)
            va.verify_attn_pages_copy([k, v], *copies, status=status)
            host[dst] = [x.copy() for x in host[src]]
        if step == 2:  # a request ends
            va.verify_attn_pages_free(pool, i32([1]), i32([0]), i32([width]), status=status)
            del host[1]
        if step != 3:
            c, m, used = va.verify_attn_pages_compact(pool, status=status)
            va.verify_attn_pages_copy([k, v], c, m, status=status)
            assert int((ref[int(used.item()):]).abs().sum()) == 0
        assert int(status.item()) == 0
        counts = np.zeros(blocks, np.int64)
        t = table.cpu().numpy()
        np.add.at(counts, t[t >= 0], 1)
        assert np.array_equal(counts, ref.cpu().numpy())
