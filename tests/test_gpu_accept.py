"""Acceptance of drafted tokens on the GPU against the fp64 oracle.

Outputs are whole numbers and have to be equal.  A decision compares numbers
of order one whose fp32 error is below 1e-5 (a sum of up to 2^20 positive
terms in pieces, each term off by at most 2^-22, the pieces' rescaling by
2^-22), and a draw's borders are off by at most 1e-9; the seeded inputs keep
every decision further from its border than that (checked with the oracle's
margin before anything is compared)."""
import numpy as np
import pytest

import oracle.step_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verify_kv_gb300 as va  # noqa: E402

MODES = {"chain": 0, "tree": 1, "mixed": 2}


class Case:
    def __init__(self, mode, rows, kinds, vocab, dtype, drawn, temperature, seed, pad=0, offset=0, spread=2.5,
                 parent=None, tokens=None):
        g = np.random.default_rng(seed)
        self.mode, self.vocab, self.kinds = mode, vocab, kinds
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        total = int(self.cu[-1])
        if parent is None:
            parent = [(-1 if j == 0 else int(g.integers(0, j))) if k else j - 1
                      for n, k in zip(rows, kinds) for j in range(n)]
        self.parent = np.asarray(parent, np.int32).reshape(-1)
        stride = vocab + pad
        self.stride = stride
        base = torch.from_numpy((g.standard_normal(total * stride + offset) * spread).astype(np.float32))
        self.base = base.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        self.offset, self.dtype = offset, dtype
        z = self.base[offset:].reshape(total, stride)[:, :vocab].float().numpy().astype(np.float64)
        self.logits = z
        self.temperature = np.broadcast_to(np.asarray(temperature, np.float32), (len(rows),)).copy()
        up = np.array([self.cu[s] + max(0, self.parent[self.cu[s] + j]) for s, n in enumerate(rows)
                       for j in range(n)], np.int64)
        self.probs = None
        if drawn:
            y = z + g.standard_normal(z.shape)
            w = np.exp(y - y.max(-1, keepdims=True))
            self.probs = (w / w.sum(-1, keepdims=True)).astype(np.float32)
        if tokens is None:
            if drawn:
                e = g.exponential(size=(total, vocab))
                tokens = (self.probs[up] / e).argmax(-1) if total else np.zeros(0)
            else:
                tokens = (z[up] + 0.5 * g.standard_normal((total, vocab))).argmax(-1) if total else np.zeros(0)
        self.tokens = np.asarray(tokens, np.int32).reshape(-1)
        self.u = g.random(total).astype(np.float32)
        self.v = g.random(len(rows)).astype(np.float32)

    def problem(self, device="cuda"):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(device)  # noqa: E731
        total = int(self.cu[-1])
        base = self.base.to(device)
        logits = base[self.offset:]
        p = va.Problem(num_seqs=len(self.cu) - 1, num_heads=1, q_dtype=va.BF16, q=None, cu_rows=t(self.cu),
                       ctx_len=None, parent=t(self.parent), seq_kind=t(np.asarray(self.kinds, np.uint8)),
                       total_rows=total, max_rows_per_seq=max(1, int(np.diff(self.cu).max())))
        probs = None
        if self.probs is not None:
            probs = torch.full((total, self.stride), 9.0)
            probs[:, :self.vocab] = torch.from_numpy(self.probs)
            probs = probs.to(device)
        d = va.Draft(logits=logits, vocab=self.vocab, tokens=t(self.tokens), accept_u=t(self.u), sample_u=t(self.v),
                     logits_dtype=va.BF16 if self.dtype == "bf16" else va.F32, logits_stride=self.stride,
                     draft_probs=probs, draft_stride=self.stride, temperature=t(self.temperature))
        return p, d

    def oracle(self):
        return so.accept(self.logits, self.probs, self.tokens, self.parent, self.kinds, self.cu, self.u, self.v,
                         self.temperature)


def run(case, status=0, **kw):
    p, d = case.problem()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    promote = torch.full((p.num_seqs,), -7, dtype=torch.int32, device="cuda")
    out = va.verify_attn_accept(p, d, MODES[case.mode], promote_len=promote, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == status, f"{int(st.item()):#x}"
    return [out[k].cpu().numpy() for k in ("accepted_len", "accepted_nodes", "promote_len", "next_token")]


def check(case, close=1e-9):
    want = case.oracle()
    assert (want[4] > close).all(), "an input next to a border"
    got = run(case)
    for g, w, what in zip(got, want, ("accepted_len", "accepted_nodes", "promote_len", "next_token")):
        assert np.array_equal(g, w), (what, g, w)
    return got


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 33, 129, 4096, 8191, 8193, 50021, 131072])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("drawn", [False, True])
def test_chains(vocab, dtype, drawn):
    check(Case("chain", [4, 1, 7, 16], [0] * 4, vocab, dtype, drawn, [1.0, 0.7, 1.3, 0.5], 10 + vocab))


@pytest.mark.parametrize("vocab,pad,offset", [(5, 0, 0), (257, 3, 1), (1000, 1, 5), (32768, 0, 0), (40001, 7, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("drawn", [False, True])
def test_trees_with_odd_strides(vocab, pad, offset, dtype, drawn):
    check(Case("tree", [8, 32, 1, 2, 19], [1] * 5, vocab, dtype, drawn, [1.0, 0.9, 0.6, 1.0, 2.0], 77 + vocab,
               pad=pad, offset=offset))


@pytest.mark.parametrize("seqs", [7, 8, 14, 15])
def test_batches_that_all_run_at_once_and_do_not(seqs):
    """The threads of a sequence follow from their number; a sequence's result
    does not."""
    c = Case("mixed", [3, 9] * 8, [0, 1] * 8, 70001, "f32", True, 0.9, 70)
    full = check(c)
    c.cu, c.kinds, c.v, c.temperature = c.cu[:seqs + 1], c.kinds[:seqs], c.v[:seqs], c.temperature[:seqs]
    n = int(c.cu[-1])
    c.parent, c.tokens, c.u, c.logits, c.probs = c.parent[:n], c.tokens[:n], c.u[:n], c.logits[:n], c.probs[:n]
    for g, w, k in zip(check(c), full, (seqs, n, seqs, seqs)):
        assert np.array_equal(g[:k], w[:k])


@pytest.mark.parametrize("vocab", [81921, 150001, 163841])
@pytest.mark.parametrize("drawn", [False, True])
def test_batches_whose_weights_fit_a_cluster_and_do_not(vocab, drawn):
    """16 sequences: clusters of 8 CTAs, whose shared memory holds the weights
    of a row of up to some 160,000 values."""
    rows = [1, 3, 2, 4] * 4
    check(Case("mixed", rows, [0, 1, 0, 1] * 4, vocab, "bf16", drawn, 1.0, vocab))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mixed_kinds_and_temperatures(dtype):
    check(Case("mixed", [8, 1, 5, 32, 40], [1, 0, 0, 1, 0], 6007, dtype, True, [0.0, 0.0, 0.8, 1.0, 0.0], 5))
    check(Case("mixed", [8, 1, 5, 32, 40], [1, 0, 0, 1, 0], 6007, dtype, False, [0.0, 1.0, 0.0, 0.3, 0.0], 6))


@pytest.mark.parametrize("drawn", [False, True])
def test_many_siblings(drawn):
    """A star: every row a child of row 0, so that residuals of up to 31
    rejected siblings are tried and drawn from."""
    parent = ([-1] + [0] * 31) * 6
    for seed in range(4):
        c = Case("tree", [32] * 6, [1] * 6, 900, "f32", drawn, 1.0, 400 + seed, parent=parent, spread=1.0)
        c.u[:] = 1.0 - 1e-3 * np.random.default_rng(seed).random(len(c.u)).astype(np.float32)
        check(c)


def test_a_chain_of_the_most_rows():
    c = Case("chain", [1024, 3], [0, 0], 301, "f32", False, 1.0, 9)
    # Proposals that are the maxima, taken with small numbers: long paths.
    c.tokens[1:1024] = c.logits[:1023].argmax(-1)
    c.u[:] *= 0.02
    got = check(c)
    assert got[0][0] > 20


def test_ties_go_to_the_lowest_index():
    c = Case("chain", [3, 3], [0, 0], 20011, "bf16", False, 0.0, 3)
    z = c.base.reshape(6, -1)
    z[:, [77, 15000, 19999]] = 30.0
    c.logits = z.float().numpy().astype(np.float64)
    c.tokens[:] = [0, 77, 77, 0, 15000, 77]
    got = check(c)
    assert got[0].tolist() == [3, 1] and got[3].tolist() == [77, 77]


def test_masked_vocabulary_and_peaked_rows():
    """-inf entries never come out; a single finite entry is certain."""
    for vocab in (40, 20000):
        c = Case("chain", [2, 2, 1], [0] * 3, vocab, "f32", False, 1.0, 21)
        z = c.base.reshape(5, vocab)
        z[0] = -np.inf
        z[0, vocab - 1] = -3.0
        z[1, ::2] = -np.inf
        z[2, 5:] = -np.inf
        z[4] = torch.finfo(torch.float32).min
        z[4, 7] = 0.0
        c.logits = z.numpy().astype(np.float64)
        c.tokens[:] = [0, vocab - 1, 0, 9, 0]
        c.u[:] = 0.999
        got = check(c)
        assert got[0].tolist() == [2, 1, 1] and got[3][2] == 7 and got[3][0] % 2 == 1


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("temperature", [0.0, 1.0])
@pytest.mark.parametrize("where", [0, 2])
def test_rows_without_a_distribution(value, temperature, where):
    """At a row with children (0) and at a leaf (2): the path ends there."""
    c = Case("chain", [3, 3], [0, 0], 9001, "f32", False, temperature, 33)
    z = c.base.reshape(6, -1)
    for r in range(6):
        z[r, 4000] = 50.0
    c.tokens[:] = 4000
    z[where] = value if value == float("-inf") else z[where]
    z[where, 8500] = value
    c.logits = z.numpy().astype(np.float64)
    want = c.oracle()
    got = run(c, status=va.DEV_BAD_LOGITS)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert got[3].tolist() == [-1, 4000]


def test_equal_distributions_take_everything_and_zero_residuals_fall_back():
    """p == g in every entry: each drafted token is taken for any u < 1."""
    c = Case("chain", [6], [0], 64, "f32", True, 1.0, 2)
    w = np.exp(c.logits - c.logits.max(-1, keepdims=True))
    c.probs = (w / w.sum(-1, keepdims=True)).astype(np.float32)
    c.tokens[1:] = c.probs[:-1].argmax(-1)
    c.u[:] = 0.75
    got = run(c)
    assert got[0].tolist() == [6]
    # g above p everywhere (not a distribution): the residual is zero, p is drawn from.
    c.probs[:] = 1.0
    c.u[:] = 0.999
    check(c)


@pytest.mark.parametrize("v", [0.0, 1.0 - 2.0 ** -24])
def test_the_ends_of_the_draw(v):
    c = Case("chain", [1, 2], [0, 0], 12345, "bf16", False, 1.0, 8)
    z = c.base.reshape(3, -1)
    z[:, :5] = -np.inf
    z[:, -9:] = -np.inf
    z[:, -10] = 0.0
    c.logits = z.float().numpy().astype(np.float64)
    c.v[:] = v
    c.u[:] = 0.9999
    c.tokens[:] = 10
    got = run(c)
    if v == 0.0:
        assert got[3].tolist() == [5, 5]
    else:
        want = c.oracle()
        assert np.array_equal(got[3], want[3])


def test_errors_and_untouched_rows():
    c = Case("mixed", [8, 3, 8, 2], [1, 0, 1, 0], 500, "f32", False, 1.0, 4)
    want = c.oracle()
    c.parent[3] = 5           # tree 0: a parent after its child
    c.tokens[9] = 500         # chain 1: no such token
    c.temperature[2] = -1.0   # tree 2
    p, d = c.problem()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = p.total_rows
    p.total_rows = rows + 2   # two rows that no sequence covers
    grow = lambda t, n: torch.cat([t, t[:n]])  # noqa: E731
    d.tokens, d.accept_u = grow(d.tokens, 2), grow(d.accept_u, 2)
    d.logits = grow(d.logits, 2 * c.stride)
    nodes = torch.full((rows + 2,), -9, dtype=torch.int32, device="cuda")
    p.parent = grow(p.parent, 2)
    out = va.verify_attn_accept(p, d, 2, accepted_nodes=nodes, status=st)
    assert int(st.item()) == va.DEV_BAD_PARENT | va.DEV_BAD_TOKEN | va.DEV_BAD_SAMPLING
    assert out["accepted_len"].tolist() == [0, 0, 0, int(want[0][3])]
    assert out["next_token"].tolist() == [-1, -1, -1, int(want[3][3])]
    assert nodes[:19].tolist() == [-1] * 19 and nodes[rows:].tolist() == [-9, -9]
    assert nodes[19:rows].tolist() == want[1][19:].tolist()


def test_bad_row_ranges_leave_the_other_sequences_alone():
    c = Case("chain", [4, 4, 4], [0] * 3, 100, "f32", False, 1.0, 4)
    want = c.oracle()
    p, d = c.problem()
    p.cu_rows = torch.tensor([0, 4, 2, 12], dtype=torch.int32, device="cuda")  # 4..2, then ten rows
    p.max_rows_per_seq = 4
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = va.verify_attn_accept(p, d, 0, status=st)
    assert int(st.item()) == va.DEV_BAD_ROWS
    assert out["accepted_len"].tolist() == [int(want[0][0]), 0, 0]
    assert out["next_token"].tolist()[1:] == [-1, -1]


def test_empty_sequences():
    c = Case("chain", [0, 3, 0], [0] * 3, 100, "f32", False, 1.0, 4)
    got = run(c)
    want = c.oracle()
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_the_result_does_not_depend_on_what_shares_the_launch():
    c = Case("mixed", [8, 1, 16, 32], [1, 0, 0, 1], 30011, "bf16", True, 1.0, 91)
    whole = run(c)
    for s in range(4):
        a, b = int(c.cu[s]), int(c.cu[s + 1])
        one = Case("mixed", [b - a], [c.kinds[s]], c.vocab, "bf16", True, 1.0, 0)
        one.base = c.base.reshape(-1, c.stride)[a:b].clone().reshape(-1)
        one.probs, one.tokens, one.parent = c.probs[a:b], c.tokens[a:b], c.parent[a:b]
        one.u, one.v = c.u[a:b], c.v[s:s + 1]
        got = run(one)
        assert got[0][0] == whole[0][s] and got[3][0] == whole[3][s]
        assert np.array_equal(got[1], whole[1][a:b])


def test_streams_and_graphs():
    """Two calls in two captured graphs, each with its own workspace, and an
    eager call on another stream: all give the same."""
    c = Case("mixed", [8, 1, 16, 32], [1, 0, 0, 1], 20000, "bf16", True, 1.0, 15)
    want = c.oracle()
    p, d = c.problem()
    calls = [va.AcceptCall(p, d, 2) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for call in calls:
            call()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for g, out in graphs:
        for t in out.values():
            t.fill_(-5)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert np.array_equal(out["accepted_nodes"].cpu().numpy(), want[1])
        assert np.array_equal(out["next_token"].cpu().numpy(), want[3])
