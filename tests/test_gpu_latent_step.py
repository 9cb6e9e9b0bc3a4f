"""A serving loop over a latent cache: prompt segments in, drafted trees verified,
the accepted path kept, pages given back (GB300)."""
import numpy as np
import pytest

from latent_util import BF16_LSE, HALF_BF16, TYPES, check, torch_dtype

import speculative_decoding_verify_kv_gb300 as va
from oracle import latent_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LATENT, HEADS, VOCAB, BLOCKS, WIDTH = 512, 8, 40, 60, 576


class Loop:
    def __init__(self, kind, seqs, seed):
        self.kind, self.dt = kind, torch_dtype(kind)
        self.g = torch.Generator().manual_seed(seed)
        self.r = np.random.default_rng(seed)
        self.table = torch.full((seqs, 12), -1, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(BLOCKS, dtype=torch.int32, device="cuda")
        self.pool = va.PagePool(self.table, self.ref)
        self.cache = torch.full((BLOCKS, 16, WIDTH), float("nan"), dtype=self.dt, device="cuda")
        self.kv = va.LatentKV(TYPES[kind], LATENT, 64, self.cache, page_size=16, block_table=self.table,
                              max_blocks_per_seq=12, num_blocks=BLOCKS)
        self.ctx = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        angle = torch.arange(200)[:, None] * 10000.0 ** (-torch.arange(32) / 32.0)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.weight = (1 + 0.1 * torch.randn(LATENT, generator=self.g)).to(self.dt).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.model = [np.zeros((0, WIDTH)) for _ in range(seqs)]  # what each sequence's cache holds, in 64 bits

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g).to(self.dt).cuda()

    def step(self, rows, mode=0, parent=None, kind=None):
        """Pages, slots and cache rows of a step, then its attention; returns what the step made."""
        total = int(sum(rows))
        dev = lambda a, t: None if a is None else torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
        parent, kind = dev(parent, torch.int32), dev(kind, torch.uint8)
        at = va.verify_attn_pages_extend(self.pool, self.ctx, dev(rows, torch.int32), total, mode, parent=parent,
                                         seq_kind=kind, status=self.status)
        new, q = self.rand(total, WIDTH), self.rand(total, HEADS, WIDTH)
        va.verify_attn_latent_append(self.kv, va.LatentRows(new, at["position"], at["slot"], self.rope,
                                                            norm_weight=self.weight, q_rope=q[..., LATENT:], q=q),
                                     status=self.status)
        p = va.Problem(num_seqs=len(rows), num_heads=HEADS, q_dtype=TYPES[self.kind], q=q, cu_rows=at["cu_rows"],
                       ctx_len=self.ctx, parent=parent, seq_kind=kind, total_rows=total, max_rows_per_seq=max(rows),
                       scale=0.07)
        p.num_splits = va.latent_splits(p, self.kv)
        out = va.verify_attn_latent(p, self.kv, mode, status=self.status)
        return at, new, q, p, out

    def rows64(self, new, position):
        """What append writes, in 64 bits."""
        cache = np.zeros((len(new), WIDTH))
        return lo.append(cache, new.double().cpu().numpy(), position, np.arange(len(new)), self.rope.double().cpu().numpy(),
                         self.weight.double().cpu().numpy())[0]

    def held(self, s, count):
        t = np.arange(count)
        page = self.table[s].cpu().numpy()[t // 16]
        return self.cache.double().cpu().numpy()[page, t % 16]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_loop(kind):
    loop = Loop(kind, 3, 5)
    # Prompt segments, one request not there yet.
    for rows in ([37, 20, 0], [5, 0, 16]):
        at, new, q, p, out = loop.step(rows)
        cu, pos = at["cu_rows"].cpu().numpy(), at["position"].cpu().numpy()
        made = loop.rows64(new, pos)
        for s, n in enumerate(rows):
            loop.model[s] = np.concatenate([loop.model[s], made[cu[s]:cu[s + 1]]])
        check(out, lo.latent(q.double().cpu().numpy(), loop.held, cu, loop.ctx.cpu().numpy(), 0.07, LATENT), kind)
        loop.ctx += torch.tensor(rows, dtype=torch.int32, device="cuda")
    step = 2.0 ** -23 if kind == "f32" else HALF_BF16
    for _ in range(3):
        # Drafted trees and a direct row; the target accepts a path of each.
        rows, kinds = [6, 1, 9], [1, 0, 1]
        parent = [-1] + [int(loop.r.integers(j)) for j in range(1, 6)] + [-1] + [-1] + [int(loop.r.integers(j)) for j in range(1, 9)]
        ctx = loop.ctx.cpu().numpy()
        at, new, q, p, out = loop.step(rows, 2, parent, kinds)
        cu = at["cu_rows"].cpu().numpy()
        check(out, lo.latent(q.double().cpu().numpy(), loop.held, cu, ctx, 0.07, LATENT, kinds, np.array(parent)), kind)
        total = int(cu[-1])
        taken = va.verify_attn_accept(p, va.Draft(torch.zeros(total, VOCAB, device="cuda"), VOCAB,
                                                  torch.randint(VOCAB, (total,), generator=loop.g, dtype=torch.int32).cuda(),
                                                  torch.rand(total, generator=loop.g).cuda() * 0.03, torch.rand(3).cuda(),
                                                  logits_dtype=va.F32), 2, status=loop.status)
        n, nodes = taken["accepted_len"], taken["accepted_nodes"]
        # The accepted rows once more, to the slots behind the context: their positions are the same.
        row = torch.arange(total, device="cuda")
        start = at["cu_rows"][at["row_seq"].long()].long()
        keep = nodes >= 0
        slot = torch.full((total,), -1, dtype=torch.int64, device="cuda")
        slot[(start + nodes)[keep].long()] = at["slot"][row[keep]]
        va.verify_attn_latent_append(loop.kv, va.LatentRows(new, at["position"], slot, loop.rope, norm_weight=loop.weight),
                                     status=loop.status)
        made = loop.rows64(new, at["position"].cpu().numpy())
        for s in range(3):
            path = nodes.cpu().numpy()[cu[s]:cu[s + 1]][:int(n[s])]
            assert len(path) >= 1
            loop.model[s] = np.concatenate([loop.model[s], made[cu[s] + path]])
        loop.ctx += n
        for s in range(3):
            want = loop.model[s]
            assert int(loop.ctx[s]) == len(want)
            got = loop.held(s, len(want))
            assert (np.abs(got - want) <= step * np.abs(want) + 3e-6 * (1 + np.abs(want))).all()
    assert loop.status.item() == 0
    # Give everything back.
    seq = torch.arange(3, dtype=torch.int32, device="cuda")
    va.verify_attn_pages_free(loop.pool, seq, torch.zeros_like(seq), torch.full_like(seq, 12), status=loop.status)
    assert loop.status.item() == 0 and not loop.ref.any() and (loop.table == -1).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_both_forms(kind):
    """A segment in the expanded form, and its rows in the absorbed form over the
    cache, are one attention; weights and their products in 64 bits."""
    g = torch.Generator().manual_seed(3)
    dt, heads, nope, ctx, n = torch_dtype(kind), 4, 128, 150, 33
    keys = ctx + n
    rows = torch.randn(keys, WIDTH, generator=g).to(dt).cuda()
    wk, wv = (torch.randn(heads, nope, LATENT, generator=g).double().cuda() / LATENT ** 0.5 for _ in range(2))
    q = torch.randn(n, heads, nope + 64, generator=g).to(dt).cuda()
    c = rows[:, :LATENT].double()
    kv = torch.cat([torch.einsum("hdl,tl->thd", w, c) for w in (wk, wv)], 2).to(dt).contiguous()
    absorbed = torch.cat([torch.einsum("nhd,hdl->nhl", q[..., :nope].double(), wk), q[..., nope:].double()], 2).to(dt)
    one = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    p = va.Problem(num_seqs=1, num_heads=heads, q_dtype=TYPES[kind], q=q, cu_rows=one(0, n), ctx_len=one(ctx), parent=None,
                   seq_kind=None, total_rows=n, max_rows_per_seq=n, scale=0.07)
    e, lse_e = va.verify_attn_latent_prompt(p, va.PromptKV(TYPES[kind], nope, 64, nope, kv, rows[:, LATENT:], one(0, keys)))
    cache = torch.zeros(1, -(-keys // 16) * 16, WIDTH, dtype=dt, device="cuda")
    cache[0, :keys] = rows
    pa = va.Problem(**{**vars(p), "q": absorbed})
    o, lse_a = va.verify_attn_latent(pa, va.LatentKV(TYPES[kind], LATENT, 64, cache, capacity=cache.shape[1]), 0)
    got = torch.einsum("nhl,hvl->nhv", o.double(), wv)
    if kind == "f32":
        # Rounding keys, values and queries to fp32 (2^-24 each) moves scores of some 10 by 1e-6.
        assert (lse_e - lse_a).abs().max() <= 5e-5 and (got - e).norm() <= 5e-5 * e.double().norm()
    else:
        # bf16 keys and absorbed queries: each score is off by 2^-9 of sqrt(sum of squares of its products),
        # some 1.5 for these; weights by as much, o by that and its own and v's rounding.
        assert (lse_e - lse_a).abs().max() <= 0.05 + BF16_LSE and (got - e).norm() <= 0.03 * e.double().norm()


def test_append_and_extend_on_another_stream():
    loop = Loop("bf16", 2, 9)
    rows = torch.tensor([30, 7], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    at = va.verify_attn_pages_extend(loop.pool, loop.ctx, rows, 40, stream=side)
    new = loop.rand(40, WIDTH)
    side.wait_stream(torch.cuda.current_stream())
    va.verify_attn_latent_append(loop.kv, va.LatentRows(new, at["position"], at["slot"], loop.rope), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert at["cu_rows"].tolist() == [0, 30, 37] and at["slot"][37:].tolist() == [-1] * 3
    flat = loop.cache.view(-1, WIDTH)
    assert torch.equal(flat[at["slot"][:37], :LATENT], new[:37, :LATENT])
    assert flat.isnan().any(1).sum() == flat.shape[0] - 37
