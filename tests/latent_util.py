"""Seeded inputs of the latent operators and their comparison with the oracle."""
from __future__ import annotations

import numpy as np

import speculative_decoding_verify_kv_gb300 as va

# Largest relative step of a rounding to bf16.
HALF_BF16 = 2.0 ** -8
TYPES = {"f32": va.F32, "bf16": va.BF16}
MODES = {"chain": 0, "tree": 1, "mixed": 2}

# fp32 results: a score is a sum of up to 576 products, whose roundings add up
# like a random walk: sqrt(576) 2^-24 times partial sums of some 6 in size,
# 9e-6 (natural units; the whole of it would stand in lse, and as a relative
# error in each weight).  o and lse are allowed twice that.
F32_O, LSE = 2e-5, 2e-5
# bf16 tensors, scores on the tensor cores, whose sums round towards zero:
# 576 2^-23 of partial sums of some 6, no more than 4e-4; half of it, since
# partial sums only grow to that, and products of one step are added first.
BF16_LSE = 2e-4


def torch_dtype(kind):
    import torch
    return torch.float32 if kind == "f32" else torch.bfloat16


def tree_parents(r, rows, kinds):
    out = []
    for n, k in zip(rows, kinds):
        out += [(-1 if j == 0 or r.random() < 0.1 else int(r.integers(j))) if k else j - 1 for j in range(n)]
    return np.array(out or [0], np.int32)


class Latent:
    """A latent cache with rows on it, on the GPU and for the oracle."""

    def __init__(self, kind, heads, latent, ctx, rows, mode="chain", paged=True, seed=0, scale=0.07, splits=1, pad=0,
                 device="cuda", extra_pages=3):
        import torch
        r = np.random.default_rng(seed)
        self.kind, self.heads, self.latent, self.mode, self.scale = kind, heads, latent, mode, scale
        seqs, width, dt = len(ctx), latent + 64, torch_dtype(kind)
        self.kinds = [1 if mode == "tree" or (mode == "mixed" and i % 2) else 0 for i in range(seqs)]
        self.ctx, self.cu = np.array(ctx, np.int32), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.parent = tree_parents(r, rows, self.kinds)
        total = int(self.cu[-1])
        g = torch.Generator().manual_seed(seed + 1)
        q = torch.randn(total + pad, heads, width, generator=g).to(dt)
        need = [-(-(c + n) // 16) for c, n in zip(ctx, rows)]
        self.table = None
        if paged:
            blocks = sum(need) + extra_pages
            order = r.permutation(blocks)
            self.table = np.full((seqs, max(need + [1])), -1, np.int32)
            at = 0
            for i, h in enumerate(need):
                self.table[i, :h] = order[at:at + h]
                at += h
            cache = torch.randn(blocks, 16, width, generator=g).to(dt)
            free = order[at:]
            cache[free] = float("nan")
            for i, (c, n) in enumerate(zip(ctx, rows)):  # what stands behind the last row is nobody's
                if (c + n) % 16:
                    cache[self.table[i, need[i] - 1], (c + n) % 16:] = float("nan")
            shape = dict(page_size=16, block_table=torch.from_numpy(self.table).to(device),
                         max_blocks_per_seq=self.table.shape[1], num_blocks=blocks)
        else:
            capacity = max(need + [1]) * 16 + 16
            cache = torch.randn(seqs, capacity, width, generator=g).to(dt)
            for i, (c, n) in enumerate(zip(ctx, rows)):
                cache[i, c + n:] = float("nan")
            shape = dict(capacity=capacity)
        self.q64, self.cache64 = q.double().numpy(), cache.double().numpy()
        self.q = q.to(device)
        self.kv = va.LatentKV(TYPES[kind], latent, 64, cache.to(device), **shape)
        dev = lambda a, t=torch.int32: torch.from_numpy(np.asarray(a)).to(t).to(device)  # noqa: E731
        self.p = va.Problem(num_seqs=seqs, num_heads=heads, q_dtype=TYPES[kind], q=self.q, cu_rows=dev(self.cu),
                            ctx_len=dev(self.ctx), parent=dev(self.parent), seq_kind=dev(self.kinds, torch.uint8),
                            total_rows=total, max_rows_per_seq=max(1, *rows) if rows else 1, scale=scale,
                            num_splits=splits)
        self.mode_code = MODES[mode]
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def rows_of(self, s, count):
        if self.table is None:
            return self.cache64[s, :count]
        return self.cache64[self.table[s, :-(-count // 16)]].reshape(-1, self.latent + 64)[:count]

    def oracle(self):
        from oracle import latent_oracle as lo
        return lo.latent(self.q64, self.rows_of, self.cu, self.ctx, self.scale, self.latent, self.kinds, self.parent)

    def run(self, **kw):
        return va.verify_attn_latent(self.p, self.kv, self.mode_code, status=self.status, **kw)


class Prompt:
    """Prompt segments over expanded keys, on the GPU and for the oracle."""

    def __init__(self, kind, heads, dim, rows, keys, seed=0, causal=True, splits=1, stride=64, scale=0.0, flags=0):
        import torch
        self.kind, self.dim, self.causal = kind, dim, causal
        dt, total, kt = torch_dtype(kind), int(sum(rows)), int(sum(keys))
        self.cu, self.cu_kv = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (rows, keys))
        g = torch.Generator().manual_seed(seed + 1)
        q = torch.randn(total, heads, dim + 64, generator=g).to(dt)
        kv = torch.randn(kt, heads, 2 * dim, generator=g).to(dt)
        wide = torch.randn(kt, stride, generator=g).to(dt)
        self.q64, self.kv64 = q.double().numpy(), kv.double().numpy()
        self.kr64 = wide[:, stride - 64:].double().numpy()
        self.scale = scale or 1.0 / np.sqrt(dim + 64)
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.kv = va.PromptKV(TYPES[kind], dim, 64, dim, kv.cuda(), wide.cuda()[:, stride - 64:], dev(self.cu_kv))
        self.p = va.Problem(num_seqs=len(rows), num_heads=heads, q_dtype=TYPES[kind], q=q.cuda(), cu_rows=dev(self.cu),
                            ctx_len=None, parent=None, seq_kind=None, total_rows=total,
                            max_rows_per_seq=max(1, *rows) if rows else 1, scale=scale, num_splits=splits, flags=flags)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def oracle(self):
        from oracle import latent_oracle as lo
        return lo.prompt(self.q64, self.kv64, self.kr64, self.cu, self.cu_kv, self.scale, self.dim, self.causal)

    def run(self, **kw):
        return va.verify_attn_latent_prompt(self.p, self.kv, causal=self.causal, status=self.status, **kw)


def check(got, want, kind):
    """o and lse against the oracle's.  bf16: a weight is rounded by at most
    2^-8 of itself, and so is o, so an element is off by at most 2^-8 (sum p
    |v| + |o|), and by the scores' part as in fp32."""
    o, lse = (t.double().cpu().numpy() for t in got)
    O, L, A = want
    o, lse = o[:len(L)], lse[:len(L)]
    none = np.isneginf(L)
    assert np.isneginf(lse[none]).all() and (o[none] == 0).all()
    assert np.isfinite(o).all() and np.isfinite(lse[~none]).all()
    if none.all():
        return 0.0, 0.0
    dl = np.abs(lse - np.where(none, 0, L))[~none].max()
    rel = np.linalg.norm(o - O) / np.linalg.norm(O)
    if kind == "f32":
        assert rel <= F32_O and dl <= LSE, (rel, dl)
    else:
        assert dl <= BF16_LSE, dl
        room = HALF_BF16 * (1 + HALF_BF16) * (A + np.abs(O)) + 2 * BF16_LSE * A + 1e-6
        assert (np.abs(o - O) <= room).all(), float((np.abs(o - O) / room).max())
        # Two roundings of at most 2^-8, spread evenly: sqrt(2 / 3) 2^-8 where all
        # weight is on one token, less elsewhere.
        assert rel <= 3.2e-3, rel
    return rel, dl
