"""Helpers of the windowed-attention tests."""
import dataclasses

import numpy as np

import oracle.step_oracle as so
import synthetic as sy


def poison_unseen(case, window, sinks, entry=-1):
    """The case with NaN in every cached token that no row sees, and with the
    block-table entries of pages without a visible token set to `entry`."""
    k, v = case.k.copy(), case.v.copy()
    table = None if case.block_table is None else case.block_table.copy()
    poison = sy._poison_row(case.kv_dtype, case.k.shape[-1])
    for s, seen in enumerate(so.seen_tokens(case, window, sinks)):
        ctx, n = int(case.ctx_len[s]), int(case.cu_rows[s + 1] - case.cu_rows[s])
        for t in range(ctx + n):
            if t in seen:
                continue
            for h in range(case.num_kv_heads):
                i = sy._cache_index(case, s, h, t)
                k[i] = poison
                v[i] = poison
        if table is not None:
            for pg in range(table.shape[1]):
                if not any(t in seen for t in range(16 * pg, 16 * pg + 16)):
                    table[s, pg] = entry
    return dataclasses.replace(case, k=k, v=v, block_table=table)


# |O - oracle| allowed per cache type, for |V| up to vmax: fp32 sums and
# exponentials of up to some thousand terms; bf16 caches carry P in 16 bits
# (hi + lo: off by at most 2^-17) and sum in fp32; Q8_0 caches round P and V
# to fp16 (2^-11 each, the half step).
def o_bound(case, out_bf16, ref):
    vmax = {"f32": 6.0, "bf16": 6.0, "q8_0": 2.6}[case.kv_dtype]
    rel = {"f32": 2.0 ** -17, "bf16": 2.0 ** -15, "q8_0": 2.0 ** -10}[case.kv_dtype]
    return vmax * rel + (np.abs(ref) * 2.0 ** -8 if out_bf16 else 0.0)


LSE_BOUND = 1e-4


def check(case, o, lse, ref, out_bf16, what=""):
    O, L = ref
    assert np.isfinite(o).all() and np.isfinite(lse).all(), what
    over = np.abs(o - O) - o_bound(case, out_bf16, O)
    assert over.max() <= 0, (what, float(over.max()), float(np.abs(o - O).max()))
    assert np.abs(lse - L).max() <= LSE_BOUND, (what, float(np.abs(lse - L).max()))
