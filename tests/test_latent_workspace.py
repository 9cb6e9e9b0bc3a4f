"""Workspaces of the latent operators by the recommended chunk counts: partials that
can exist, not a slot for every row and chunk (host only)."""
import ctypes

import pytest

import speculative_decoding_verify_kv_gb300 as va

FAKE = 1 << 20


def problem(dtype, heads, seqs, rows, splits=1):
    return va.VaProblem(**dict(num_seqs=seqs, num_heads=heads, q_dtype=dtype, q=FAKE, cu_rows=FAKE, ctx_len=FAKE,
                               total_rows=seqs * rows, max_rows_per_seq=rows, scale=0.1, num_splits=splits))


def latent(dtype, dim):
    return va.VaLatent(dtype=dtype, latent_dim=dim, rope_dim=64, cache=FAKE, page_size=16, block_table=FAKE,
                       max_blocks_per_seq=1000, num_blocks=5000)


def prompt(dtype, dim):
    return va.VaPrompt(dtype=dtype, nope_dim=dim, rope_dim=64, value_dim=dim, kv=FAKE, k_rope=FAKE, k_rope_stride=64,
                       cu_kv=FAKE, total_kv=1 << 20, causal=1)


@pytest.mark.parametrize("dtype", [va.F32, va.BF16])
@pytest.mark.parametrize("dim", [256, 512])
@pytest.mark.parametrize("heads,seqs,rows", [(128, 1, 300), (128, 1, 1024), (64, 4, 16), (128, 1, 200), (16, 64, 1), (5, 3, 7)])
def test_latent(dtype, dim, heads, seqs, rows):
    """Chunks fill the GPU once, so partials are no more than the CTAs' rows: 128 for
    each of some 150 SMs on the tensor cores, 16 for each of two a SM in fp32."""
    p, kv = problem(dtype, heads, seqs, rows), latent(dtype, dim)
    p.num_splits = va.lib.va_latent_splits(ctypes.byref(p), ctypes.byref(kv))
    need = va.lib.va_latent_workspace_size(ctypes.byref(p), ctypes.byref(kv))
    block = 16 if dtype == va.F32 else 128
    assert p.num_splits >= 1
    assert need <= p.num_splits * min(seqs * block, seqs * rows * heads) * (dim + 2) * 4 + 512
    assert need <= 160 * 128 * (dim + 2) * 4 + 512


@pytest.mark.parametrize("dtype", [va.F32, va.BF16])
@pytest.mark.parametrize("heads,seqs,rows", [(1, 1, 2048), (4, 2, 700), (2, 1, 1 << 18), (3, 5, 9)])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt(dtype, heads, seqs, rows, dim):
    p, kv = problem(dtype, heads, seqs, rows), prompt(dtype, dim)
    p.num_splits = va.lib.va_latent_prompt_splits(ctypes.byref(p), ctypes.byref(kv))
    need = va.lib.va_latent_prompt_workspace_size(ctypes.byref(p), ctypes.byref(kv))
    block = 16 if dtype == va.F32 else 128
    assert need <= p.num_splits * min(seqs * block, seqs * rows) * heads * (dim + 2) * 4 + 512


def test_any_count_is_no_more_than_before():
    """Partials never need more than a slot for every row and chunk."""
    for dtype, heads, seqs, rows, splits in [(va.BF16, 16, 60, 3, 5), (va.F32, 2, 9, 4, 256), (va.BF16, 256, 7, 1024, 256)]:
        p, kv = problem(dtype, heads, seqs, rows, splits), latent(dtype, 512)
        need = va.lib.va_latent_workspace_size(ctypes.byref(p), ctypes.byref(kv))
        assert 0 < need <= splits * seqs * rows * heads * 514 * 4 + 512
