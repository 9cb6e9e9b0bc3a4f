"""Host-only checks of the acceptance and page entry points: every refusal
comes before any CUDA call."""
import ctypes

import pytest

import speculative_decoding_verify_kv_gb300 as va

torch = pytest.importorskip("torch")

FAKE = 1 << 20  # aligned, never dereferenced on the host path


def _accept(mode=0, ws=FAKE, ws_bytes=1 << 40, out=(FAKE, FAKE, None, FAKE), **kw):
    p = dict(num_seqs=2, cu_rows=FAKE, parent=FAKE, seq_kind=FAKE, total_rows=8, max_rows_per_seq=4)
    d = dict(vocab=100, logits_dtype=va.BF16, logits=FAKE, logits_stride=100, draft_probs=None, draft_stride=0,
             tokens=FAKE, accept_u=FAKE, sample_u=FAKE, temperature=None)
    for k, v in kw.items():
        (p if k in p else d)[k] = v
    pc = va.VaProblem(p["num_seqs"], 1, va.BF16, None, p["cu_rows"], None, p["parent"], p["seq_kind"],
                      p["total_rows"], p["max_rows_per_seq"], 0.0, 1, 0)
    dc = va.VaDraft(*[d[f] for f, _ in va.VaDraft._fields_])
    return va.lib.verify_attn_accept(ctypes.byref(pc), ctypes.byref(dc), mode, ws, ws_bytes, *out, None, None), \
        va.lib.verify_attn_accept_workspace_size(ctypes.byref(pc), ctypes.byref(dc))


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), 1), (dict(total_rows=-1), 1), (dict(max_rows_per_seq=0), 1), (dict(cu_rows=None), 1),
    (dict(mode=3), 1), (dict(mode=1, parent=None), 1), (dict(mode=2, seq_kind=None), 1), (dict(vocab=0), 1),
    (dict(logits_stride=99), 1), (dict(draft_probs=FAKE, draft_stride=99), 1), (dict(logits_dtype=5), 1),
    (dict(logits=None), 1), (dict(tokens=None), 1), (dict(accept_u=None), 1), (dict(sample_u=None), 1),
    (dict(logits_dtype=va.Q8_0), 2), (dict(vocab=(1 << 20) + 1, logits_stride=1 << 21), 2),
    (dict(max_rows_per_seq=1025), 2), (dict(mode=1, max_rows_per_seq=33), 2), (dict(num_seqs=65536), 2),
    (dict(logits=FAKE + 1), 3), (dict(logits=FAKE + 2, logits_dtype=va.F32), 3),
    (dict(draft_probs=FAKE + 2, draft_stride=100), 3), (dict(ws_bytes=100), 4), (dict(ws=None), 4),
    (dict(ws=FAKE + 64), 3), (dict(out=(None, FAKE, None, FAKE)), 1), (dict(out=(FAKE, None, None, FAKE)), 1),
    (dict(out=(FAKE, FAKE, None, None)), 1),
])
def test_accept_refusals(kw, code):
    assert _accept(**kw)[0] == code


def test_accept_workspace():
    # One 16-byte record per row and piece of 4,096 values (a row may start 7 values past a boundary).
    size = lambda **kw: _accept(ws_bytes=0, **kw)[1]  # noqa: E731
    assert size(vocab=100, total_rows=8) == 256
    assert size(vocab=4089, logits_stride=4089, total_rows=64) == 1024
    assert size(vocab=4090, logits_stride=4090, total_rows=64) == 2048
    assert size(max_rows_per_seq=1) == 0 and size(vocab=0) == 0


def _pool(**kw):
    d = dict(num_seqs=4, max_blocks_per_seq=8, num_blocks=32, block_table=FAKE, ref_count=FAKE)
    d.update(kw)
    return va.VaPagePool(*[d[f] for f, _ in va.VaPagePool._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), 1), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1), (dict(block_table=None), 1),
    (dict(ref_count=None), 1), (dict(num_blocks=(1 << 30) + 1), 2), (dict(num_seqs=(1 << 30) + 1), 2), (dict(max_blocks_per_seq=(1 << 26) + 1), 2), (dict(block_table=FAKE + 2), 3),
    (dict(ref_count=FAKE + 1), 3),
])
def test_pool_refusals(kw, code):
    g = ctypes.byref(_pool(**kw))
    assert va.lib.verify_attn_pages_fork(g, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None, None) == code
    assert va.lib.verify_attn_pages_free(g, 1, FAKE, FAKE, FAKE, None, None) == code
    assert va.lib.verify_attn_pages_compact(g, FAKE, FAKE, None, FAKE, 1 << 30, None, None) == code
    assert va.lib.verify_attn_pages_workspace_size(g, 1) == 0


def test_plan_refusals():
    g = ctypes.byref(_pool())
    need = va.lib.verify_attn_pages_workspace_size(g, 3)
    assert need == 256  # 4 + 2 * 3 + 32 words
    fork = lambda n=1, a=FAKE, copies=FAKE, num=FAKE, ws=FAKE, b=1 << 30: va.lib.verify_attn_pages_fork(  # noqa: E731
        g, n, a, FAKE, FAKE, FAKE, copies, num, ws, b, None, None)
    assert fork(n=-1) == 1 and fork(a=None) == 1 and fork(copies=None) == 1 and fork(num=None) == 1
    assert fork(ws=None) == 4 and fork(b=255) == 4 and fork(ws=FAKE + 16) == 3 and fork(n=1 << 29) == 2
    assert va.lib.verify_attn_pages_free(g, -1, FAKE, FAKE, FAKE, None, None) == 1
    assert va.lib.verify_attn_pages_free(g, 1, None, FAKE, FAKE, None, None) == 1
    assert va.lib.verify_attn_pages_free(g, 0, None, None, None, None, None) == 0
    assert va.lib.verify_attn_pages_compact(g, None, FAKE, None, FAKE, 1 << 30, None, None) == 1
    assert va.lib.verify_attn_pages_compact(g, FAKE, None, None, FAKE, 1 << 30, None, None) == 1
    assert va.lib.verify_attn_pages_compact(g, FAKE, FAKE, None, FAKE, 16, None, None) == 4


def test_copy_refusals():
    def copy(pools=(FAKE,), n=None, bytes_=32, blocks=8, copies=FAKE, num=FAKE, most=4):
        a = (ctypes.c_void_p * max(1, len(pools)))(*pools)
        return va.lib.verify_attn_pages_copy(a, len(pools) if n is None else n, bytes_, blocks, copies, num, most,
                                             None, None)
    assert copy(n=-1) == 1 and copy(bytes_=0) == 1 and copy(blocks=0) == 1 and copy(most=-1) == 1
    assert copy(num=None) == 1 and copy(copies=None) == 1 and copy(pools=(FAKE, None)) == 1
    assert copy(bytes_=24) == 2 and copy(pools=(FAKE, FAKE + 8)) == 3
    assert copy(pools=()) == 0 and copy(most=0) == 0


def test_bound_calls_check_their_tensors():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    pool = va.PagePool(z(2, 4), z(16))
    with pytest.raises(TypeError):
        va.ForkCall(pool, z(1, dt=torch.int64), z(1), z(1), z(1))
    with pytest.raises(ValueError):
        va.ForkCall(pool, z(2), z(1), z(1), z(1))
    with pytest.raises(ValueError):
        va.ForkCall(va.PagePool(z(8), z(16)), z(1), z(1), z(1), z(1))
    with pytest.raises(ValueError):
        va.ForkCall(pool, z(2, 2).t()[0], z(2), z(2), z(2))
    with pytest.raises(ValueError):
        va.CompactCall(pool, copies=z(3, 2))
    with pytest.raises(ValueError, match="not on a GPU"):
        va.CompactCall(pool)()
    with pytest.raises(ValueError):
        va.PageCopyCall([], z(1, 2), z(1))
    with pytest.raises(ValueError):
        va.PageCopyCall([z(4, 8), z(4, 4)], z(1, 2), z(1))
    p = va.Problem(num_seqs=2, num_heads=1, q_dtype=va.BF16, q=None, cu_rows=z(3), ctx_len=None, parent=z(4),
                   seq_kind=z(2, dt=torch.uint8), total_rows=4, max_rows_per_seq=2)
    f = torch.float32
    good = dict(logits=z(4, 10, dt=torch.bfloat16), vocab=10, tokens=z(4), accept_u=z(4, dt=f), sample_u=z(2, dt=f))
    va.AcceptCall(p, va.Draft(**good), 0)
    for k, v in [("logits", z(4, 10, dt=f)), ("logits", z(39, dt=torch.bfloat16)), ("tokens", z(3)),
                 ("accept_u", z(4)), ("sample_u", z(1, dt=f)), ("draft_probs", z(39, dt=f)),
                 ("temperature", z(1, dt=f)), ("logits_dtype", va.Q8_0)]:
        with pytest.raises((TypeError, ValueError, va.VaError)):
            va.AcceptCall(p, va.Draft(**{**good, k: v}), 0)


def _window(w=(128, 4, va.F32), fn="verify_attn_window", p=None, kv=None, mode=0, ws=FAKE, b=1 << 40, o=FAKE, lse=FAKE):
    d = dict(num_seqs=2, num_heads=8, q_dtype=va.BF16, q=FAKE, cu_rows=FAKE, ctx_len=FAKE, parent=FAKE, seq_kind=FAKE,
             total_rows=8, max_rows_per_seq=4, scale=0.0, num_splits=2, flags=0)
    d.update(p or {})
    c = dict(dtype=va.BF16, num_kv_heads=2, head_dim=128, k=FAKE, v=FAKE, page_size=16, capacity=0, block_table=FAKE,
             max_blocks_per_seq=9, num_blocks=99, draft_k=None, draft_v=None)
    c.update(kv or {})
    pc, kc, wc = va.VaProblem(*d.values()), va.VaKV(*c.values()), va.VaWindow(*w)
    a = (ctypes.byref(pc), ctypes.byref(kc))
    if fn != "verify_attn_window":
        return getattr(va.lib, fn)(*a, ctypes.byref(wc))
    return va.lib.verify_attn_window(*a, mode, ctypes.byref(wc), ws, b, o, lse, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=(0, 4, 0)), 1), (dict(w=(-1, 4, 0)), 1), (dict(w=(8, -1, 0)), 1), (dict(w=(8, 0, 9)), 1),
    (dict(w=(8, 0, va.Q8_0)), 2), (dict(mode=7), 1), (dict(p=dict(num_seqs=0)), 1), (dict(kv=dict(head_dim=96)), 2),
    (dict(p=dict(q_dtype=va.F32)), 2), (dict(p=dict(num_splits=257)), 2), (dict(p=dict(num_seqs=65536)), 2), (dict(o=None), 1), (dict(lse=None), 1),
    (dict(o=FAKE + 8), 3), (dict(ws=None), 4), (dict(b=1000), 4), (dict(ws=FAKE + 16), 3), (dict(kv=dict(k=FAKE + 4)), 3),
])
def test_window_refusals(kw, code):
    assert _window(**kw) == code
    if "w" in kw:
        assert _window(w=kw["w"], fn="va_window_workspace_size") == 0
        assert _window(w=kw["w"], fn="va_window_splits") == 0


def test_window_workspace_and_splits():
    # slots * rows * heads * (D + 2) floats, each part a multiple of 256 bytes.
    assert _window(fn="va_window_workspace_size") == 2 * 8 * 8 * 130 * 4
    assert _window(fn="va_window_splits") == 1                       # 136 tokens
    assert _window(w=(4096, 0, 0), fn="va_window_splits") == 16
    assert _window(w=(4096, 0, 0), p=dict(num_seqs=300), fn="va_window_splits") == 1


def test_window_calls_check_their_tensors():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    p = lambda **kw: va.Problem(**{**dict(  # noqa: E731
        num_seqs=2, num_heads=4, q_dtype=va.BF16, q=z(3, 4, 64, dt=torch.bfloat16), cu_rows=z(3), ctx_len=z(2),
        parent=z(3), seq_kind=z(2, dt=torch.uint8), total_rows=3, max_rows_per_seq=2), **kw})
    kv = lambda **kw: va.KV(**{**dict(  # noqa: E731
        dtype=va.BF16, num_kv_heads=2, head_dim=64, k=z(5, 2, 16, 64, dt=torch.bfloat16),
        v=z(5, 2, 16, 64, dt=torch.bfloat16), page_size=16, block_table=z(2, 4), max_blocks_per_seq=4, num_blocks=5),
        **kw})
    w = va.Window(8, 1, va.BF16)
    call = va.WindowCall(p(), kv(), 0, w)
    assert call._out[0].dtype == torch.bfloat16
    with pytest.raises(ValueError, match="not on a GPU"):
        call()
    for bad in (dict(p=p(q=z(3, 4, 63, dt=torch.bfloat16))), dict(p=p(ctx_len=z(1))), dict(p=p(cu_rows=z(2))),
                dict(kv=kv(k=z(5, 2, 16, 63, dt=torch.bfloat16))), dict(kv=kv(block_table=z(7))),
                dict(kv=kv(draft_k=z(3, 2, 60, dt=torch.bfloat16), draft_v=z(3, 2, 64, dt=torch.bfloat16))),
                dict(w=va.Window(8, 1, va.Q8_0)), dict(o=z(3, 4, 64, dt=torch.float32)), dict(status=z(1, dt=torch.int64))):
        kw = {k: v for k, v in bad.items() if k not in ("p", "kv", "w")}
        with pytest.raises((TypeError, ValueError, va.VaError)):
            va.WindowCall(bad.get("p", p()), bad.get("kv", kv()), 0, bad.get("w", w), **kw)


def test_bound_calls_hold_the_tensors_they_were_given():
    """The argument objects may get other tensors later: the addresses are bound."""
    import gc
    import weakref
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    pool = va.PagePool(i32(-1, -1).view(1, 2), i32(0, 0))
    pools = [torch.zeros(2, 16)]
    call, free, copy = va.CompactCall(pool), va.FreeCall(pool, i32(0), i32(0), i32(1)), va.PageCopyCall(pools, i32(0, 1), i32(1))
    p = va.Problem(num_seqs=1, num_heads=1, total_rows=1, max_rows_per_seq=1, q=None, q_dtype=va.F32, cu_rows=i32(0, 1),
                   ctx_len=None, parent=None, seq_kind=None)
    draft = va.Draft(torch.zeros(1, 8), 8, i32(0), torch.zeros(1), torch.zeros(1), logits_dtype=va.F32)
    accept = va.AcceptCall(p, draft, 0)
    held = [weakref.ref(t) for t in (pool.block_table, pool.ref_count, pools[0], draft.logits, draft.tokens, p.cu_rows)]
    pool.block_table = pool.ref_count = draft.logits = draft.tokens = p.cu_rows = None
    pools.clear()
    gc.collect()
    assert all(r() is not None for r in held)
    del call, free, copy, accept
    gc.collect()
    assert all(r() is None for r in held)
