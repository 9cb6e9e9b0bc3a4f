"""Host-only checks of the latent entry points: every refusal comes before any
CUDA call."""
import ctypes

import pytest

import speculative_decoding_verify_kv_gb300 as va

torch = pytest.importorskip("torch")

FAKE = 1 << 20  # aligned, never dereferenced on the host path
BIG = 1 << 40


def fill(cls, base, kw):
    d = {**base, **{k: kw.pop(k) for k in list(kw) if k in base}}
    return cls(*[d[f] for f, _ in cls._fields_])


PROBLEM = dict(num_seqs=2, num_heads=16, q_dtype=va.BF16, q=FAKE, cu_rows=FAKE, ctx_len=FAKE, parent=FAKE,
               seq_kind=FAKE, total_rows=8, max_rows_per_seq=4, scale=0.1, num_splits=4, flags=0)
LATENT = dict(dtype=va.BF16, latent_dim=512, rope_dim=64, cache=FAKE, page_size=16, capacity=0, block_table=FAKE,
              max_blocks_per_seq=10, num_blocks=50)
PROMPT = dict(dtype=va.BF16, nope_dim=128, rope_dim=64, value_dim=128, kv=FAKE, k_rope=FAKE, k_rope_stride=576,
              cu_kv=FAKE, total_kv=100, causal=1)
ROWS = dict(num_rows=3, kv=FAKE, kv_stride=576, norm_weight=FAKE, norm_eps=1e-6, rope=FAKE, rope_positions=10,
            interleaved=0, position=FAKE, slot=FAKE, num_slots=100, num_heads=4, q_rope=FAKE, q_row_stride=256,
            q_head_stride=64, q=FAKE)
POOL = dict(num_seqs=4, max_blocks_per_seq=8, num_blocks=32, block_table=FAKE, ref_count=FAKE)
EXTEND = dict(ctx_len=FAKE, rows=FAKE, parent=FAKE, seq_kind=FAKE, max_rows=9)


def attend(fn, cls, base, mode=(), o=FAKE, lse=FAKE, ws=FAKE, ws_bytes=BIG, **kw):
    p, k = fill(va.VaProblem, PROBLEM, kw), fill(cls, base, kw)
    assert not kw, kw
    return fn(ctypes.byref(p), ctypes.byref(k), *mode, ws, ws_bytes, o, lse, None, None)


COMMON = [
    (dict(num_seqs=0), 1), (dict(num_heads=0), 1), (dict(total_rows=-1), 1), (dict(max_rows_per_seq=0), 1),
    (dict(num_splits=0), 1), (dict(num_splits=257), 2), (dict(num_heads=257), 2), (dict(num_seqs=65536), 2),
    (dict(q_dtype=7), 1), (dict(dtype=-1), 1), (dict(q_dtype=va.F32), 2), (dict(dtype=va.Q8_0), 2),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(flags=2), 1),
    (dict(cu_rows=None), 1), (dict(q=None), 1), (dict(q=FAKE + 8), 3), (dict(rope_dim=32), 2), (dict(o=None), 1),
    (dict(lse=None), 1), (dict(o=FAKE + 4), 3), (dict(ws=None), 4), (dict(ws_bytes=1000), 4), (dict(ws=FAKE + 16), 3),
    (dict(total_rows=1 << 30, num_heads=4), 2),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(mode=(3,)), 1), (dict(mode=(1,), parent=None), 1), (dict(mode=(2,), seq_kind=None), 1),
    (dict(latent_dim=128), 2), (dict(max_rows_per_seq=1025), 2), (dict(mode=(1,), max_rows_per_seq=33), 2),
    (dict(scale=0.0), 1), (dict(ctx_len=None), 1), (dict(cache=None), 1), (dict(cache=FAKE + 8), 3),
    (dict(page_size=8), 2), (dict(block_table=None), 1), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1),
    (dict(page_size=0, capacity=0), 1), (dict(page_size=0, capacity=24), 2), (dict(page_size=0, capacity=1 << 31), 2),
    (dict(max_blocks_per_seq=(1 << 26) + 1), 2),
])
def test_latent_refusals(kw, code):
    kw = dict(kw)
    assert attend(va.lib.verify_attn_latent, va.VaLatent, LATENT, kw.pop("mode", (0,)), **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(nope_dim=96), 2), (dict(value_dim=64), 2), (dict(max_rows_per_seq=(1 << 22) + 1), 2), (dict(total_kv=-1), 1),
    (dict(cu_kv=None), 1), (dict(causal=2), 1), (dict(kv=None), 1), (dict(k_rope=None), 1), (dict(k_rope_stride=32), 1),
    (dict(k_rope_stride=68), 3), (dict(kv=FAKE + 2), 3), (dict(k_rope=FAKE + 8), 3), (dict(total_kv=(1 << 30) + 1), 2),
])
def test_prompt_refusals(kw, code):
    assert attend(va.lib.verify_attn_latent_prompt, va.VaPrompt, PROMPT, **dict(kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_rows=-1), 1), (dict(num_heads=-1), 1), (dict(num_heads=257), 2), (dict(dtype=3), 1),
    (dict(dtype=va.Q8_0), 2), (dict(latent_dim=384), 2), (dict(rope_dim=128), 2), (dict(norm_eps=-1.0), 1),
    (dict(norm_eps=float("nan")), 1), (dict(rope_positions=0), 1), (dict(num_slots=0), 1), (dict(interleaved=2), 1),
    (dict(kv_stride=575), 1), (dict(cache=None), 1), (dict(kv=None), 1), (dict(rope=None), 1), (dict(position=None), 1),
    (dict(slot=None), 1), (dict(q_rope=None), 1), (dict(q=None), 1), (dict(q_head_stride=63), 1),
    (dict(q_row_stride=60), 1), (dict(cache=FAKE + 8), 3), (dict(q=FAKE + 8), 3), (dict(rope=FAKE + 4), 3),
    (dict(kv=FAKE + 1), 3), (dict(slot=FAKE + 4), 3), (dict(norm_weight=FAKE + 1), 3),
])
def test_append_refusals(kw, code):
    kw = dict(kw)
    k, n = fill(va.VaLatent, LATENT, kw), fill(va.VaLatentRows, ROWS, kw)
    assert not kw
    assert va.lib.verify_attn_latent_append(ctypes.byref(k), ctypes.byref(n), None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), 1), (dict(block_table=None), 1), (dict(ctx_len=None), 1), (dict(rows=None), 1),
    (dict(max_rows=-1), 1), (dict(max_rows=(1 << 30) + 1), 2), (dict(mode=-1), 1), (dict(mode=1, parent=None), 1),
    (dict(mode=2, seq_kind=None), 1), (dict(cu=None), 1), (dict(out=None), 1), (dict(out=FAKE + 4), 3),
    (dict(ws=None), 4), (dict(ws_bytes=10), 4), (dict(ws=FAKE + 64), 3),
])
def test_extend_refusals(kw, code):
    kw = dict(kw)
    mode, cu, out = kw.pop("mode", 0), kw.pop("cu", FAKE), kw.pop("out", FAKE)
    ws, n = kw.pop("ws", FAKE), kw.pop("ws_bytes", BIG)
    g, x = fill(va.VaPagePool, POOL, kw), fill(va.VaExtend, EXTEND, kw)
    assert not kw
    assert va.lib.verify_attn_pages_extend(ctypes.byref(g), ctypes.byref(x), mode, cu, out, out, out, ws, n, None,
                                           None) == code


def test_workspaces():
    size = lambda **kw: va.lib.va_latent_workspace_size(  # noqa: E731
        ctypes.byref(fill(va.VaProblem, PROBLEM, dict(kw))), ctypes.byref(fill(va.VaLatent, LATENT, {})))
    assert size(num_splits=1) == 0 and size(num_splits=0) == 0
    assert size(num_splits=3) == 3 * 8 * 16 * 514 * 4
    p = fill(va.VaProblem, PROBLEM, dict(num_splits=2))
    assert va.lib.va_latent_prompt_workspace_size(ctypes.byref(p), ctypes.byref(fill(va.VaPrompt, PROMPT, {}))) \
        == 2 * 8 * 16 * 130 * 4
    g = fill(va.VaPagePool, POOL, {})
    assert va.lib.verify_attn_pages_extend_workspace_size(ctypes.byref(g)) == 256


def test_no_rows_no_launch():
    assert attend(va.lib.verify_attn_latent, va.VaLatent, LATENT, (0,), total_rows=0, o=None) == 0
    assert attend(va.lib.verify_attn_latent_prompt, va.VaPrompt, PROMPT, total_rows=0, o=None) == 0
    k, n = fill(va.VaLatent, LATENT, {}), fill(va.VaLatentRows, ROWS, dict(num_rows=0, kv=None, q=None))
    assert va.lib.verify_attn_latent_append(ctypes.byref(k), ctypes.byref(n), None, None) == 0


def _latent_call(**kw):
    bf = torch.bfloat16
    d = dict(num_seqs=2, num_heads=3, q_dtype=va.BF16, q=torch.zeros(4, 3, 320, dtype=bf),
             cu_rows=torch.zeros(3, dtype=torch.int32), ctx_len=torch.zeros(2, dtype=torch.int32), parent=None,
             seq_kind=None, total_rows=4, max_rows_per_seq=2, scale=1.0)
    k = dict(dtype=va.BF16, latent_dim=256, rope_dim=64, cache=torch.zeros(2, 16, 320, dtype=bf), capacity=16)
    for name, v in kw.items():
        (d if name in d else k)[name] = v
    return va.LatentCall(va.Problem(**d), va.LatentKV(**k), 0)


@pytest.mark.parametrize("kw,error", [
    (dict(q=torch.zeros(4, 3, 320)), TypeError), (dict(q=torch.zeros(3, 3, 320, dtype=torch.bfloat16)), ValueError),
    (dict(cache=torch.zeros(2, 15, 320, dtype=torch.bfloat16)), ValueError), (dict(ctx_len=None), TypeError),
    (dict(cu_rows=torch.zeros(2, dtype=torch.int32)), ValueError), (dict(dtype=va.Q8_0), va.VaError),
    (dict(max_blocks_per_seq=1 << 32), ValueError), (dict(cache=torch.zeros(320, 32, dtype=torch.bfloat16).T), ValueError),
])
def test_bound_calls_check_tensors(kw, error):
    _latent_call()
    with pytest.raises(error):
        _latent_call(**kw)


def test_bound_append_checks():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    base = dict(kv=z(3, 330)[:, 5:325], position=z(3, t=torch.int32), slot=z(3, t=torch.int64),
                rope=z(7, 64, t=torch.float32), q_rope=z(3, 2, 80)[..., :64], q=z(3, 2, 320))
    make = lambda **kw: va.LatentAppendCall(va.LatentKV(va.BF16, 256, 64, z(5, 320)), va.LatentRows(**{**base, **kw}))  # noqa: E731
    make()
    for kw, error in [(dict(kv=z(3, 319)), ValueError), (dict(kv=z(320, 3).T), ValueError), (dict(q=None), ValueError),
                      (dict(slot=z(3, t=torch.int32)), TypeError), (dict(rope=z(7, 32, t=torch.float32)), ValueError),
                      (dict(q_rope=z(3, 3, 64)), ValueError), (dict(q=z(3, 2, 256)), ValueError),
                      (dict(kv=z(2, 320)), ValueError), (dict(norm_weight=z(255)), ValueError),
                      (dict(q=z(3, 2, 320, t=torch.float32)), TypeError)]:
        with pytest.raises(error):
            make(**kw)
