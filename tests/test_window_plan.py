"""The most chunks of a windowed call, as the header states them, read from its
workspace: chunks x rows x heads x (D + 2) floats.  No GPU."""
import pytest

import speculative_decoding_verify_kv_gb300 as va
from test_step_abi import _window


def chunks(window, out, splits, rows, kv=va.BF16, pages=1 << 16):
    size = _window(w=(window, 4, out), fn="va_window_workspace_size",
                   p=dict(num_splits=splits, max_rows_per_seq=rows, total_rows=64, q_dtype=va.F32 if kv == va.F32 else va.BF16),
                   kv=dict(dtype=kv, max_blocks_per_seq=pages, num_blocks=1 << 20))
    per = 64 * 8 * 130 * 4
    assert size and size % per == 0
    return size // per


@pytest.mark.parametrize("window,most", [(1000, 2), (2000, 2), (2100, 2), (4000, 2), (9000, 5), (500000, 245),
                                         (524288, 256), (1 << 30, 256)])
@pytest.mark.parametrize("kv", [va.BF16, va.Q8_0])
def test_fp32_outputs_of_the_128_row_kernel(window, most, kv):
    """A chunk per 2,048 tokens at least (what the rows may see beyond the
    window counted in), 256 at most; bf16 outputs keep what was asked for."""
    assert chunks(window, va.F32, 2, 16, kv) == most
    assert chunks(window, va.BF16, 2, 16, kv) == 2
    assert chunks(window, va.F32, 256, 16, kv) == 256


@pytest.mark.parametrize("window", [100, 9000, 1 << 30])
def test_other_kernels_keep_what_was_asked_for(window):
    for out in (va.F32, va.BF16):
        assert chunks(window, out, 2, 4) == 2            # 16 rows per KV head
        assert chunks(window, out, 2, 8) == 2            # 32: row tiles at D = 128
        assert chunks(window, out, 2, 200, va.F32) == 2  # CUDA cores


def test_a_short_cache_bounds_the_chunks():
    assert chunks(1 << 30, va.F32, 1, 16, pages=200) == 2  # 3,200 tokens
