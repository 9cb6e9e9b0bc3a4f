"""Windowed verify attention: every output of a sequence that fails, and of
those beside it, by every kernel, joined in a cluster and merged."""
import dataclasses

import numpy as np
import pytest

import oracle.step_oracle as so
import synthetic as sy
from window_util import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verify_kv_gb300 as va  # noqa: E402
from test_gpu_window import make  # noqa: E402

# (cache, heads, KV heads, D, rows of a sequence, flags): few rows, row tiles, the 128-row kernel, CUDA cores.
KERNELS = [("bf16", 8, 2, 64, 4, 0), ("q8_0", 4, 1, 128, 4, 0), ("bf16", 5, 1, 256, 3, 0), ("bf16", 4, 1, 64, 8, 0),
           ("bf16", 4, 1, 64, 12, 0), ("bf16", 4, 1, 128, 8, 0), ("bf16", 6, 1, 256, 8, 0), ("q8_0", 6, 1, 256, 8, 0),
           ("f32", 4, 1, 64, 8, 0), ("bf16", 4, 2, 128, 8, va.FLAG_CUDA_CORES)]
WINDOW, SINKS = 600, 3


def launch(p, kv, mode, out=va.F32):
    """Outputs that hold 7 where the call does not write, and the status."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    shape = (p.total_rows, p.num_heads, kv.head_dim)
    o = torch.full(shape, 7.0, dtype=torch.float32 if out == va.F32 else torch.bfloat16, device="cuda")
    lse = torch.full(shape[:2], 7.0, device="cuda")
    va.verify_attn_window(p, kv, mode, va.Window(WINDOW, SINKS, out), o=o, lse=lse, status=st)
    return o.float().cpu().numpy(), lse.cpu().numpy(), int(st.item())


@pytest.fixture(scope="module")
def cases():
    made = {}

    def get(kernel):
        if kernel not in made:
            kv, heads, kvh, dim, rows, _ = kernel
            case = make(kv, heads, kvh, dim, [900, 640, 64], [rows] * 3, kinds=[0, 1, 0], mode="mixed", paged=True, seed=dim)
            made[kernel] = case, so.window_case(case, WINDOW, SINKS)
        return made[kernel]
    return get


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("splits", [1, 2, 7, 20])
@pytest.mark.parametrize("out", [va.F32, va.BF16])
def test_a_failed_sequence_is_nan(cases, kernel, splits, out):
    case, ref = cases(kernel)
    n, flags = kernel[4], kernel[5]
    for what, bit in (("block", va.DEV_BAD_BLOCK), ("ctx", va.DEV_CTX_OVERFLOW), ("negative ctx", va.DEV_CTX_OVERFLOW),
                      ("parent", va.DEV_BAD_PARENT)):
        p, kv, mode = va.upload(case, "cuda", num_splits=splits, flags=flags)
        lost = set(range(n, 2 * n))  # rows that have to be NaN
        if what == "block":  # within every row's window
            kv.block_table[1, 30] = kv.num_blocks
        elif what == "ctx":
            p.ctx_len[1] = 10 ** 6
        elif what == "negative ctx":
            p.ctx_len[1] = -1
        else:  # the rows below node 1 of the tree, itself among them
            p.parent[n + 1] = n
            par = p.parent[n:2 * n].tolist()
            lost = set()
            for j in range(n):
                a = j
                while a > 1 or a == 0 and par[0] >= 0:
                    a = par[a]
                if a == 1:
                    lost.add(n + j)
        o, lse, st = launch(p, kv, mode, out)
        assert st == bit, (what, hex(st))
        for r in lost:
            assert np.isnan(o[r]).all() and np.isnan(lse[r]).all(), (what, r)
        keep = [r for r in range(3 * n) if not n <= r < 2 * n]
        check(case, o[keep], lse[keep], (ref[0][keep], ref[1][keep]), out == va.BF16, what)


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("splits", [1, 2, 7, 20])
def test_a_bad_row_range_is_nan(cases, kernel, splits):
    case, _ = cases(kernel)
    n, flags = kernel[4], kernel[5]
    # One row too many in the second sequence; then one behind the launch's rows in the third.
    for cu, bad in (([0, n, 2 * n + 1, 3 * n], 1), ([0, n, 2 * n, 3 * n + 1], 2)):
        p, kv, mode = va.upload(case, "cuda", num_splits=splits, flags=flags)
        p.cu_rows = torch.tensor(cu, dtype=torch.int32, device="cuda")
        moved = dataclasses.replace(case, cu_rows=np.minimum(cu, 3 * n).astype(np.int32))
        ref = so.window_case(moved, WINDOW, SINKS)
        o, lse, st = launch(p, kv, mode)
        assert st == va.DEV_BAD_ROWS
        rows = np.arange(3 * n)
        lost = (rows >= cu[bad]) & (rows < cu[bad + 1])
        assert np.isnan(o[lost]).all() and np.isnan(lse[lost]).all()
        check(case, o[~lost], lse[~lost], (ref[0][~lost], ref[1][~lost]), False, str(cu))


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("splits", [1, 2, 20])
def test_sequences_of_no_rows(kernel, splits):
    """A padded batch: empty sequences first, between others and last."""
    kv, heads, kvh, dim, rows, flags = kernel
    case = make(kv, heads, kvh, dim, [50, 700, 90, 64, 300], [0, rows, 0, 1, 0], kinds=[1, 1, 0, 0, 1], mode="mixed",
                paged=True, seed=dim + 1)
    p, kvs, mode = va.upload(case, "cuda", num_splits=splits, flags=flags)
    o, lse, st = launch(p, kvs, mode)
    assert st == 0
    check(case, o, lse, so.window_case(case, WINDOW, SINKS), False)
