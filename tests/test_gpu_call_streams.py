"""Calls on a given stream beside earlier work of another stream on memory
that the allocator hands out again."""
import numpy as np
import pytest

import oracle.step_oracle as so
import synthetic as sy
from window_util import check as check_window

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verify_kv_gb300 as va  # noqa: E402
from test_gpu_accept import Case  # noqa: E402


def sizes(call):
    return [t.numel() * t.element_size() for t in call._own]


def busy_blocks(lengths):
    """Blocks of the sizes of a call's own buffers, dropped while the current
    stream, asleep for half a second, has yet to fill them; their addresses."""
    blocks = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in lengths for _ in range(2)]
    blocks[0].fill_(255)  # (loaded by now)
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)
    for b in blocks:
        b.fill_(255)
    return {b.data_ptr() for b in blocks}


def window():
    case = sy.make_case("streams", num_heads=8, num_kv_heads=2, head_dim=128, kv_dtype="bf16", q_dtype="bf16",
                        ctx=[3000, 500, 90], rows=[4, 1, 2], paged=True, seed=11)
    p, kv, mode = va.upload(case, "cuda", num_splits=20)  # (more chunks than a cluster joins: the workspace is used)
    ref = so.window_case(case, 2600, 4)

    def right(out):
        check_window(case, out[0].cpu().numpy(), out[1].cpu().numpy(), ref, False)
    return va.WindowCall, va.verify_attn_window, (p, kv, mode, va.Window(2600, 4)), right


def accept():
    c = Case("mixed", [8, 1, 16, 32], [1, 0, 0, 1], 20000, "bf16", True, 1.0, 15)
    p, d = c.problem()
    want = c.oracle()

    def right(out):
        for k, w in zip(("accepted_len", "accepted_nodes", "next_token"), (want[0], want[1], want[3])):
            assert np.array_equal(out[k].cpu().numpy(), w)
    return va.AcceptCall, va.verify_attn_accept, (p, d, 2), right


def fork():
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((3, 64), -1, dtype=torch.int32, device="cuda")
    table[0, :3] = torch.arange(3, device="cuda")
    ref = torch.zeros(1 << 16, dtype=torch.int32, device="cuda")
    ref[:3] = 1
    before = table.clone(), ref.clone()

    def right(out):
        assert table[1].tolist() == [0, 1, 3] + list(range(4, 41)) + [-1] * 24
        assert out[0].tolist() == [[2, 3]] and out[1].tolist() == [1]
        table.copy_(before[0]), ref.copy_(before[1])
    return va.ForkCall, va.verify_attn_pages_fork, (va.PagePool(table, ref), i32(0), i32(1), i32(40), i32(40)), right


def compact():
    table = torch.full((1, 64), -1, dtype=torch.int32, device="cuda")
    table[0, :40] = torch.arange(40000, 40040, device="cuda")
    ref = torch.zeros(1 << 16, dtype=torch.int32, device="cuda")
    ref[40000:40040] = 1
    before = table.clone(), ref.clone()

    def right(out):
        assert table[0].tolist() == list(range(40)) + [-1] * 24
        assert out[1].tolist() == [40] and out[2].tolist() == [40]
        assert out[0][:40].tolist() == [[40000 + i, i] for i in range(40)]
        table.copy_(before[0]), ref.copy_(before[1])
    return va.CompactCall, va.verify_attn_pages_compact, (va.PagePool(table, ref),), right


@pytest.mark.parametrize("make", [window, accept, fork, compact])
def test_a_call_in_one_go_does_not_write_into_another_streams_memory(make):
    call, function, args, right = make()
    side = torch.cuda.Stream()
    out = call(*args)()  # (loaded, and the sizes of its buffers)
    right(out)
    del out
    busy = busy_blocks(sizes(call(*args)))
    out = function(*args, stream=side)
    side.synchronize()
    for t in out.values() if isinstance(out, dict) else out:
        assert t.data_ptr() not in busy
    torch.cuda.synchronize()  # the fills are done
    right(out)


@pytest.mark.parametrize("make", [window, accept, fork, compact])
def test_a_bound_call_runs_behind_what_its_buffers_held(make):
    call, _, args, right = make()
    side = torch.cuda.Stream()
    right(call(*args)())
    busy = busy_blocks(sizes(call(*args)))
    bound = call(*args)
    assert {t.data_ptr() for t in bound._own} & busy  # its buffers are such blocks
    out = bound(side)
    torch.cuda.synchronize()
    right(out)


@pytest.mark.parametrize("make", [window, accept, fork, compact])
def test_outputs_dropped_while_the_current_stream_reads_them(make):
    """The outputs of a call on a given stream are not handed out to that
    stream's next call before the current stream's work on them is done."""
    call, function, args, right = make()
    side = torch.cuda.Stream()
    out = function(*args, stream=side)
    side.synchronize()
    right(out)
    where = {t.data_ptr() for t in (out.values() if isinstance(out, dict) else out)}
    for t in out.values() if isinstance(out, dict) else out:
        t.sum()  # (loaded by now)
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)
    for t in out.values() if isinstance(out, dict) else out:
        t.sum()
    del out, t
    again = function(*args, stream=side)
    assert not torch.cuda.current_stream().query()  # still asleep
    assert not where & {t.data_ptr() for t in (again.values() if isinstance(again, dict) else again)}
    side.synchronize()
    right(again)


@pytest.mark.parametrize("make", [window, accept])
def test_a_stream_that_captures(make):
    """The first call on a capturing stream, given as an argument, of a call
    bound before the capture and of one bound in it."""
    call, function, args, right = make()
    right(call(*args)())
    bound = call(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        first = bound(side)
        second = function(*args, stream=side)
    for out in (first, second):
        for t in out.values() if isinstance(out, dict) else out:
            t.zero_()
    g.replay()
    torch.cuda.synchronize()
    right(first)
    right(second)


def test_an_unwindowed_call_does_not_write_into_another_streams_memory():
    import oracle
    case = sy.mixed_tree_direct(ctx=[40, 300, 17, 130], direct=(0, 2), num_splits=2, seed=7)
    p, kv, mode = va.upload(case, "cuda")
    ref = oracle.verify_case(case)
    side = torch.cuda.Stream()
    ws = va.alloc_workspace(p, kv)
    out = va.verify_attn(p, kv, mode, ws=ws)
    check_window(case, out[0].cpu().numpy(), out[1].cpu().numpy(), ref, False)
    lengths = [t.numel() * t.element_size() for t in (ws, *out)]
    del ws, out
    busy = busy_blocks(lengths)
    out = va.verify_attn(p, kv, mode, stream=side)
    assert not {t.data_ptr() for t in out} & busy
    torch.cuda.synchronize()
    check_window(case, out[0].cpu().numpy(), out[1].cpu().numpy(), ref, False)
