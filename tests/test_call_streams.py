"""Where a call on a given stream takes its buffers from: memory that the
allocator hands out belongs to the stream that was current then, whose earlier
work may still be using it.  Fake streams; no GPU."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verify_kv_gb300 as va
from speculative_decoding_verify_kv_gb300 import _calls


class Stream:
    def __init__(self, handle, capturing=False):
        self.cuda_stream, self.capturing, self.waited = handle, capturing, []

    def wait_stream(self, other):
        self.waited.append(other.cuda_stream)


@pytest.fixture
def world(monkeypatch):
    """The current stream is `home` unless another one is made current; what
    is allocated is noted with the stream that was current."""
    w = type("World", (), {})()
    w.home, w.now, w.allocated = Stream(7), None, []
    w.now = w.home

    @contextlib.contextmanager
    def stream(s):
        before, w.now = w.now, s
        yield
        w.now = before

    new = _calls._Call._new

    def noted(self, shape, dtype):
        w.allocated.append(w.now.cuda_stream)
        self._home = w.now.cuda_stream
        return new(self, shape, dtype)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(_calls, "_stream_of", lambda handle, device: {7: w.home}[handle])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.now.capturing)
    monkeypatch.setattr(_calls._Call, "_new", noted)
    return w


z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731


def arguments():
    bf, f = torch.bfloat16, torch.float32
    p = va.Problem(num_seqs=2, num_heads=4, q_dtype=va.BF16, q=z(3, 4, 64, dt=bf), cu_rows=z(3), ctx_len=z(2), parent=z(3),
                   seq_kind=z(2, dt=torch.uint8), total_rows=3, max_rows_per_seq=2)
    kv = va.KV(dtype=va.BF16, num_kv_heads=2, head_dim=64, k=z(5, 2, 16, 64, dt=bf), v=z(5, 2, 16, 64, dt=bf),
               page_size=16, block_table=z(2, 4), max_blocks_per_seq=4, num_blocks=5)
    draft = va.Draft(z(3, 10, dt=f), 10, z(3), z(3, dt=f), z(2, dt=f), logits_dtype=va.F32)
    pool = va.PagePool(z(2, 4), z(16))
    return {"window": (va.verify_attn_window, (p, kv, 0, va.Window(8)), 3),
            "accept": (va.verify_attn_accept, (p, draft, 0), 4),
            "fork": (va.verify_attn_pages_fork, (pool, z(1), z(1), z(1), z(1)), 3),
            "compact": (va.verify_attn_pages_compact, (pool,), 4)}


@pytest.mark.parametrize("name", sorted(arguments()))
@pytest.mark.parametrize("given", [False, True])
def test_a_call_in_one_go_allocates_on_its_stream(world, name, given):
    fn, args, buffers = arguments()[name]
    side = Stream(9)
    with pytest.raises(ValueError, match="not on a GPU"):  # raised by the call: everything is bound by then
        fn(*args, stream=side if given else None)
    assert world.allocated == [side.cuda_stream if given else world.home.cuda_stream] * buffers
    assert world.now is world.home


def test_a_bound_call_waits_once_for_the_stream_of_its_buffers(world):
    call = va.CompactCall(va.PagePool(z(2, 4), z(16)))
    side, other = Stream(9), Stream(11)
    for s in (side, side, other, world.home):
        call._order(s)
    assert side.waited == [7] and other.waited == [7] and world.home.waited == []


def test_a_captured_stream_waits_for_captured_work_only(world):
    call = va.CompactCall(va.PagePool(z(2, 4), z(16)))
    side = Stream(9, capturing=True)
    call._order(side)
    assert side.waited == []
    side.capturing = False  # the same stream, eager again
    call._order(side)
    assert side.waited == [7]
    world.home.capturing = True
    other = Stream(11, capturing=True)
    call._order(other)
    assert other.waited == [7]


def test_a_call_with_all_buffers_given_waits_for_nothing(world):
    pool = va.PagePool(z(2, 4), z(16))
    call = va.CompactCall(pool, copies=z(8, 2), num_copies=z(1), live_blocks=z(1), ws=z(1024, dt=torch.uint8))
    side = Stream(9)
    call._order(side)
    assert side.waited == [] and world.allocated == []


class Library:
    """Every entry point succeeds; the split plan has one slot."""
    def __getattr__(self, name):
        def call(*args):
            if name == "va_plan":
                args[3]._obj.slots = 1
            return 1000 if name == "va_workspace_size" else 0
        return call


@pytest.mark.parametrize("given", [False, True])
def test_verify_calls_allocate_on_their_stream(world, monkeypatch, given):
    """The unwindowed calls and the debug exports."""
    _, (p, kv, _, _), _ = arguments()["window"]
    side = Stream(9)
    made = []
    for name in ("empty", "full", "zeros"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, real=real, **k: made.append(world.now.cuda_stream) or real(*a, **k))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: made.append(("seen by", s.cuda_stream)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: world.now)
    monkeypatch.setattr(va, "lib", Library())
    monkeypatch.setattr(va, "_stream_handle", lambda s: None)
    kw = {"stream": side} if given else {}
    at = 9 if given else 7
    for call, buffers, outputs in ((lambda: va.verify_attn_chain(p, kv, **kw), 3, 2), (lambda: va.debug_row_map(p, 0, **kw), 2, 2),
                                   (lambda: va.debug_gather_index(p, kv, 0, 10, **kw), 1, 1),
                                   (lambda: va.debug_split_ranges(p, kv, 0, **kw), 1, 1)):
        made.clear()
        call()
        assert made == [at] * buffers + ([("seen by", 7)] * outputs if given else [])
    o, lse, ws = z(3, 4, 64), z(3, 4), z(1000)
    made.clear()
    va.verify_attn_chain(p, kv, o=o, lse=lse, ws=ws, **kw)
    assert made == []
