"""Bound calls of the operators around a verify step: windowed verify
attention, acceptance of drafted tokens and the pages of a paged cache.

A serving loop makes the same call step after step over buffers that it
keeps.  Each ``...Call`` object checks its tensors, allocates what the
caller left out (outputs, workspace) and fills the C structs once; calling
it launches on the current stream (or the one given) and returns the output
tensors, which the next call of the same object overwrites.  The functions
of the C names bind and call in one go.  Two calls that may overlap in time
need two objects (the workspace is the object's).  A stream given to a call
is recorded with its tensors (they may be dropped before it gets there).  It
also waits for the earlier work of the stream that the object's own buffers
were allocated on (which still has to exist), whose memory they may be; a
function of a C name allocates them on the stream that it is given.  A
stream that captures waits for captured work only: what the replay runs
behind is the caller's.  One made current follows the rules of any PyTorch
operation.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import BF16, F32, KV, Q8_0, Problem, VaDraft, VaError, VaPagePool, VaWindow, _ptr, lib

_FLOAT = {F32: torch.float32, BF16: torch.bfloat16}


def _tensor(name, t, dtype, numel, device=None, optional=False):
    """Check one argument: a contiguous tensor of the type, with at least
    numel elements, on the given device."""
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, {numel} needed")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the other arguments on {device}")
    return t


def _i32(name, x):
    """A number for a 32-bit field: ctypes would cut it to that silently."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


# The current stream's handle without a Stream object around it (2.9 us of
# the 7 that a bound call took on the host).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_of(handle, device):
    """A stream object of a raw handle (0: the default stream)."""
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


def _capturing(stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _in_one_go(cls, stream, *args, **kw):
    """Bind a call and make it.  What it allocates belongs to the stream that
    it runs on (memory of another one may still be in use by that one's work),
    and the outputs are read on the stream that is current here."""
    if stream is None:
        return cls(*args, **kw)()
    with torch.cuda.stream(stream):
        call = cls(*args, **kw)
    out = call(stream)
    for t in _flat(out):
        t.record_stream(torch.cuda.current_stream(t.device))
    return out


def _flat(*todo):
    """The tensors of nested tuples, lists and dicts."""
    found, todo = [], list(todo)
    while todo:
        x = todo.pop()
        if isinstance(x, torch.Tensor):
            found.append(x)
        elif isinstance(x, (tuple, list)):
            todo.extend(x)
        elif isinstance(x, dict):
            todo.extend(x.values())
    return found


class _Call:
    """Arguments of one entry point, bound.  Subclasses fill ``_fn``,
    ``_args`` (all but the stream), ``_out``, ``_keep`` (every tensor whose
    address is bound) and ``device``."""
    _where = ""
    _own = ()  # buffers that the call allocated itself
    _home = None  # handle of the stream that they were allocated on
    _ordered = frozenset()  # handles of the streams that have waited for it

    def __call__(self, stream=None):
        dev = self.device
        if dev.type != "cuda":
            raise ValueError(f"{self._where}: tensors on {dev}, not on a GPU")
        index = torch.cuda.current_device()
        if index != dev.index:
            raise ValueError(f"{self._where}: tensors on {dev}, current device cuda:{index}")
        if stream is None:
            st = self._fn(*self._args, _current_stream(index))
        else:
            self._order(stream)
            st = self._fn(*self._args, stream.cuda_stream)
            for t in _flat(self._keep, self._own, self._out):  # may be freed with the call, before the stream gets to it
                t.record_stream(stream)
        if st:
            raise VaError(st, self._where)
        return self._out

    def _order(self, stream):
        """Once per stream: what ran on the memory of the call's own buffers
        before they were allocated comes before what this stream does there."""
        if self._home is None or stream.cuda_stream == self._home or stream.cuda_stream in self._ordered:
            return
        home = _stream_of(self._home, self.device)
        if _capturing(stream) != _capturing(home):
            return
        stream.wait_stream(home)
        if not _capturing(stream):
            self._ordered |= {stream.cuda_stream}

    def _new(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        self._own += (t,)
        if self._home is None and t.is_cuda:
            self._home = _current_stream(t.device.index)
        return t

    def _buffer(self, name, t, shape, dtype):
        n = 1
        for d in shape:
            n *= d
        if t is None:
            return self._new(shape, dtype)
        return _tensor(name, t, dtype, n, self.device)

    def _workspace(self, ws, need):
        if ws is None:
            return self._new(max(need, 256), torch.uint8)
        return _tensor("ws", ws, torch.uint8, need, self.device)


def _held(*holders):
    """The values of argument objects as they are now: the objects may be given
    other tensors later, the addresses are bound."""
    return tuple(t for h in holders for t in vars(h).values())


@dataclass
class Window:
    """Sliding window and first visible tokens of a windowed call (va_window)."""
    window: int
    sinks: int = 0
    o_dtype: int = F32

    def c(self) -> VaWindow:
        return VaWindow(_i32("window", self.window), _i32("sinks", self.sinks), self.o_dtype)


_ELEMENT = {F32: 4, BF16: 2}


def _row_bytes(kv: KV) -> int:
    return kv.head_dim // 32 * 34 if kv.dtype == Q8_0 else kv.head_dim * _ELEMENT.get(kv.dtype, 4)


def _check_bytes(name, t, need, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, the other arguments on {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if t.numel() * t.element_size() < need:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, {need} needed")


class WindowCall(_Call):
    """verify_attn_window.  Returns (o, lse)."""
    _where = "verify_attn_window"

    def __init__(self, p: Problem, kv: KV, mode: int, window: Window, *, ws=None, o=None, lse=None, status=None):
        self.device = dev = p.q.device
        rows, heads, dim = p.total_rows, p.num_heads, kv.head_dim
        _check_rows(p, mode, dev)
        _tensor("ctx_len", p.ctx_len, torch.int32, p.num_seqs, dev)
        _check_bytes("q", p.q, rows * heads * dim * _ELEMENT.get(p.q_dtype, 4), dev)
        if kv.page_size:
            _tensor("block_table", kv.block_table, torch.int32, p.num_seqs * kv.max_blocks_per_seq, dev)
            cells = kv.num_blocks * kv.page_size
        else:
            cells = p.num_seqs * kv.capacity
        for name, t in (("k", kv.k), ("v", kv.v)):
            _check_bytes(name, t, cells * kv.num_kv_heads * _row_bytes(kv), dev)
        for name, t in (("draft_k", kv.draft_k), ("draft_v", kv.draft_v)):
            if t is not None:
                _check_bytes(name, t, rows * kv.num_kv_heads * _row_bytes(kv), dev)
        _tensor("status", status, torch.int32, 1, dev, optional=True)
        if window.o_dtype not in _FLOAT:
            raise VaError(2, self._where)
        o = self._buffer("o", o, (rows, heads, dim), _FLOAT[window.o_dtype])
        lse = self._buffer("lse", lse, (rows, heads), torch.float32)
        pc, kc, wc = p.c(), kv.c(), window.c()
        ws = self._workspace(ws, int(lib.va_window_workspace_size(ctypes.byref(pc), ctypes.byref(kc),
                                                                  ctypes.byref(wc))))
        self._fn, self._out = lib.verify_attn_window, (o, lse)
        self._args = (ctypes.byref(pc), ctypes.byref(kc), mode, ctypes.byref(wc), _ptr(ws), ws.numel(), _ptr(o),
                      _ptr(lse), _ptr(status))
        self._keep = (_held(p, kv), ws, status, pc, kc, wc)


def verify_attn_window(p: Problem, kv: KV, mode: int, window: Window, *, stream=None, **kw):
    """Verify attention through a sliding window with a few first tokens that
    stay visible; returns (o, lse)."""
    return _in_one_go(WindowCall, stream, p, kv, mode, window, **kw)


def window_splits(p: Problem, kv: KV, window: Window) -> int:
    """A num_splits that fills the current GPU once (va_window_splits)."""
    return int(lib.va_window_splits(ctypes.byref(p.c()), ctypes.byref(kv.c()), ctypes.byref(window.c())))


@dataclass
class Draft:
    """Logits, proposals and random numbers of an acceptance step (va_draft)."""
    logits: object                  # [total_rows][logits_stride]
    vocab: int
    tokens: object                  # int32 [total_rows]
    accept_u: object                # float32 [total_rows]
    sample_u: object                # float32 [num_seqs]
    logits_dtype: int = BF16
    logits_stride: int = 0          # 0: vocab
    draft_probs: object = None      # float32 [total_rows][draft_stride]
    draft_stride: int = 0           # 0: vocab
    temperature: object = None      # float32 [num_seqs]

    def c(self) -> VaDraft:
        return VaDraft(_i32("vocab", self.vocab), self.logits_dtype, _ptr(self.logits), self.logits_stride or self.vocab,
                       _ptr(self.draft_probs), self.draft_stride or self.vocab, _ptr(self.tokens),
                       _ptr(self.accept_u), _ptr(self.sample_u), _ptr(self.temperature))


def _check_rows(p: Problem, mode: int, dev):
    _tensor("cu_rows", p.cu_rows, torch.int32, p.num_seqs + 1, dev)
    _tensor("parent", p.parent, torch.int32, p.total_rows if mode else 0, dev, optional=mode == 0)
    _tensor("seq_kind", p.seq_kind, torch.uint8, p.num_seqs if mode == 2 else 0, dev, optional=mode != 2)


class AcceptCall(_Call):
    """verify_attn_accept.  Returns a dict of accepted_len, accepted_nodes,
    next_token (and promote_len where given)."""
    _where = "verify_attn_accept"

    def __init__(self, p: Problem, draft: Draft, mode: int, *, accepted_len=None, accepted_nodes=None,
                 promote_len=None, next_token=None, ws=None, status=None):
        self.device = dev = draft.logits.device
        rows, seqs = p.total_rows, p.num_seqs
        _check_rows(p, mode, dev)
        if draft.logits_dtype not in _FLOAT:
            raise VaError(2, self._where)
        span = lambda stride: (rows - 1) * (stride or draft.vocab) + draft.vocab if rows else 0  # noqa: E731
        _tensor("logits", draft.logits, _FLOAT[draft.logits_dtype], span(draft.logits_stride), dev)
        _tensor("draft_probs", draft.draft_probs, torch.float32, span(draft.draft_stride), dev, optional=True)
        _tensor("tokens", draft.tokens, torch.int32, rows, dev)
        _tensor("accept_u", draft.accept_u, torch.float32, rows, dev)
        _tensor("sample_u", draft.sample_u, torch.float32, seqs, dev)
        _tensor("temperature", draft.temperature, torch.float32, seqs, dev, optional=True)
        _tensor("status", status, torch.int32, 1, dev, optional=True)
        _tensor("promote_len", promote_len, torch.int32, seqs, dev, optional=True)
        out = {"accepted_len": self._buffer("accepted_len", accepted_len, (seqs,), torch.int32),
               "accepted_nodes": self._buffer("accepted_nodes", accepted_nodes, (rows,), torch.int32),
               "next_token": self._buffer("next_token", next_token, (seqs,), torch.int32)}
        if promote_len is not None:
            out["promote_len"] = promote_len
        pc, dc = p.c(), draft.c()
        need = int(lib.verify_attn_accept_workspace_size(ctypes.byref(pc), ctypes.byref(dc)))
        ws = self._workspace(ws, need)
        self._fn, self._out = lib.verify_attn_accept, out
        self._args = (ctypes.byref(pc), ctypes.byref(dc), mode, _ptr(ws), ws.numel(), _ptr(out["accepted_len"]),
                      _ptr(out["accepted_nodes"]), _ptr(promote_len), _ptr(out["next_token"]), _ptr(status))
        self._keep = (_held(p, draft), ws, status, pc, dc)


def verify_attn_accept(p: Problem, draft: Draft, mode: int, *, stream=None, **kw):
    """Which drafted rows the target accepts, and the next token of each
    sequence (see verify_attn_accept in the header)."""
    return _in_one_go(AcceptCall, stream, p, draft, mode, **kw)


@dataclass
class PagePool:
    """Block table (int32 [num_seqs][max_blocks]) and reference counts
    (int32 [num_blocks]) of a paged cache, on the device."""
    block_table: object
    ref_count: object

    def c(self) -> VaPagePool:
        t = self.block_table
        return VaPagePool(_i32("block_table", t.shape[0]), _i32("block_table", t.shape[1]),
                          _i32("ref_count", self.ref_count.numel()), _ptr(t), _ptr(self.ref_count))


class _PageCall(_Call):
    def _bind(self, pool: PagePool, status):
        if not isinstance(pool.block_table, torch.Tensor) or pool.block_table.dim() != 2:
            raise ValueError("block_table: expected a tensor of two dimensions")
        self.device = pool.block_table.device
        _tensor("block_table", pool.block_table, torch.int32, 1)
        _tensor("ref_count", pool.ref_count, torch.int32, 1, self.device)
        _tensor("status", status, torch.int32, 1, self.device, optional=True)
        return pool.c()

    def _commands(self, **kw):
        n = None
        for name, t in kw.items():
            _tensor(name, t, torch.int32, 0, self.device)
            if n is not None and t.numel() != n:
                raise ValueError(f"{name}: {t.numel()} commands, the others have {n}")
            n = _i32(name, t.numel())
        return n


class ForkCall(_PageCall):
    """verify_attn_pages_fork.  Returns (copies, num_copies)."""
    _where = "verify_attn_pages_fork"

    def __init__(self, pool: PagePool, src, dst, length, pages, *, copies=None, num_copies=None, ws=None,
                 status=None):
        c = self._bind(pool, status)
        n = self._commands(src=src, dst=dst, length=length, pages=pages)
        copies = self._buffer("copies", copies, (n, 2), torch.int32)
        num_copies = self._buffer("num_copies", num_copies, (1,), torch.int32)
        ws = self._workspace(ws, int(lib.verify_attn_pages_workspace_size(ctypes.byref(c), n)))
        self._fn, self._out = lib.verify_attn_pages_fork, (copies, num_copies)
        self._args = (ctypes.byref(c), n, _ptr(src), _ptr(dst), _ptr(length), _ptr(pages), _ptr(copies),
                      _ptr(num_copies), _ptr(ws), ws.numel(), _ptr(status))
        self._keep = (_held(pool), src, dst, length, pages, ws, status, c)


class FreeCall(_PageCall):
    """verify_attn_pages_free.  Returns nothing."""
    _where = "verify_attn_pages_free"

    def __init__(self, pool: PagePool, seq, first, last, *, status=None):
        c = self._bind(pool, status)
        n = self._commands(seq=seq, first=first, last=last)
        self._fn, self._out = lib.verify_attn_pages_free, None
        self._args = (ctypes.byref(c), n, _ptr(seq), _ptr(first), _ptr(last), _ptr(status))
        self._keep = (_held(pool), seq, first, last, status, c)


class CompactCall(_PageCall):
    """verify_attn_pages_compact.  Returns (copies, num_copies, live_blocks)."""
    _where = "verify_attn_pages_compact"

    def __init__(self, pool: PagePool, *, copies=None, num_copies=None, live_blocks=None, ws=None, status=None):
        c = self._bind(pool, status)
        copies = self._buffer("copies", copies, (pool.ref_count.numel() // 2, 2), torch.int32)
        num_copies = self._buffer("num_copies", num_copies, (1,), torch.int32)
        live_blocks = self._buffer("live_blocks", live_blocks, (1,), torch.int32)
        ws = self._workspace(ws, int(lib.verify_attn_pages_workspace_size(ctypes.byref(c), 0)))
        self._fn, self._out = lib.verify_attn_pages_compact, (copies, num_copies, live_blocks)
        self._args = (ctypes.byref(c), _ptr(copies), _ptr(num_copies), _ptr(live_blocks), _ptr(ws), ws.numel(),
                      _ptr(status))
        self._keep = (_held(pool), ws, status, c)


class PageCopyCall(_Call):
    """verify_attn_pages_copy over a list of pools, tensors whose first
    dimension is the pages (the K and V arrays of every layer)."""
    _where = "verify_attn_pages_copy"

    def __init__(self, pools, copies, num_copies, *, status=None):
        if not pools:
            raise ValueError("pools: none given")
        self.device = dev = copies.device
        blocks = pools[0].shape[0]
        bytes_of = lambda t: t.numel() * t.element_size()  # noqa: E731
        for i, t in enumerate(pools):
            _tensor(f"pools[{i}]", t, pools[0].dtype, 1, dev)
            if t.shape[0] != blocks or bytes_of(t) != bytes_of(pools[0]):
                raise ValueError(f"pools[{i}]: another size than pools[0]")
        _tensor("copies", copies, torch.int32, 0)
        _tensor("num_copies", num_copies, torch.int32, 1, dev)
        _tensor("status", status, torch.int32, 1, dev, optional=True)
        ptrs = (ctypes.c_void_p * len(pools))(*[_ptr(t) for t in pools])
        self._fn, self._out = lib.verify_attn_pages_copy, None
        self._args = (ptrs, len(pools), bytes_of(pools[0]) // blocks, _i32("pools", blocks), _ptr(copies),
                      _ptr(num_copies), _i32("copies", copies.numel() // 2), _ptr(status))
        self._keep = (tuple(pools), copies, num_copies, status)


def verify_attn_pages_fork(pool: PagePool, src, dst, length, pages, *, stream=None, **kw):
    """Fork and grow sequences of a paged cache; returns (copies, num_copies)
    for verify_attn_pages_copy."""
    return _in_one_go(ForkCall, stream, pool, src, dst, length, pages, **kw)


def verify_attn_pages_free(pool: PagePool, seq, first, last, *, status=None, stream=None):
    """Give back table entries first[i] .. last[i] - 1 of sequence seq[i]."""
    return _in_one_go(FreeCall, stream, pool, seq, first, last, status=status)


def verify_attn_pages_compact(pool: PagePool, *, stream=None, **kw):
    """Pull the pages in use together at the front of the pool; returns
    (copies, num_copies, live_blocks)."""
    return _in_one_go(CompactCall, stream, pool, **kw)


def verify_attn_pages_copy(pools, copies, num_copies, *, status=None, stream: Optional[object] = None):
    """Copy the page pairs in every pool."""
    return _in_one_go(PageCopyCall, stream, pools, copies, num_copies, status=status)
