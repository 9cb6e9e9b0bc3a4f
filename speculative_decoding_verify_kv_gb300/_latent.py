"""Bound calls of the operators of a latent cache: rows into it, verify
attention over it (absorbed form), and attention of prompt segments over
expanded keys and values.  Bound calls, streams and workspaces are those of
the operators around a verify step.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import Problem, VaError, VaLatent, VaLatentRows, VaPrompt, _ptr, lib
from ._calls import _FLOAT, _Call, _check_rows, _held, _i32, _in_one_go, _tensor


def _strided(name, t, dtype, shape, device):
    """A tensor of at least the shape in its first dimension and exactly that in
    the others but the last, which may be wider; the last is dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the other arguments on {device}")
    fits = t.dim() == len(shape) and t.shape[0] >= shape[0] and t.shape[-1] >= shape[-1] and \
        tuple(t.shape[1:-1]) == tuple(shape[1:-1])
    if not fits:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, {tuple(shape)} needed")
    if t.numel() and (t.stride(-1) != 1 or min(t.stride()) < 0):
        raise ValueError(f"{name}: the last dimension has to be dense")
    return t


def _where_dtype(where, code):
    if code not in _FLOAT:
        raise VaError(2, where)
    return _FLOAT[code]


@dataclass
class LatentKV:
    """A latent cache (va_latent): rows of latent_dim + rope_dim values,
    contiguous [num_seqs][capacity] or paged [num_blocks][16]."""
    dtype: int
    latent_dim: int
    rope_dim: int
    cache: object
    page_size: int = 0
    capacity: int = 0
    block_table: object = None
    max_blocks_per_seq: int = 0
    num_blocks: int = 0

    def c(self) -> VaLatent:
        return VaLatent(self.dtype, self.latent_dim, self.rope_dim, _ptr(self.cache), self.page_size, self.capacity,
                        _ptr(self.block_table), _i32("max_blocks_per_seq", self.max_blocks_per_seq),
                        _i32("num_blocks", self.num_blocks))


@dataclass
class LatentRows:
    """Rows for a latent cache (va_latent_rows): kv [rows][>= latent_dim +
    rope_dim] and q_rope [rows][heads][rope_dim] may be parts of wider rows; q
    is [rows][heads][latent_dim + rope_dim]."""
    kv: object
    position: object                # int32 [rows]
    slot: object                    # int64 [rows]
    rope: object                    # float32 [positions][rope_dim]: cosines, then sines
    norm_weight: object = None      # [latent_dim]
    norm_eps: float = 1e-6
    interleaved: bool = False
    q_rope: object = None
    q: object = None


class LatentAppendCall(_Call):
    """verify_attn_latent_append.  Returns the cache, or (cache, q) where
    queries are given."""
    _where = "verify_attn_latent_append"

    def __init__(self, kv: LatentKV, new: LatentRows, *, status=None):
        dt = _where_dtype(self._where, kv.dtype)
        self.device = dev = new.kv.device
        width = kv.latent_dim + kv.rope_dim
        rows = _i32("position", new.position.numel())
        _tensor("cache", kv.cache, dt, width, dev)
        _strided("kv", new.kv, dt, (rows, width), dev)
        _tensor("position", new.position, torch.int32, rows, dev)
        _tensor("slot", new.slot, torch.int64, rows, dev)
        _tensor("rope", new.rope, torch.float32, kv.rope_dim, dev)
        if new.rope.dim() != 2 or new.rope.shape[1] != kv.rope_dim:
            raise ValueError(f"rope: shape {tuple(new.rope.shape)}, (positions, {kv.rope_dim}) needed")
        _tensor("norm_weight", new.norm_weight, dt, kv.latent_dim, dev, optional=True)
        _tensor("status", status, torch.int32, 1, dev, optional=True)
        heads = row_stride = head_stride = 0
        if (new.q_rope is None) != (new.q is None):
            raise ValueError("q_rope, q: one of them given")
        if new.q is not None:
            heads = _i32("q", new.q.shape[1]) if new.q.dim() == 3 else 0
            _strided("q_rope", new.q_rope, dt, (rows, heads, kv.rope_dim), dev)
            _tensor("q", new.q, dt, rows * heads * width, dev)
            if new.q.dim() != 3 or new.q.shape[2] != width:
                raise ValueError(f"q: shape {tuple(new.q.shape)}, (rows, heads, {width}) needed")
            row_stride, head_stride = new.q_rope.stride(0), new.q_rope.stride(1)
        kc = kv.c()
        nc = VaLatentRows(rows, _ptr(new.kv), new.kv.stride(0), _ptr(new.norm_weight), float(new.norm_eps),
                          _ptr(new.rope), _i32("rope", new.rope.shape[0]), int(bool(new.interleaved)),
                          _ptr(new.position), _ptr(new.slot), kv.cache.numel() // width, heads, _ptr(new.q_rope),
                          row_stride, head_stride, _ptr(new.q))
        self._fn = lib.verify_attn_latent_append
        self._out = kv.cache if new.q is None else (kv.cache, new.q)
        self._args = (ctypes.byref(kc), ctypes.byref(nc), _ptr(status))
        self._keep = (_held(kv, new), status, kc, nc)


def verify_attn_latent_append(kv: LatentKV, new: LatentRows, *, status=None, stream=None):
    """Normalise and rotate rows and write them to their slots of a latent
    cache (see verify_attn_latent_append in the header)."""
    return _in_one_go(LatentAppendCall, stream, kv, new, status=status)


class _Attention(_Call):
    def _outputs(self, p, value_dim, dt, need, ws, o, lse):
        rows, heads = p.total_rows, p.num_heads
        return (self._workspace(ws, need), self._buffer("o", o, (rows, heads, value_dim), dt),
                self._buffer("lse", lse, (rows, heads), torch.float32))


class LatentCall(_Attention):
    """verify_attn_latent.  Returns (o, lse)."""
    _where = "verify_attn_latent"

    def __init__(self, p: Problem, kv: LatentKV, mode: int, *, ws=None, o=None, lse=None, status=None):
        dt = _where_dtype(self._where, kv.dtype)
        self.device = dev = p.q.device
        width = kv.latent_dim + kv.rope_dim
        _check_rows(p, mode, dev)
        _tensor("ctx_len", p.ctx_len, torch.int32, p.num_seqs, dev)
        _tensor("q", p.q, dt, p.total_rows * p.num_heads * width, dev)
        if kv.page_size:
            _tensor("block_table", kv.block_table, torch.int32, p.num_seqs * kv.max_blocks_per_seq, dev)
        cells = kv.num_blocks * kv.page_size if kv.page_size else p.num_seqs * kv.capacity
        _tensor("cache", kv.cache, dt, cells * width, dev)
        _tensor("status", status, torch.int32, 1, dev, optional=True)
        pc, kc = p.c(), kv.c()
        need = int(lib.va_latent_workspace_size(ctypes.byref(pc), ctypes.byref(kc)))
        ws, o, lse = self._outputs(p, kv.latent_dim, dt, need, ws, o, lse)
        self._fn, self._out = lib.verify_attn_latent, (o, lse)
        self._args = (ctypes.byref(pc), ctypes.byref(kc), mode, _ptr(ws), ws.numel(), _ptr(o), _ptr(lse), _ptr(status))
        self._keep = (_held(p, kv), ws, status, pc, kc)


def verify_attn_latent(p: Problem, kv: LatentKV, mode: int, *, stream=None, **kw):
    """Verify attention over a latent cache in the absorbed form; returns (o, lse)."""
    return _in_one_go(LatentCall, stream, p, kv, mode, **kw)


def latent_splits(p: Problem, kv: LatentKV) -> int:
    """A num_splits that fills the current GPU once (va_latent_splits)."""
    return int(lib.va_latent_splits(ctypes.byref(p.c()), ctypes.byref(kv.c())))


@dataclass
class PromptKV:
    """Expanded keys and values of prompt segments (va_prompt): kv
    [tokens][heads][nope_dim + value_dim], k_rope [tokens][rope_dim] (its rows
    may be parts of wider ones), cu_kv int32 [num_seqs + 1]."""
    dtype: int
    nope_dim: int
    rope_dim: int
    value_dim: int
    kv: object
    k_rope: object
    cu_kv: object

    def c(self, causal: bool = True) -> VaPrompt:
        return VaPrompt(self.dtype, self.nope_dim, self.rope_dim, self.value_dim, _ptr(self.kv), _ptr(self.k_rope),
                        self.k_rope.stride(0) if self.k_rope.dim() else 0, _ptr(self.cu_kv),
                        _i32("k_rope", self.k_rope.shape[0]), int(bool(causal)))


class PromptCall(_Attention):
    """verify_attn_latent_prompt.  Returns (o, lse)."""
    _where = "verify_attn_latent_prompt"

    def __init__(self, p: Problem, kv: PromptKV, *, causal: bool = True, ws=None, o=None, lse=None, status=None):
        dt = _where_dtype(self._where, kv.dtype)
        self.device = dev = p.q.device
        _check_rows(p, 0, dev)
        _tensor("q", p.q, dt, p.total_rows * p.num_heads * (kv.nope_dim + kv.rope_dim), dev)
        _strided("k_rope", kv.k_rope, dt, (0, kv.rope_dim), dev)
        _tensor("kv", kv.kv, dt, kv.k_rope.shape[0] * p.num_heads * (kv.nope_dim + kv.value_dim), dev)
        _tensor("cu_kv", kv.cu_kv, torch.int32, p.num_seqs + 1, dev)
        _tensor("status", status, torch.int32, 1, dev, optional=True)
        pc, kc = p.c(), kv.c(causal)
        need = int(lib.va_latent_prompt_workspace_size(ctypes.byref(pc), ctypes.byref(kc)))
        ws, o, lse = self._outputs(p, kv.value_dim, dt, need, ws, o, lse)
        self._fn, self._out = lib.verify_attn_latent_prompt, (o, lse)
        self._args = (ctypes.byref(pc), ctypes.byref(kc), _ptr(ws), ws.numel(), _ptr(o), _ptr(lse), _ptr(status))
        self._keep = (_held(p, kv), ws, status, pc, kc)


def verify_attn_latent_prompt(p: Problem, kv: PromptKV, *, causal: bool = True, stream=None, **kw):
    """Attention of prompt segments over expanded keys and values; returns (o, lse)."""
    return _in_one_go(PromptCall, stream, p, kv, causal=causal, **kw)


def prompt_splits(p: Problem, kv: PromptKV) -> int:
    """A num_splits that fills the current GPU once (va_latent_prompt_splits)."""
    return int(lib.va_latent_prompt_splits(ctypes.byref(p.c()), ctypes.byref(kv.c())))
