"""Serving sets of sequences that change and that are drafted ahead: the gated delta rule over fp32 states in slots, verification
of drafted tokens, the pages of the caches.

Binding of include/pace_serve.h, in the manner of kv.py: the pace_* functions marshal tensors (shape, type, device and stride
checks happen here, value ranges in the library), PaceDelta and PacePages own their regions. Tensors are [batch, tokens, heads,
d] views with d contiguous; counts, slots, tables, masks and paths are contiguous int32 tensors; all of a call is on the current
device.
"""
from __future__ import annotations

import ctypes as C

import torch

from ._lib import (PACE_ERR_STATE, PACE_ERR_TIMEOUT, PACE_IO_BF16, PACE_IO_F32, check, lib, pace_delta_config, pace_delta_step,
                   pace_pages_config, pace_pages_layout, pace_tensor)
from .kv import _device, _fn, _ints, _Memory, _stream, _tensor

PACE_DELTA_BAD_SLOT, PACE_DELTA_BAD_KEEP, PACE_DELTA_TIMEOUT = 1, 2, 4
PACE_DELTA_MAX_DRAFT = 64
PACE_VERIFY_MAX_NODES, PACE_VERIFY_MAX_VOCAB = 256, 1 << 24
PACE_PAGES_BAD_CELL, PACE_PAGES_BAD_ROW = 1, 2

__all__ = ["make_delta_config", "pace_delta_config", "pace_delta_bytes", "pace_delta_alloc", "pace_delta_free", "pace_delta_chunk",
           "pace_delta_draft", "pace_delta_keep", "pace_delta_get_status", "PaceDelta", "pace_verify", "pace_pages_config",
           "pace_pages_get_layout", "pace_pages_alloc", "pace_pages_free", "pace_pages_select", "pace_pages_take",
           "pace_pages_compact", "pace_pages_get_status", "PacePages", "PACE_DELTA_BAD_SLOT",
           "PACE_DELTA_BAD_KEEP", "PACE_DELTA_TIMEOUT", "PACE_DELTA_MAX_DRAFT", "PACE_VERIFY_MAX_NODES", "PACE_VERIFY_MAX_VOCAB",
           "PACE_PAGES_BAD_CELL", "PACE_PAGES_BAD_ROW"]


def _gate(t, shape, name):
    """pace_tensor of an fp32 [batch, tokens, heads] view of any strides."""
    if t.dtype is not torch.float32 or t.get_device() != _device() or t.shape != shape:
        raise ValueError(f"{name}: expected a float32 tensor on the current CUDA device, of shape {tuple(shape)}, got {t.dtype} on "
                         f"{t.device}, shape {tuple(t.shape)}")
    return pace_tensor(t.data_ptr(), *t.stride())


def _status(name, handle, clear, stream):
    out = C.c_int()
    st = _fn(name)(handle, int(clear), C.byref(out), _stream(stream))
    if st not in (PACE_ERR_STATE, PACE_ERR_TIMEOUT):
        check(st)
    return out.value


# ---- the gated delta rule over states in slots ---------------------------------------------------------------------------------
def make_delta_config(heads: int, d: int, n_slots: int, key_heads: int = 0, io_dtype: int = PACE_IO_BF16) -> pace_delta_config:
    return pace_delta_config(heads, key_heads, d, n_slots, io_dtype)


def pace_delta_bytes(cfg: pace_delta_config) -> int:
    out = C.c_size_t()
    check(lib().pace_delta_bytes(C.byref(cfg), C.byref(out)))
    return out.value


def pace_delta_alloc(cfg: pace_delta_config, device_mem: int, nbytes: int, stream=None) -> int:
    h = C.c_void_p()
    check(lib().pace_delta_alloc(C.byref(cfg), device_mem, nbytes, _stream(stream), C.byref(h)))
    return h.value


def pace_delta_free(handle) -> None:
    if handle:
        lib().pace_delta_free(handle)


def _delta_step(B, T, slots, lens, n_new):
    return pace_delta_step(B, T, _ints(slots, (B,), "slots", True), _ints(lens, (B,), "lens", True), _ints(n_new, (B,), "n_new", True))


def pace_delta_chunk(handle, cfg, q, k, v, a, beta, o, slots=None, lens=None, n_new=None, stream=None) -> None:
    B, T, H, d = v.shape
    ks, vs, io = (B, T, cfg.key_heads or cfg.heads, cfg.d), (B, T, cfg.heads, cfg.d), cfg.io_dtype
    check(_fn("pace_delta_chunk")(handle, _delta_step(B, T, slots, lens, n_new), _tensor(q, io, ks, "q"), _tensor(k, io, ks, "k"),
                                  _tensor(v, io, vs, "v"), _gate(a, vs[:3], "a"), _gate(beta, vs[:3], "beta"),
                                  _tensor(o, io, vs, "o"), _stream(stream)))


def pace_delta_draft(handle, cfg, q, k, v, a, beta, o, slots=None, lens=None, n_new=None, mask=None, stream=None) -> None:
    B, T, H, d = v.shape
    ks, vs, io = (B, T, cfg.key_heads or cfg.heads, cfg.d), (B, T, cfg.heads, cfg.d), cfg.io_dtype
    check(_fn("pace_delta_draft")(handle, _delta_step(B, T, slots, lens, n_new), _tensor(q, io, ks, "q"), _tensor(k, io, ks, "k"),
                                  _tensor(v, io, vs, "v"), _gate(a, vs[:3], "a"), _gate(beta, vs[:3], "beta"),
                                  _ints(mask, (B, T, (T + 31) // 32), "mask", True), _tensor(o, io, vs, "o"), _stream(stream)))


def pace_delta_keep(handle, cfg, k, v, a, beta, idx, n_keep, slots=None, lens=None, n_new=None, stream=None) -> None:
    B, T, H, d = v.shape
    ks, vs, io = (B, T, cfg.key_heads or cfg.heads, cfg.d), (B, T, cfg.heads, cfg.d), cfg.io_dtype
    n = idx.shape[1]
    check(_fn("pace_delta_keep")(handle, _delta_step(B, T, slots, lens, n_new), _tensor(k, io, ks, "k"), _tensor(v, io, vs, "v"),
                                 _gate(a, vs[:3], "a"), _gate(beta, vs[:3], "beta"), _ints(idx, (B, n), "idx"), n,
                                 _ints(n_keep, (B,), "n_keep"), _stream(stream)))


def pace_delta_get_status(handle, clear: bool = False, stream=None) -> int:
    """The handle's device status bits (synchronises the stream). The bits are returned, not raised; other errors raise."""
    return _status("pace_delta_get_status", handle, clear, stream)


def pace_test_delta_wait_probe(handle, ns: int) -> None:
    """Failure-detection hook for tests: while ns > 0, calls by chunks of this handle wait that long for what nothing signals, give up and leave the
    states as they are. 0 turns it off."""
    fn = lib().pace_test_delta_wait_probe
    fn.restype, fn.argtypes = C.c_int, [C.c_void_p, C.c_uint32]
    check(fn(handle, int(ns)))


class PaceDelta:
    """The fp32 states of one gated-delta layer, [n_slots, heads, d, d] (`states`, key index first), bound to a handle.

    A prompt or a token is chunk; a step of drafts is draft, then keep along the accepted path. Tensors passed in are the caller's to
    keep until a call's stream has done with them; the states' memory waits for the streams of their calls.
    """

    def __init__(self, cfg: pace_delta_config, device="cuda", stream=None):
        self.cfg = cfg
        self.nbytes = pace_delta_bytes(cfg)
        self._memory = _Memory(self.nbytes + 256, torch.uint8, device, stream)
        self.mem, self._on = self._memory.tensor, self._memory.on
        off = -self.mem.data_ptr() % 256
        self.handle = pace_delta_alloc(cfg, self.mem.data_ptr() + off, self.nbytes, self._on(stream))
        shape = (cfg.n_slots, cfg.heads, cfg.d, cfg.d)
        self.states = self.mem[off:off + self.nbytes - 256].view(torch.float32).view(shape)

    def chunk(self, q, k, v, a, beta, o, slots=None, lens=None, n_new=None, stream=None):
        pace_delta_chunk(self.handle, self.cfg, q, k, v, a, beta, o, slots, lens, n_new, self._on(stream))

    def draft(self, q, k, v, a, beta, o, slots=None, lens=None, n_new=None, mask=None, stream=None):
        pace_delta_draft(self.handle, self.cfg, q, k, v, a, beta, o, slots, lens, n_new, mask, self._on(stream))

    def keep(self, k, v, a, beta, idx, n_keep, slots=None, lens=None, n_new=None, stream=None):
        pace_delta_keep(self.handle, self.cfg, k, v, a, beta, idx, n_keep, slots, lens, n_new, self._on(stream))

    def status(self, clear: bool = False, stream=None) -> int:
        return pace_delta_get_status(self.handle, clear, self._on(stream))

    def close(self):
        if getattr(self, "handle", None):
            pace_delta_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- verification -----------------------------------------------------------------------------------------------------------------
def _probabilities(t, io, shape, name):
    st = t.stride()
    want = torch.float32 if io == PACE_IO_F32 else torch.bfloat16
    if t.dtype is not want or t.get_device() != _device() or t.shape != shape or (st[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name}: expected a {want} tensor on the current CUDA device, of shape {tuple(shape)} with its last dimension "
                         f"contiguous, got {t.dtype} on {t.device}, shape {tuple(t.shape)}, strides {st}")
    return pace_tensor(t.data_ptr(), st[0], st[1], 0)


def pace_verify(tokens, p, q, u, idx, n_keep, next, mask=None, n_new=None, stream=None) -> None:
    """Keeps the drafts of tokens [B, N] (node 0: the last token) that the target's probabilities p [B, N, V] (fp32 or bf16) accept
    against the draft model's q (None: drafts named without probabilities), by the random numbers u [B, N] (fp32). Writes the
    kept nodes to idx [B, N], their number to n_keep [B] and the next token to next [B]."""
    if p.dim() != 3:
        raise ValueError("p: expected [batch, nodes, vocabulary]")
    B, N, V = p.shape
    if N < 1 or V < 1:
        raise ValueError("p: expected at least one node and one token")
    io = PACE_IO_F32 if p.dtype is torch.float32 else PACE_IO_BF16
    if u.dtype is not torch.float32 or u.get_device() != _device() or u.shape != (B, N) or not u.is_contiguous():
        raise ValueError(f"u: expected a contiguous float32 tensor on the current CUDA device, of shape {(B, N)}, got {u.dtype} on "
                         f"{u.device}, shape {tuple(u.shape)}, strides {u.stride()}")
    check(_fn("pace_verify")(B, N, V, io, _ints(tokens, (B, N), "tokens"), _probabilities(p, io, (B, N, V), "p"),
                             None if q is None else _probabilities(q, io, (B, N, V), "q"), u.data_ptr(),
                             _ints(mask, (B, N, (N + 31) // 32), "mask", True), _ints(n_new, (B,), "n_new", True),
                             _ints(idx, (B, N), "idx"), _ints(n_keep, (B,), "n_keep"), _ints(next, (B,), "next"), _stream(stream)))


# ---- pages ------------------------------------------------------------------------------------------------------------------------
def pace_pages_get_layout(cfg: pace_pages_config) -> pace_pages_layout:
    out = pace_pages_layout()
    check(lib().pace_pages_get_layout(C.byref(cfg), C.byref(out)))
    return out


def pace_pages_alloc(cfg: pace_pages_config, device_mem: int, nbytes: int, stream=None) -> int:
    h = C.c_void_p()
    check(lib().pace_pages_alloc(C.byref(cfg), device_mem, nbytes, _stream(stream), C.byref(h)))
    return h.value


def pace_pages_free(handle) -> None:
    if handle:
        lib().pace_pages_free(handle)


def _table(table):
    if table is None or table.dim() != 2:
        raise ValueError("table: expected [batch, columns]")
    B, cols = table.shape
    return B, cols, _ints(table, (B, cols), "table")


def pace_pages_select(handle, table, lens, src=None, stream=None) -> None:
    B, cols, at = _table(table)
    check(_fn("pace_pages_select")(handle, B, at, cols, _ints(lens, (B,), "lens"), _ints(src, (B,), "src", True), _stream(stream)))


def pace_pages_take(handle, table, lens, n_new, fits, stream=None) -> None:
    B, cols, at = _table(table)
    check(_fn("pace_pages_take")(handle, B, at, cols, _ints(lens, (B,), "lens"), _ints(n_new, (B,), "n_new"), _ints(fits, (B,), "fits"),
                                 _stream(stream)))


def pace_pages_compact(handle, table, stream=None) -> None:
    B, cols, at = _table(table)
    check(_fn("pace_pages_compact")(handle, B, at, cols, _stream(stream)))


def pace_pages_get_status(handle, clear: bool = False, stream=None) -> int:
    """The handle's device status bits (synchronises the stream). The bits are returned, not raised; other errors raise."""
    return _status("pace_pages_get_status", handle, clear, stream)


class PacePages:
    """Counts which pages of the caches are held, by the rows of a table [batch, columns] (-1: no page).

    A step of a serving loop is take (pages for the new tokens), copy_pages of each layer's cache where rows share their last page,
    the layers' calls, and select (fork, reorder, shorten, free rows). `refs` [n_pages] are the counts; src and dst [n_pages] hold the
    last call's n_moves [1] moves.
    """

    def __init__(self, n_pages: int, page_tokens: int, max_batch: int, device="cuda", stream=None):
        self.cfg = pace_pages_config(n_pages, page_tokens, max_batch)
        lay = pace_pages_get_layout(self.cfg)
        self._memory = _Memory(lay.total_bytes + 256, torch.uint8, device, stream)
        self.mem, self._on = self._memory.tensor, self._memory.on
        off = -self.mem.data_ptr() % 256
        self.handle = pace_pages_alloc(self.cfg, self.mem.data_ptr() + off, lay.total_bytes, self._on(stream))
        ints = lambda at, n: self.mem[off + at:off + at + 4 * n].view(torch.int32)
        self.refs, self.src, self.dst = (ints(at, n_pages) for at in (lay.refs, lay.src, lay.dst))
        self.n_moves = ints(lay.n_moves, 1)

    def select(self, table, lens, src=None, stream=None):
        pace_pages_select(self.handle, table, lens, src, self._on(stream))

    def take(self, table, lens, n_new, fits, stream=None):
        pace_pages_take(self.handle, table, lens, n_new, fits, self._on(stream))

    def compact(self, table, stream=None):
        pace_pages_compact(self.handle, table, self._on(stream))

    def status(self, clear: bool = False, stream=None) -> int:
        return pace_pages_get_status(self.handle, clear, self._on(stream))

    def close(self):
        if getattr(self, "handle", None):
            pace_pages_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
