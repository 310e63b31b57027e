"""Attention layers of a hybrid model: rotary positions, the quantized paged KV cache and attention over it.

Binding of include/pace_kv.h: the pace_* functions marshal tensors (shape, type, device and stride checks happen here, value
ranges in the library), PaceRope and PaceKV own the table and the cache region. Tensors are [batch, tokens, heads, d] views
with d contiguous; lengths, page tables, masks and paths are contiguous int32 tensors; all of a call is on the current device.
"""
from __future__ import annotations

import ctypes as C
import functools

import torch

from ._lib import (PACE_ERR_STATE, PACE_ERR_TIMEOUT, PACE_IO_BF16, PACE_IO_F32, check, lib, pace_kv_config, pace_kv_step,
                   pace_rope_config, pace_tensor)

PACE_KV_BAD_PAGE, PACE_KV_BAD_POSITION, PACE_KV_BAD_KEEP, PACE_KV_TIMEOUT = 1, 2, 4, 8
PACE_KV_MAX_BATCH, PACE_KV_MAX_NEW = 1024, 4096
_INTS = (torch.int32, torch.uint32)
_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}

__all__ = ["make_rope_config", "pace_rope_bytes", "pace_rope_table", "pace_rope_apply", "PaceRope", "make_kv_config",
           "pace_kv_bytes", "pace_kv_tile_bytes", "pace_kv_alloc", "pace_kv_free", "pace_kv_append", "pace_kv_read",
           "pace_kv_attend", "pace_kv_keep", "pace_kv_get_status", "PaceKV", "pace_kv_config", "pace_rope_config",
           "PACE_KV_BAD_PAGE", "PACE_KV_BAD_POSITION", "PACE_KV_BAD_KEEP", "PACE_KV_TIMEOUT", "PACE_KV_MAX_BATCH",
           "PACE_KV_MAX_NEW"]


# The calls below are made for every layer and token, so their marshalling is kept short: raw stream handles, one stride() per
# tensor, library functions looked up once.
_device = getattr(torch._C, "_cuda_getDevice", None)     # the current device's index


def _stream(s):
    if s is None:
        return torch._C._cuda_getCurrentRawStream(_device())
    return s if isinstance(s, int) else s.cuda_stream


class _Memory:
    """Device memory that calls on several streams use: its allocator learns of each stream, so that what is dropped while one of
    them still works on it is not given out again before that work has ended."""

    def __init__(self, shape, dtype, device, stream):
        self.tensor = torch.empty(shape, dtype=dtype, device=device)
        own = torch.cuda.current_stream(self.tensor.device)
        self.streams = {own.cuda_stream}
        s = self.on(stream)
        if s != own.cuda_stream:         # (it may be memory that `own` has not done with)
            torch.cuda.ExternalStream(s, self.tensor.device).wait_stream(own)

    def on(self, stream):
        """The raw handle of `stream` (None: the current one), which the memory is now known to be used on."""
        if self.tensor.get_device() != _device():
            raise ValueError(f"memory on {self.tensor.device}, but the current device is {_device()}")
        s = _stream(stream)
        if s not in self.streams:
            self.tensor.record_stream(torch.cuda.ExternalStream(s, self.tensor.device))
            self.streams.add(s)
        return s


@functools.lru_cache(maxsize=None)
def _fn(name):
    return getattr(lib(), name)


@functools.lru_cache(maxsize=None)
def _dtype(io):
    return torch.float32 if io == PACE_IO_F32 else torch.bfloat16


def _tensor(t, io, shape, name):
    """pace_tensor of a [.., tokens, heads, d] view, or a ValueError that says what is wrong with it."""
    if t is None:
        return None
    st = t.stride()
    if t.dtype is not _dtype(io) or t.get_device() != _device() or t.shape != shape or (st[-1] != 1 and shape[-1] > 1 and t.numel()):
        raise ValueError(f"{name}: expected a {_dtype(io)} tensor on the current CUDA device, of shape {tuple(shape)} with its last "
                         f"dimension contiguous, got {t.dtype} on {t.device}, shape {tuple(t.shape)}, strides {st}")
    if 1 in shape:                       # the stride of a single element is anything
        st = [0 if n == 1 else x for n, x in zip(shape, st)]
    return pace_tensor(t.data_ptr(), st[0] if len(st) == 4 else 0, st[-3], st[-2])


def _ints(t, shape, name, optional=False):
    """Pointer of a contiguous int32 (masks: also uint32) CUDA tensor of the given shape."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is missing")
    if t.dtype not in _INTS or t.get_device() != _device() or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor on the current CUDA device, of shape {tuple(shape)}, got {t.dtype} on "
                         f"{t.device}, shape {tuple(t.shape)}, strides {t.stride()}")
    return t.data_ptr()


# ---- rotary positions -------------------------------------------------------------------------------------------------------
def make_rope_config(rot: int, max_pos: int, base: float = 10000.0, layout: str = "half", scaling: str = "none",
                     factor: float = 1.0, orig_pos: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     mscale: float = 0.0) -> pace_rope_config:
    if layout not in _LAYOUTS or scaling not in _SCALINGS:
        raise ValueError(f"layout is one of {sorted(_LAYOUTS)}, scaling one of {sorted(_SCALINGS)}")
    return pace_rope_config(rot, max_pos, _LAYOUTS[layout], _SCALINGS[scaling], base, factor, orig_pos, beta_fast, beta_slow,
                            mscale)


def pace_rope_bytes(cfg: pace_rope_config) -> int:
    out = C.c_size_t()
    check(lib().pace_rope_bytes(C.byref(cfg), C.byref(out)))
    return out.value


def pace_rope_table(cfg: pace_rope_config, table, nbytes: int, stream=None) -> None:
    check(lib().pace_rope_table(C.byref(cfg), table if isinstance(table, int) else table.data_ptr(), nbytes, _stream(stream)))


class PaceRope:
    """A cos/sin table: `rot` elements of a head, positions 0..max_pos-1, built once."""

    def __init__(self, rot: int, max_pos: int, device="cuda", stream=None, **kw):
        self.cfg = make_rope_config(rot, max_pos, **kw)
        self.nbytes = pace_rope_bytes(self.cfg)
        self._memory = _Memory((max_pos, rot // 2, 2), torch.float32, device, stream)
        self.table, self._on = self._memory.tensor, self._memory.on
        self.ptr = self.table.data_ptr()
        pace_rope_table(self.cfg, self.ptr, self.nbytes, self._on(stream))


def pace_rope_apply(rope: PaceRope, x, positions, out, inverse: bool = False, stream=None) -> None:
    """Rotates x [n, heads, d] (bf16 or fp32) at positions [n] into out (x itself is allowed). inverse: the gradient."""
    if x.dim() != 3:
        raise ValueError("x: expected [n, heads, d]")
    io = PACE_IO_F32 if x.dtype is torch.float32 else PACE_IO_BF16
    shape = n, h, d = x.shape
    check(_fn("pace_rope_apply")(rope.cfg, rope.ptr, n, h, d, io, _tensor(x, io, shape, "x"), _ints(positions, (n,), "positions"),
                                 _tensor(out, io, shape, "out"), inverse, rope._on(stream)))


# ---- the cache ----------------------------------------------------------------------------------------------------------------
def make_kv_config(q_heads: int, kv_heads: int, d: int, n_pages: int, max_batch: int, bits: int = 4, page_tokens: int = 64,
                   max_new: int = 256, io_dtype: int = PACE_IO_BF16) -> pace_kv_config:
    return pace_kv_config(q_heads, kv_heads, d, bits, page_tokens, n_pages, max_batch, max_new, io_dtype)


def pace_kv_bytes(cfg: pace_kv_config) -> int:
    out = C.c_size_t()
    check(lib().pace_kv_bytes(C.byref(cfg), C.byref(out)))
    return out.value


def pace_kv_tile_bytes(cfg: pace_kv_config) -> int:
    return lib().pace_kv_tile_bytes(C.byref(cfg))


def pace_kv_alloc(cfg: pace_kv_config, device_mem: int, nbytes: int, stream=None) -> int:
    h = C.c_void_p()
    check(lib().pace_kv_alloc(C.byref(cfg), device_mem, nbytes, _stream(stream), C.byref(h)))
    return h.value


def pace_kv_free(handle) -> None:
    if handle:
        lib().pace_kv_free(handle)


def _step(B, T, lens, table, n_new):
    if table is None or table.dim() != 2:
        raise ValueError("table: expected [batch, columns]")
    cols = table.shape[1]
    return pace_kv_step(B, T, None if lens is None else _ints(lens, (B,), "lens"), _ints(n_new, (B,), "n_new", True),
                        _ints(table, (B, cols), "table"), cols)


def pace_kv_append(handle, cfg, q, k, v, lens, table, rope=None, positions=None, n_new=None, q_out=None, stream=None) -> None:
    B, T = k.shape[0], k.shape[1]
    io = cfg.io_dtype
    kv, qs = (B, T, cfg.kv_heads, cfg.d), (B, T, cfg.q_heads, cfg.d)
    check(_fn("pace_kv_append")(handle, _step(B, T, lens, table, n_new), _tensor(q, io, qs, "q"), _tensor(k, io, kv, "k"),
                                _tensor(v, io, kv, "v"), _tensor(q_out, io, qs, "q_out"), rope.cfg if rope else None,
                                rope.ptr if rope else None, _ints(positions, (B, T), "positions", True),
                                rope._on(stream) if rope else _stream(stream)))


def pace_kv_read(handle, cfg, k_out, v_out, table, first=None, end=None, stream=None) -> None:
    B, n = k_out.shape[0], k_out.shape[1]
    shape = (B, n, cfg.kv_heads, cfg.d)
    check(_fn("pace_kv_read")(handle, _step(B, n, None, table, None), _ints(first, (B,), "first", True),
                              _ints(end, (B,), "end", True), _tensor(k_out, cfg.io_dtype, shape, "k_out"),
                              _tensor(v_out, cfg.io_dtype, shape, "v_out"), _stream(stream)))


def pace_kv_attend(handle, cfg, q, o, lens, table, mask=None, n_new=None, scale=None, stream=None) -> None:
    B, T = q.shape[0], q.shape[1]
    d = cfg.d
    shape = (B, T, cfg.q_heads, d)
    check(_fn("pace_kv_attend")(handle, _step(B, T, lens, table, n_new), _tensor(q, cfg.io_dtype, shape, "q"),
                                _ints(mask, (B, T, (T + 31) // 32), "mask", True), d ** -0.5 if scale is None else scale,
                                _tensor(o, cfg.io_dtype, shape, "o"), _stream(stream)))


def pace_kv_keep(handle, lens, table, idx, n_keep, stream=None) -> None:
    B, K = idx.shape
    check(_fn("pace_kv_keep")(handle, _step(B, K, lens, table, None), _ints(idx, (B, K), "idx"), _ints(n_keep, (B,), "n_keep"),
                              _stream(stream)))


def pace_kv_get_status(handle, clear: bool = False, stream=None) -> int:
    """The cache's device status bits (synchronises the stream). The bits are returned, not raised; other errors raise."""
    out = C.c_int()
    st = lib().pace_kv_get_status(handle, int(clear), C.byref(out), _stream(stream))
    if st not in (PACE_ERR_STATE, PACE_ERR_TIMEOUT):
        check(st)
    return out.value


class PaceKV:
    """Owns a device region (a torch uint8 tensor) bound to a KV-cache handle.

    One cache serves one attention layer; lens [B] and table [B, columns] are the caller's and may serve all layers. A step is
    append (k rotated and quantized, q rotated), attend, and, for drafted trees, keep; the caller then advances lens. The cache's
    memory waits for the streams of its calls; tensors passed in are the caller's to keep until a call's stream has done with them.
    """

    def __init__(self, cfg: pace_kv_config, device="cuda", stream=None):
        self.cfg = cfg
        self.nbytes = pace_kv_bytes(cfg)
        self._memory = _Memory(self.nbytes + 256, torch.uint8, device, stream)
        self.mem, self._on = self._memory.tensor, self._memory.on
        base = (self.mem.data_ptr() + 255) // 256 * 256
        self.handle = pace_kv_alloc(cfg, base, self.nbytes, self._on(stream))

    def append(self, q, k, v, lens, table, rope=None, positions=None, n_new=None, q_out=None, stream=None):
        pace_kv_append(self.handle, self.cfg, q, k, v, lens, table, rope, positions, n_new, q_out, self._on(stream))

    def read(self, k_out, v_out, table, first=None, end=None, stream=None):
        pace_kv_read(self.handle, self.cfg, k_out, v_out, table, first, end, self._on(stream))

    def attend(self, q, o, lens, table, mask=None, n_new=None, scale=None, stream=None):
        pace_kv_attend(self.handle, self.cfg, q, o, lens, table, mask, n_new, scale, self._on(stream))

    def keep(self, lens, table, idx, n_keep, stream=None):
        pace_kv_keep(self.handle, lens, table, idx, n_keep, self._on(stream))

    def status(self, clear: bool = False, stream=None) -> int:
        return pace_kv_get_status(self.handle, clear, self._on(stream))

    def close(self):
        if getattr(self, "handle", None):
            pace_kv_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
