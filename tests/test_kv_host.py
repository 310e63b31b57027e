"""Host side of include/pace_kv.h: exported names, sizes and refusals. CPU only: no call reaches a GPU."""
import ctypes as C
import os
import re

import numpy as np
import pytest

import kv_testlib as K
from pace_testlib import ensure_built

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    P.lib()
    return P


def test_library_exports_what_the_header_declares(P):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pace_kv.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(pace_[a-z0-9_]+)\s*\(", text)))
    assert set(names) == set(P._lib.exported_kv_symbols()) and len(names) == 12
    for n in names:
        assert hasattr(P.lib(), n)


def config(P, **kw):
    return P.make_kv_config(**{**dict(q_heads=8, kv_heads=2, d=128, n_pages=10, max_batch=4), **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(kv_heads=16), INVALID),
    (dict(q_heads=257), INVALID), (dict(d=96), UNSUPPORTED), (dict(bits=5), UNSUPPORTED), (dict(page_tokens=48), INVALID),
    (dict(page_tokens=0), INVALID), (dict(page_tokens=8192), INVALID), (dict(n_pages=0), INVALID),
    (dict(max_batch=0), INVALID), (dict(max_batch=1025), INVALID), (dict(max_new=0), INVALID), (dict(max_new=5000), INVALID),
    (dict(io_dtype=7), INVALID)])
def test_cache_configs_are_refused(P, kw, status):
    with pytest.raises(P.PaceError) as e:
        P.pace_kv_bytes(config(P, **kw))
    assert e.value.status == status and P.pace_last_error()
    assert P.pace_kv_tile_bytes(config(P, **kw)) == 0


@pytest.mark.parametrize("d,bits", [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8)])
def test_cache_bytes(P, d, bits):
    cfg = config(P, d=d, bits=bits, page_tokens=64, n_pages=1000)
    row = 2 * (d * bits // 8 + d // 64 * (2 + (bits == 4)))
    assert P.pace_kv_tile_bytes(cfg) == 32 * row
    pool = 1000 * 2 * 2 * 32 * row
    work = P.pace_kv_bytes(config(P, d=d, bits=bits, page_tokens=64, n_pages=1)) - 2 * 2 * 32 * row
    assert 0 <= P.pace_kv_bytes(cfg) - pool - work <= 512


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), INVALID), (dict(rot=24), INVALID), (dict(rot=512), INVALID), (dict(max_pos=0), INVALID),
    (dict(base=1.0), INVALID), (dict(base=float("nan")), INVALID), (dict(scaling="linear", factor=0.5), INVALID),
    (dict(scaling="ntk", factor=float("inf")), INVALID), (dict(mscale=-1.0), INVALID),
    (dict(scaling="parts", factor=4.0), INVALID),
    (dict(scaling="parts", factor=4.0, orig_pos=4096, beta_fast=1.0, beta_slow=2.0), INVALID)])
def test_rope_configs_are_refused(P, kw, status):
    with pytest.raises(P.PaceError) as e:
        P.pace_rope_bytes(P.make_rope_config(**{**dict(rot=64, max_pos=100), **kw}))
    assert e.value.status == status
    with pytest.raises(ValueError):
        P.make_rope_config(64, 100, layout="spiral")


def test_rope_table_and_apply_refuse_before_any_launch(P):
    L = P._lib
    cfg = P.make_rope_config(64, 100)
    assert P.pace_rope_bytes(cfg) == 100 * 32 * 8
    lib = P.lib()
    assert lib.pace_rope_table(C.byref(cfg), None, 1 << 20, None) == INVALID
    assert lib.pace_rope_table(C.byref(cfg), 4096, 100 * 32 * 8 - 1, None) == INVALID
    assert lib.pace_rope_table(C.byref(cfg), 4104, 1 << 20, None) == INVALID
    t = L.pace_tensor(4096, 0, 512, 128)

    def apply(table=4096, n=2, heads=2, d=128, io=0, x=t, pos=4096, out=t):
        return lib.pace_rope_apply(C.byref(cfg), table, n, heads, d, io, x and C.byref(x), pos, out and C.byref(out), 0, None)

    assert apply(n=-1) == INVALID and apply(heads=-1) == INVALID and apply(io=9) == INVALID
    assert apply(d=48) == INVALID                       # rot 64 > d
    assert apply(d=100) == UNSUPPORTED and apply(d=264) == UNSUPPORTED
    assert apply(table=None) == INVALID and apply(pos=None) == INVALID and apply(pos=4098) == INVALID
    assert apply(x=None) == INVALID and apply(out=L.pace_tensor(4100, 0, 512, 128)) == INVALID
    assert apply(x=L.pace_tensor(4096, 0, 516, 128)) == INVALID and apply(x=L.pace_tensor(4096, 0, 512, 130)) == INVALID
    assert apply(n=0, x=None, pos=None) == 0 and apply(heads=0) == 0



def test_cache_calls_refuse_before_any_launch(P):
    L, lib = P._lib, P.lib()
    cfg = config(P)
    n = P.pace_kv_bytes(cfg)
    h = C.c_void_p()
    assert lib.pace_kv_alloc(C.byref(cfg), None, n, None, C.byref(h)) == INVALID
    assert lib.pace_kv_alloc(C.byref(cfg), 4096 + 16, n, None, C.byref(h)) == INVALID
    assert lib.pace_kv_alloc(C.byref(cfg), 4096, n - 1, None, C.byref(h)) == INVALID
    assert lib.pace_kv_alloc(C.byref(cfg), 4096, n, None, None) == INVALID and not h.value
    lib.pace_kv_free(None)
    st = L.pace_kv_step(1, 1, 4096, None, 4096, 4)
    t = L.pace_tensor(4096, 0, 0, 0)
    out = C.c_int()
    assert lib.pace_kv_append(None, C.byref(st), None, C.byref(t), C.byref(t), None, None, None, None, None) == INVALID
    assert lib.pace_kv_read(None, C.byref(st), None, None, C.byref(t), C.byref(t), None) == INVALID
    assert lib.pace_kv_attend(None, C.byref(st), C.byref(t), None, 1.0, C.byref(t), None) == INVALID
    assert lib.pace_kv_keep(None, C.byref(st), 4096, 4096, None) == INVALID
    assert lib.pace_kv_get_status(None, 0, C.byref(out), None) == INVALID


def test_quantizer_statement_by_hand():
    """The tests' own quantizer on groups worked by hand."""
    x = np.zeros(64, np.float32)
    x[:4] = [127.0, -63.5, 0.5, 1.5]
    c, s, z = K.quantize(x, 8)                          # s = 1: ties to even
    assert s[0] == 1.0 and list(c[0, :4]) == [127, -64, 0, 2]
    x[:4] = [10.0, -5.0, 0.5, 1.5]
    c, s, z = K.quantize(x, 4)                          # range 15 over 15 steps: s = 1, z = 5
    assert s[0] == 1.0 and z[0] == 5 and list(c[0, :4]) == [15, 0, 5, 7]
    assert list(K.held(x, 4)[:4]) == [10.0, -5.0, 0.0, 2.0]
    assert (K.held(np.full(64, 1e-41, np.float32), 8) == 0).all()


def test_attention_statement_by_hand():
    q = np.ones((1, 2, 2))
    k = np.zeros((3, 1, 2))
    k[2] = np.log(2) / 2
    v = np.array([1.0, 2.0, 4.0]).reshape(3, 1, 1) * np.ones((3, 1, 2))
    see = np.array([[True, False, True]])
    assert np.allclose(K.attend(q, k, v, see, 1.0), (1 + 2 * 4) / 3)
    assert (K.attend(q, k, v, np.zeros((1, 3), bool), 1.0) == 0).all()


class OnDevice:
    """What the binding looks at of a tensor, on a device that need not exist."""

    def __init__(self, shape, dtype, device):
        import torch
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device("cuda", device), True

    def get_device(self):
        return self.device.index

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def test_tensors_of_another_device_are_refused(P, monkeypatch):
    """A call runs on the current device's stream: tensors, caches and tables of another one are refused before any launch."""
    import torch

    from bit_gated_delta_gb300 import kv
    monkeypatch.setattr(kv, "_device", lambda: 0, raising=False)
    shape = (1, 2, 2, 64)
    assert kv._tensor(OnDevice(shape, torch.bfloat16, 0), P.PACE_IO_BF16, shape, "q").data == 4096
    assert kv._ints(OnDevice((2,), torch.int32, 0), (2,), "lens") == 4096
    with pytest.raises(ValueError, match="current CUDA device"):
        kv._tensor(OnDevice(shape, torch.bfloat16, 1), P.PACE_IO_BF16, shape, "q")
    with pytest.raises(ValueError, match="current CUDA device"):
        kv._ints(OnDevice((2,), torch.int32, 1), (2,), "lens")
    memory = object.__new__(kv._Memory)
    memory.tensor, memory.streams = OnDevice((64,), torch.uint8, 1), {7}
    with pytest.raises(ValueError, match="current device"):
        memory.on(7)
    memory.tensor = OnDevice((64,), torch.uint8, 0)
    assert memory.on(7) == 7
