"""Host side of include/pace_serve.h: exported names, sizes and refusals. CPU only: no call reaches a GPU."""
import ctypes as C
import os
import re

import pytest

from pace_testlib import ensure_built

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 2
MEM = 1 << 20                     # an address that no refused call reads


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    P.lib()
    return P


def test_library_exports_what_the_header_declares(P):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pace_serve.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(pace_[a-z0-9_]+)\s*\(", text))
    assert names == set(P._lib.exported_serve_symbols()) and len(names) == 17
    for n in names:
        assert hasattr(P.lib(), n)


def test_public_names_resolve(P):
    assert all(hasattr(P, n) for n in P.__all__) and len(set(P.__all__)) == len(P.__all__)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), INVALID), (dict(heads=257), INVALID), (dict(key_heads=3), INVALID), (dict(key_heads=16), INVALID),
    (dict(key_heads=-1), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(n_slots=0), INVALID),
    (dict(io_dtype=2), INVALID)])
def test_delta_configs_are_refused(P, kw, status):
    cfg = P.make_delta_config(**{**dict(heads=8, d=128, n_slots=4), **kw})
    with pytest.raises(P.PaceError) as e:
        P.pace_delta_bytes(cfg)
    assert e.value.status == status and P.pace_last_error()


def test_sizes(P):
    assert P.pace_delta_bytes(P.make_delta_config(6, 64, 5, key_heads=2)) == 5 * 6 * 64 * 64 * 4 + 256
    lay = P.pace_pages_get_layout(P.pace_pages_config(1000, 64, 8))
    assert lay.refs % 256 == lay.src % 256 == lay.dst % 256 == lay.n_moves % 256 == 0
    assert lay.src - lay.refs >= 4000 and lay.dst - lay.src >= 4000 and lay.total_bytes > lay.n_moves > lay.dst + 4000


@pytest.mark.parametrize("args", [(0, 64, 8), ((1 << 30) + 1, 64, 8), (10, 48, 8), (10, 0, 8), (10, 8192, 8), (10, 64, 0), (10, 64, 1025)])
def test_pages_configs_are_refused(P, args):
    with pytest.raises(P.PaceError) as e:
        P.pace_pages_get_layout(P.pace_pages_config(*args))
    assert e.value.status == INVALID


def refused(P, name, *args, status=INVALID):
    assert getattr(P.lib(), name)(*args) == status
    return P.pace_last_error()


def test_handles_are_refused(P):
    out = C.c_void_p()
    cfg = P.make_delta_config(2, 64, 1)
    assert "aligned" in refused(P, "pace_delta_alloc", cfg, MEM + 8, 1 << 30, None, C.byref(out))
    assert "smaller" in refused(P, "pace_delta_alloc", cfg, MEM, 100, None, C.byref(out))
    assert "out is NULL" in refused(P, "pace_delta_alloc", cfg, MEM, 1 << 30, None, None)
    assert "smaller" in refused(P, "pace_pages_alloc", P.pace_pages_config(10, 64, 1), MEM, 100, None, C.byref(out))
    assert not out.value
    for name, n in (("pace_delta_get_status", 1), ("pace_pages_get_status", 1)):
        assert "NULL" in refused(P, name, None, 0, None, None)
    assert "NULL" in refused(P, "pace_kv_pool", None, None, None)
    assert "NULL" in refused(P, "pace_kv_copy_pages", None, MEM, MEM, None, 1, None)
    step, t = P._lib.pace_delta_step(1, 1, None, None, None), P._lib.pace_tensor(MEM, 0, 0, 0)
    assert "handle" in refused(P, "pace_delta_chunk", None, step, t, t, t, t, t, t, None)
    assert "handle" in refused(P, "pace_pages_take", None, 1, MEM, 1, MEM, MEM, MEM, None)


VERIFY = dict(batch=1, n_nodes=2, vocab=10, io=1, tokens=MEM, p=True, q=None, u=MEM, mask=None, n_new=None, idx=MEM, n_keep=MEM, next=MEM)


@pytest.mark.parametrize("kw,say", [
    (dict(batch=-1), "batch"), (dict(batch=1025), "batch"), (dict(n_nodes=0), "n_nodes"), (dict(n_nodes=257), "n_nodes"),
    (dict(vocab=0), "vocab"), (dict(vocab=(1 << 24) + 1), "vocab"), (dict(io=2), "io_dtype"), (dict(p=None), "p is NULL"),
    (dict(p=MEM + 2), "aligned"), (dict(q=MEM + 1), "aligned"), (dict(tokens=None), "NULL"), (dict(u=None), "NULL"), (dict(idx=None), "NULL"),
    (dict(n_keep=None), "NULL"), (dict(next=None), "NULL"), (dict(mask=MEM + 2), "aligned"), (dict(u=MEM + 1), "aligned")])
def test_verification_is_refused(P, kw, say):
    a = {**VERIFY, **kw}
    tensor = lambda x: None if x is None else P._lib.pace_tensor(MEM if x is True else x, 20, 10, 0)
    assert say in refused(P, "pace_verify", a["batch"], a["n_nodes"], a["vocab"], a["io"], a["tokens"], tensor(a["p"]), tensor(a["q"]),
                          a["u"], a["mask"], a["n_new"], a["idx"], a["n_keep"], a["next"], None)


def test_binding_refuses_tensors_off_the_device(P, monkeypatch):
    import torch
    from bit_gated_delta_gb300 import serve
    monkeypatch.setattr(serve, "_device", lambda: 0)
    f, i = torch.zeros(1, 2, 10), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        serve.pace_verify(i, f, None, f[..., 0], i, i[:, 0], i[:, 0])
    with pytest.raises(ValueError, match="batch, nodes"):
        serve.pace_verify(i, f[0], None, f[0, :, 0], i, i[:, 0], i[:, 0])
    with pytest.raises(ValueError, match="columns"):
        serve.pace_pages_compact(1, i[0])
    with pytest.raises(ValueError, match="float32"):
        serve._gate(f.double(), (1, 2, 10), "a")
