"""Attention-layer operators on the GPU against the plain statement in tests/kv_testlib.py."""
import numpy as np
import pytest

import kv_testlib as K
from pace_testlib import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    P.lib()
    return P


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.float().cpu().numpy()


def io_of(P, io):
    import torch
    return (P.PACE_IO_F32, torch.float32) if io == "f32" else (P.PACE_IO_BF16, torch.bfloat16)


class Layer:
    """A cache with scattered pages whose unwritten bytes are all ones (NaN scales), and the values it should hold."""

    def __init__(self, P, B, Hq, Hkv, d, bits, io, page, cap, seed, max_new=256, spare=3):
        import torch
        self.P, self.rng = P, np.random.default_rng(seed)
        self.B, self.Hq, self.Hkv, self.d, self.bits, self.page = B, Hq, Hkv, d, bits, page
        self.io, self.dt = io_of(P, io)
        cols = (cap + page - 1) // page
        n_pages = B * cols + spare
        self.cfg = P.make_kv_config(Hq, Hkv, d, n_pages, B, bits=bits, page_tokens=page, max_new=max_new, io_dtype=self.io)
        self.kv = P.PaceKV(self.cfg)
        pool = n_pages * Hkv * (page // 32) * P.pace_kv_tile_bytes(self.cfg)
        base = (self.kv.mem.data_ptr() + 255) // 256 * 256 - self.kv.mem.data_ptr()
        end = base + self.kv.nbytes
        start = end - (pool + 255) // 256 * 256
        self.kv.mem[start:end] = 0xFF
        self.pool = self.kv.mem[start:start + pool]
        self.table_np = self.rng.permutation(n_pages)[:B * cols].reshape(B, cols).astype(np.int32)
        self.table = dev(self.table_np)
        self.k = np.zeros((B, cols * page, Hkv, d))
        self.v = np.zeros_like(self.k)
        torch.cuda.synchronize()

    def rand(self, *shape, amp=1.0):
        x = self.rng.standard_normal(shape).astype(np.float32) * np.float32(amp)
        return K.bf16(x) if self.io == self.P.PACE_IO_BF16 else x

    def append(self, lens, T, n_new=None, k=None, v=None):
        k = self.rand(self.B, T, self.Hkv, self.d, amp=1.5) if k is None else k
        v = self.rand(self.B, T, self.Hkv, self.d) if v is None else v
        self.kv.append(None, dev(k, self.dt), dev(v, self.dt), dev(np.asarray(lens, np.int32)), self.table,
                       n_new=None if n_new is None else dev(np.asarray(n_new, np.int32)))
        for b in range(self.B):
            n = T if n_new is None else min(max(n_new[b], 0), T)
            self.k[b, lens[b]:lens[b] + n] = K.held(k[b, :n], self.bits)
            self.v[b, lens[b]:lens[b] + n] = K.held(v[b, :n], self.bits)

    def read(self, n, first=None, end=None):
        import torch
        k, v = (torch.full((self.B, n, self.Hkv, self.d), 7.0, dtype=self.dt, device="cuda") for _ in range(2))
        self.kv.read(k, v, self.table, None if first is None else dev(np.asarray(first, np.int32)),
                     None if end is None else dev(np.asarray(end, np.int32)))
        return host(k), host(v)


def as_io(L, x):
    return K.bf16(x.astype(np.float32)) if L.io == L.P.PACE_IO_BF16 else x.astype(np.float32)


# ---- rotary positions ----------------------------------------------------------------------------------------------------------
ROPES = [dict(rot=64, d=64, layout="half"), dict(rot=128, d=128, layout="interleaved"),
         dict(rot=32, d=128, layout="half", scaling="linear", factor=4.0),
         dict(rot=64, d=256, layout="interleaved", scaling="ntk", factor=8.0),
         dict(rot=256, d=256, layout="half", scaling="parts", factor=4.0, orig_pos=4096),
         dict(rot=16, d=96, layout="half"), dict(rot=48, d=80, layout="interleaved", base=1e6)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kw", ROPES, ids=lambda k: f"{k['layout']}{k['rot']}of{k['d']}{k.get('scaling', '')}")
@pytest.mark.parametrize("n,heads", [(1, 1), (5, 3), (700, 9)])
def test_rope_forward_inverse_and_in_place(P, kw, io, n, heads):
    import torch
    kw = dict(kw)
    d, rot = kw.pop("d"), kw.pop("rot")
    rng = np.random.default_rng(n + d)
    x = rng.standard_normal((n, heads, d)).astype(np.float32)
    if io == "bf16":
        x = K.bf16(x)
    pos = rng.integers(0, 32768, n).astype(np.int32)
    pos[0] = 32767
    rope = P.PaceRope(rot, 32768, **kw)
    dt = io_of(P, io)[1]
    # a slice of a wider tensor: token and head strides other than the dense ones
    wide = torch.zeros(n, heads + 2, d + 8, dtype=dt, device="cuda")
    xin = wide[:, 1:heads + 1, :d]
    xin.copy_(dev(x, dt))
    out = torch.empty(n, heads, d, dtype=dt, device="cuda")
    for inverse in (False, True):
        P.pace_rope_apply(rope, xin, dev(pos), out, inverse=inverse)
        want = K.rotate(x, pos, rot, inverse=inverse, **kw)
        # two products and a sum rounded to fp32, with cos and sin rounded too: 4 half-ulps of |a| m + |b| m, m < 1.5
        tol = 1.5 * 2.0 ** -22 * np.abs(x).max()
        if io == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(want)
        assert (np.abs(host(out) - want) <= tol).all()
        assert np.array_equal(host(out)[..., rot:], x[..., rot:])
    P.pace_rope_apply(rope, xin, dev(pos), xin)
    want = K.rotate(x, pos, rot, **kw)
    assert (np.abs(host(xin) - want) <= 1.5 * 2.0 ** -22 * np.abs(x).max() + (2.0 ** -8 * np.abs(want) if io == "bf16" else 0)).all()
    assert (host(wide[:, 0]) == 0).all() and (host(wide[..., d:]) == 0).all()


def test_rope_inverse_is_the_gradient(P):
    """For y = rope(x) and L = sum(w y): dL/dx is the inverse rotation of w (m = 1), and agrees with differences of L."""
    rng = np.random.default_rng(3)
    n, h, d, rot = 4, 2, 64, 32
    x, w = rng.standard_normal((2, n, h, d)).astype(np.float32)
    pos = np.array([0, 1, 77, 999], np.int32)
    import torch
    rope = P.PaceRope(rot, 1000, layout="half")
    g = torch.empty(n, h, d, device="cuda")
    P.pace_rope_apply(rope, dev(w), dev(pos), g, inverse=True)
    loss = lambda z: float((K.rotate(z, pos, rot) * w).sum())
    eps = 1e-3
    for i in [(0, 0, 0), (1, 1, 5), (2, 0, 17), (3, 1, 31), (3, 0, 40)]:
        dx = np.zeros((n, h, d))
        dx[i] = eps
        diff = (loss(x.astype(np.float64) + dx) - loss(x.astype(np.float64) - dx)) / (2 * eps)
        # the loss is linear in x: the difference is exact but for 64-bit rounding; the kernel rounds three times to fp32
        assert abs(float(g[i]) - diff) <= 2.0 ** -21 * np.abs(w).max()


# ---- cache: write, read back, keep ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,bits,page", [(64, 4, 32), (64, 8, 64), (128, 4, 64), (128, 8, 128), (256, 4, 96), (256, 8, 32)])
def test_append_then_read_is_the_quantizer_bit_for_bit(P, d, bits, page, io):
    L = Layer(P, 4, 6, 3, d, bits, io, page, 400, seed=d + bits)
    k = L.rand(4, 200, 3, d, amp=2.0)
    k[0, 3] = 0.0                       # a zero vector
    k[1, 5, 0, :64] = 1e-41             # a group below the smallest normal scale
    k[2, 7, 1] = np.abs(k[2, 7, 1])     # one sign only (zero point at the end of its range)
    k[2, 8, 1] = -np.abs(k[2, 8, 1])
    k[3, 9, 2, 0] = 1e30                # one outlier
    lens = [0, 1, 31, 160]
    L.append(lens, 200, n_new=[200, 199, 33, 0], k=as_io(L, k))
    L.append([200, 200, 64, 160], 1)
    end = [201, 201, 65, 161]
    rk, rv = L.read(230, end=end)
    for b in range(4):
        s0 = lens[b]                    # slots below were never written
        assert np.array_equal(rk[b, s0:end[b]], as_io(L, L.k[b, s0:end[b]]))
        assert np.array_equal(rv[b, s0:end[b]], as_io(L, L.v[b, s0:end[b]]))
        assert (rk[b, end[b]:] == 0).all() and (rv[b, end[b]:] == 0).all()
    first = [5, 17, 33, 160]
    rk2, rv2 = L.read(3, first=first, end=end)
    for b in range(4):
        n = min(3, end[b] - first[b])
        assert np.array_equal(rk2[b, :n], rk[b, first[b]:first[b] + n]) and (rk2[b, n:] == 0).all()
        assert np.array_equal(rv2[b, :n], rv[b, first[b]:first[b] + n])
    assert L.kv.status() == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_non_finite_elements_stay_in_their_row(P, bits):
    L = Layer(P, 1, 2, 2, 128, bits, "f32", 32, 64, seed=1)
    k = L.rand(1, 9, 2, 128)
    k[0, 4, 1, 3], k[0, 4, 1, 70], k[0, 5, 0, 0] = np.nan, np.inf, -np.inf
    L.append([0], 9, k=k)
    rk, rv = L.read(9)
    assert np.isfinite(rk).all() and np.array_equal(rk[0], L.k[0, :9].astype(np.float32))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout,rot,d,bits", [("half", 64, 64, 8), ("interleaved", 32, 128, 4), ("half", 128, 256, 4),
                                               ("interleaved", 256, 256, 8), ("half", 16, 128, 8)])
@pytest.mark.parametrize("T,fused", [(1, False), (7, True), (150, True)])
def test_append_rotates_queries_and_keys(P, layout, rot, d, bits, io, T, fused):
    import torch
    B, Hq, Hkv = 3, 10, 2
    L = Layer(P, B, Hq, Hkv, d, bits, io, 64, 300, seed=T)
    rope = P.PaceRope(rot, 5000, layout=layout)
    lens = np.array([0, 33, 100], np.int32)
    pos = None if T == 1 else L.rng.integers(0, 5000, (B, T)).astype(np.int32)
    at = lens[:, None] + np.arange(T) if pos is None else pos
    q, k, v = L.rand(B, T, Hq, d), L.rand(B, T, Hkv, d), L.rand(B, T, Hkv, d)
    if fused:                           # views into one projection output [B, T, (Hq + 2 Hkv) d]
        qkv = dev(np.concatenate([q, k, v], 2), L.dt).reshape(B, T, -1, d)
        tq, tk, tv = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    else:
        tq, tk, tv = dev(q, L.dt), dev(k, L.dt), dev(v, L.dt)
    qo = tq if fused else torch.empty_like(tq)
    L.kv.append(tq, tk, tv, dev(lens), L.table, rope=rope, positions=None if pos is None else dev(pos), q_out=qo)
    want = K.rotate(q, at, rot, layout=layout)
    tol = 2.0 ** -22 * np.abs(q).max() + (2.0 ** -8 * np.abs(want) if io == "bf16" else 0)
    assert (np.abs(host(qo) - want) <= tol).all()
    rk, rv = L.read(T, first=lens)
    assert np.array_equal(rv, as_io(L, K.held(v, bits)))
    # keys: the fp32 rotation, then the quantizer; cos and sin of the 64-bit angle may round the other way, which can move a
    # code by one step where x/s is near a half (an fp32 error of about 2^-22 * 127 steps: well under one code in a thousand)
    kr = K.rotate(k, at, rot, layout=layout, dtype=np.float32)
    _, s, _ = K.quantize(kr, bits)
    wk = as_io(L, K.held(kr, bits))
    off = np.abs(rk - wk)
    step = np.repeat(s, 64, -1) * 1.02 + 2.0 ** -8 * np.abs(wk)
    assert (off <= step).all() and (off > 2.0 ** -7 * np.abs(wk)).mean() <= 1e-3
    assert L.kv.status() == 0


@pytest.mark.parametrize("d,bits,page", [(64, 4, 32), (128, 4, 64), (64, 8, 32), (128, 8, 32), (256, 4, 128), (256, 8, 32)])
def test_keep_moves_the_path_and_nothing_else(P, d, bits, page):
    B, Hkv = 5, 2
    L = Layer(P, B, 2, Hkv, d, bits, "f32", page, 320, seed=9)
    lens = [0, 31, 32, 90, 100]
    L.append([0] * B, 200)
    L.append(lens, 70)
    idx = np.zeros((B, 45), np.int32)
    nk = np.array([45, 1, 0, 40, 3], np.int32)
    for b in range(B):
        idx[b, :nk[b]] = np.sort(L.rng.permutation(70)[:nk[b]])
    idx[4, :3] = [0, 1, 69]
    L.kv.keep(dev(np.asarray(lens, np.int32)), L.table, dev(idx), dev(nk))
    rk, rv = L.read(200)
    for b in range(B):
        wk, wv = L.k[b].copy(), L.v[b].copy()
        wk[lens[b]:lens[b] + nk[b]] = L.k[b, lens[b] + idx[b, :nk[b]]]
        wv[lens[b]:lens[b] + nk[b]] = L.v[b, lens[b] + idx[b, :nk[b]]]
        assert np.array_equal(rk[b], wk[:200].astype(np.float32)) and np.array_equal(rv[b], wv[:200].astype(np.float32))
    assert L.kv.status() == 0


# ---- attention -------------------------------------------------------------------------------------------------------------------
def tree_mask(rng, B, T, empty=False):
    see = np.zeros((B, T, T), bool)
    for b in range(B):
        for t in range(T):
            p = int(rng.integers(-1, t)) if t else -1
            if p >= 0:
                see[b, t] = see[b, p]
            see[b, t, t] = True
    if empty:
        see[:, T // 2] = False
    words = np.zeros((B, T, (T + 31) // 32), np.uint32)
    for j in range(T):
        words[:, :, j // 32] |= see[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return see, words.view(np.int32)


def check_attend(L, T, lens, n_new=None, mask="causal", q=None, scale=None, view=False, out=None):
    import torch
    B, Hq, d = L.B, L.Hq, L.d
    q = L.rand(B, T, Hq, d, amp=1.5) if q is None else q
    if mask == "causal":
        see, words = np.broadcast_to(np.tril(np.ones((T, T), bool)), (B, T, T)), None
    else:
        see, words = tree_mask(L.rng, B, T, empty=mask == "empty")
    tq = dev(q, L.dt)
    o = torch.full((B, T, Hq, d), 7.0, dtype=L.dt, device="cuda")
    if view:                            # heads-major outputs and queries
        tq = tq.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        o = o.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    L.kv.attend(tq, o, dev(np.asarray(lens, np.int32)), L.table, mask=None if words is None else dev(words),
                n_new=None if n_new is None else dev(np.asarray(n_new, np.int32)), scale=scale)
    got = host(o)
    assert L.kv.status() == 0
    sc = d ** -0.5 if scale is None else scale
    bf = L.io == L.P.PACE_IO_BF16
    num = den = 0.0
    for b in range(B):
        n = T if n_new is None else min(max(n_new[b], 0), T)
        total = lens[b] + n
        vis = np.concatenate([np.ones((T, lens[b]), bool), see[b][:, :n]], 1)
        vis[n:] = False
        k, v = L.k[b, :total], L.v[b, :total]
        want = K.attend(q[b].astype(np.float64), k, v, vis, sc)
        assert (got[b][~vis.any(1)] == 0).all()
        if not total:
            continue
        # a score is a sum of products: its error is at most eps * sum|q||k| * scale, eps = 2^-20 for fp32 queries (sums of
        # exact parts in fp32) and 2^-11 for bf16 ones (keys may be rounded to 11 bits for the tensor cores); a weight is
        # off by that relative to itself, twice after normalising; weights are rounded to 8 bits (bf16 I/O), and so is o.
        G = L.Hq // L.Hkv
        mag = np.abs(q[b]).transpose(1, 0, 2) @ np.repeat(np.abs(k).transpose(1, 2, 0), G, 0)      # [Hq, T, total]
        ds = (2.0 ** -11 if bf else 2.0 ** -20) * abs(sc) * mag.max()
        vmax = np.abs(v).max()
        tol = 2 * ds * vmax + (2.0 ** -8 if bf else 2.0 ** -19) * vmax
        assert np.abs(got[b] - want).max() <= tol, (b, np.abs(got[b] - want).max(), tol)
        num += ((got[b] - want) ** 2).sum()
        den += (want ** 2).sum()
    # rms of the same: 8-bit weights and 8-bit outputs are each off by about 2^-9 of themselves, fp32 by a few 1e-7 of scores
    # of about ten
    if den:
        assert np.sqrt(num / den) <= (4e-3 if bf else 1e-5), np.sqrt(num / den)
    return got


SHAPES = [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,bits", SHAPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (8, 1), (14, 2), (32, 2)])
def test_attend_single_tokens(P, d, bits, Hq, Hkv, io):
    lens = [0, 1, 30, 31, 32, 33, 100, 257]
    L = Layer(P, 8, Hq, Hkv, d, bits, io, 32 if bits == 8 else 64, 300, seed=d)
    L.append([0] * 8, 256)
    L.append([256] * 8, 1)
    L.append(lens, 1)
    check_attend(L, 1, lens)
    check_attend(L, 1, lens, n_new=[1, 0, 1, 0, 1, 1, 0, 1], scale=0.3)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,bits", SHAPES)
@pytest.mark.parametrize("T,G", [(2, 4), (5, 3), (16, 1), (25, 4), (40, 8)])
def test_attend_trees_with_empty_rows(P, d, bits, T, G, io):
    lens = [0, 31, 60, 200]
    L = Layer(P, 4, 2 * G, 2, d, bits, io, 32, 300, seed=T)
    L.append([0] * 4, 256)
    L.append(lens, T)
    check_attend(L, T, lens, mask="tree")
    check_attend(L, T, lens, mask="empty", n_new=[T, T - 1, 0, 1], view=True)
    check_attend(L, T, lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,bits", SHAPES)
def test_attend_prompt_chunks(P, d, bits, io):
    lens = [0, 100, 333]
    L = Layer(P, 3, 6, 2, d, bits, io, 64, 700, seed=4)
    L.append([0] * 3, 256)
    L.append([256] * 3, 100)
    L.append(lens, 256)
    check_attend(L, 256, lens)
    check_attend(L, 193, lens, n_new=[193, 77, 1], view=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,T,n", [(1, 8, 1, 1, 20000), (1, 4, 4, 3, 9000), (2, 8, 2, 20, 5000), (1, 2, 1, 100, 6000)])
def test_attend_long_contexts_are_split_and_joined(P, B, Hq, Hkv, T, n, io):
    L = Layer(P, B, Hq, Hkv, 128, 4 if T != 3 else 8, io, 128, n + T, seed=n, max_new=4096)
    for at in range(0, n, 4000):
        L.append([at] * B, min(4000, n - at))
    lens = [n - 37 * b for b in range(B)]
    L.append(lens, T)
    a = check_attend(L, T, lens, mask="tree" if T > 1 else "causal")
    L.rng = np.random.default_rng(0)
    x = check_attend(L, T, lens)
    L.rng = np.random.default_rng(0)
    y = check_attend(L, T, lens)
    assert np.array_equal(x, y)         # the same call gives the same bits


@pytest.mark.parametrize("T", [1, 30, 256])
@pytest.mark.parametrize("bits", [4, 8])
def test_attend_ignores_what_the_mask_hides(P, bits, T):
    """Huge and non-finite drafts that a row does not see, and unwritten slots with NaN scales, leave that row unchanged."""
    import torch
    L = Layer(P, 2, 8, 2, 128, bits, "bf16", 64, 500, seed=2)
    L.append([0, 0], 180)
    lens = [150, 64]
    k, v = L.rand(2, T, 2, 128), L.rand(2, T, 2, 128)
    hide = T // 2 if T > 1 else None
    if hide:
        k[:, hide], v[:, hide] = np.inf, np.nan
        v[:, hide, :, ::2] = np.inf
    L.append(lens, T, k=k, v=v)
    q = L.rand(2, T, 8, 128)
    words = np.zeros((2, T, (T + 31) // 32), np.uint32)
    vis = np.tril(np.ones((T, T), bool))
    if hide:
        vis[:, hide] = False
    for j in range(T):
        words[:, :, j // 32] |= vis[None, :, j].astype(np.uint32) << np.uint32(j % 32)
    o = torch.empty(2, T, 8, 128, dtype=torch.bfloat16, device="cuda")
    L.kv.attend(dev(q, L.dt), o, dev(np.asarray(lens, np.int32)), L.table, mask=dev(words.view(np.int32)))
    got = host(o)
    for b in range(2):
        want = K.attend(q[b].astype(np.float64), L.k[b, :lens[b] + T], L.v[b, :lens[b] + T],
                        np.concatenate([np.ones((T, lens[b]), bool), vis], 1), 128 ** -0.5)
        assert np.sqrt(((got[b] - want) ** 2).sum() / (want ** 2).sum()) <= 4e-3


@pytest.mark.parametrize("T", [1, 40])
def test_attend_sink_tokens_with_tiny_values(P, T):
    """A first token that takes nearly all of the weight and holds values a million times smaller than the others."""
    L = Layer(P, 1, 16, 2, 128, 4, "bf16", 64, 400, seed=5)
    k, v = L.rand(1, 300, 2, 128), L.rand(1, 300, 2, 128)
    q = L.rand(1, T, 16, 128)
    q[..., 0] = 8.0
    k[0, 0, :, 0], v[0, 0] = 16.0, v[0, 0] * np.float32(2.0 ** -20)
    L.append([0], 256, k=k[:, :256], v=v[:, :256])
    L.append([256], T, k=L.rand(1, T, 2, 128), v=L.rand(1, T, 2, 128))
    check_attend(L, T, [256], q=q)


def test_calls_run_on_their_stream_and_replay_from_a_graph(P):
    import torch
    L = Layer(P, 2, 8, 2, 128, 4, "bf16", 64, 300, seed=8)
    L.append([0, 0], 200)
    lens = dev(np.array([200, 150], np.int32))
    s = torch.cuda.Stream()
    q, k, v = (dev(L.rand(2, 1, h, 128), L.dt) for h in (8, 2, 2))
    rope = P.PaceRope(128, 400)
    qo, o = torch.empty_like(q), torch.empty_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        L.kv.append(q, k, v, lens, L.table, rope=rope, q_out=qo)
        L.kv.attend(qo, o, lens, L.table)
    s.synchronize()
    want = host(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        L.kv.append(q, k, v, lens, L.table, rope=rope, q_out=qo)
        L.kv.attend(qo, o, lens, L.table)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(o), want)


def test_bad_device_indices_are_reported_and_touch_nothing(P):
    import torch
    L = Layer(P, 2, 2, 2, 64, 8, "f32", 32, 64, seed=6)
    L.append([0, 0], 40)
    before = L.pool.clone()
    x = torch.zeros(2, 4, 2, 64, device="cuda")
    bad = L.table.clone()
    bad[0, 1], bad[1, 1] = -1, L.cfg.n_pages
    L.kv.append(None, x, x, dev(np.array([40, 40], np.int32)), bad)
    assert L.kv.status(clear=True) == P.PACE_KV_BAD_PAGE
    L.kv.append(None, x, x, dev(np.array([64, -3], np.int32)), L.table)
    assert L.kv.status(clear=True) == P.PACE_KV_BAD_PAGE
    L.kv.keep(dev(np.array([40, 40], np.int32)), L.table, dev(np.array([[1, 1], [-1, 2]], np.int32)), dev(np.array([2, 2], np.int32)))
    assert L.kv.status(clear=True) == P.PACE_KV_BAD_KEEP
    after = L.pool.clone()
    # (the first kept index of sequence 0 is good: slot 41 moved to 40)
    assert (before != after).sum() <= 2 * 2 * (64 + 2)
    o = torch.full((2, 4, 2, 64), 7.0, device="cuda")
    L.kv.attend(x, o, dev(np.array([40, 10], np.int32)), bad)
    assert L.kv.status(clear=True) == P.PACE_KV_BAD_PAGE
    assert torch.isfinite(o).all()
    k, v = torch.empty_like(x), torch.empty_like(x)
    L.kv.read(k, v, bad, first=dev(np.array([30, 30], np.int32)))
    assert L.kv.status(clear=True) == P.PACE_KV_BAD_PAGE
    assert (k[:, 2:] == 0).all()
    rope = P.PaceRope(64, 10)
    L.kv.append(x, x, x, dev(np.array([8, 0], np.int32)), L.table, rope=rope, q_out=torch.empty_like(x))
    assert L.kv.status(clear=True) == P.PACE_KV_BAD_POSITION
    assert L.kv.status() == 0


def test_calls_refuse_wrong_arguments(P):
    import torch
    L = Layer(P, 2, 4, 2, 64, 8, "bf16", 32, 64, seed=6, max_new=8)
    lens = dev(np.array([0, 0], np.int32))
    q, k = (torch.zeros(2, 3, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    rope = P.PaceRope(64, 100)
    for bad in (k.float(), k[:, :, :1], k.cpu(), torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16, device="cuda")[..., ::2]):
        with pytest.raises(ValueError):
            L.kv.append(None, bad, k, lens, L.table)
    wide = torch.zeros(2, 3, 2, 72, dtype=torch.bfloat16, device="cuda")
    L.kv.append(None, wide[..., 8:], k, lens, L.table)                     # 16-byte offset and strides: fine
    wide = torch.zeros(2, 3, 2, 68, dtype=torch.bfloat16, device="cuda")
    for fn in (lambda: L.kv.append(None, wide[..., :64], k, lens, L.table),  # strides of 136 bytes
               lambda: L.kv.append(q, k, k, lens, L.table, q_out=q),         # rotation without a table
               lambda: L.kv.append(q, k, k, lens, L.table, rope=rope),       # q without q_out
               lambda: L.kv.append(None, k, k, lens, L.table, rope=P.PaceRope(128, 100)),
               lambda: L.kv.attend(q, q, lens, L.table, scale=float("inf")),
               lambda: L.kv.append(None, *(2 * [torch.zeros(2, 9, 2, 64, dtype=torch.bfloat16, device="cuda")]), lens, L.table),
               lambda: L.kv.append(None, *(2 * [torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16, device="cuda")]),
                                   torch.zeros(3, dtype=torch.int32, device="cuda"),
                                   torch.zeros(3, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(P.PaceError) as e:
            fn()
        assert e.value.status == 1
    for fn in (lambda: L.kv.append(None, k, k, lens.long(), L.table), lambda: L.kv.append(None, k, k, lens[:1], L.table),
               lambda: L.kv.append(None, k, k, lens, L.table[0]), lambda: L.kv.append(None, k, k, lens, L.table.t()),
               lambda: L.kv.attend(q, q, lens, L.table, mask=torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fn()
    empty = torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    L.kv.append(None, empty, empty, lens, L.table)                          # no tokens: nothing to do
    e4 = torch.zeros(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    L.kv.attend(e4, e4, lens, L.table)
    assert L.kv.status() == 0
