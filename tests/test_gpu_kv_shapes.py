"""Attention over the cache where the work is split unusually: very many short sequences, tables and pools beyond 32 bits, odd pages,
scales of any sign, tokens of very different size, random shapes. Tolerances are those of test_gpu_kv.check_attend unless stated."""
import numpy as np
import pytest

import kv_testlib as K
from test_gpu_kv import P, Layer, check_attend, dev, host  # noqa: F401  (P is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,Hkv,T,d,bits,io", [(330, 16, 16, 1, 256, 8, "f32"), (1000, 4, 2, 1, 64, 4, "bf16"), (90, 6, 3, 5, 128, 8, "bf16"),
                                                  (300, 8, 2, 12, 128, 4, "bf16"), (70, 2, 1, 130, 64, 8, "bf16"), (200, 8, 1, 6, 256, 4, "bf16")])
def test_attend_many_short_sequences(P, B, Hq, Hkv, T, d, bits, io):
    """More sequences, and more items a block, than the kernels keep at hand at a time; a third of the sequences are empty."""
    cap = 32 if T == 1 else 128 + T
    L = Layer(P, B, Hq, Hkv, d, bits, io, 32, cap, seed=B)
    n = cap - T
    L.append([0] * B, min(n, 200))
    lens = np.where(L.rng.random(B) < 0.33, 0, L.rng.integers(0, min(n, 200) + 1, B)).tolist()
    L.append(lens, T)
    n_new = L.rng.integers(0, T + 1, B).tolist()
    check_attend(L, T, lens, mask="tree" if T > 1 else "causal")
    check_attend(L, T, lens, n_new=n_new)


@pytest.mark.parametrize("T", [1, 130])
def test_attend_with_tables_for_2_to_the_30_tokens(P, T):
    """What the tables could hold passes 2^31 tiles, and the call is split over the sequences."""
    import torch
    B = 40
    L = Layer(P, B, 8, 2, 64, 4, "bf16", 4096, 300 + T, seed=7)
    L.append([0] * B, 256)
    lens = L.rng.integers(0, 257, B).tolist()
    L.append(lens, T)
    table = torch.full((B, 1 << 18), -1, dtype=torch.int32, device="cuda")
    table[:, :L.table.shape[1]] = L.table
    L.table = table
    check_attend(L, T, lens)


@pytest.mark.parametrize("T", [1, 40])
def test_pool_beyond_4_gb(P, T):
    L = Layer(P, 2, 8, 2, 256, 8, "bf16", 4096, 300, seed=9, spare=1100)
    last = L.cfg.n_pages - 1
    L.table_np = np.array([[last], [last - 1]], np.int32)
    L.table = dev(L.table_np)
    assert L.pool.numel() > 2 ** 32
    lens = [200, 131]
    L.append([0, 0], 200)
    L.append(lens, T)
    check_attend(L, T, lens)
    k, _ = L.read(200)
    assert np.array_equal(k[0], K.bf16(L.k[0, :200].astype(np.float32)))


@pytest.mark.parametrize("page", [96, 160])
@pytest.mark.parametrize("d,bits,T", [(64, 8, 1), (128, 4, 1), (128, 4, 40), (64, 4, 150), (256, 8, 40)])
def test_attend_pages_of_odd_tiles(P, page, d, bits, T):
    L = Layer(P, 3, 8, 2, d, bits, "bf16", page, 700, seed=page + T)
    L.append([0] * 3, 256)
    L.append([256] * 3, 256)
    lens = [511, 95, 320]
    L.append(lens, T)
    check_attend(L, T, lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.11])
@pytest.mark.parametrize("d,T", [(64, 1), (128, 1), (128, 40), (64, 100), (256, 20)])
def test_attend_any_scale(P, io, scale, d, T):
    L = Layer(P, 2, 8, 2, d, 4, io, 64, 400, seed=11)
    L.append([0, 0], 200)
    L.append([200, 77], T)
    check_attend(L, T, [200, 77], scale=scale, mask="tree" if T > 1 else "causal")


@pytest.mark.parametrize("d,bits,T,G", [(128, 4, 40, 4), (64, 8, 60, 8), (256, 4, 70, 1), (128, 8, 200, 2), (128, 4, 6, 4)])
def test_attend_new_tokens_of_very_different_size(P, d, bits, T, G):
    """Rows that see one new token each, of sizes from 2^-40 to 2^20: each gets that token's values. One weight and its sum are 2^-11
    apart at most and a value rounded to 11 bits is off by 2^-11, so an output is the bf16 of something within 2^-10 of the value."""
    import torch
    L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, 400, seed=13)
    size = (2.0 ** L.rng.integers(-40, 21, T)).astype(np.float32)
    k = K.bf16(L.rand(1, T, 2, d) * 2.0 ** L.rng.integers(-40, 0, T).astype(np.float32)[None, :, None, None])
    v = K.bf16(L.rand(1, T, 2, d) * size[None, :, None, None])
    L.append([0], T, k=k, v=v)
    q = L.rand(1, T, 2 * G, d)
    words = np.zeros((1, T, (T + 31) // 32), np.uint32)
    for t in range(T):
        words[0, t, t // 32] = np.uint32(1) << np.uint32(t % 32)
    o = torch.empty(1, T, 2 * G, d, dtype=torch.bfloat16, device="cuda")
    L.kv.attend(dev(q, L.dt), o, dev(np.array([0], np.int32)), L.table, mask=dev(words.view(np.int32)))
    want = np.repeat(L.v[0, :T], G, axis=1)
    got = np.abs(host(o)[0])
    low, high = (K.bf16((np.abs(want) * f).astype(np.float32)) for f in (1 - 2.0 ** -10, 1 + 2.0 ** -10))
    assert ((low <= got) & (got <= high)).all() and (np.sign(host(o)[0]) == np.sign(want)).all()


@pytest.mark.parametrize("d,bits,T,G,B", [(128, 4, 600, 2, 1), (64, 8, 1000, 1, 2), (256, 4, 300, 4, 1), (128, 8, 120, 1, 40), (128, 4, 30, 1, 1)])
def test_attend_rows_that_see_only_late_tokens(P, d, bits, T, G, B):
    """Rows that see nothing in the first tiles of an item, or of a block's share of it, and a few tokens with very low scores later:
    the weights are relative to those, and the share counts when the results are joined."""
    import torch
    L = Layer(P, B, 2 * G, 2, d, bits, "bf16", 64, T, seed=17, max_new=1024)
    L.append([0] * B, T)
    q = L.rand(B, T, 2 * G, d)
    q[..., :8] = -3.0
    k = L.rand(B, T, 2, d)
    k[..., :8] = 6.0                                       # scores of about -144 / sqrt(d), all alike
    L.append([0] * B, T, k=k)
    words = np.zeros((B, T, (T + 31) // 32), np.uint32)
    vis = np.zeros((T, T), bool)
    for t in range(T):
        vis[t, max(0, t - 2):t + 1] = True
    for j in range(T):
        words[:, :, j // 32] |= vis[:, j].astype(np.uint32) << np.uint32(j % 32)
    o = torch.empty(B, T, 2 * G, d, dtype=torch.bfloat16, device="cuda")
    L.kv.attend(dev(q, L.dt), o, dev(np.zeros(B, np.int32)), L.table, mask=dev(words.view(np.int32)))
    got = host(o)
    for b in range(0, B, 13):
        want = K.attend(q[b].astype(np.float64), L.k[b, :T], L.v[b, :T], vis, d ** -0.5)
        # as in check_attend: scores off by 2^-11 of the sums of their products' sizes, weights and outputs by 8 bits
        mag = (np.abs(q[b]).max(0) @ np.abs(L.k[b, :T]).max((0, 1))).max() * d ** -0.5
        assert np.abs(got[b] - want).max() <= (2 * 2.0 ** -11 * mag + 2.0 ** -8) * np.abs(L.v[b, :T]).max()
        assert np.sqrt(((got[b] - want) ** 2).sum() / (want ** 2).sum()) <= 4e-3


@pytest.mark.parametrize("T", [1, 40, 200])
def test_attend_bad_pages_and_lengths_are_reported(P, T):
    import torch
    L = Layer(P, 2, 8, 2, 128, 4, "bf16", 32, 300, seed=6)
    L.append([0, 0], 90)
    L.append([90, 90], T)
    q = torch.ones(2, T, 8, 128, dtype=torch.bfloat16, device="cuda")
    bad = L.table.clone()
    bad[0, 1], bad[1, 2] = -1, L.cfg.n_pages
    for lens, table in (([90, 90], bad), ([10 ** 9, -5], L.table), ([2 ** 31 - 1, 2 ** 31 - 1], L.table)):
        o = torch.full_like(q, 7.0)
        L.kv.append(None, q[:, :, :2].contiguous() * 0, q[:, :, :2].contiguous() * 0, dev(np.zeros(2, np.int32)), L.table)
        L.kv.attend(q, o, dev(np.array(lens, np.int32)), table)
        assert L.kv.status(clear=True) == P.PACE_KV_BAD_PAGE
        if table is bad:
            assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("seed", range(32))
def test_attend_random_shapes(P, seed):
    r = np.random.default_rng(1000 + seed)
    d, bits, io = int(r.choice([64, 128, 256])), int(r.choice([4, 8])), str(r.choice(["f32", "bf16", "bf16"]))
    Hkv, G = int(r.integers(1, 5)), int(r.integers(1, 9))
    T = int(np.exp(r.uniform(0, np.log(200))))
    B = int(np.exp(r.uniform(0, np.log(24))))
    page = 32 * int(r.integers(1, 6))
    n = int(np.exp(r.uniform(np.log(20), np.log(2000))))
    L = Layer(P, B, G * Hkv, Hkv, d, bits, io, page, n + T, seed=seed, max_new=2048)
    L.append([0] * B, n)
    lens = r.integers(0, n + 1, B).tolist()
    lens[0] = n
    L.append(lens, T)
    n_new = None if seed % 3 else r.integers(0, T + 1, B).tolist()
    check_attend(L, T, lens, n_new=n_new, mask=["causal", "tree", "empty"][seed % 3] if T > 1 else "causal", view=bool(seed % 2))


@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4)])
def test_fp32_over_long_stretches_of_tiles(P, d, bits):
    """So many tokens that each warp adds up over a hundred tiles: rounding errors may grow like a random walk but not all lean one way.
    Scores of up to about 16 bits are off by a few 2^-21 of one, a weight by as much of itself and by ex2's 2^-22; averaged over the
    rows' many tokens that stays below 1.5e-6 of the outputs."""
    import torch
    B, Hq, Hkv, n = 16, 16, 8, 16000
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cols = n // 128 + 1
    kv = P.PaceKV(P.make_kv_config(Hq, Hkv, d, B * cols, B, bits=bits, page_tokens=128, max_new=4096, io_dtype=P.PACE_IO_F32))
    table = torch.randperm(B * cols, generator=g, device="cuda").int().view(B, cols)
    for at in range(0, n, 4000):
        kv.append(None, rand(B, 4000, Hkv, d), rand(B, 4000, Hkv, d), torch.full((B,), at, dtype=torch.int32, device="cuda"), table)
    lens = torch.full((B,), n - 2, dtype=torch.int32, device="cuda")
    q = 2 * rand(B, 2, Hq, d)
    o = torch.empty_like(q)
    kv.attend(q, o, lens, table)
    k, v = torch.empty(2, B, n, Hkv, d, device="cuda")
    kv.read(k, v, table)
    num = den = 0.0
    for b in range(B):
        for h in range(Hq):
            s = (q[b, :, h].double() @ k[b, :, h // 2].double().t()) * d ** -0.5
            s[0, n - 1] = -torch.inf
            want = torch.softmax(s, -1) @ v[b, :, h // 2].double()
            num += float(((o[b, :, h].double() - want) ** 2).sum())
            den += float((want ** 2).sum())
    assert (num / den) ** 0.5 <= 1.5e-6


@pytest.mark.parametrize("d,T", [(128, 40), (64, 200), (256, 20)])
def test_many_rows_on_another_stream_and_from_a_graph(P, d, T):
    import torch
    L = Layer(P, 3, 8, 2, d, 4, "bf16", 64, 700, seed=21)
    L.append([0] * 3, 256)
    L.append([256] * 3, 200)
    lens = dev(np.array([456, 100, 333], np.int32))
    q, k, v = (dev(L.rand(3, T, h, d), L.dt) for h in (8, 2, 2))
    qo, o = torch.empty_like(q), torch.empty_like(q)
    rope = P.PaceRope(64, 1000)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step():
        L.kv.append(q, k, v, lens, L.table, rope=rope, q_out=qo)
        L.kv.attend(qo, o, lens, L.table)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    want = host(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(o), want)
    assert np.isfinite(want).all() and L.kv.status() == 0
