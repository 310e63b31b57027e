"""Attention-layer operators at the edges of what they accept: padding rows that hold anything, values hidden, lost, empty, infinite or of
very different size."""
import os
import subprocess
import sys

import numpy as np
import pytest

import kv_testlib as K
from test_gpu_kv import P, Layer, dev, host  # noqa: F401  (P is a fixture)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def words_of(see):
    """Mask words [B, T, words] (int32) of see [B, T, T]."""
    B, T, _ = see.shape
    words = np.zeros((B, T, (T + 31) // 32), np.uint32)
    for j in range(T):
        words[:, :, j // 32] |= see[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return words.view(np.int32)


def attend(L, q, lens, see=None, n_new=None, table=None):
    import torch
    o = torch.full(q.shape, 7.0, dtype=L.dt, device="cuda")
    L.kv.attend(dev(q, L.dt), o, dev(np.asarray(lens, np.int32)), L.table if table is None else table,
                mask=None if see is None else dev(words_of(see)), n_new=None if n_new is None else dev(np.asarray(n_new, np.int32)))
    return host(o)


def relative(got, want):
    return float(np.sqrt(((got.astype(np.float64) - want) ** 2).sum() / (want ** 2).sum()))


def expected(L, b, q, len_, T, see=None, hidden=()):
    """The attention of sequence b's T new tokens in 64 bits; `hidden` slots are seen by no row."""
    vis = np.concatenate([np.ones((T, len_), bool), np.tril(np.ones((T, T), bool)) if see is None else see], 1)
    vis[:, list(hidden)] = False
    return K.attend(q[b].astype(np.float64), L.k[b, :len_ + T], L.v[b, :len_ + T], vis, L.d ** -0.5)


# Root mean square errors. bf16: rounding an output to 8 bits is 2^-9.2 of it; queries, weights and held values of 11 bits an eighth of that
# each, and twice as much by way of the scores (of a few units): all together below 1.2 times 2^-9. fp32: as in check_attend.
LIMIT = {"bf16": 1.2 * 2.0 ** -9, "f32": 1e-5}


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("d,bits,T,G,io,n", [(128, 4, 3, 4, "bf16", 100), (64, 8, 6, 4, "f32", 100), (64, 8, 30, 1, "bf16", 100), (128, 8, 40, 2, "bf16", 150),
                                             (64, 4, 100, 4, "bf16", 150), (256, 4, 60, 1, "bf16", 150), (128, 4, 5, 1, "bf16", 6000),
                                             (64, 4, 5, 1, "f32", 6000), (128, 4, 100, 2, "bf16", 6000)])
def test_padding_rows_may_hold_anything(P, d, bits, T, G, io, n, fill):
    """Queries of rows at and past n_new are not looked at: those rows are zeros, and the others as if the padding were zeros."""
    L = Layer(P, 3, 2 * G, 2, d, bits, io, 64, n + T, seed=T)
    for at in range(0, n, 256):
        L.append([at] * 3, min(256, n - at))
    lens, n_new = [n, n // 2, 0], [T - 1, T // 2, 0]
    L.append(lens, T)
    q = L.rand(3, T, 2 * G, d)
    for b in range(3):
        q[b, n_new[b]:] = 0
    want = attend(L, q, lens, n_new=n_new)
    for b in range(3):
        q[b, n_new[b]:] = fill
    got = attend(L, q, lens, n_new=n_new)
    for b in range(3):
        assert (got[b, n_new[b]:] == 0).all()
        assert np.array_equal(got[b, :n_new[b]], want[b, :n_new[b]])
    assert np.isfinite(want).all() and L.kv.status() == 0


@pytest.mark.parametrize("size", [np.inf, 2.0 ** 40])
@pytest.mark.parametrize("d,bits,G", [(128, 4, 2), (64, 8, 1), (256, 4, 1), (256, 8, 1)])
def test_whole_tiles_that_the_mask_hides(P, d, bits, G, size):
    """Drafts 64..127, hidden from the rows behind them, hold huge keys and values; those rows see what they see without them."""
    T, ctx = 192, 64
    L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, ctx + T, seed=d)
    L.append([0], ctx)
    k, v = L.rand(1, T, 2, d), L.rand(1, T, 2, d)
    k[:, 64:128], v[:, 64:128] = (np.inf, np.inf) if np.isinf(size) else (k[:, 64:128] * np.float32(size), v[:, 64:128] * np.float32(size))
    L.append([ctx], T, k=k, v=v)
    q = L.rand(1, T, 2 * G, d)
    see = np.tril(np.ones((T, T), bool))
    see[128:, :128] = False
    got = attend(L, q, [ctx], see[None])
    want = expected(L, 0, q, ctx, T, see)
    assert relative(got[0, 128:], want[128:]) <= LIMIT["bf16"]
    # rows that see the new tokens behind the hidden ones alone
    L2 = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, T, seed=d)
    L2.append([0], T, k=k, v=v)
    got = attend(L2, q, [0], see[None])
    assert relative(got[0, 128:], expected(L2, 0, q, 0, T, see)[128:]) <= LIMIT["bf16"]


@pytest.mark.parametrize("d,bits,T,G", [(128, 4, 1, 4), (128, 4, 40, 2), (64, 8, 100, 2), (128, 8, 150, 1), (256, 4, 50, 1), (256, 8, 50, 1)])
def test_zero_values_beside_tiny_ones(P, d, bits, T, G):
    """A context whose first tiles hold zero values, and the others 2^-30: the weights of the others keep their bits."""
    L = Layer(P, 2, 2 * G, 2, d, bits, "bf16", 64, 512 + T, seed=3)
    lens = [512, 300]
    for at in (0, 256):
        v = L.rand(2, 256, 2, d) * np.float32(2.0 ** -30)
        if at == 0:
            v[:, :128] = 0
        L.append([at] * 2, 256, v=K.bf16(v))
    L.append(lens, T, v=K.bf16(L.rand(2, T, 2, d) * np.float32(2.0 ** -30)))
    q = L.rand(2, T, 2 * G, d)
    got = attend(L, q, lens)
    for b in range(2):
        assert relative(got[b], expected(L, b, q, lens[b], T)) <= LIMIT["bf16"]


@pytest.mark.parametrize("d,bits,T,G", [(128, 4, 40, 2), (64, 8, 100, 2), (256, 4, 50, 1)])
def test_a_zero_draft_beside_tiny_ones(P, d, bits, T, G):
    """New tokens of very different size (one of them hidden and large), among them one whose values are zero."""
    L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, T, seed=4)
    v = L.rand(1, T, 2, d) * np.float32(2.0 ** -30)
    v[0, 1], v[0, 2] = 0, 1e3
    L.append([0], T, v=K.bf16(v))
    q = L.rand(1, T, 2 * G, d)
    see = np.tril(np.ones((T, T), bool))
    see[:, 2] = False
    got = attend(L, q, [0], see[None])
    want = expected(L, 0, q, 0, T, see)
    assert relative(got[0, 3:], want[3:]) <= LIMIT["bf16"]


CONTEXTS = [(128, 4, 1, 4), (64, 8, 20, 1), (128, 4, 40, 2), (64, 8, 100, 2), (128, 8, 150, 1), (256, 4, 50, 1), (256, 8, 50, 1)]


@pytest.mark.parametrize("d,bits,T,G", CONTEXTS)
def test_large_context_tiles_of_no_weight(P, d, bits, T, G):
    """The first 128 context tokens hold values 2^30 times larger than the others' and take no weight worth naming."""
    L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, 512 + T, seed=7)
    q = L.rand(1, T, 2 * G, d)
    q[..., 0] = 8.0
    for at in (0, 256):
        k, v = L.rand(1, 256, 2, d), L.rand(1, 256, 2, d)
        k[..., 0] = 0
        if at == 0:
            v[0, :128] *= np.float32(2.0 ** 30)
            k[0, :128, :, 0] = -12.0 * d ** 0.5
        L.append([at], 256, k=k, v=v)
    L.append([512], T, k=L.rand(1, T, 2, d) * 0.1)
    got = attend(L, q, [512])
    assert relative(got[0], expected(L, 0, q, 512, T)) <= LIMIT["bf16"]


@pytest.mark.parametrize("d,bits,T,G", CONTEXTS)
def test_tiny_values_of_much_weight_after_others(P, d, bits, T, G):
    """A context whose later tokens score 60 bits higher but hold values 2^-80 of the first ones': both sides of the product count."""
    L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, 512 + T, seed=8)
    q = L.rand(1, T, 2 * G, d, amp=0.1)
    q[..., 0] = 8.0
    for at in (0, 256):
        k, v = L.rand(1, 256, 2, d, amp=0.1), L.rand(1, 256, 2, d)
        k[..., 0] = 0
        if at == 256:
            v *= np.float32(2.0 ** -80)
            k[..., 0] = 41.6 / 8 * d ** 0.5                 # 41.6 nats
        L.append([at], 256, k=K.bf16(k), v=K.bf16(v))
    k = L.rand(1, T, 2, d, amp=0.1)
    k[..., 0] = 41.6 / 8 * d ** 0.5
    L.append([512], T, k=K.bf16(k), v=K.bf16(L.rand(1, T, 2, d) * np.float32(2.0 ** -80)))
    got = attend(L, q, [512])
    # the first tokens' part is e^-41.6 2^80 times the others': it alone is the output. Its scores differ from the others' by a key element of
    # up to 84 in products with 8, rounded to 11 bits: 2^-11 of 60 bits, which moves every weight of the first tokens alike
    assert relative(got[0], expected(L, 0, q, 512, T)) <= LIMIT["bf16"] + 60 * 2.0 ** -11


@pytest.mark.parametrize("what", ["value", "key"])
@pytest.mark.parametrize("d,bits,T,G", CONTEXTS)
def test_a_large_context_token_of_no_weight(P, d, bits, T, G, what):
    """One context token holds values 2^30 times larger than its neighbours', or an infinite key, and takes no weight worth naming."""
    L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, 256 + T, seed=6)
    k, v = L.rand(1, 256, 2, d), L.rand(1, 256, 2, d)
    q = L.rand(1, T, 2 * G, d)
    q[..., 0] = 8.0
    k[..., 0] = 0
    if what == "value":
        v[0, 70] *= np.float32(2.0 ** 30)
        k[0, 70, :, 0] = -12.0 * d ** 0.5                   # a score near -96: e^-96 2^30 is below 2^-108
    else:
        k[0, 70, :, 0] = -np.inf
    L.append([0], 256, k=k, v=v)
    L.append([256], T, k=L.rand(1, T, 2, d) * 0.1)
    got = attend(L, q, [256])
    assert relative(got[0], expected(L, 0, q, 256, T)) <= LIMIT["bf16"]


@pytest.mark.parametrize("d,bits,G", [(128, 4, 1), (64, 8, 1), (256, 4, 1)])
def test_slots_without_a_page_are_not_seen(P, d, bits, G):
    """The same, whether a KV head has few rows or many: pages outside the pool, and tokens past an odd table's end."""
    n, page = 160, 32
    for T in (20, 32, 33, 130):
        L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", page, n + T, seed=9)
        L.append([0], n)
        L.append([n], T)
        q = L.rand(1, T, 2 * G, d)
        bad = L.table.clone()
        bad[0, 1], bad[0, 4] = -1, L.cfg.n_pages
        got = attend(L, q, [n], table=bad)
        assert L.kv.status(clear=True) == P.PACE_KV_BAD_PAGE
        want = expected(L, 0, q, n, T, hidden=[*range(32, 64), *range(128, 160)])
        assert relative(got[0], want) <= LIMIT["bf16"]
        short = L.table[:, :5].contiguous()                 # (160 tokens: the new ones have no slots)
        got = attend(L, q, [150], table=short)
        assert L.kv.status(clear=True) == P.PACE_KV_BAD_PAGE
        assert relative(got[0], expected(L, 0, q, 150, T, hidden=range(160, 150 + T))) <= LIMIT["bf16"]


@pytest.mark.parametrize("n", [200, 6000])
@pytest.mark.parametrize("d,bits,T,G,io", [(128, 4, 1, 4, "bf16"), (64, 8, 5, 2, "f32"), (128, 4, 2, 2, "f32"), (256, 8, 1, 1, "f32"), (64, 8, 16, 2, "bf16"),
                                           (128, 4, 40, 2, "bf16"), (64, 8, 150, 1, "bf16"), (256, 4, 50, 1, "bf16")])
def test_visible_infinite_values_count_as_their_clamp(P, d, bits, T, G, io, n):
    """Infinite values are held as 2^120 (as near as their scale comes), and a weighted mean of such values is finite."""
    L = Layer(P, 1, 2 * G, 2, d, bits, io, 64, n + T, seed=10)
    v0 = None
    for at in range(0, n, 250):
        v0 = L.rand(1, min(250, n - at), 2, d)
        v0[0, 7::20] = np.inf
        v0[0, 9::40] = -np.inf
        L.append([at], v0.shape[1], v=v0)
    v1 = L.rand(1, T, 2, d)
    v1[0, 0] = np.inf
    L.append([n], T, v=v1)
    q = L.rand(1, T, 2 * G, d)
    got = attend(L, q, [n])
    assert np.isfinite(got).all()
    want = expected(L, 0, q, n, T)
    scale = 2.0 ** -100                                     # (squares of the errors stay within 64 bits)
    assert relative(got[0] * scale, want * scale) <= LIMIT[io]


SAME_BITS = """
import sys
import numpy as np
import torch
sys.path[:0] = [%r, %r]
import bit_gated_delta_gb300 as P
from test_gpu_kv import Layer, dev, host
first = int(sys.argv[1])
def call(B):
    L = Layer(P, B, 8, 2, 64, 4, "f32" if sys.argv[2] == "f32" else "bf16", 64, 400, seed=B)
    L.append([0] * B, 256)
    L.append([256] * B, 144)
    lens = L.rng.integers(0, 400, B).tolist()
    q = L.rand(B, 1, 8, 64)
    o = torch.empty(B, 1, 8, 64, dtype=L.dt, device="cuda")
    L.kv.attend(dev(q, L.dt), o, dev(np.asarray(lens, np.int32)), L.table)
    return host(o)
if first:
    call(first)
np.save(sys.argv[3], call(300))
"""


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_bits_do_not_depend_on_earlier_calls(tmp_path, P, io):
    """A call of 300 sequences in a process of its own, and after a call of 200 or 20."""
    outs = []
    for first in (0, 200, 20):
        at = str(tmp_path / f"o{first}.npy")
        code = SAME_BITS % (ROOT, os.path.join(ROOT, "tests"))
        r = subprocess.run([sys.executable, "-c", code, str(first), io, at], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        outs.append(np.load(at))
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


@pytest.mark.parametrize("Hkv,G,T,io", [(1, 8, 600, "f32"), (8, 8, 600, "bf16")])
def test_one_sequence_in_several_launches(P, Hkv, G, T, io):
    """Where a table could hold 2^30 tokens, the items of one sequence pass what a launch counts, and go out in ranges."""
    import torch
    L = Layer(P, 2, Hkv * G, Hkv, 64, 4, io, 4096, 100 + T, seed=12, max_new=600)
    L.append([0, 0], 100)
    lens = [100, 33]
    L.append(lens, T)
    table = torch.full((2, 1 << 18), -1, dtype=torch.int32, device="cuda")
    table[:, :L.table.shape[1]] = L.table
    q = L.rand(2, T, Hkv * G, 64)
    got = attend(L, q, lens, table=table)
    assert L.kv.status() == 0
    for b in range(2):
        assert relative(got[b], expected(L, b, q, lens[b], T)) <= LIMIT[io]


def test_kept_counts_outside_the_path_are_reported(P):
    L = Layer(P, 3, 2, 2, 64, 8, "f32", 32, 64, seed=6)
    L.append([0] * 3, 40)
    before = L.pool.clone()
    idx = dev(np.tile(np.arange(4, dtype=np.int32), (3, 1)))
    L.kv.keep(dev(np.array([20] * 3, np.int32)), L.table, idx, dev(np.array([0, 4, 3], np.int32)))
    assert L.kv.status() == 0
    for n in ([5, 0, 0], [0, -1, 0], [0, 0, 2 ** 31 - 1]):
        L.kv.keep(dev(np.array([20] * 3, np.int32)), L.table, idx, dev(np.array(n, np.int32)))
        assert L.kv.status(clear=True) == P.PACE_KV_BAD_KEEP
    assert bool((before == L.pool).all())                   # (the paths keep every row where it is)


@pytest.mark.parametrize("rot,scaling", [(256, "ntk"), (64, "parts")])
def test_an_angle_table_is_built_as_fast_as_by_tensor_operations(P, rot, scaling):
    """The table's 64-bit powers are formed once a pair, not once an entry (which took four to six times as long)."""
    import torch
    n = 32768 * 128 // (rot // 2)
    rope = P.PaceRope(rot, n, scaling=scaling, factor=4.0, orig_pos=4096)
    theta = torch.from_numpy(K.thetas(rot, scaling=scaling, factor=4.0, orig_pos=4096)[0]).cuda()

    def plain():
        angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * theta
        return torch.cos(angle).float(), torch.sin(angle).float()

    def best(call):
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert best(lambda: P.pace_rope_table(rope.cfg, rope.ptr, rope.nbytes)) <= best(plain)


def test_memory_of_a_cache_waits_for_the_streams_that_use_it(P):
    """A cache and a table that are dropped while another stream still works on them keep their memory until it is done."""
    import torch
    cfg = P.make_kv_config(2, 2, 64, 64, 1, bits=8, page_tokens=64)
    kv, rope = P.PaceKV(cfg), P.PaceRope(64, 5000)
    lens, table = dev(np.zeros(1, np.int32)), dev(np.arange(64, dtype=np.int32)[None])
    q, k, v, qo = (torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)                      # (about 0.2 s)
        kv.append(q, k, v, lens, table, rope=rope, q_out=qo)
    sizes = {x.data_ptr(): x.numel() * x.element_size() for x in (kv.mem, rope.table)}
    del kv, rope
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for size in sizes.values()]
    busy = not s.query()
    assert busy and not {o.data_ptr() for o in others} & set(sizes)
    s.synchronize()


# What is left beside the rounding of the output, as a root mean square of the difference from the output type's rounding of the exact
# value. A rounding to p bits is 0.42 2^-p of a value, so 2e-4 for weights of 11 bits (few rows); with held values of 11 bits and scores that move
# by twice that, 4e-4 (many rows; held 4-bit values have few bits to lose). An error e moves a bf16 output to its neighbour, 5.6e-3 away, once
# in 5.6e-3 / 0.8 e: 1e-3 of the output (few rows) and 1.4e-3 (many). Weights of 8 bits would give 2.4e-3 or more. fp32: sums of exact
# products and the exponential, each a few 2^-23; a lost third part of a query or weight would give 6e-6.
@pytest.mark.parametrize("d,bits,T,G,io,limit", [
    (64, 4, 1, 8, "bf16", 1.3e-3), (128, 8, 1, 6, "bf16", 1.3e-3), (128, 4, 4, 4, "bf16", 1.3e-3), (256, 8, 7, 1, "bf16", 1.3e-3), (64, 8, 32, 1, "bf16", 1.3e-3),
    (128, 4, 25, 4, "bf16", 1.5e-3), (64, 4, 100, 4, "bf16", 1.5e-3), (256, 4, 40, 2, "bf16", 1.5e-3), (128, 8, 60, 4, "bf16", 2e-3), (256, 8, 40, 2, "bf16", 2e-3),
    (64, 8, 1, 4, "f32", 2e-6), (128, 4, 5, 2, "f32", 2e-6), (256, 8, 20, 1, "f32", 2e-6), (128, 8, 40, 2, "f32", 2e-6)])
def test_bits_that_queries_weights_and_values_keep(P, d, bits, T, G, io, limit):
    L = Layer(P, 2, 2 * G, 2, d, bits, io, 64, 750 + T, seed=14)
    for at in (0, 250, 500):
        L.append([at] * 2, 250)
    lens = [750, 611]
    L.append(lens, T)
    q = L.rand(2, T, 2 * G, d)
    got = attend(L, q, lens)
    for b in range(2):
        want = expected(L, b, q, lens[b], T)
        to = K.bf16(want.astype(np.float32)) if io == "bf16" else want
        assert relative(got[b], to.astype(np.float64)) <= limit


@pytest.mark.parametrize("d,bits,T,G", [(128, 4, 1, 4), (128, 8, 20, 1), (256, 8, 1, 4), (128, 4, 40, 2), (128, 8, 150, 1), (256, 4, 50, 1), (256, 8, 50, 1)])
def test_groups_of_very_different_size(P, d, bits, T, G):
    """A group 2^-12 of its head vector's largest keeps its bits; one of 2^-30 is within 2^-22 of the vector's largest element."""
    for ratio in (2.0 ** -12, 2.0 ** -30):
        L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, 256 + T, seed=15)
        k, v = L.rand(1, 256 + T, 2, d), L.rand(1, 256 + T, 2, d)
        v[..., d - 64:] *= np.float32(ratio)
        L.append([0], 256, k=k[:, :256], v=v[:, :256])
        L.append([256], T, k=k[:, 256:], v=v[:, 256:])
        q = L.rand(1, T, 2 * G, d)
        got, want = attend(L, q, [256])[0], expected(L, 0, q, 256, T)
        assert relative(got[..., :d - 64], want[..., :d - 64]) <= LIMIT["bf16"]
        if ratio == 2.0 ** -12:
            assert relative(got[..., d - 64:], want[..., d - 64:]) <= LIMIT["bf16"]
        else:
            assert np.abs(got[..., d - 64:] - want[..., d - 64:]).max() <= 2.0 ** -22 * np.abs(L.v).max()


@pytest.mark.parametrize("d,bits,T,G,size", [(128, 4, 1, 4, 2.0 ** -70), (64, 8, 16, 1, 2.0 ** -70), (128, 8, 40, 2, 2.0 ** -110), (64, 4, 100, 2, 2.0 ** -110),
                                             (256, 4, 50, 1, 2.0 ** -110)])
def test_tiny_values_alone(P, d, bits, T, G, size):
    L = Layer(P, 1, 2 * G, 2, d, bits, "bf16", 64, 256 + T, seed=16)
    v = K.bf16(L.rand(1, 256 + T, 2, d) * np.float32(size))
    L.append([0], 256, v=v[:, :256])
    L.append([256], T, v=v[:, 256:])
    q = L.rand(1, T, 2 * G, d)
    got, want = attend(L, q, [256])[0].astype(np.float64) / size, expected(L, 0, q, 256, T) / size
    assert relative(got, want) <= LIMIT["bf16"]
