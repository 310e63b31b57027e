"""The gated delta rule over states in slots against its recurrence in 64 bits.

Tolerances. Everything is held in fp32 or in three bf16 parts (24 bits), but for what the second paragraph names, so that an output differs by the rounding of the I/O type (half a step: 2^-8 of
the value for bf16, 2^-24 for fp32) and by what the sums of up to 128 products and the tokens before carry: 2^-18 of the rows' rms (64 half
steps of fp32; n random roundings of a dot of n terms come to sqrt(n) = 11 half steps, and decays below 1 keep those of earlier
tokens bounded). States are held to the second part alone.

bf16 outputs of calls by chunks are formed from two bf16 parts of S, P and u: a part takes half a step of 2^-8, so that two leave at most 2^-18
of an element, and an output differs by at most 2^-18 sum_i |S_ij q_i| + 3 * 2^-18 sum_s |P_ts u_s| beside the above (S; P, u and the product
of their second parts). With |q| = 1 the first sum is at most |S_j|, sqrt(d) times the rms of S_j, which is that of S_j^T q over
directions q: 11.3 at d = 128. The second has at most as many terms of the same size as make up S. 4 * 11.3 * 2^-18 < 2^-12 of the rms.
"""
import numpy as np
import pytest

import serve_testlib as T
from pace_testlib import ensure_built

pytestmark = pytest.mark.gpu
CARRY, CARRY_BF16 = 2.0 ** -18, 2.0 ** -12


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    return P


def inputs(torch, B, n, H, Hk, d, io, seed=0, a_lo=0.9):
    """One packed projection [B, n, ..] (so that q, k and v are views with strides), gates by strides too."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    dt = torch.float32 if io else torch.bfloat16
    x = r(B, n, 2 * Hk + H, d)
    x[:, :, :2 * Hk] /= x[:, :, :2 * Hk].norm(dim=-1, keepdim=True)
    q, k, v = x.to(dt).cuda().split([Hk, Hk, H], 2)
    gates = torch.rand(B, 2, n, H, generator=g)
    gates[:, 0] = a_lo + (1 - a_lo) * gates[:, 0]
    gates = gates.cuda()
    return q, k, v, gates[:, 0], gates[:, 1]


def f64(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def close(got, want, step, what):
    got, want = f64(got), np.asarray(want)
    rms = np.sqrt((want ** 2).mean()) if want.size else 0.0
    off = np.abs(got - want) - step * np.abs(want) - (CARRY_BF16 if step == 2.0 ** -8 else CARRY) * rms
    assert np.isfinite(got).all() and (off <= 0).all(), f"{what}: off by {np.abs(got - want).max():.3e} of {rms:.3e} (worst {off.max():.3e} over)"


def make(P, torch, H, Hk, d, io, slots, seed=1, scale=0.5):
    D = P.PaceDelta(P.make_delta_config(H, d, slots, key_heads=Hk, io_dtype=P.PACE_IO_F32 if io else P.PACE_IO_BF16))
    D.states.copy_(torch.randn(D.states.shape, generator=torch.Generator().manual_seed(seed)) * scale)
    return D


def ints(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_chunk(P, torch, B, n, H, Hk, d, io, counts=None, lens=None, seed=0, a_lo=0.9, gates=None):
    slots = np.random.default_rng(seed).permutation(B + 2)[:B]
    D = make(P, torch, H, Hk, d, io, B + 2)
    before = f64(D.states)
    q, k, v, a, beta = inputs(torch, B, n, H, Hk, d, io, seed, a_lo)
    if gates is not None:
        gates(a, beta)
    m = [n] * B if counts is None else counts
    pad = torch.zeros(B, n, dtype=torch.bool, device="cuda")
    for b in range(B):
        pad[b, m[b]:] = True
    for x in (q, k, v, a, beta):                 # rows that do not exist hold anything
        x[pad] = float("nan")
    o = torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
    D.chunk(q, k, v, a, beta, o, slots=ints(torch, slots), lens=None if lens is None else ints(torch, lens),
            n_new=None if counts is None else ints(torch, counts))
    after = f64(D.states)
    want_o, want_S = np.zeros(v.shape), before.copy()
    qn, kn, vn, an, bn = map(f64, (q, k, v, a, beta))
    for b in range(B):
        for h in range(H):
            S = before[slots[b], h] * (lens is None or lens[b] > 0)
            t, hk = slice(0, m[b]), h // (H // Hk)
            if m[b]:
                want_o[b, t, h], want_S[slots[b], h] = T.chunk(S, qn[b, t, hk], kn[b, t, hk], vn[b, t, h], an[b, t, h], bn[b, t, h])
    close(o, want_o, 2.0 ** -24 if io else 2.0 ** -8, "outputs")
    close(torch.tensor(after), want_S, 0.0, "states")
    for b in range(B):
        assert not f64(o)[b, m[b]:].any()
    idle = [s for s in range(B + 2) if s not in [slots[b] for b in range(B) if m[b]]]
    assert np.array_equal(after[idle], before[idle])
    assert D.status() == 0


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 7, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 129, 200])
def test_chunk_lengths(P, n, d, io):
    import torch
    check_chunk(P, torch, 2, n, 2, 1, d, io, seed=n)


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("H,Hk,d", [(1, 1, 128), (3, 3, 64), (6, 2, 128), (5, 1, 64)])
def test_ragged_batches_and_heads(P, H, Hk, d, io):
    import torch
    check_chunk(P, torch, 6, 150, H, Hk, d, io, counts=[150, 0, 1, 64, 149, 70], lens=[0, 5, 0, 9, 1, 0], seed=3)
    check_chunk(P, torch, 5, 3, H, Hk, d, io, counts=[3, 0, 1, 2, 3], lens=[0, 0, 4, 0, 1], seed=4)


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("n", [5, 130])
def test_decays_and_strengths_at_their_ends(P, n, io):
    import torch

    def gates(a, beta):
        a[:, ::7] = 0.0                          # forget everything
        a[:, 1::5] = 1.0
        a[:, 3::11] = 1e-30
        beta[:, ::4] = 1.0
        beta[:, 2::6] = 0.0                      # no update
    check_chunk(P, torch, 2, n, 2, 2, 128, io, seed=8, gates=gates)
    check_chunk(P, torch, 2, n, 2, 2, 64, io, seed=9, a_lo=0.0)


def test_counts_past_the_rows_are_clamped(P):
    import torch
    D = make(P, torch, 2, 2, 64, 1, 3)
    x = inputs(torch, 3, 4, 2, 2, 64, 1)
    o, o2 = torch.zeros_like(x[2]), torch.zeros_like(x[2])
    S = D.states.clone()
    D.chunk(*x, o, n_new=ints(torch, [9, -4, 4]))
    got = D.states.clone()
    D.states.copy_(S)
    D.chunk(*x, o2, n_new=ints(torch, [4, 0, 4]))
    assert torch.equal(o, o2) and torch.equal(got, D.states) and D.status() == 0


def test_states_only(P):
    import torch
    for n in (3, 100):
        q, k, v, a, beta = inputs(torch, 2, n, 4, 2, 128, 0)
        one, two = make(P, torch, 4, 2, 128, 0, 2), make(P, torch, 4, 2, 128, 0, 2)
        one.chunk(q, k, v, a, beta, torch.empty_like(v))
        two.chunk(None, k, v, a, beta, None)
        assert torch.equal(one.states, two.states)


def tree(rng, n):
    see = np.eye(n, dtype=bool)
    for t in range(1, n):
        parent = rng.integers(-1, t)
        if parent >= 0:
            see[t] |= see[parent]
    return see


def words(torch, see):
    n = see.shape[-1]
    W = (n + 31) // 32
    bits = np.zeros(see.shape[:-1] + (W * 32,), np.uint64)
    bits[..., :n] = see
    w = (bits.reshape(see.shape[:-1] + (W, 32)) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.from_numpy(w.view(np.int32)).cuda()


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 5, 16, 25, 33, 64])
def test_drafts(P, n, d, io):
    import torch
    B, H, Hk = 3, 2, 1
    D = make(P, torch, H, Hk, d, io, 4)
    before = D.states.clone()
    q, k, v, a, beta = inputs(torch, B, n, H, Hk, d, io, n)
    rng = np.random.default_rng(n)
    see = np.stack([tree(rng, n) for _ in range(B)])
    count = [n, max(n - 1, 0), (n + 1) // 2]
    for b in range(B):
        for x in (q, k, v, a, beta):
            x[b, count[b]:] = float("inf")
    slots = [2, 0, 2]                            # two trees from one state
    qn, kn, vn, an, bn = map(f64, (q, k, v, a, beta))
    S = f64(before)
    for mask, what in ((words(torch, see), see), (None, np.ones_like(see))):
        o = torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
        D.draft(q, k, v, a, beta, o, slots=ints(torch, slots), n_new=ints(torch, count), mask=mask)
        want = np.zeros(v.shape)
        for b in range(B):
            t = slice(0, count[b])
            for h in range(H):
                want[b, t, h] = T.draft(S[slots[b], h], qn[b, t, h // 2], kn[b, t, h // 2], vn[b, t, h], an[b, t, h], bn[b, t, h], what[b])
        close(o, want, 2.0 ** -24 if io else 2.0 ** -8, "outputs")
        assert all(not f64(o)[b, count[b]:].any() for b in range(B))
    # bits of a token's own and of later ones do not matter
    i = np.arange(n)
    other = np.where(i[None, :] >= i[:, None], rng.random((B, n, n)) < 0.5, see)
    o2 = torch.empty_like(o)
    D.draft(q, k, v, a, beta, o, slots=ints(torch, slots), n_new=ints(torch, count), mask=words(torch, see))
    D.draft(q, k, v, a, beta, o2, slots=ints(torch, slots), n_new=ints(torch, count), mask=words(torch, other))
    assert torch.equal(o, o2) and torch.equal(D.states, before) and D.status() == 0


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 20, 64, 100])
def test_kept_paths(P, n, d, io):
    import torch
    B, H, Hk = 4, 4, 2
    D = make(P, torch, H, Hk, d, io, 5)
    before = f64(D.states)
    q, k, v, a, beta = inputs(torch, B, n, H, Hk, d, io, n + 50)
    rng = np.random.default_rng(n)
    keep = [min(n, m) for m in (n, 0, 1, (n + 1) // 2)]
    paths = [sorted(rng.choice(n, m, replace=False)) for m in keep]
    idx = np.zeros((B, n), np.int32)
    for b in range(B):
        idx[b, :keep[b]] = paths[b]
    slots = [4, 1, 0, 2]
    D.keep(k, v, a, beta, ints(torch, idx), ints(torch, keep), slots=ints(torch, slots))
    kn, vn, an, bn = map(f64, (k, v, a, beta))
    want = before.copy()
    for b in range(B):
        for h in range(H):
            for i in paths[b]:
                want[slots[b], h] = T.rule(want[slots[b], h], kn[b, i, h // 2], vn[b, i, h], an[b, i, h], bn[b, i, h])
    close(D.states, want, 0.0, "states")
    assert np.array_equal(f64(D.states)[[1, 3]], before[[1, 3]]) and D.status() == 0


def test_a_draft_and_its_path_are_a_chunk(P):
    """Tokens drafted in a row give the outputs, and kept the state, that the same tokens give one by one."""
    import torch
    B, n, H, d = 2, 6, 4, 128
    x = inputs(torch, B, n, H, H, d, 1, 4)
    one, two = make(P, torch, H, H, d, 1, B), make(P, torch, H, H, d, 1, B)
    o, o2 = torch.empty_like(x[2]), torch.empty_like(x[2])
    for t in range(n):
        y = torch.empty(B, 1, H, d, device="cuda")
        one.chunk(*(z[:, t:t + 1] for z in x), y)
        o[:, t:t + 1] = y
    two.draft(*x, o2)
    two.keep(*x[1:], ints(torch, [list(range(n))] * B), ints(torch, [n] * B))
    close(o2, f64(o), 2.0 ** -24, "outputs")
    close(two.states, f64(one.states), 0.0, "states")


def test_bad_slots_and_paths_are_left_out(P):
    import torch
    H, d = 2, 64
    for n in (2, 80):
        D = make(P, torch, H, H, d, 0, 4)
        S = D.states.clone()
        x = inputs(torch, 4, n, H, H, d, 0)
        o, ref = torch.empty_like(x[2]), torch.empty_like(x[2])
        D.chunk(*x, o, slots=ints(torch, [1, 7, 1, -1]))
        assert D.status() == P.PACE_DELTA_BAD_SLOT and D.status(clear=True) and D.status() == 0
        assert not o[1:].any()
        got = D.states.clone()
        D.states.copy_(S)
        D.chunk(*(y[:1] for y in x), ref[:1], slots=ints(torch, [1]))
        assert torch.equal(o[0], ref[0]) and torch.equal(got, D.states)
        # a sequence without tokens claims no slot
        D.states.copy_(S)
        D.chunk(*x, o, slots=ints(torch, [1, 1, 99, 2]), n_new=ints(torch, [0, n, 0, n]))
        assert D.status() == 0
        D.states.copy_(S)
        idx = [[0, 1], [1, 1], [0, 5000], [0, 1]]
        D.keep(*x[1:], ints(torch, idx), ints(torch, [2, 2, 2, 9]))
        assert D.status(clear=True) == P.PACE_DELTA_BAD_KEEP
        got = D.states.clone()
        D.states.copy_(S)
        D.keep(*x[1:], ints(torch, [[0, 1], [1, 0], [0, 0], [0, 1]]), ints(torch, [2, 1, 1, 2]))
        assert torch.equal(got, D.states) and D.status() == 0


def test_same_call_same_bits_on_any_stream_and_in_a_graph(P):
    import torch
    B, H, d = 3, 4, 128
    for n in (1, 100):
        x = inputs(torch, B, n, H, H, d, 0, 2)
        D = make(P, torch, H, H, d, 0, B)
        S = D.states.clone()
        want = torch.empty_like(x[2])
        D.chunk(*x, want)
        final = D.states.clone()
        side, o = torch.cuda.Stream(), torch.empty_like(want)
        D.states.copy_(S)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            D.chunk(*x, o)
        side.synchronize()
        assert torch.equal(o, want) and torch.equal(D.states, final)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            D.chunk(*x, o)
        for _ in range(2):
            D.states.copy_(S)
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(D.states, final)


def test_empty_calls(P):
    import torch
    D = make(P, torch, 2, 2, 64, 0, 2)
    S = D.states.clone()
    x = inputs(torch, 2, 0, 2, 2, 64, 0)
    D.chunk(*x, torch.empty_like(x[2]))
    D.draft(*x, torch.empty_like(x[2]))
    x = inputs(torch, 2, 3, 2, 2, 64, 0)
    D.keep(*x[1:], torch.zeros(2, 0, dtype=torch.int32, device="cuda"), ints(torch, [0, 0]))
    D.chunk(*(y[:0] for y in x), torch.empty_like(x[2][:0]))
    assert torch.equal(S, D.states) and D.status() == 0


def test_refusals(P):
    import torch
    D = make(P, torch, 4, 2, 64, 0, 2)
    q, k, v, a, beta = inputs(torch, 2, 3, 4, 2, 64, 0)
    o = torch.empty_like(v)
    for bad in (dict(q=v), dict(k=k.float()), dict(v=v[:, :, :2]), dict(a=a.double()), dict(a=a[:, :2]), dict(beta=beta.cpu()),
                dict(o=torch.empty(2, 3, 4, 128, dtype=v.dtype, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            D.chunk(**{**dict(q=q, k=k, v=v, a=a, beta=beta, o=o), **bad})
    with pytest.raises(ValueError):
        D.chunk(q, k, v, a, beta, o, slots=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(P.PaceError, match="go together"):
        D.chunk(q, k, v, a, beta, None)
    with pytest.raises(P.PaceError, match="without slots"):
        D.chunk(*(torch.cat((x, x)) for x in (q, k, v, a, beta, o)))
    big = inputs(torch, 2, 65, 4, 2, 64, 0)
    with pytest.raises(P.PaceError, match="n_tokens 65"):
        D.draft(*big, torch.empty_like(big[2]))
    odd = torch.empty(2, 3, 4, 68, dtype=v.dtype, device="cuda")[..., 4:]
    with pytest.raises(P.PaceError, match="16-byte"):
        D.chunk(q, k, odd, a, beta, o)
    assert D.status() == 0


@pytest.mark.parametrize("n", [3, 40, 130])
def test_outputs_into_part_of_a_tensor(P, n):
    """o is a view with gaps: what lies between its rows stays as it was."""
    import torch
    B, H, d = 3, 2, 64
    for io in (0, 1):
        x = inputs(torch, B, n, H, H, d, io, 6)
        D, E = make(P, torch, H, H, d, io, B), make(P, torch, H, H, d, io, B)
        want = torch.empty_like(x[2])
        counts = ints(torch, [n, n // 2, 0])
        D.chunk(*x, want, n_new=counts)
        wide = torch.full((B + 1, n + 2, H + 1, d + 16), 9.0, dtype=x[2].dtype, device="cuda")
        o = wide[1:, 1:1 + n, :H, 8:8 + d]
        E.chunk(*x, o, n_new=counts)
        assert torch.equal(o, want) and torch.equal(D.states, E.states)
        o.fill_(9.0)
        assert (wide == 9.0).all()


@pytest.mark.parametrize("n", [2, 30, 100])
def test_what_is_not_finite_stays_with_its_sequence_and_head(P, n):
    """More sequences and heads than multiprocessors, so that blocks go on from a spoiled one to the next."""
    import torch
    B, H, d = 40, 8, 64
    x = inputs(torch, B, n, H, H, d, 0, 7)
    good, bad = make(P, torch, H, H, d, 0, B), make(P, torch, H, H, d, 0, B)
    want, got = torch.empty_like(x[2]), torch.empty_like(x[2])
    good.chunk(*x, want)
    x = [y.clone() for y in x]
    spoiled = torch.zeros(B, H, dtype=torch.bool, device="cuda")
    for b in range(0, B, 3):
        spoiled[b, b % H] = True
        x[b % 3][b, n - 1, b % H] = float("nan") if b % 2 else float("inf")
        x[2][b, 0, b % H] = float("inf")
    bad.chunk(*x, got)
    keep = ~spoiled[:, None, :, None].expand(want.shape)
    assert torch.equal(got[keep], want[keep]) and torch.equal(good.states[~spoiled], bad.states[~spoiled])
    assert bad.status() == 0


@pytest.mark.parametrize("n", [1, 20, 70])
def test_many_sequences_of_all_lengths(P, n):
    """Sequences and heads of every length below n, more than the multiprocessors hold at once: the same bits as each sequence alone."""
    import torch
    B, H, d = 70, 6, 64
    x = inputs(torch, B, n, H, 3, d, 0, 9)
    count = np.random.default_rng(n).integers(0, n + 1, B)
    D, E = make(P, torch, H, 3, d, 0, B), make(P, torch, H, 3, d, 0, B)
    o = torch.empty_like(x[2])
    D.chunk(*x, o, n_new=ints(torch, count))
    for b in range(0, B, 7):
        one = torch.empty_like(o[b:b + 1])
        E.chunk(*(y[b:b + 1] for y in x), one, slots=ints(torch, [b]), n_new=ints(torch, count[b:b + 1]))
        assert torch.equal(one, o[b:b + 1]) and torch.equal(E.states[b], D.states[b])
    assert D.status() == E.status() == 0


def test_slow_decays_over_a_long_prompt(P):
    """Decays of 0.999 and more keep errors of hundreds of tokens. bf16 I/O by chunks forms w = S^T k from two parts of S: off by at most 2^-18 |S_j|
    |k| = 2^-18 sqrt(d) rms, a token's share of which, beta k_i of it, enters the state; n random shares of k_i = 1 / sqrt(d) each come to
    sqrt(n) 2^-18 rms, 2^-13.4 at n = 600 if none were undone by later tokens."""
    import torch
    n, d = 600, 128
    x = inputs(torch, 1, n, 2, 1, d, 0, 3, a_lo=0.999)
    D = make(P, torch, 2, 1, d, 0, 1)
    S = f64(D.states)[0]
    o = torch.empty_like(x[2])
    D.chunk(*x, o)
    q, k, v, a, beta = map(f64, x)
    for h in range(2):
        want, end = T.chunk(S[h], q[0, :, 0], k[0, :, 0], v[0, :, h], a[0, :, h], beta[0, :, h])
        close(o[0, :, h], want, 2.0 ** -8, "outputs")
        off = np.abs(f64(D.states)[0, h] - end).max() / np.sqrt((end ** 2).mean())
        assert off < 2.0 ** -13, off


def test_memory_waits_for_the_streams_that_use_it(P):
    import torch
    side = torch.cuda.Stream()
    for make_one in (lambda: P.PaceDelta(P.make_delta_config(8, 64, 4)), lambda: P.PacePages(200000, 64, 8)):
        for first in (True, False):                             # (a kernel's first launch loads it, which may wait for the stream)
            one = make_one()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                if not first:
                    torch.cuda._sleep(400_000_000)              # (about 0.2 s)
                if isinstance(one, P.PaceDelta):
                    x = torch.zeros(4, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
                    gate = torch.ones(4, 1, 8, device="cuda")
                    one.chunk(x, x, x, gate, gate, torch.empty_like(x))
                else:
                    one.compact(torch.full((8, 4), -1, dtype=torch.int32, device="cuda"))
            if first:
                torch.cuda._sleep(1000)
                side.synchronize()
                continue
            at, size = one.mem.data_ptr(), one.mem.numel()
            del one
            other = torch.empty(size, dtype=torch.uint8, device="cuda")
            busy = not side.query()
            assert busy and other.data_ptr() != at
            side.synchronize()


def test_longest_offsets(P):
    """A tensor whose last sequence lies past 2^32 bytes, and states past 2^32 bytes."""
    import torch
    H, d = 4, 128
    D = P.PaceDelta(P.make_delta_config(H, d, 17000))                     # 4.5 GB
    x = inputs(torch, 1, 70, H, H, d, 0, 5)
    o, ref = torch.empty_like(x[2]), torch.empty_like(x[2])
    wide = torch.empty(2, 1 << 31, dtype=torch.bfloat16, device="cuda")   # 8 GB: the second row begins 4 GB in
    views = [wide[:, i * 40000:i * 40000 + 70 * H * d].view(2, 70, H, d) for i in range(3)]
    for view, y in zip(views, x):
        view.zero_()
        view[1] = y[0]
    out = wide[:, 200000:200000 + 70 * H * d].view(2, 70, H, d)
    gates = [g.expand(2, -1, -1) for g in x[3:]]
    D.chunk(*views, *gates, out, slots=ints(torch, [0, 16999]))
    D.chunk(*x, ref, slots=ints(torch, [5]))
    assert torch.equal(out[1], ref[0]) and torch.equal(D.states[16999], D.states[5])
    D.states.zero_()
    D.chunk(*(v[:, :1] for v in views), *(g[:, :1] for g in gates), out[:, :1], slots=ints(torch, [0, 16999]))
    D.chunk(*(y[:, :1] for y in x), ref[:, :1], slots=ints(torch, [5]))
    assert torch.equal(out[1, :1], ref[0, :1]) and torch.equal(D.states[16999], D.states[5])
