"""More of the gated delta rule over states in slots: order between chunks, blocks that go on from one sequence and head to the next at every
instantiation, errors of the states, waits that run out. Inputs, tolerances and statements are those of test_gpu_delta.py and
serve_testlib.py."""
import numpy as np
import pytest

import serve_testlib as T
from pace_testlib import ensure_built
from test_gpu_delta import close, f64, inputs, ints, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    return P


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_long_prompts_repeat_themselves(P, d, io):
    """Every multiprocessor goes through 14 chunks, whose u is written where the outputs before were: the same bits at each of eight calls, and
    those of the first half and of the second half of the chunks' tokens as the rule gives them."""
    import torch
    B, n, H, Hk = 10, 14 * 64 - 5, 16, 8
    D = make(P, torch, H, Hk, d, io, B)
    x = inputs(torch, B, n, H, Hk, d, io, 11)
    S = D.states.clone()
    want, end = None, None
    for _ in range(8):
        D.states.copy_(S)
        o = torch.empty_like(x[2])
        D.chunk(*x, o)
        if want is None:
            want, end = o, D.states.clone()
        assert torch.equal(o, want) and torch.equal(D.states, end)
    q, k, v, a, beta = (f64(y) for y in x)
    for b, h in ((0, 0), (4, 7), (9, 15)):
        o, last = T.chunk(f64(S[b, h]), q[b, :, h // 2], k[b, :, h // 2], v[b, :, h], a[b, :, h], beta[b, :, h])
        for first in (0, 32):
            at = np.arange(n) % 64 // 32 * 32 == first
            close(want[b, torch.from_numpy(at).cuda(), h], o[at], 2.0 ** -24 if io else 2.0 ** -8, f"outputs of tokens {first}..{first + 31} of the chunks")
        close(end[b, h], last, 0.0, "states")
    assert D.status() == 0


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("strong", [False, True])
def test_states_of_slow_decays_are_held_in_32_bits(P, d, io, strong):
    """Decays of 0.999 and more, so that hundreds of tokens' errors meet. What fp32 accumulation costs: a sum of the tensor cores takes its largest
    parts in steps of 16 terms, d / 16 <= 8 for w = S^T k, 4 for u and 4 for the increment, each cut off by half a unit of 2^-23 on average: at most 16 * 2^-24 =
    2^-20 of the values. A token's error of w enters the state times beta, and takes beta (2 - beta) / d of the error's square along k away: what
    stays is sqrt(beta / (2 - beta)) <= 1 of it. The three bf16 parts of an operand leave 2^-25, which is small beside that; two would leave 2^-18."""
    import torch
    n, H = 900, 4
    x = inputs(torch, 1, n, H, 2, d, io, 5, a_lo=0.999)
    if strong:
        x[4].fill_(1.0)
    D = make(P, torch, H, 2, d, io, 1)
    S = f64(D.states)[0]
    D.chunk(*x, torch.empty_like(x[2]))
    q, k, v, a, beta = map(f64, x)
    got = f64(D.states)[0]
    for h in range(H):
        _, want = T.chunk(S[h], q[0, :, h // 2], k[0, :, h // 2], v[0, :, h], a[0, :, h], beta[0, :, h])
        off = np.linalg.norm(got[h] - want) / np.linalg.norm(want)
        assert off < 2.0 ** -20, off


def alone(P, torch, kind, D, S, x, o, rows, counts, mask, idx, keep, slots):
    """Sequences `rows` of a call, each in a call of its own: their outputs and states, from the states S."""
    E = P.PaceDelta(D.cfg)
    E.states.copy_(S)
    for b in rows:
        one = slice(b, b + 1)
        y, s = [z[one] for z in x], slots[one]
        c = None if counts is None else counts[one]
        got = torch.full_like(o[one], 7.0)
        if kind == "chunk":
            E.chunk(*y, got, slots=s, n_new=c)
        elif kind == "draft":
            E.draft(*y, got, slots=s, n_new=c, mask=None if mask is None else mask[one].contiguous())
        else:
            E.keep(*y[1:], idx[one].contiguous(), keep[one].contiguous(), slots=s, n_new=c)
        if kind != "keep":
            assert torch.equal(got, o[one]), f"outputs of sequence {b}"
        assert torch.equal(E.states[int(s)], D.states[int(s)]), f"state of sequence {b}"


def lasting(P, kind, B, n, H, Hk, d, io, seed, every):
    """A call of many sequences of all lengths and counts, with every few of them against calls of their own and one against the rule."""
    import torch
    from test_gpu_delta import tree, words
    rng = np.random.default_rng(seed)
    D = make(P, torch, H, Hk, d, io, B + 3, seed)
    S = D.states.clone()
    x = inputs(torch, B, n, H, Hk, d, io, seed)
    counts = rng.integers(0, n + 1, B)
    counts[0], counts[-1] = n, n
    slots = rng.permutation(B + 3)[:B]
    cn, sl = ints(torch, counts), ints(torch, slots)
    mask = idx = keep = None
    o = torch.full_like(x[2], 7.0)
    if kind == "chunk":
        D.chunk(*x, o, slots=sl, n_new=cn)
    elif kind == "draft":
        see = np.stack([tree(rng, n) for _ in range(B)])
        mask = words(torch, see)
        D.draft(*x, o, slots=sl, n_new=cn, mask=mask)
    else:
        kept = np.minimum(rng.integers(0, n + 1, B), counts)
        kept[0] = n
        path = np.zeros((B, n), np.int32)
        for b in range(B):
            path[b, :kept[b]] = np.sort(rng.choice(counts[b], kept[b], replace=False)) if kept[b] else []
        idx, keep = ints(torch, path), ints(torch, kept)
        D.keep(*x[1:], idx, keep, slots=sl, n_new=cn)
    assert D.status() == 0
    alone(P, torch, kind, D, S, x, o, [0, *range(1, B - 1, every), B - 1], cn, mask, idx, keep, sl)
    q, k, v, a, beta = (f64(y[0]) for y in x)
    h, hk, before = H - 1, (H - 1) // (H // Hk), f64(S[int(slots[0]), H - 1])
    t = slice(None) if kind != "keep" else path[0, :kept[0]]
    if kind == "draft":
        want, end = T.draft(before, q[:, hk], k[:, hk], v[:, h], a[:, h], beta[:, h], see[0]), before
    else:
        want, end = T.chunk(before, q[t, hk], k[t, hk], v[t, h], a[t, h], beta[t, h])
    if kind != "keep":
        close(o[0, :, h], want, 2.0 ** -24 if io else 2.0 ** -8, "outputs")
    close(D.states[int(slots[0]), h], end, 0.0, "states")
    untouched = [s for s in range(B + 3) if s not in set(slots)] + [int(slots[b]) for b in range(B) if (counts if kind != "keep" else kept)[b] == 0]
    assert torch.equal(D.states[untouched], S[untouched])


@pytest.mark.parametrize("kind", ["chunk", "draft", "keep"])
@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [33, 64])
def test_blocks_that_go_on(P, n, d, io, kind):
    lasting(P, kind, 60, n, 6, 3, d, io, n + d, 7)


@pytest.mark.parametrize("kind", ["chunk", "keep"])
@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_blocks_that_go_on_over_several_chunks(P, d, io, kind):
    lasting(P, kind, 40, 200, 5, 5, d, io, d, 6)


@pytest.mark.parametrize("kind,d,io", [("chunk", 64, 0), ("draft", 128, 0), ("keep", 128, 1)])
def test_more_than_256_sequences(P, kind, d, io):
    """Sequences that are not sorted by their length."""
    lasting(P, kind, 300, 20, 2, 1, d, io, 3, 40)


@pytest.mark.parametrize("kind,io", [("chunk", 0), ("draft", 1), ("keep", 0)])
def test_more_than_64_units_a_multiprocessor(P, kind, io):
    """16,000 sequences and heads: more blocks than multiprocessors, each with as many units as it can list."""
    lasting(P, kind, 1000, 17, 16, 4, 64, io, 4, 150)


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind,B,n", [("chunk", 3, 200), ("chunk", 50, 70), ("draft", 50, 20), ("keep", 50, 20), ("keep", 3, 300)])
def test_waits_that_run_out(P, kind, B, n, d, io):
    """Each block waits 2 ms for what nothing signals: the call ends, says so, and leaves the states and what lies around the outputs as they were; the next
    call is like any other. (50 x 4 sequences and heads: blocks that go on from one to the next.)"""
    import torch
    H = 4
    D, E = make(P, torch, H, H, d, io, B), make(P, torch, H, H, d, io, B)
    S = D.states.clone()
    x = inputs(torch, B, n, H, H, d, io, 12)
    idx, keep = ints(torch, np.tile(np.arange(n), (B, 1))), ints(torch, [n] * B)
    wide = torch.full((B, n + 2, H, d), 7.0, dtype=x[2].dtype, device="cuda")
    o, want = wide[:, 1:-1], torch.empty_like(x[2])

    def call(to, out):
        if kind == "keep":
            to.keep(*x[1:], idx, keep)
        else:
            getattr(to, kind)(*x, out)
    call(E, want)
    P.serve.pace_test_delta_wait_probe(D.handle, 2_000_000)
    call(D, o)
    assert D.status(clear=True) == P.PACE_DELTA_TIMEOUT and D.status() == 0
    assert torch.equal(D.states, S) and (wide[:, 0] == 7.0).all() and (wide[:, -1] == 7.0).all()
    P.serve.pace_test_delta_wait_probe(D.handle, 0)
    call(D, o)
    assert D.status() == 0 and torch.equal(D.states, E.states) and (kind == "keep" or torch.equal(o, want))
