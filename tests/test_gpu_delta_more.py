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
