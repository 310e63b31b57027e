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
