"""More of the verification of drafts: random numbers at their ends with every row's token, rows that are no distributions."""
import numpy as np
import pytest

from pace_testlib import ensure_built
from test_gpu_verify import call, check, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    return P


def test_every_row_of_random_numbers_at_their_ends(P):
    """p has 1/4 at token 5 and 3/4 at 2990. Named drafts: 2990 is kept where u < 3/4; where it is refused only 5 is left; 7 is never kept."""
    import torch
    V = 3000
    p = torch.zeros(3, 2, V, device="cuda")
    p[:, :, 5], p[:, :, 2990] = 0.25, 0.75
    tok = torch.tensor([[0, 2990], [0, 2990], [0, 7]], dtype=torch.int32, device="cuda")
    last = float(np.nextafter(np.float32(1), np.float32(0)))
    for u, want, kept in ((0.0, [5, 5, 5], [2, 2, 1]), (last, [5, 5, 2990], [1, 1, 1]), (1.0, [5, 5, 2990], [1, 1, 1])):
        idx, n, nxt = call(P, torch, tok, p, None, torch.full((3, 2), u, device="cuda"))
        assert n.tolist() == kept and nxt.tolist() == want


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [1 << 17, (1 << 17) + 3, 1 << 18, 1000003])
def test_rows_of_ones(P, V, dtype):
    """Rows that sum to the size of the vocabulary (all ones, or infinities, which count as ones), far above a distribution's 1: the formulas hold
    for them. Values are 0, 1/2 and 1, so that every sum is exact."""
    import torch
    dt = getattr(torch, dtype)
    B, N = 4, 4
    p = torch.ones(B, N, V, dtype=dt, device="cuda")
    p[1] = float("inf")
    p[2, :, : V // 2] = 0.5
    q = torch.full((B, N, V), 0.5, dtype=dt, device="cuda")
    tok = torch.tensor([[0, 5, 9, V - 1]] * B, dtype=torch.int32, device="cuda")
    q[:, :, 5] = q[:, :, 9] = 1.0
    see = np.eye(N, dtype=bool)
    see[1:, 0] = True                                    # three drafts of one node
    mask = words(torch, np.tile(see, (B, 1, 1)))
    parents = np.tile(np.array([-1, 0, 0, 0]), (B, 1))
    for u in ([0.3, 1.0, 1.0, 1.0], [0.999, 1.0, 0.5, 1e-9], [0.75, 0.25, 0.5, 0.5]):
        uu = torch.tensor([u] * B, device="cuda")
        for draft in (q, None):
            check(P, torch, tok, p, draft, uu, parents, mask)


def test_ones_over_the_largest_vocabulary(P):
    import torch
    V = P.PACE_VERIFY_MAX_VOCAB
    p = torch.ones(1, 1, V, dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for u, want in ((0.0, 0), (0.5, V // 2), (0.75, 3 * (V // 4)), (1.0, V - 1)):
        _, n, nxt = call(P, torch, tok, p, None, torch.full((1, 1), u, device="cuda"))
        assert n.tolist() == [1] and nxt.tolist() == [want]
