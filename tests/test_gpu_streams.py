"""A state that is dropped while another stream still works on it keeps its memory until that work is done."""
import pytest

from pace_testlib import ensure_built

pytestmark = pytest.mark.gpu


def test_memory_of_a_state_waits_for_the_streams_that_use_it():
    import torch

    ensure_built()
    import bit_gated_delta_gb300 as P
    B, H, D = 4, 8, 64
    state = P.PaceState(P.make_config(H, D, B), B)
    q, k, v, o = (torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    a, beta = torch.ones(2, B, H, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)                      # (about 0.2 s)
        state.decode_step(q, k, v, a, beta, o)
    at, size = state.mem.data_ptr(), state.mem.numel()
    del state
    other = torch.empty(size, dtype=torch.uint8, device="cuda")
    busy = not s.query()
    assert busy and other.data_ptr() != at
    s.synchronize()
