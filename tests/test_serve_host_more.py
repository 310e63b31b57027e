"""More of the host side of include/pace_serve.h. CPU only: no call reaches a GPU."""
import ctypes as C

import pytest

from pace_testlib import ensure_built

INVALID = 1
MEM = 1 << 20                     # an address that no refused call reads


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    P.lib()
    return P


def test_the_probe_of_waits_is_refused(P):
    with pytest.raises(P.PaceError) as e:
        P.serve.pace_test_delta_wait_probe(None, 1000)
    assert e.value.status == INVALID
