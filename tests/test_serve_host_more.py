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


class Handle(C.Structure):
    """As much of a pace_pages as a refused call reads: its configuration, and nothing that points anywhere."""
    _fields_ = [("n_pages", C.c_int), ("page_tokens", C.c_int), ("max_batch", C.c_int), ("rest", C.c_byte * 500)]


def test_tables_whose_cells_pass_32_bits_are_not_taken_from(P):
    pages = Handle(1 << 30, 32, 1024)
    for batch, cols in ((1024, 1 << 21), (64, 1 << 25), (1024, 1 << 25)):
        assert P.lib().pace_pages_take(C.byref(pages), batch, MEM, cols, MEM, MEM, MEM, None) == 2, (batch, cols)
        assert "cells" in P.pace_last_error()
    assert P.lib().pace_pages_take(C.byref(pages), 1, MEM, (1 << 25) + 1, MEM, MEM, MEM, None) == INVALID
