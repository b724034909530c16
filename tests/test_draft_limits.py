"""CPU checks of limits of the draft model's operators (fake pointers, never
dereferenced)."""
import ctypes

import pytest

import row_reduction_pass_gb300 as rr_pkg


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return rr_pkg.load_library()


@pytest.mark.parametrize("T,status", [(2.0 ** -120, 0), (2.0 ** 120, 0), (1e-37, 1), (1e-40, 1),
                                      (2e36, 1), (3e38, 1), (-0.0, 1)])
def test_distill_temperature_limits(lib, T, status):
    """(rows == 0: nothing is launched)"""
    p = [ctypes.c_void_p(0x100000000 * (i + 1)) for i in range(6)]
    assert lib.rr_distill_fwd_bwd(p[0], p[1], p[2], None, p[3], p[4], 0, 8, 2, ctypes.c_float(T), 0,
                                  None, 0, ctypes.c_void_p(0)) == status
