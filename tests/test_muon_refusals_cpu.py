"""What zero_newton_schulz refuses and what it takes, on the host: every call here
ends in a check, before anything is launched."""
import ctypes as C

import pytest


def _call(L, mats=0, rows=64, cols=96, irow=96, imat=0, orow=96, omat=0, coefs=(3.4445, -4.7750, 2.0315) * 5,
          nbytes=1 << 40):
    c = (C.c_float * len(coefs))(*coefs)
    return L.zero_newton_schulz(1 << 40, 0, irow, imat, 1 << 50, orow, omat, mats, rows, cols, c, len(coefs) // 3, 1.0,
                                1 << 30, nbytes, None)


# ------------------------------------------------------------ coefficients
@pytest.mark.parametrize("c", [1e-45, 1e-38, -1e-38, 1e-20, -1e-20, 1e-12, 0.0])
def test_a_maximum_inside_is_seen_whatever_the_last_coefficient(libzero, c):
    # p(s) = a (s - s^3) has its maximum 0.385 a at s = 0.577 and is 0 at 1
    assert _call(libzero, coefs=(7.9, -7.9, c)) == -1
    assert b"singular values" in libzero.zero_last_error()
    assert _call(libzero, coefs=(5.0, -5.0, c)) == 0
