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


# ----------------------------------------------------------------- strides
# A workspace of 256 bytes is refused after the strides have passed.
def _strides(L, mats, rows, cols, irow, imat, orow=None, omat=None):
    orow, omat = (cols, rows * cols) if orow is None else (orow, omat)
    st = _call(L, mats=mats, rows=rows, cols=cols, irow=irow, imat=imat, orow=orow, omat=omat, nbytes=256)
    assert st == -3
    return L.zero_last_error().decode()


def test_matrices_side_by_side_in_a_wider_buffer(libzero):
    # heads, or gate and up, as column ranges of one buffer
    assert "needed" in _strides(libzero, 2, 64, 96, 192, 96)
    assert "needed" in _strides(libzero, 2, 64, 96, 96, 64 * 96, 192, 96)     # the output
    assert "needed" in _strides(libzero, 32, 4096, 128, 32 * 128, 128)
    assert "overlap" in _strides(libzero, 2, 64, 96, 191, 96)
    assert "overlap" in _strides(libzero, 2, 64, 96, 192, 95)
    assert "overlap" in _strides(libzero, 3, 64, 96, 192, 96)
    assert "overlap" in _strides(libzero, 2, 64, 96, 96, 64 * 96, 192, 95)


def _disjoint(mats, rows, cols, row, mat):
    seen = set()
    for q in range(mats):
        for i in range(rows):
            for j in range(cols):
                at = q * mat + i * row + j
                if at in seen:
                    return False
                seen.add(at)
    return True


def test_strides_pass_exactly_where_no_two_elements_meet(libzero):
    for mats in (1, 2, 3, 4):
        for rows in (1, 2, 3, 5):
            for cols in (1, 2, 4):
                for row in range(cols if rows > 1 else 0, 14):
                    for mat in range(0, 34):
                        msg = _strides(libzero, mats, rows, cols, row, mat)
                        assert ("needed" in msg) == _disjoint(mats, rows, cols, row, mat), (mats, rows, cols, row, mat, msg)


def test_strides_at_the_limits(libzero):
    big = (1 << 62) // 70000
    assert "needed" in _strides(libzero, 65535, 2, 3, 3 * 65535, 3)
    assert "overlap" in _strides(libzero, 65535, 2, 3, 3 * 65535 - 1, 3)
    for row, mat in ((big, 1), (1, big), (big, big), (1 << 62, 0), (0, 1 << 62), (1 << 62, 1 << 62)):
        msg = _strides(libzero, 65535, 262144, 1, row, mat)
        assert "overlap" in msg or "out of range" in msg or "below cols" in msg or "needed" in msg


# ------------------------------------------------- coefficients and roundings
# Five steps, each the best quintic for the range that the last one leaves: results
# reach 1.99, where the next polynomial's slope is 10.
MINIMAX = ((8.28721201814563, -23.595886519098837, 17.300387312530933),
           (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
           (3.9486908534822946, -2.908902115962949, 0.5518191394370137),
           (3.3184196573706015, -2.488488024314874, 0.51004894012372),
           (2.300652019954817, -1.6689039845749493, 0.4188073119525673))


def _divided(by):
    return [v for a, b, c in MINIMAX for v in (a / by, b / by ** 3, c / by ** 5)]


def test_a_set_without_room_for_a_rounding_is_refused(libzero):
    assert _call(libzero, coefs=_divided(1.0)) == -1
    assert b"rounding" in libzero.zero_last_error()
    for by in (1.01, 1.02, 1.05):
        assert _call(libzero, coefs=_divided(by)) == 0
    assert _call(libzero, coefs=_divided(1.0)[:3]) == 0      # what grows is the steps after the first


@pytest.mark.parametrize("coefs", [(3.4445, -4.7750, 2.0315) * 16, (1.5, -0.5, 0.0) * 16, (1.875, -1.25, 0.375) * 16,
                                   (3.4445, -4.7750, 2.0315) * 5 + (1.5, -0.5, 0.0) * 5, (1e-3, 0.0, 0.0),
                                   (0.0, 0.0, 0.0) * 3, (-1.0, 0.0, 0.0) * 4, (5.125, -5.125, 0.0)])
def test_sets_with_room_are_taken(libzero, coefs):
    assert _call(libzero, coefs=coefs) == 0
