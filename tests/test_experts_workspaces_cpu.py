"""Refusals of missing, short, misaligned and overlapping workspaces of the gradients of grouped products, in calls that do
need one, and the message of an overlap.  CPU only; pointers are never read."""
import ctypes

import pytest

import submanifold_sparse_convolution_submconv3d_amd as sc

E_INVALID_ARG, E_ALIAS = -1, -5
P = lambda i: ctypes.c_void_p(i << 36)  # noqa: E731  (addresses 64 GiB apart)
X_ROW = G_ROW = 4096


@pytest.fixture(scope="module")
def lib():
    return sc.load_library()


def backward(lib, n, cin, cout, groups, dtype, g=P(1), x=P(2), w=P(4), offsets=P(5), dx=P(6), dw=P(7), db=P(8), ws=P(9), nbytes=1 << 34):
    return lib.submconv_grouped_linear_backward(g, G_ROW, x, X_ROW, n, P(3), w, offsets, groups, n, cin, cout, dtype, dx, cin, dw, db, ws, nbytes,
                                                None)


# pieces of groups in each of the kernels, aligned and not, in both types
CALLS = [(20000, 64, 32, 4, 1), (20000, 64, 32, 4, 0), (20384, 123, 501, 5, 0), (20384, 123, 501, 5, 1), (60000, 264, 520, 2, 1),
         (20000, 264, 516, 3, 0), (65000, 256, 256, 70, 1), (90000, 3, 517, 3, 0), (512, 1, 1, 1, 1)]


@pytest.mark.parametrize("n,cin,cout,groups,dtype", CALLS)
def test_workspace_refusals(lib, n, cin, cout, groups, dtype):
    need = lib.submconv_grouped_linear_backward_workspace(groups, n, cin, cout, dtype)
    assert need > 0 and need % 4 == 0
    call = lambda **k: backward(lib, n, cin, cout, groups, dtype, **k)  # noqa: E731
    for bad in (dict(nbytes=need - 1), dict(nbytes=0), dict(ws=None), dict(ws=None, nbytes=need), dict(ws=None, db=None), dict(nbytes=need - 1, dx=None),
                dict(nbytes=need - 1, db=None), dict(ws=ctypes.c_void_p((9 << 36) + 8)), dict(ws=ctypes.c_void_p((9 << 36) + 4), nbytes=need)):
        assert call(**bad) == E_INVALID_ARG, bad
    assert b"workspace" in lib.submconv_last_error() or b"misaligned" in lib.submconv_last_error()
    last = lambda at, size: ctypes.c_void_p((at << 36) + (size - 1) // 16 * 16)  # noqa: E731  (its last 16 bytes)
    es = 2 if dtype else 4
    for bad in (dict(ws=P(1)), dict(ws=P(2)), dict(ws=P(3)), dict(ws=P(4)), dict(ws=P(5)), dict(ws=P(6)), dict(ws=P(7)), dict(ws=P(8)),
                dict(ws=last(2, ((n - 1) * X_ROW + cin) * es)), dict(ws=last(1, ((n - 1) * G_ROW + cout) * es)), dict(ws=last(3, 4 * n)),
                dict(ws=last(7, groups * cin * cout * es)), dict(dw=last(9, need)), dict(db=last(9, need))):
        assert call(**bad) == E_ALIAS, bad


def test_sizes_without_a_workspace(lib):
    """Below 512 positions, or where whole groups fill the card, there is none, and none is asked for."""
    for args in ((4, 511, 64, 32, 1), (16, 8000, 1024, 1024, 1), (1, 0, 64, 32, 1)):
        assert lib.submconv_grouped_linear_backward_workspace(*args) == 0
    # a refusal of something else comes with ws = NULL: the workspace is not what is missing
    assert backward(lib, 511, 64, 32, 4, 1, ws=None, nbytes=0, dx=P(1)) == E_ALIAS
    assert b"workspace" not in lib.submconv_last_error()


def test_an_overlap_names_both(lib):
    code = lib.submconv_combine(P(1), 64, 200, P(2), P(3), 100, 2, 64, 0, P(1), 64, None)
    assert code == E_ALIAS
    assert b"out overlaps y" in lib.submconv_last_error() or b"y overlaps out" in lib.submconv_last_error()
    assert backward(lib, 20000, 64, 32, 4, 1, ws=P(2)) == E_ALIAS
    message = lib.submconv_last_error()
    assert b"workspace" in message and b"x" in message
