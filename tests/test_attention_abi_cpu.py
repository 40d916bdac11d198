"""Arguments of the attention entry points at the edge of what they take.  CPU only: every call here is
refused, or accepted without work, before any HIP call."""
import ctypes

import pytest

import submanifold_sparse_convolution_submconv3d_amd as sc

from test_block_abi_cpu import E_ALIAS, E_INVALID_ARG, E_UNSUPPORTED, attention, attention_bwd


@pytest.fixture(scope="module")
def lib():
    return sc.load_library()


@pytest.mark.parametrize("scale", [1.01e38, 2.4e38, 3.4e38])
def test_scales_whose_exponents_overflow_are_refused(lib, scale):
    """scale times log2 e has to stay finite: weights are formed as powers of two."""
    assert attention(lib, scale=scale) == E_INVALID_ARG
    assert b"scale" in lib.submconv_last_error()
    assert attention_bwd(lib, scale=scale) == E_INVALID_ARG
    assert b"scale" in lib.submconv_last_error()
    assert attention(lib, scale=1e38, nq=0) == 0 and attention_bwd(lib, scale=1e38, nq=0, nk=0) == 0


def at(base, elements):
    """`elements` bf16 past the address that stands for tensor number `base`."""
    return ctypes.c_void_p((base << 32) + 2 * elements)


def test_interleaved_outputs_that_overlap_are_refused(lib):
    """Gradients packed head by head ([heads, 3, n, dim] and [n, heads, 3, dim]): one element too near is
    an overlap.  (What lies clear of each other is run on the GPU.)"""
    n, h, d = 100, 2, 64
    sizes = dict(entries=1, nq=n, nk=n, heads=h, kv_heads=h, dim=d)
    for row, head, step in ((d, 3 * n * d, n * d), (3 * h * d, 3 * d, d)):
        strides = (h * d, d) * 5 + (row, head) * 3
        for dq, dk, dv in ((0, step - 1, 2 * step), (0, step, 2 * step - 1), (1, step, 2 * step), (0, step, 2 * step + 1), (0, step + row, step)):
            assert attention_bwd(lib, strides=strides, dq=at(9, dq), dk=at(9, dk), dv=at(9, dv), **sizes) == E_ALIAS, (row, dq, dk, dv)
    # a written tensor between the heads of one that is read, the last of its rows one element too far
    strides = (d, 2 * n * d) + (h * d, d) * 2 + (d, 2 * n * d)
    assert attention(lib, strides=strides, out=at(1, n * d + 1), **sizes) == E_ALIAS


def test_fp32_out_flag(lib):
    """SUBMCONV_OUT_F32 beside a known type; an fp32 out has twice the bytes of a bf16 one."""
    flag = sc.OUT_F32
    sizes = (2, 100, 100, 4, 2, 64)
    for dtype in (0, 1):
        assert attention(lib, nq=0, dtype=dtype | flag) == 0
        assert lib.submconv_attention_backward_workspace(*sizes, dtype | flag) == lib.submconv_attention_backward_workspace(*sizes, dtype) > 0
    for dtype in (2 | flag, flag << 1, 1 | flag << 1, -1, -1 & ~flag):
        assert attention(lib, nq=0, dtype=dtype) == E_UNSUPPORTED, dtype
        assert lib.submconv_attention_backward_workspace(*sizes, dtype) == 0
    # 100 rows of 256: past 51200 bytes only if they are fp32
    near = ctypes.c_void_p((6 << 32) + 60000)
    assert attention(lib, lse=near, dtype=1 | flag) == E_ALIAS
    assert attention(lib, out=ctypes.c_void_p((6 << 32) + 2), dtype=1 | flag) == E_INVALID_ARG
