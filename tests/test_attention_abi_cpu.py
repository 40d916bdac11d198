"""Arguments of the attention entry points at the edge of what they take.  CPU only: every call here is
refused, or accepted without work, before any HIP call."""
import ctypes

import pytest

import submanifold_sparse_convolution_submconv3d_amd as sc

from test_block_abi_cpu import E_INVALID_ARG, attention, attention_bwd


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
