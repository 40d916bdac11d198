"""Gradients of ragged attention where a key holds an infinity that gives it no weight."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import block_reference as ref
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq,h", [(1, 1), (32, 2), (33, 2), (11, 3), (130, 2), (20011, 2)])
def test_attention_gradients_of_a_key_without_weight(nq, h, dtype):
    """A key with an element of -inf where all queries are positive has scores of -inf and weights of
    zero: dk and dv are zero for it, and for the others what they are without it, whatever the number of
    query rows (20011: split between blocks).  (dq is 0 times inf there, which has no value.)"""
    nk, d, gone = 70, 64, 9
    rng = np.random.default_rng([nq, h])
    make = lambda n, m: torch.from_numpy(rng.standard_normal((n, m, d)).astype(np.float32)).to(DEV).to(TYPES[dtype])  # noqa: E731
    q, k, v, g = make(nq, h), make(nk, 1), make(nk, 1), make(nq, h)
    q[..., 5] = q[..., 5].abs() + 0.5
    k[gone, 0, 5] = -float("inf")
    qo, ko = np.array([0, nq]), np.array([0, nk])
    tq, tk = (torch.from_numpy(o.astype(np.int32)).to(DEV) for o in (qo, ko))
    note("attention key without weight nq=%d h=%d %s" % (nq, h, dtype))
    out, lse = sc.submconv_attention(q, k, v, tq, tk, return_lse=True)
    _, dk, dv = (to_f64(t) for t in sc.submconv_attention_backward(g, q, k, v, out, lse, tq, tk))
    assert (dk[gone] == 0).all() and (dv[gone] == 0).all()
    rest = np.arange(nk) != gone
    expect, bounds = ref.attention_backward(to_f64(g), to_f64(q), to_f64(k)[rest], to_f64(v)[rest], qo, ko - [0, 1], d ** -0.5, ref.UNIT[dtype])
    for name, got, e, b in (("dk", dk[rest], expect[1], bounds[1]), ("dv", dv[rest], expect[2], bounds[2])):
        assert (np.abs(got - e) <= b).all(), name
