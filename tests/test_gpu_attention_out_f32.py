"""Attention of bf16 tensors with its result kept in fp32: the same result without the last rounding, and
gradients that are spared that rounding."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import block_reference as ref
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def heads(rng, n, h, d, std=1.0, mean=0.0, dtype=BF16):
    return torch.from_numpy((std * rng.standard_normal((n, h, d)) + mean).astype(np.float32)).to(DEV).to(dtype)


def offsets(lengths):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).to(DEV)


# one pass; split along the keys; split along the queries in the backward pass; the last round of tiles cut
@pytest.mark.parametrize("lq,lk,h,hk,d", [([70, 0, 133], [40, 5, 90], 4, 2, 72), ([3, 2], [9000, 4001], 4, 1, 64),
                                          ([9000, 21], [5, 140], 2, 2, 128), ([3900], [3900], 13, 13, 32), ([33, 60], [0, 50], 2, 2, 24)])
def test_out_in_fp32_is_the_result_before_rounding(lq, lk, h, hk, d):
    rng = np.random.default_rng([sum(lq), h, d])
    q, k, v, g = heads(rng, sum(lq), h, d), heads(rng, sum(lk), hk, d), heads(rng, sum(lk), hk, d), heads(rng, sum(lq), h, d)
    qo, ko = offsets(lq), offsets(lk)
    note("attention fp32 out %s %s h=%d/%d d=%d" % (lq, lk, h, hk, d))
    low, llse = sc.submconv_attention(q, k, v, qo, ko, return_lse=True)
    out, lse = sc.submconv_attention(q, k, v, qo, ko, return_lse=True, out_dtype=F32)
    assert out.dtype == F32 and low.dtype == BF16
    assert torch.equal(out.to(BF16), low) and torch.equal(lse, llse)
    held = torch.full((sum(lq), h, d + 3), 7.0, device=DEV)
    sc.submconv_attention(q, k, v, qo, ko, out=held[..., 1:d + 1])      # an fp32 tensor at any alignment
    assert torch.equal(held[..., 1:d + 1], out) and bool((held[..., 0] == 7).all()) and bool((held[..., d + 1:] == 7).all())
    # a result that bf16 holds gives the same gradients in either type
    want = sc.submconv_attention_backward(g, q, k, v, low, lse, qo, ko)
    assert all(torch.equal(a, b) for a, b in zip(sc.submconv_attention_backward(g, q, k, v, low.float(), lse, qo, ko), want))
    again = [sc.submconv_attention_backward(g, q, k, v, out, lse, qo, ko) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*again)) and torch.equal(again[0][2], want[2])


def test_gradients_of_values_with_an_offset():
    """Values around `mean`: dp and delta are both near mean sum(grad) and cancel.  What a bf16 out loses
    (2^-9 of it on average, at random) stays; an fp32 out leaves the sums' roundings and those of the weights,
    which average out over 200 nearly equal ones.  So dq's error is several times smaller; here it has to be
    at most a third."""
    rng = np.random.default_rng(3)
    n, d, mean = 200, 64, 8.0
    q, k, g = (heads(rng, n, 1, d) for _ in range(3))
    v = heads(rng, n, 1, d, mean=mean)
    off, o = offsets([n]), np.array([0, n])
    note("attention values with an offset")
    expect, _ = ref.attention_backward(*(to_f64(t) for t in (g, q, k, v)), o, o, d ** -0.5, ref.UNIT["bf16"])
    error = {}
    for kind in (BF16, F32):
        out, lse = sc.submconv_attention(q, k, v, off, return_lse=True, out_dtype=kind)
        dq, dk, _ = (to_f64(t) for t in sc.submconv_attention_backward(g, q, k, v, out, lse, off))
        error[kind] = [np.linalg.norm(a - b) / np.linalg.norm(b) for a, b in ((dq, expect[0]), (dk, expect[1]))]
        print("  out %s: dq off by %.5f, dk by %.5f" % (kind, *error[kind]), flush=True)
    assert error[F32][0] <= error[BF16][0] / 3 and error[F32][1] <= error[BF16][1] / 3


def test_refused_types_of_out():
    rng = np.random.default_rng(4)
    h = heads(rng, 6, 2, 16)
    off = offsets([6])
    out, lse = sc.submconv_attention(h, h, h, off, return_lse=True)
    note("attention types of out")
    for call in (lambda: sc.submconv_attention(h, h, h, off, out_dtype=torch.float16),
                 lambda: sc.submconv_attention(h, h, h, off, out=torch.empty_like(h, dtype=F32), out_dtype=BF16),
                 lambda: sc.submconv_attention(h.float(), h.float(), h.float(), off, out=torch.empty_like(h)),
                 lambda: sc.submconv_attention_backward(h, h, h, h, out.double(), lse, off),
                 lambda: sc.submconv_attention_backward(h.float(), h.float(), h.float(), h.float(), out, lse, off)):
        with pytest.raises(TypeError):
            call()
