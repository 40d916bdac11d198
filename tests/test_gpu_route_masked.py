"""Gradients of a routing whose rows have fewer open experts than k: what the gradient holds at pairs without an
expert is never used."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import experts_reference as ex
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("experts,k", [(3, 2), (8, 2), (9, 4), (40, 8), (130, 16), (512, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradients_of_pairs_without_an_expert(experts, k, dtype, normalize):
    """Their gates are 0, so a loss of the gates' logarithms gives infinities or NaN there: the same bits as with zeros."""
    n = 500
    rng = np.random.default_rng([11, experts, k])
    x = rng.standard_normal((n, experts)).astype(np.float32)
    for i in range(n):  # 0 .. k + 1 open experts
        x[i, rng.permutation(experts)[:max(0, experts - int(rng.integers(0, k + 2)))]] = -np.inf
    x = torch.from_numpy(x).to(DEV).to(TYPES[dtype])
    grad = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).to(DEV)
    note("route masked gradients experts=%d k=%d %s normalize=%s" % (experts, k, dtype, normalize))
    r = sc.submconv_route(x, k, normalize=normalize)
    none = r.experts < 0
    assert bool(none.any()) and bool(none.all(dim=1).any()) and not bool(r.gates[none].any())
    clean = grad.masked_fill(none, 0.0)
    expect = sc.submconv_route_backward(clean, x, r.experts, r.gates, normalize=normalize)
    want, bound = ex.route_backward(to_f64(clean), to_f64(x), r.experts.cpu().numpy(), to_f64(r.gates), normalize, ex.UNIT[dtype])
    assert (np.abs(to_f64(expect) - want) <= bound).all()
    for bad in (float("nan"), float("inf"), -float("inf"), 3.4e38):
        got = sc.submconv_route_backward(grad.masked_fill(none, bad), x, r.experts, r.gates, normalize=normalize)
        assert torch.equal(got, expect), "gradient %s at pairs without an expert" % bad


def test_a_gradient_of_an_expert_still_counts():
    """A NaN or infinity beside an expert is the row's, also where the gate has become 0."""
    x = torch.tensor([[0.0, 1.0, 2.0], [0.0, -300.0, -400.0]], device=DEV)
    note("route gradients beside experts")
    for normalize in (False, True):
        r = sc.submconv_route(x, 2, normalize=normalize)
        for row, j in ((0, 0), (0, 1), (1, 1)):
            grad = torch.ones((2, 2), device=DEV)
            grad[row, j] = float("nan")
            d = sc.submconv_route_backward(grad, x, r.experts, r.gates, normalize=normalize)
            assert bool(torch.isnan(d[row]).any()) and bool(torch.isfinite(d[1 - row]).all())
