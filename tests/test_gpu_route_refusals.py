"""Numbers of experts a row that the library does not take come back as its refusal."""
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

from gpu_common import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_many_experts_a_row_are_refused():
    """k past what the library takes is refused before anything of that size is allocated, however large."""
    x = torch.zeros((100000, 8), device=DEV)
    note("route of too many experts a row")
    for k in (9, 17, 1 << 20, 2 ** 31 - 1, 2 ** 32 + 2, 1 << 40, -(2 ** 32) + 2):
        before = torch.cuda.max_memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        with pytest.raises(sc.SubmconvError):
            sc.submconv_route(x, k)
        with pytest.raises(sc.SubmconvError):
            sc.submconv_route(x[:0], k)
        assert torch.cuda.max_memory_allocated() < before + (64 << 20)
