"""The heads' norm of heads whose squares leave the range of fp32, against its definition in 64 bits: the result is
of ordinary size, whatever the head's."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import experts_reference as ex
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
N, H = 37, 5


def heads(dim, dtype, sizes, seed):
    """Heads of the given sizes in turn, so that the lanes of a wave have different ones."""
    rng = np.random.default_rng([seed, dim])
    x = np.clip(rng.standard_normal((N, H, dim)), -3, 3)
    x[np.abs(x) < 1e-3] = 1e-3
    x *= np.resize(np.asarray(sizes), (N, H))[..., None]
    g = rng.standard_normal((N, H, dim))
    pos = torch.from_numpy(rng.integers(0, 64, (N, 2), dtype=np.int32)).to(DEV)
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal((H, dim))).astype(np.float32)).to(DEV)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV).to(TYPES[dtype])  # noqa: E731
    return t(x), t(g), w, pos


@pytest.mark.parametrize("dim,sections", [(2, (1, 0)), (8, (2, 2)), (16, (2, 3)), (48, (8, 8)), (64, (16, 16)), (128, (32, 30)), (256, (50, 50)),
                                          (510, (100, 100))])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("eps,sizes", [(0.0, (1.0, 1e-17, 1e-22, 1e-30)), (0.0, (1.0, 1e18, 1e20, 1e30)), (1e-6, (1.0, 1e18, 1e20, 1e36)),
                                       (1e-36, (1.0, 1e-17, 1e-19, 1e-25)), (1e-6, (1.0, 1e-10, 1e-25, 1e25))])
def test_heads_of_any_size(dim, sections, dtype, split, eps, sizes):
    """Bounds as for ordinary heads: scaling by a power of two is exact."""
    x, g, w, pos = heads(dim, dtype, sizes, 1)
    freqs = sc.rotary_freqs(sections, device=DEV)
    args = (w, pos, freqs, sections)
    note("head norm range d=%d %s split=%s eps=%g sizes %s" % (dim, dtype, split, eps, sizes))
    y, rstd = sc.submconv_head_norm_rotary(x, *args, eps=eps, split=split, return_rstd=True)
    x64, g64, w64 = to_f64(x), to_f64(g), to_f64(w)
    host = (pos.cpu().numpy(), freqs.cpu().numpy(), sections)
    eps64 = float(np.float32(eps))
    expect, er, bound = ex.head_norm(x64, w64, 0, *host, eps64, split, ex.UNIT[dtype])
    err = np.abs(to_f64(y) - expect)
    assert (err <= bound).all(), "y off by %.3e" % np.nanmax(err - bound)
    assert (np.abs(to_f64(rstd) - er) <= (dim / 2 + 8) * ex.U32 * er).all()
    # gradients: of size 1 / rms, so only where that is far from the smallest normal number
    if max(sizes) <= 1e30:
        dx, dw = sc.submconv_head_norm_rotary_backward(g, x, rstd, *args, split=split)
        (edx, edw), (bx, bw) = ex.head_norm_backward(g64, x64, w64, 0, *host, eps64, split, ex.UNIT[dtype], ex.U32)
        assert (np.abs(to_f64(dx) - edx) <= bx).all() and (np.abs(to_f64(dw) - edw) <= bw).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_values(dtype):
    """A head of the type's largest values, and one of a single value among zeros."""
    top = torch.finfo(TYPES[dtype]).max
    x = torch.full((3, 2, 64), top, dtype=TYPES[dtype], device=DEV)
    x[1] = 0
    x[1, :, 7] = -top
    x[2] = 0
    note("head norm of the largest values %s" % dtype)
    y, rstd = sc.submconv_head_norm_rotary(x, return_rstd=True)
    # 1 / rms below 2^-126 has steps of 2^-149: at 2^-128 half a step is 2^-22; with the norm's own roundings 2^-18
    assert bool(((y[0].double() - 1).abs() <= 2.0 ** -18 + ex.UNIT[dtype]).all())
    assert bool(((y[1, :, 7].double() + 8).abs() <= 8 * (2.0 ** -18 + ex.UNIT[dtype])).all())
    y[1, :, 7] = 0
    assert not bool(y[1:].any()) and bool((rstd[2] == 1e3).all() | ((rstd[2] - 1e3).abs() < 1e-3).all())


def test_infinities_and_nan_stay_what_they_were():
    x = torch.ones((4, 2, 24), device=DEV)
    x[0, 0, 3], x[1, 1, 5], x[2, 0, 1], x[2, 0, 2] = float("inf"), float("nan"), float("inf"), float("nan")
    note("head norm of infinities")
    y, rstd = sc.submconv_head_norm_rotary(x, return_rstd=True)
    assert bool(torch.isnan(y[0, 0, 3])) and not bool(y[0, 0, 4:].any()) and float(rstd[0, 0]) == 0.0
    assert bool(torch.isnan(y[1, 1]).all()) and bool(torch.isnan(y[2, 0]).all())
    ok = torch.ones((4, 2), dtype=torch.bool, device=DEV)
    ok[0, 0] = ok[1, 1] = ok[2, 0] = False
    assert bool(torch.isfinite(y[ok]).all())
    zero = torch.zeros((1, 1, 24), device=DEV)
    assert not bool(sc.submconv_head_norm_rotary(zero).any())
    assert bool(torch.isnan(sc.submconv_head_norm_rotary(zero, eps=0.0)).all())
