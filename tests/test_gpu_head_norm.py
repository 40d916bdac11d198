"""The heads' norm with rotation on the GPU against its definition in 64 bits (bounds in experts_reference.py)."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import experts_reference as ex
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(n, h, d, dtype, many, seed, axes=3, wtype=torch.float32, res=64):
    rng = np.random.default_rng([seed, n, h, d])
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV)  # noqa: E731
    pos = torch.from_numpy(rng.integers(0, res, (n, axes), dtype=np.int32)).to(DEV)
    return f(n, h, d).to(TYPES[dtype]), f(n, h, d).to(TYPES[dtype]), (1 + 0.3 * f(many, d)).to(wtype), pos


def within(got, expect, bound, what):
    err = np.abs(to_f64(got) - expect)
    assert (err <= bound).all(), "%s off by %.3e" % (what, (err - bound).max())


def check(x, g, w, q_heads, pos, freqs, sections, dtype, split, eps=1e-6):
    args = (w, pos, freqs, sections)
    y, rstd = sc.submconv_head_norm_rotary(x, *args, eps=eps, q_heads=q_heads, split=split, return_rstd=True)
    dx, dw = sc.submconv_head_norm_rotary_backward(g, x, rstd, *args, q_heads=q_heads, split=split)
    x64, g64, w64 = to_f64(x), to_f64(g), to_f64(w)
    host = (pos.cpu().numpy(), freqs.cpu().numpy(), sections)
    unit = ex.UNIT[dtype]
    ey, er, by = ex.head_norm(x64, w64, q_heads, *host, eps, split, unit)
    within(y, ey, by, "y")
    assert (np.abs(to_f64(rstd) - er) <= (x64.shape[2] / 2 + 8) * ex.U32 * er).all()
    (edx, edw), (bx, bw) = ex.head_norm_backward(g64, x64, w64, q_heads, *host, eps, split, unit,
                                                 ex.UNIT["f32" if w.dtype == torch.float32 else "bf16"])
    within(dx, edx, bx, "dx")
    within(dw, edw, bw, "dweight")
    return y, rstd, dx, dw


@pytest.mark.parametrize("dim,sections", [(2, (1,)), (6, (1, 1, 1)), (16, (2, 2, 2)), (30, (5, 5, 5)), (64, (10, 10, 10)), (64, (32,)),
                                          (80, (0, 40)), (96, (16, 16, 16)), (128, (21, 21, 21)), (250, (30, 30, 30, 35)), (258, (43, 43, 43)),
                                          (512, (85, 85, 85))])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("split", [False, True])
def test_head_norm(dim, sections, dtype, split):
    freqs = sc.rotary_freqs(sections, device=DEV)
    for n, h, many, q_heads, wtype in ((1, 1, 1, 0, torch.float32), (3, 5, 5, 0, torch.bfloat16), (257, 8, 2, 6, torch.float32),
                                       (130, 33, 1, 0, torch.float32), (61, 130, 130, 0, torch.float32), (40, 70, 2, 1, torch.bfloat16)):
        x, g, w, pos = make(n, h, dim, dtype, many, 1, len(sections), wtype)
        note("head norm n=%d h=%d d=%d %s %s split=%s weights %d q_heads %d" % (n, h, dim, sections, dtype, split, many, q_heads))
        check(x, g, w, q_heads, pos, freqs, sections, dtype, split)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_norm_many_rows(dtype):
    """More rows than blocks take at once: sums over blocks and the walk along the rows."""
    sections = (5, 5, 5)
    freqs = sc.rotary_freqs(sections, device=DEV)
    for h, many, q_heads in ((1, 1, 0), (3, 3, 0), (70, 2, 64)):
        x, g, w, pos = make(40001 if h < 70 else 4001, h, 32, dtype, many, 2)
        note("head norm many rows h=%d %s" % (h, dtype))
        check(x, g, w, q_heads, pos, freqs, sections, dtype, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("split", [False, True])
def test_head_norm_without_rotation_or_weight(dtype, split):
    x, g, w, _ = make(77, 6, 40, dtype, 6, 3)
    zero = torch.zeros((77, 1), dtype=torch.int32, device=DEV)
    note("head norm alone %s" % dtype)
    plain, rstd = sc.submconv_head_norm_rotary(x, w, split=split, return_rstd=True)
    assert torch.equal(plain, sc.submconv_head_norm_rotary(x, w, zero, torch.ones(3, device=DEV), (3,), split=split))
    one = sc.submconv_head_norm_rotary(x, split=split)
    assert torch.equal(one, sc.submconv_head_norm_rotary(x, torch.ones(40, device=DEV), split=split))
    dx, dw = sc.submconv_head_norm_rotary_backward(g, x, rstd, split=split)
    assert dw is None
    assert torch.equal(dx, sc.submconv_head_norm_rotary_backward(g, x, rstd, torch.ones(40, device=DEV), split=split)[0])
    dx, dw = sc.submconv_head_norm_rotary_backward(g, x, rstd, w, split=split, need_weight=False)
    assert dw is None and torch.equal(dx, sc.submconv_head_norm_rotary_backward(g, x, rstd, w, split=split)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("split", [False, True])
def test_head_norm_views_and_in_place(dtype, split):
    """Queries and keys inside a packed projection, coordinate columns, odd offsets, head-major order, in place."""
    n, h, d, sections = 211, 6, 48, (8, 8, 8)
    freqs = sc.rotary_freqs(sections, device=DEV)
    qkv, grad, w, _ = make(n, 3 * h, d, dtype, 2, 4)
    coords = torch.from_numpy(np.random.default_rng(5).integers(0, 100, (n, 4), dtype=np.int32)).to(DEV)
    pos = coords[:, 1:]
    args = (w, pos, freqs, sections)
    more = dict(q_heads=h, split=split)
    note("head norm views %s split=%s" % (dtype, split))
    qk, g = qkv[:, :2 * h], grad[:, :2 * h]
    y, rstd, dx, dw = check(qk.contiguous(), g.contiguous(), w, h, pos.contiguous(), freqs, sections, dtype, split)
    got, r = sc.submconv_head_norm_rotary(qk, *args, return_rstd=True, **more)
    assert torch.equal(got, y) and torch.equal(r, rstd)
    major = torch.empty((2 * h, n, d), dtype=qkv.dtype, device=DEV)
    sc.submconv_head_norm_rotary(qk, *args, out=major.transpose(0, 1), **more)
    assert torch.equal(major.transpose(0, 1), y)
    odd = torch.zeros((n, 2 * h, d + 3), dtype=qkv.dtype, device=DEV)
    odd[:, :, 1:1 + d] = qk
    assert torch.equal(sc.submconv_head_norm_rotary(odd[:, :, 1:1 + d], *args, **more), y)
    for a, b in zip(sc.submconv_head_norm_rotary_backward(g, odd[:, :, 1:1 + d], rstd, *args, dx=major.transpose(0, 1), **more), (dx, dw)):
        assert torch.equal(a, b)
    values = grad[:, 2 * h:].clone()
    sc.submconv_head_norm_rotary_backward(g, qk, rstd, *args, dx=g, **more)
    assert torch.equal(g, dx) and torch.equal(grad[:, 2 * h:], values)
    values = qkv[:, 2 * h:].clone()
    sc.submconv_head_norm_rotary(qk, *args, out=qk, **more)
    assert torch.equal(qk, y) and torch.equal(qkv[:, 2 * h:], values)


def test_head_norm_agrees_with_the_rotation_alone():
    """Positions that turn far: the same angles as submconv_rotary's."""
    sections = (8, 8)
    freqs = sc.rotary_freqs(sections, device=DEV)
    x, _, _, _ = make(64, 2, 32, "f32", 1, 6)
    pos = torch.from_numpy(np.random.default_rng(3).integers(-2 ** 31, 2 ** 31 - 1, (64, 2)).astype(np.int32)).to(DEV)
    note("head norm large positions")
    got = sc.submconv_head_norm_rotary(x, None, pos, freqs, sections)
    two = sc.submconv_rotary(sc.submconv_head_norm_rotary(x), pos, freqs, sections)
    assert (got - two).abs().max() <= 4 * ex.U32 * got.abs().max()


def test_head_norm_rows_apart_and_zero_rows():
    """A head of zeros gives zeros; infinities and NaN stay in their own head."""
    sections = (4, 4, 4)
    freqs = sc.rotary_freqs(sections, device=DEV)
    x, g, w, pos = make(50, 4, 24, "f32", 4, 7)
    plain = sc.submconv_head_norm_rotary(x, w, pos, freqs, sections)
    x[3, 1] = 0
    x[7, 2, 5] = float("inf")
    x[9, 0, 23] = float("nan")
    note("head norm special heads")
    y, rstd = sc.submconv_head_norm_rotary(x, w, pos, freqs, sections, return_rstd=True)
    dx, _ = sc.submconv_head_norm_rotary_backward(g, x, rstd, w, pos, freqs, sections)
    bad = torch.zeros((50, 4), dtype=torch.bool, device=DEV)
    bad[3, 1] = bad[7, 2] = bad[9, 0] = True
    assert torch.equal(y[~bad], plain[~bad]) and bool((y[3, 1] == 0).all()) and bool(torch.isnan(y[9, 0]).any())
    assert bool(torch.isfinite(dx[~bad]).all()) and bool(torch.isfinite(dx[3, 1]).all())


def test_head_norm_empty():
    sections = (2, 2, 2)
    freqs = sc.rotary_freqs(sections, device=DEV)
    x = torch.zeros((0, 4, 12), device=DEV)
    pos = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    w = torch.ones((4, 12), device=DEV)
    note("head norm empty")
    y, rstd = sc.submconv_head_norm_rotary(x, w, pos, freqs, sections, return_rstd=True)
    dx, dw = sc.submconv_head_norm_rotary_backward(x, x, rstd, w, pos, freqs, sections)
    assert y.shape == dx.shape == (0, 4, 12) and bool((dw == 0).all())


def test_head_norm_offsets_past_32_bits():
    sections = (2, 2, 2)
    freqs = sc.rotary_freqs(sections, device=DEV)
    n, ld = 270001, 8192
    wide = torch.empty((n, ld), dtype=torch.bfloat16, device=DEV)
    x0, g, w, pos = make(n, 2, 12, "bf16", 2, 9)
    x = wide[:, 100:124].view(n, 2, 12)
    x.copy_(x0)
    note("head norm offsets past 32 bits")
    a, ra = sc.submconv_head_norm_rotary(x, w, pos, freqs, sections, return_rstd=True)
    b, rb = sc.submconv_head_norm_rotary(x0, w, pos, freqs, sections, return_rstd=True)
    assert torch.equal(a, b) and torch.equal(ra, rb)
    for p, q in zip(sc.submconv_head_norm_rotary_backward(g, x, ra, w, pos, freqs, sections),
                    sc.submconv_head_norm_rotary_backward(g, x0, rb, w, pos, freqs, sections)):
        assert torch.equal(p, q)
    del wide, x
    torch.cuda.empty_cache()
