"""Rotary positions on the GPU against the 64-bit definition.

Bound: sine and cosine of a phase reduced in fp64 are good to a few fp32 roundings (8 u,
u = 2^-24), the two products and their sum add three, and the result is rounded once:
|error| <= unit(type) |y| + 16 u (|a| + |b|)."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import block_reference as ref
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(n, h, d, dtype, seed, res=64, axes=3):
    rng = np.random.default_rng([seed, n, h, d])
    x = torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(DEV).to(TYPES[dtype])
    pos = torch.from_numpy(rng.integers(0, res, (n, axes), dtype=np.int32)).to(DEV)
    return x, pos


def check(out, x, pos, freqs, sections, dtype, inverse=False, split=False):
    x64 = to_f64(x)
    expect = ref.rotary(x64, pos.cpu().numpy(), freqs.cpu().numpy(), sections, inverse, split)
    d = x64.shape[2]
    mate = np.concatenate([x64[..., d // 2:], x64[..., :d // 2]], axis=-1) if split else \
        x64.reshape(x64.shape[:2] + (d // 2, 2))[..., ::-1].reshape(x64.shape)
    bound = ref.UNIT[dtype] * np.abs(expect) + 16 * ref.U32 * (np.abs(x64) + np.abs(mate))
    err = np.abs(to_f64(out) - expect)
    assert (err <= bound).all(), "off by %.3e" % (err - bound).max()
    used = sum(sections)
    rest = np.r_[used:d // 2, d // 2 + used:d] if split else np.r_[2 * used:d]
    assert (to_f64(out)[..., rest] == x64[..., rest]).all(), "pairs past the sections are copied"


@pytest.mark.parametrize("dim,sections", [(2, (1,)), (6, (1, 1, 1)), (16, (2, 2, 2)), (30, (5, 5, 5)), (64, (10, 10, 10)),
                                          (64, (32,)), (96, (16, 16, 16)), (128, (21, 21, 21)), (128, (16, 24, 24)),
                                          (80, (0, 40)), (250, (30, 30, 30, 35)), (512, (85, 85, 85))])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("split", [False, True])
def test_rotary(dim, sections, dtype, split):
    freqs = sc.rotary_freqs(sections, device=DEV)
    for n, h in ((1, 1), (3, 5), (257, 8), (130, 33)):
        x, pos = make(n, h, dim, dtype, 1, axes=len(sections))
        note("rotary n=%d h=%d d=%d %s %s split=%s" % (n, h, dim, sections, dtype, split))
        out = sc.submconv_rotary(x, pos, freqs, sections, split=split)
        check(out, x, pos, freqs, sections, dtype, split=split)
        check(sc.submconv_rotary(x, pos, freqs, sections, split=split, inverse=True), x, pos, freqs, sections, dtype,
              inverse=True, split=split)


def test_rotary_freqs():
    f = sc.rotary_freqs((21, 21, 21), 10000.0, DEV).cpu().numpy()
    assert f.shape == (63,) and f.dtype == np.float32
    for p in range(63):
        assert f[p] == np.float32(10000.0 ** (-(p % 21) / 21.0))
    assert sc.rotary_freqs((0, 2), device=DEV).shape == (2,)


def test_rotary_large_positions():
    """The phase is formed in fp64: a position of 10^9 steps is as exact as one of 10."""
    sections = (8, 8)
    freqs = sc.rotary_freqs(sections, device=DEV)
    x, _ = make(64, 2, 32, "f32", 2)
    rng = np.random.default_rng(3)
    pos = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31 - 1, (64, 2)).astype(np.int32)).to(DEV)
    note("rotary large positions")
    out = to_f64(sc.submconv_rotary(x, pos, freqs, sections))
    x64 = to_f64(x)
    # numpy's own fp64 product is off by half an ulp of 2^31, 2.4e-7 of a radian
    expect = ref.rotary(x64, pos.cpu().numpy(), freqs.cpu().numpy(), sections, False, False)
    assert np.abs(out - expect).max() <= (5e-7 + 16 * ref.U32) * 2 * np.abs(x64).max()


def test_rotary_integer_turn():
    """Hand-worked: freq pi/2 turns a pair by a quarter for every step."""
    x = torch.tensor([[[1.0, 2.0]]] * 4, device=DEV)
    pos = torch.tensor([[0], [1], [2], [3]], dtype=torch.int32, device=DEV)
    freqs = torch.tensor([np.pi / 2], dtype=torch.float32, device=DEV)
    note("rotary quarter turns")
    out = sc.submconv_rotary(x, pos, freqs, (1,)).cpu().numpy()[:, 0]
    assert np.allclose(out, [[1, 2], [-2, 1], [-1, -2], [2, -1]], atol=2e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("split", [False, True])
def test_rotary_views_in_place_and_inverse(dtype, split):
    """Queries and keys inside a packed projection, coordinate columns, odd offsets, head-major order."""
    n, h, d, sections = 211, 6, 48, (8, 8, 8)
    freqs = sc.rotary_freqs(sections, device=DEV)
    qkv, _ = make(n, 3 * h, d, dtype, 4)
    coords = torch.from_numpy(np.random.default_rng(5).integers(0, 100, (n, 4), dtype=np.int32)).to(DEV)
    note("rotary views %s split=%s" % (dtype, split))
    pos = coords[:, 1:]
    plain = sc.submconv_rotary(qkv[:, :2 * h].contiguous(), pos.contiguous(), freqs, sections, split=split)
    assert torch.equal(sc.submconv_rotary(qkv[:, :2 * h], pos, freqs, sections, split=split), plain)
    major = torch.empty((2 * h, n, d), dtype=qkv.dtype, device=DEV)
    sc.submconv_rotary(qkv[:, :2 * h], pos, freqs, sections, split=split, out=major.transpose(0, 1))
    assert torch.equal(major.transpose(0, 1), plain)
    odd = torch.zeros((n, 2 * h, d + 3), dtype=qkv.dtype, device=DEV)
    odd[:, :, 1:1 + d] = qkv[:, :2 * h]
    assert torch.equal(sc.submconv_rotary(odd[:, :, 1:1 + d], pos, freqs, sections, split=split), plain)
    values = qkv[:, 2 * h:].clone()
    before = qkv[:, :2 * h].clone()
    sc.submconv_rotary(qkv[:, :2 * h], pos, freqs, sections, split=split, out=qkv[:, :2 * h])
    assert torch.equal(qkv[:, :2 * h], plain) and torch.equal(qkv[:, 2 * h:], values)
    back = sc.submconv_rotary(plain, pos, freqs, sections, split=split, inverse=True)
    check(back, plain, pos, freqs, sections, dtype, inverse=True, split=split)
    top = float(before.float().abs().max())
    assert float((back.float() - before.float()).abs().max()) <= 4 * ref.UNIT[dtype] * top + 64 * ref.U32 * top


def test_rotary_gradient_against_differences():
    """The map is linear, so its gradient is exact in any step: <g, R x> = <R^T g, x>."""
    sections = (10, 10, 10)
    freqs = sc.rotary_freqs(sections, device=DEV)
    x, pos = make(57, 3, 64, "f32", 6)
    g, _ = make(57, 3, 64, "f32", 7)
    note("rotary differences")
    back = to_f64(sc.submconv_rotary(g, pos, freqs, sections, inverse=True))
    x64, g64 = to_f64(x), to_f64(g)
    rng = np.random.default_rng(8)
    f = lambda a: float((ref.rotary(a, pos.cpu().numpy(), freqs.cpu().numpy(), sections, False, False) * g64).sum())  # noqa: E731
    for _ in range(3):
        d = rng.standard_normal(x64.shape)
        slope = (f(x64 + 0.5 * d) - f(x64 - 0.5 * d))
        assert abs(slope - float((back * d).sum())) <= 32 * ref.U32 * float((np.abs(back) * np.abs(d)).sum())


def test_rotary_empty_and_offsets_past_32_bits():
    sections = (2, 2, 2)
    freqs = sc.rotary_freqs(sections, device=DEV)
    note("rotary empty")
    empty = torch.zeros((0, 4, 12), device=DEV)
    assert sc.submconv_rotary(empty, torch.zeros((0, 3), dtype=torch.int32, device=DEV), freqs, sections).shape == (0, 4, 12)
    note("rotary offsets past 32 bits")
    n, ld = 270001, 8192
    wide = torch.empty((n, ld), dtype=torch.bfloat16, device=DEV)
    x0, pos = make(n, 2, 12, "bf16", 9)
    x = wide[:, 100:124].view(n, 2, 12)
    x.copy_(x0)
    assert torch.equal(sc.submconv_rotary(x, pos, freqs, sections), sc.submconv_rotary(x0, pos, freqs, sections))
    del wide, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("split", [False, True])
def test_rotary_copies_what_does_not_turn(split):
    """Infinities and NaN in the pairs past the sections stay where they are and reach nothing else."""
    sections, n, h, d = (3, 2), 40, 2, 16                     # 5 of 8 pairs turn
    freqs = sc.rotary_freqs(sections, device=DEV)
    x, pos = make(n, h, d, "f32", 10, axes=2)
    plain = sc.submconv_rotary(x, pos, freqs, sections, split=split)
    at = 6 if split else 12                                   # the first element of pair 6
    x[:, :, at] = float("inf")
    x[3, 1, at] = float("nan")
    note("rotary copies split=%s" % split)
    out = sc.submconv_rotary(x, pos, freqs, sections, split=split)
    rest = [i for i in range(d) if i != at]
    assert torch.equal(out[..., rest], plain[..., rest])
    assert bool(torch.isnan(out[3, 1, at])) and int(torch.isinf(out[..., at]).sum()) == n * h - 1
