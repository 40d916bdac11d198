"""Grouped matrix products on the GPU against their definitions in 64 bits (bounds in experts_reference.py)."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import experts_reference as ex
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(rng, *shape, dtype="f32"):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV).to(TYPES[dtype])


def ints(v):
    return torch.as_tensor(v, dtype=torch.int32, device=DEV)


def within(got, expect, bound, what):
    err = np.abs(to_f64(got) - expect)
    assert not np.isnan(to_f64(got)).any() and (err <= bound).all(), "%s off by %.3e" % (what, (err - bound).max())


def check(x, w, b, offsets, rows, g, dtype):
    unit = ex.UNIT[dtype]
    out = sc.submconv_grouped_linear(x, w, offsets, bias=b, rows=rows)
    dx, dw, db = sc.submconv_grouped_linear_backward(g, x, w, offsets, rows=rows, need_bias=True)
    x64, w64, off = to_f64(x), to_f64(w), offsets.cpu().numpy()
    r = None if rows is None else rows.cpu().numpy()
    within(out, *ex.grouped_linear(x64, w64, None if b is None else to_f64(b), off, r, out.shape[0], unit), "out")
    expect, bound = ex.grouped_linear_backward(to_f64(g), x64, w64, off, r, unit)
    for got, e, d, what in zip((dx, dw, db), expect, bound, ("dx", "dweight", "dbias")):
        within(got, e, d, what)
    return out, dx, dw, db


def lengths(rng, groups, most, empty=True):
    n = rng.integers(0 if empty else 1, most + 1, groups)
    if empty and groups > 2:
        n[rng.integers(groups)] = 0
    return np.concatenate([[0], np.cumsum(n)])


@pytest.mark.parametrize("cin,cout", [(1, 1), (8, 8), (3, 130), (64, 32), (123, 7), (65, 129), (128, 256), (200, 264), (333, 517)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_linear(cin, cout, dtype):
    for groups, most in ((1, 1), (3, 5), (4, 200), (70, 20), (2, 700)):
        rng = np.random.default_rng([1, cin, cout, groups])
        off = lengths(rng, groups, most)
        many, nx = int(off[-1]), max(1, int(off[-1]) // 2)
        w, b = rand(rng, groups, cout, cin, dtype=dtype), rand(rng, groups, cout)
        g = rand(rng, many, cout, dtype=dtype)
        note("linear %d -> %d %s groups=%d n=%d" % (cin, cout, dtype, groups, many))
        check(rand(rng, many, cin, dtype=dtype), w, b, ints(off), None, g, dtype)
        check(rand(rng, nx, cin, dtype=dtype), w, None, ints(off), ints(rng.integers(0, nx, many)), g, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cin,cout,groups,most", [(256, 512, 3, 1500), (1024, 768, 2, 600), (768, 1024, 5, 300), (72, 2056, 2, 900),
                                                  (512, 256, 1, 4000)])
def test_grouped_linear_wide(dtype, cin, cout, groups, most):
    """Whole tiles and their ends, along every axis."""
    rng = np.random.default_rng([2, cin, cout])
    off = lengths(rng, groups, most, empty=False)
    many = int(off[-1])
    x = rand(rng, many, cin, dtype=dtype)
    rows = ints(rng.permutation(many))
    note("linear wide %d -> %d %s n=%d" % (cin, cout, dtype, many))
    check(x, rand(rng, groups, cout, cin, dtype=dtype), rand(rng, groups, cout), ints(off), rows, rand(rng, many, cout, dtype=dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cin,cout", [(64, 96), (1024, 512), (77, 130), (2048, 64)])
def test_grouped_linear_few_rows(dtype, cin, cout):
    """Single tokens: a row or a few for each of some groups."""
    for off in ([0, 1], [0, 1, 1, 2, 4], [0, 0, 0, 3], [0, 16, 17], [0, 2, 15, 33]):
        rng = np.random.default_rng([3, cin, len(off)])
        groups, many = len(off) - 1, off[-1]
        x = rand(rng, 3, cin, dtype=dtype)
        note("linear few rows %d -> %d %s %s" % (cin, cout, dtype, off))
        check(x, rand(rng, groups, cout, cin, dtype=dtype), rand(rng, groups, cout), ints(off), ints(rng.integers(0, 3, many)),
              rand(rng, many, cout, dtype=dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cin,cout", [(64, 128), (45, 51), (256, 256)])
def test_grouped_linear_bad_offsets_and_rows(dtype, cin, cout):
    """Descending, negative and far offsets, positions of no group and rows out of range: zeros, and nothing outside."""
    many, nx, groups = 700, 300, 6
    rng = np.random.default_rng([4, cin])
    w, b = rand(rng, groups, cout, cin, dtype=dtype), rand(rng, groups, cout)
    x, g = rand(rng, nx, cin, dtype=dtype), rand(rng, many, cout, dtype=dtype)
    rows = rng.integers(-50, nx + 50, many)
    rows[5], rows[6] = 2 ** 31 - 1, -2 ** 31
    for off in ([10, 100, 50, 50, 300, 200, 400], [-5, 100, 100, 100, 100, 650, 10 ** 6], [700] * 7, [0] * 7, [2 ** 31 - 1, 0, 0, 0, 0, 0, 0],
                [0, -2 ** 31, 5, 600, 400, 500, 690]):
        note("linear offsets %s %s %d -> %d" % (off, dtype, cin, cout))
        check(x, w, b, ints(off), ints(rows), g, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cin,cout", [(64, 128), (45, 51), (320, 264)])
def test_grouped_linear_keeps_groups_apart(dtype, cin, cout):
    """Infinities and NaN in one group's rows, weight, bias and gradient, and in rows of no group, reach no other group."""
    rng = np.random.default_rng([5, cin])
    off, many = [3, 60, 61, 400], 403
    x, w, b = rand(rng, many, cin, dtype=dtype), rand(rng, 3, cout, cin, dtype=dtype), rand(rng, 3, cout)
    g = rand(rng, many, cout, dtype=dtype)
    note("linear groups apart %s %d -> %d" % (dtype, cin, cout))
    out, dx, dw, db = check(x, w, b, ints(off), None, g, dtype)
    for t in (x, g):
        t[:3], t[60], t[400:] = float("nan"), float("inf"), float("nan")
    w[1], b[1] = float("nan"), float("-inf")
    out2 = sc.submconv_grouped_linear(x, w, ints(off), bias=b)
    dx2, dw2, db2 = sc.submconv_grouped_linear_backward(g, x, w, ints(off), need_bias=True)
    keep = [i for i in range(many) if i != 60]
    assert torch.equal(out2[keep], out[keep]) and torch.equal(dx2[keep], dx[keep])
    assert torch.equal(dw2[[0, 2]], dw[[0, 2]]) and torch.equal(db2[[0, 2]], db[[0, 2]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cin,cout", [(64, 128), (45, 51), (256, 512)])
def test_grouped_linear_strides_and_marks(dtype, cin, cout):
    """Rows inside wider tensors at odd places; memory beside the results stays as it was."""
    rng = np.random.default_rng([6, cin])
    off, many = ints([0, 130, 130, 300]), 300
    wide, grads = rand(rng, many, 2 * cin + 5, dtype=dtype), rand(rng, many, cout + 3, dtype=dtype)
    w, b = rand(rng, 3, cout, cin, dtype=dtype), rand(rng, 3, cout)
    for a in (0, 1, 3, 4, 8):
        x, g = wide[:, a:a + cin], grads[:, 3:]
        note("linear strided by %d %s %d -> %d" % (a, dtype, cin, cout))
        expect = sc.submconv_grouped_linear(x.contiguous(), w, off, bias=b)
        out = torch.full((many + 2, cout + 8), 7.0, dtype=x.dtype, device=DEV)
        sc.submconv_grouped_linear(x, w, off, bias=b, out=out[1:-1, a:a + cout])
        unit = ex.UNIT[dtype]
        e64, bound = ex.grouped_linear(to_f64(x), to_f64(w), to_f64(b), off.cpu().numpy(), None, many, unit)
        within(out[1:-1, a:a + cout], e64, bound, "strided out")
        within(expect, e64, bound, "out")
        marks = out.clone()
        marks[1:-1, a:a + cout] = 7.0
        assert bool((marks == 7.0).all())
        check(x, w, b, off, None, g, dtype)
    # one row for all positions
    x = wide[:1, :cin].expand(many, cin)
    check(x, w, b, off, None, grads[:, 3:].contiguous(), dtype)


def test_grouped_linear_exact_sums():
    """Small whole numbers are exact in every type and order, so any shift, loss or doubling of a term shows."""
    rng = np.random.default_rng(7)
    for dtype, cin, cout, off in (("bf16", 264, 520, [0, 300, 301, 777]), ("f32", 136, 250, [0, 5, 400]), ("bf16", 1000, 24, [0, 2, 3, 9])):
        groups, many = len(off) - 1, off[-1]
        f = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).to(DEV).to(TYPES[dtype])  # noqa: E731
        x, w, g = f(many, cin), f(groups, cout, cin), f(many, cout)
        note("linear exact %s" % dtype)
        out = sc.submconv_grouped_linear(x, w, ints(off))
        dx, dw, db = sc.submconv_grouped_linear_backward(g, x, w, ints(off), need_bias=True)
        top = 2 ** 8 if dtype == "bf16" else 2 ** 24   # whole numbers up to here are kept
        for got, (e, d) in zip((out, dx, dw, db), (ex.grouped_linear(to_f64(x), to_f64(w), None, off, None, many, 0.0),
                                                   *zip(*ex.grouped_linear_backward(to_f64(g), to_f64(x), to_f64(w), off, None, 0.0)))):
            small = np.abs(e) <= top
            assert small.mean() > 0.9 and (to_f64(got)[small] == e[small]).all()


def test_grouped_linear_empty():
    w, b = torch.ones((3, 20, 12), device=DEV), torch.ones((3, 20), device=DEV)
    off = ints([0, 0, 0, 0])
    x, g = torch.zeros((0, 12), device=DEV), torch.zeros((0, 20), device=DEV)
    note("linear empty")
    assert sc.submconv_grouped_linear(x, w, off, bias=b).shape == (0, 20)
    dx, dw, db = sc.submconv_grouped_linear_backward(g, x, w, off, need_bias=True)
    assert dx.shape == (0, 12) and bool((dw == 0).all()) and bool((db == 0).all())
    rows = ints([0, 5, -1])
    out = sc.submconv_grouped_linear(x, w, ints([0, 1, 2, 3]), bias=b, rows=rows)   # no row to take: the bias alone
    assert torch.equal(out, torch.ones((3, 20), device=DEV))


def test_grouped_linear_parts_of_the_gradient():
    rng = np.random.default_rng(8)
    x, w, g, off = rand(rng, 90, 24), rand(rng, 2, 40, 24), rand(rng, 90, 40), ints([0, 50, 90])
    note("linear parts")
    dx, dw, db = sc.submconv_grouped_linear_backward(g, x, w, off, need_bias=True)
    a = sc.submconv_grouped_linear_backward(g, x, w, off, need_weight=False)
    c = sc.submconv_grouped_linear_backward(g, x, w, off, need_x=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    assert c[0] is None and torch.equal(c[1], dw) and c[2] is None
    assert all(torch.equal(p, q) for p, q in zip(sc.submconv_grouped_linear_backward(g, x, w, off, need_bias=True), (dx, dw, db)))
    with pytest.raises(ValueError):
        sc.submconv_grouped_linear_backward(g, x, w, off, need_weight=False, need_bias=True)


@pytest.mark.parametrize("cin", [3, 64, 77])
def test_grouped_linear_rows_of_no_positions(cin):
    """The library's function with rows, but no positions: the weight's gradients are zeros and no row number is read."""
    import ctypes
    from submanifold_sparse_convolution_submconv3d_amd import load_library
    x, rows, off = torch.ones((4, cin), device=DEV), ints([0, 1]), ints([0, 0, 0])
    dw, db = torch.full((2, 5, cin), 7.0, device=DEV), torch.full((2, 5), 7.0, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    note("linear rows of no positions %d" % cin)
    code = load_library().submconv_grouped_linear_backward(
        None, 5, x.data_ptr(), cin, 4, rows.data_ptr(), None, off.data_ptr(), 2, 0, cin, 5, sc.F32, None, cin, dw.data_ptr(),
        ctypes.cast(db.data_ptr(), ctypes.c_void_p), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert code == 0 and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_linear_offsets_past_32_bits(dtype):
    """Rows that lie more than 2^32 elements into their tensors."""
    n, ld, cin, cout = 270001, 16384, 40, 48
    rng = np.random.default_rng(9)
    wide = torch.empty((n, ld), dtype=TYPES[dtype], device=DEV)
    x0 = rand(rng, n, cin, dtype=dtype)
    x = wide[:, 16000:16000 + cin]
    x.copy_(x0)
    w, off = rand(rng, 2, cout, cin, dtype=dtype), ints([0, 135000, n])
    note("linear offsets past 32 bits %s" % dtype)
    assert torch.equal(sc.submconv_grouped_linear(x, w, off), sc.submconv_grouped_linear(x0, w, off))
    g0 = rand(rng, n, cout, dtype=dtype)
    g = wide[:, 200:200 + cout]
    g.copy_(g0)
    for a, b in zip(sc.submconv_grouped_linear_backward(g, x, w, off, need_bias=True),
                    sc.submconv_grouped_linear_backward(g0, x0, w, off, need_bias=True)):
        assert torch.equal(a, b)
    del wide, x, g
    torch.cuda.empty_cache()
