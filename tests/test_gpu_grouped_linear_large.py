"""Grouped matrix products of sizes that take the kernels for long calls, against their definitions in 64 bits on the
GPU (bounds as in experts_reference.py): ends inside tiles on every axis, empty groups, positions of no group, rows out of
range, more groups than a wave has lanes, whole groups and pieces of groups."""
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import experts_reference as ex
from gpu_common import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def within(got, expect, bound, what):
    over = (got.double() - expect).abs() - bound
    assert not bool(torch.isnan(over).any()) and float(over.max()) <= 0, "%s off by %.3e" % (what, float(over.max()))


def plan(groups, n, nx, seed):
    g = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(5, n - 7, (groups + 1,), generator=g)).values
    cuts[0], cuts[-1] = 5, n - 7
    cuts[groups // 2 + 1] = cuts[groups // 2] if groups > 1 else cuts[groups // 2 + 1]   # an empty group
    rows = torch.randint(-3, nx + 3, (n,), generator=g)
    return cuts.to(DEV, torch.int32), rows.to(DEV, torch.int32)


CASES = [("bf16", 200, 2056, 3, 9001), ("bf16", 2056, 200, 3, 9001), ("bf16", 72, 2048, 2, 8300), ("bf16", 128, 1024, 70, 17000),
         ("bf16", 1024, 1024, 16, 3000), ("bf16", 512, 512, 70, 9000), ("bf16", 264, 520, 2, 40000), ("bf16", 1000, 200, 5, 12345),
         ("f32", 264, 516, 3, 9000), ("f32", 516, 264, 3, 9000), ("f32", 300, 520, 2, 14000), ("f32", 512, 512, 20, 9000),
         ("f32", 132, 1028, 70, 8000), ("bf16", 257, 1023, 3, 11000), ("bf16", 515, 1023, 3, 9000), ("f32", 257, 1023, 3, 11000),
         ("f32", 515, 1023, 3, 9000), ("bf16", 200, 2056, 3, 20001), ("bf16", 2056, 200, 3, 20001), ("bf16", 264, 520, 2, 60000),
         ("bf16", 512, 512, 70, 31000), ("bf16", 1024, 1024, 16, 8000), ("bf16", 136, 520, 70, 9000), ("bf16", 520, 136, 5, 40000),
         ("f32", 3, 517, 3, 90000), ("bf16", 515, 5, 3, 90000)]


@pytest.mark.parametrize("dtype,cin,cout,groups,n", CASES)
@pytest.mark.parametrize("gather", [False, True])
def test_long_calls(dtype, cin, cout, groups, n, gather):
    kind, unit, u = TYPES[dtype], ex.UNIT[dtype], ex.U32
    gen = torch.Generator(device="cuda").manual_seed(cin + cout)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    nx = n // 2 if gather else n
    off, rows = plan(groups, n, nx, 1)
    x, w, b, g = rand(nx, cin).to(kind), rand(groups, cout, cin).to(kind), rand(groups, cout), rand(n, cout).to(kind)
    rows = rows if gather else None
    note("linear long %s %d -> %d groups=%d n=%d gather=%s" % (dtype, cin, cout, groups, n, gather))
    out = sc.submconv_grouped_linear(x, w, off, bias=b, rows=rows)
    dx, dw, db = sc.submconv_grouped_linear_backward(g, x, w, off, rows=rows, need_bias=True)
    xr = x.double()
    if gather:
        there = (rows >= 0) & (rows < nx)
        xr = xr[rows.long().clamp(0, nx - 1)] * there[:, None]
    ends = off.tolist()
    outside = torch.ones(n, dtype=torch.bool, device=DEV)
    outside[ends[0]:ends[-1]] = False
    assert bool((out[outside] == 0).all()) and bool((dx[outside] == 0).all())
    for i in range(groups):
        p = slice(ends[i], ends[i + 1])
        many = ends[i + 1] - ends[i]
        a, m, gg, bb = xr[p], w[i].double(), g[p].double(), b[i].double()
        y = a @ m.t() + bb
        within(out[p], y, unit * y.abs() + (cin + 8) * u * (a.abs() @ m.abs().t() + bb.abs()), "out of group %d" % i) if many else None
        y = gg @ m
        within(dx[p], y, unit * y.abs() + (cout + 8) * u * (gg.abs() @ m.abs()), "dx of group %d" % i) if many else None
        y = gg.t() @ a
        within(dw[i], y, unit * y.abs() + (many + 8) * u * (gg.abs().t() @ a.abs()), "dweight of group %d" % i)
        y = gg.sum(0)
        within(db[i], y, u * y.abs() + (many + 8) * u * gg.abs().sum(0), "dbias of group %d" % i)


@pytest.mark.parametrize("dtype,cin,cout,groups,n", [("bf16", 256, 2048, 4, 9000), ("bf16", 512, 512, 3, 12000), ("f32", 256, 520, 4, 9000),
                                                     ("f32", 512, 512, 3, 9000)])
def test_groups_stay_apart(dtype, cin, cout, groups, n):
    """Infinities and NaN in one group's rows, weight, bias and gradient, and in rows of no group, reach no other group."""
    kind = TYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w, b, g = rand(n, cin).to(kind), rand(groups, cout, cin).to(kind), rand(groups, cout), rand(n, cout).to(kind)
    ends = [3, 1001, 1002] + [n - 5] * (groups - 2)
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    note("linear long, groups apart %s %d -> %d" % (dtype, cin, cout))
    out = sc.submconv_grouped_linear(x, w, off, bias=b)
    grads = sc.submconv_grouped_linear_backward(g, x, w, off, need_bias=True)
    for t in (x, g):
        t[:3], t[1001], t[n - 5:] = float("nan"), float("inf"), float("nan")
    w[1], b[1] = float("nan"), float("-inf")
    out2 = sc.submconv_grouped_linear(x, w, off, bias=b)
    grads2 = sc.submconv_grouped_linear_backward(g, x, w, off, need_bias=True)
    keep = [i for i in range(n) if i != 1001]
    others = [i for i in range(groups) if i != 1]
    assert torch.equal(out2[keep], out[keep]) and torch.equal(grads2[0][keep], grads[0][keep])
    for a, c in zip(grads2[1:], grads[1:]):
        assert torch.equal(a[others], c[others])


@pytest.mark.parametrize("dtype,cin,cout", [("bf16", 128, 2048), ("f32", 128, 520)])
def test_long_calls_keep_to_their_memory(dtype, cin, cout):
    """Results inside wider tensors: what lies beside them stays as it was, also at ends inside tiles."""
    kind, n = TYPES[dtype], 9003
    gen = torch.Generator(device="cuda").manual_seed(8)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(kind)  # noqa: E731
    wide, w = rand(n, 2 * cin), rand(3, cout, cin)
    off = torch.tensor([0, 4000, 4001, n - 2], dtype=torch.int32, device=DEV)
    note("linear long, marks %s" % dtype)
    x = wide[:, 8:8 + cin]
    expect = sc.submconv_grouped_linear(x.contiguous(), w, off)
    out = torch.full((n + 2, cout + 16), 7.0, dtype=kind, device=DEV)
    sc.submconv_grouped_linear(x, w, off, out=out[1:-1, 8:8 + cout])
    assert torch.equal(out[1:-1, 8:8 + cout], expect)
    out[1:-1, 8:8 + cout] = 7.0
    assert bool((out == 7.0).all())
