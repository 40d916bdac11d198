"""Long calls of the operators with experts where a lost, doubled or misplaced row has to show: products of whole
numbers, whose sums are exact in every type and order; gradients of weights with and without the bias' in whole groups and
in pieces of groups, of more groups than a wave has lanes; and the walks of the routing's and the combination's gradients
past one turn of their blocks."""
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import experts_reference as ex
import whole_numbers
from gpu_common import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def exact(x, w, b, g, off, rows):
    """(out, dx, dw, db) in 64 bits; sums of whole numbers below 2^53 have no error."""
    n, groups = g.shape[0], w.shape[0]
    xr = x.double()
    if rows is not None:
        there = (rows >= 0) & (rows < x.shape[0])
        xr = xr[rows.long().clamp(0, x.shape[0] - 1)] * there[:, None]
    out, dx = torch.zeros((n, w.shape[1]), dtype=torch.float64, device=DEV), torch.zeros((n, w.shape[2]), dtype=torch.float64, device=DEV)
    dw, db = torch.zeros(w.shape, dtype=torch.float64, device=DEV), torch.zeros(b.shape, dtype=torch.float64, device=DEV)
    for i in range(groups):
        p = slice(off[i], off[i + 1])
        if off[i] == off[i + 1]:
            continue
        gg = g[p].double()
        out[p] = xr[p] @ w[i].double().t() + b[i].double()
        dx[p] = gg @ w[i].double()
        dw[i] = gg.t().contiguous() @ xr[p]
        db[i] = gg.sum(0)
    return out, dx, dw, db


@pytest.mark.parametrize("dtype,cin,cout,groups,n", whole_numbers.CASES)
@pytest.mark.parametrize("gather", [False, True])
def test_products_of_whole_numbers(dtype, cin, cout, groups, n, gather):
    """Every sum is a whole number below 2^24, exact in fp32 whatever the order; the one rounding to the type is torch's."""
    kind = TYPES[dtype]
    x, w, b, g, off, rows = (t.to(DEV) for t in whole_numbers.inputs(cin, cout, groups, n, gather))
    rows = rows if gather else None
    note("linear whole numbers %s %d -> %d groups=%d n=%d gather=%s" % (dtype, cin, cout, groups, n, gather))
    expect = exact(x, w, b, g, off.tolist(), rows)
    assert all(float(t.abs().max()) < 2 ** 24 for t in expect)
    x, w, g = x.to(kind), w.to(kind), g.to(kind)
    out = sc.submconv_grouped_linear(x, w, off, bias=b, rows=rows)
    assert torch.equal(out, expect[0].float().to(kind)), "out"
    for need_bias in (True, False):
        dx, dw, db = sc.submconv_grouped_linear_backward(g, x, w, off, rows=rows, need_bias=need_bias)
        assert torch.equal(dx, expect[1].float().to(kind)), "dx"
        assert torch.equal(dw, expect[2].float().to(kind)), "dweight, need_bias=%s" % need_bias
        assert db is None or torch.equal(db, expect[3].float()), "dbias"


@pytest.mark.parametrize("experts,n", [(512, 20000), (8, 1100003)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradients_of_more_rows_than_one_turn(experts, n, dtype, normalize):
    """4096 blocks of 256 / (experts / 8) rows a turn: 16,384 rows of 512 experts, 1,048,576 of 8.  Bounds of experts_reference.py."""
    k, kind, unit, u = 3, TYPES[dtype], ex.UNIT[dtype], ex.U32
    gen = torch.Generator(device="cuda").manual_seed(experts)
    x = torch.randn((n, experts), generator=gen, device="cuda").to(kind)
    grad = torch.randn((n, k), generator=gen, device="cuda")
    note("route gradients %d rows of %d experts %s normalize=%s" % (n, experts, dtype, normalize))
    r = sc.submconv_route(x, k, normalize=normalize)
    got = sc.submconv_route_backward(grad, x, r.experts, r.gates, normalize=normalize).double()
    x64, at, gates = x.double(), r.experts.long(), r.gates.double()
    top = x64.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(top, at)
    d = grad.double() * gates
    if normalize:
        p, rel = torch.zeros_like(x64).scatter_(1, at, gates), 2.0
    else:
        p, rel = x64.softmax(dim=1), experts + 12 + 2 * (x64.amax(dim=1, keepdim=True) - x64.amin(dim=1, keepdim=True))
    expect = (-p * d.sum(dim=1, keepdim=True)).scatter_add_(1, at, d)
    size = d.abs().sum(dim=1, keepdim=True)
    bound = p * (k + 6 + rel) * u * size
    bound += torch.zeros_like(p).scatter_(1, at, 6 * u * (d.abs() + size * p.gather(1, at))) + unit * expect.abs()
    assert bool(((got - expect).abs() <= bound).all())


@pytest.mark.parametrize("c", [64, 1000, 2056])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_combine_gradients_of_more_rows_than_one_turn(c, dtype):
    """8192 blocks of 32, 4 or 1 rows a turn, by the rows' width."""
    kind, unit, u, k = TYPES[dtype], ex.UNIT[dtype], ex.U32, 2
    v = 4 if dtype == "f32" else 8
    pieces = (c + v - 1) // v
    n = 8192 * (32 if pieces <= 8 else 4 if pieces <= 128 else 1) + 1001
    gen = torch.Generator(device="cuda").manual_seed(c)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    r = sc.submconv_route(rand(n, 5), k)
    y, g = rand(n * k, c).to(kind), rand(n, c).to(kind)
    note("combine gradients of %d rows of %d %s" % (n, c, dtype))
    dy, dgates = sc.submconv_combine_backward(g, y, r.slots, r.rows, r.gates)
    for j in range(k):
        at, f, g64 = r.slots[:, j].long(), r.gates[:, j:j + 1].double(), g.double()
        expect = f * g64
        assert bool(((dy[at].double() - expect).abs() <= (unit + 2 * k * u) * expect.abs()).all()), "dy"
        y64 = y[at].double()
        assert bool(((dgates[:, j].double() - (g64 * y64).sum(dim=1)).abs() <= (c + 8) * u * (g64 * y64).abs().sum(dim=1)).all()), "dgates"
