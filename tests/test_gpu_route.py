"""Routing, and the combination of experts' results, on the GPU against their definitions in 64 bits (bounds in
experts_reference.py).  Plans are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import experts_reference as ex
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def scores(n, e, dtype, seed, closed=0.0):
    rng = np.random.default_rng([seed, n, e])
    x = rng.standard_normal((n, e)).astype(np.float32)
    if closed:
        x[rng.random((n, e)) < closed] = -np.inf
        x[rng.random(n) < 0.1] = -np.inf
    return torch.from_numpy(x).to(DEV).to(TYPES[dtype])


def check_plan(r, logits, k, normalize):
    experts, gates, offsets, rows, slots, bound = ex.route(to_f64(logits), k, normalize)
    for name, got, expect in (("experts", r.experts, experts), ("offsets", r.offsets, offsets), ("rows", r.rows, rows), ("slots", r.slots, slots)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), expect), name
    err = np.abs(to_f64(r.gates) - gates)
    assert (err <= bound).all(), "gates off by %.3e" % (err - bound).max()


@pytest.mark.parametrize("experts,k", [(1, 1), (2, 1), (3, 3), (7, 2), (8, 2), (64, 8), (65, 5), (100, 16), (255, 4), (257, 3), (512, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_route(experts, k, dtype, normalize):
    for n, closed in ((1, 0.0), (2, 0.5), (300, 0.0), (301, 0.7)):
        x = scores(n, experts, dtype, 1, closed)
        note("route n=%d experts=%d k=%d %s normalize=%s closed=%s" % (n, experts, k, dtype, normalize, closed))
        r = sc.submconv_route(x, k, normalize=normalize)
        check_plan(r, x, k, normalize)
        g = torch.from_numpy(np.random.default_rng(n).standard_normal((n, k)).astype(np.float32)).to(DEV)
        d = sc.submconv_route_backward(g, x, r.experts, r.gates, normalize=normalize)
        expect, bound = ex.route_backward(to_f64(g), to_f64(x), r.experts.cpu().numpy(), to_f64(r.gates), normalize, ex.UNIT[dtype])
        err = np.abs(to_f64(d) - expect)
        assert (err <= bound).all(), "dlogits off by %.3e" % (err - bound).max()


@pytest.mark.parametrize("n,experts,k", [(30011, 16, 3), (9000, 200, 8), (70001, 2, 1)])
def test_route_many_blocks(n, experts, k):
    """The plan of many blocks, against a stable sort on the host."""
    x = scores(n, experts, "f32", 2, 0.3)
    note("route many blocks n=%d experts=%d k=%d" % (n, experts, k))
    r = sc.submconv_route(x, k)
    x64 = to_f64(x)
    order = np.argsort(-x64, axis=1, kind="stable")[:, :k]
    expect = np.where(np.take_along_axis(x64, order, axis=1) == -np.inf, -1, order)
    assert np.array_equal(r.experts.cpu().numpy(), expect)
    keys = np.where(expect < 0, experts, expect).reshape(-1)
    places = np.argsort(keys, kind="stable")
    assert np.array_equal(r.rows.cpu().numpy(), places // k)
    slots = np.empty(n * k, dtype=np.int64)
    slots[places] = np.arange(n * k)
    assert np.array_equal(r.slots.cpu().numpy().reshape(-1), slots)
    assert np.array_equal(r.offsets.cpu().numpy(), np.searchsorted(keys[places], np.arange(experts + 1)))
    again = sc.submconv_route(x, k)
    assert all(torch.equal(a, b) for a, b in zip(r, again))


def test_route_ties_and_signed_zeros():
    x = torch.zeros((5, 9), device=DEV)
    x[1] = torch.tensor([0.0, -0.0] * 4 + [0.0], device=DEV)
    x[2, 4:] = 1.0
    x[3] = -3.0e38
    x[4] = torch.tensor([-0.0] * 8 + [0.0], device=DEV)
    for dtype in ("f32", "bf16"):
        note("route ties %s" % dtype)
        r = sc.submconv_route(x.to(TYPES[dtype]), 3)
        assert r.experts.tolist() == [[0, 1, 2], [0, 1, 2], [4, 5, 6], [0, 1, 2], [0, 1, 2]]
        assert torch.allclose(r.gates, torch.full_like(r.gates, 1 / 3))


@pytest.mark.parametrize("normalize", [False, True])
def test_route_infinities_and_nan(normalize):
    """A NaN or +inf spoils its own row's gates, and nothing else; the plan stays a plan."""
    x = scores(200, 12, "f32", 3)
    x[5, 3], x[9, 1], x[11, :6] = float("nan"), float("inf"), float("inf")
    x[17, 2], x[17, 8] = -float("nan"), float("nan")
    note("route special scores")
    r = sc.submconv_route(x, 2, normalize=normalize)
    check_plan_rows = ex.route(to_f64(x), 2, normalize)
    for got, expect in ((r.experts, check_plan_rows[0]), (r.offsets, check_plan_rows[2]), (r.rows, check_plan_rows[3]), (r.slots, check_plan_rows[4])):
        assert np.array_equal(got.cpu().numpy(), expect)
    bad = torch.zeros(200, dtype=torch.bool, device=DEV)
    bad[[5, 9, 11, 17]] = True
    assert bool(torch.isnan(r.gates[bad]).all()) and bool(torch.isfinite(r.gates[~bad]).all())
    g = torch.ones((200, 2), device=DEV)
    d = sc.submconv_route_backward(g, x, r.experts, r.gates, normalize=normalize)
    assert bool(torch.isfinite(d[~bad]).all())


def test_route_large_scores():
    """Gates depend on differences alone: scores near the largest value neither overflow nor vanish."""
    x = torch.full((3, 4), -3.3e38, device=DEV)
    x[0], x[2, 1] = 3.3e38, 3.3e38
    note("route large scores")
    for normalize in (False, True):
        r = sc.submconv_route(x, 4, normalize=normalize)
        assert torch.equal(r.gates[0], torch.full((4,), 0.25, device=DEV)) and torch.equal(r.gates[1], r.gates[0])
        assert r.gates[2].tolist() == [1.0, 0.0, 0.0, 0.0] and r.experts[2].tolist() == [1, 0, 2, 3]


def test_route_strided_and_empty():
    wide = scores(300, 40, "bf16", 4)
    x = wide[:, 3:14]
    note("route strided")
    assert all(torch.equal(a, b) for a, b in zip(sc.submconv_route(x, 3), sc.submconv_route(x.contiguous(), 3)))
    r = sc.submconv_route(x, 3, normalize=False)
    g = torch.ones((300, 3), device=DEV)
    assert torch.equal(sc.submconv_route_backward(g, x, r.experts, r.gates, normalize=False),
                       sc.submconv_route_backward(g, x.contiguous(), r.experts, r.gates, normalize=False))
    note("route empty")
    r = sc.submconv_route(x[:0], 3)
    assert r.experts.shape == (0, 3) and r.rows.shape == (0,) and r.offsets.tolist() == [0] * 12
    assert sc.submconv_route_backward(g[:0], x[:0], r.experts, r.gates).shape == (0, 11)


def test_route_backward_of_foreign_numbers():
    """Numbers outside the experts stand for none; an expert named twice takes both."""
    x = scores(3, 5, "f32", 5)
    experts = torch.tensor([[1, 1], [-7, 4], [5, 2 ** 30]], dtype=torch.int32, device=DEV)
    gates = torch.tensor([[0.5, 0.25], [0.5, 0.5], [0.5, 0.5]], device=DEV)
    g = torch.tensor([[1.0, 2.0], [1.0, 3.0], [1.0, 1.0]], device=DEV)
    note("route backward foreign numbers")
    for normalize in (False, True):
        d = sc.submconv_route_backward(g, x, experts, gates, normalize=normalize)
        expect, bound = ex.route_backward(to_f64(g), to_f64(x), experts.cpu().numpy(), to_f64(gates), normalize, ex.U32)
        if normalize:  # d_j - gate_j sum(d) at each expert that is there
            expect[:] = 0
            expect[0, 1] = (0.5 - 0.5) + (0.5 - 0.25)
            expect[1, 4] = 1.5 - 0.5 * 2.0
            bound = np.full_like(expect, 8 * ex.U32)
        assert (np.abs(to_f64(d) - expect) <= bound).all()


# ----------------------------------------------------------------------------
# combination
# ----------------------------------------------------------------------------


def plan(n, k, e, seed):
    rng = np.random.default_rng([seed, n, k])
    return sc.submconv_route(torch.from_numpy(rng.standard_normal((n, e)).astype(np.float32)).to(DEV), k)


def rows_of(n, c, dtype, seed):
    return torch.from_numpy(np.random.default_rng([seed, n, c]).standard_normal((n, c)).astype(np.float32)).to(DEV).to(TYPES[dtype])


def check_combine(y, slots, rows, gates, g, dtype):
    unit = ex.UNIT[dtype]
    out = sc.submconv_combine(y, slots, gates)
    dy, dgates = sc.submconv_combine_backward(g, y, slots, rows, gates)
    y64, s, w = to_f64(y), slots.cpu().numpy(), None if gates is None else to_f64(gates)
    expect, bound = ex.combine(y64, s, w, unit)
    assert (np.abs(to_f64(out) - expect) <= bound).all(), "out"
    (edy, edg), (by, bg) = ex.combine_backward(to_f64(g), y64, s, rows.cpu().numpy(), w, unit)
    assert (np.abs(to_f64(dy) - edy) <= by).all(), "dy"
    if gates is None:
        assert dgates is None
    else:
        assert (np.abs(to_f64(dgates) - edg) <= bg).all(), "dgates"


@pytest.mark.parametrize("channels", [1, 5, 8, 33, 64, 250, 520, 1024, 2056, 4099])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_combine(channels, dtype):
    for n, k in ((1, 1), (3, 2), (40, 3), (70, 4), (33, 7), (20, 16)):
        r = plan(n, k, 17, 1)
        y, g = rows_of(n * k, channels, dtype, 2), rows_of(n, channels, dtype, 3)
        note("combine n=%d k=%d c=%d %s" % (n, k, channels, dtype))
        check_combine(y, r.slots, r.rows, r.gates, g, dtype)
        check_combine(y, r.slots, r.rows, None, g, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_combine_of_slots_that_are_no_plan(dtype):
    """Slots out of range add nothing, a place named twice in its row takes both gates, places that no row owns get zeros."""
    n, k, many, c = 50, 4, 130, 72
    rng = np.random.default_rng(6)
    slots = torch.from_numpy(rng.integers(-20, many + 20, (n, k)).astype(np.int32)).to(DEV)
    slots[3] = torch.tensor([7, 9, 7, 7], device=DEV)
    rows = torch.from_numpy(rng.integers(-5, n + 5, many).astype(np.int32)).to(DEV)
    for i in range(0, n, 2):  # some places are owned
        p = int(slots[i, 0])
        if 0 <= p < many:
            rows[p] = i
    rows[7] = 3
    y, g, gates = rows_of(many, c, dtype, 4), rows_of(n, c, dtype, 5), torch.from_numpy(rng.random((n, k)).astype(np.float32)).to(DEV)
    note("combine foreign slots %s" % dtype)
    check_combine(y, slots, rows, gates, g, dtype)
    check_combine(y, slots, rows, None, g, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_combine_strided_and_empty(dtype):
    n, k, c = 60, 2, 100
    r = plan(n, k, 5, 7)
    wide, g = rows_of(n * k, 2 * c + 7, dtype, 8), rows_of(n, c + 1, dtype, 9)
    y = wide[:, 5:5 + c]
    note("combine strided %s" % dtype)
    out = torch.zeros((n, c + 9), dtype=y.dtype, device=DEV)
    sc.submconv_combine(y, r.slots, r.gates, out=out[:, 3:3 + c])
    assert torch.equal(out[:, 3:3 + c], sc.submconv_combine(y.contiguous(), r.slots, r.gates))
    assert bool((out[:, :3] == 0).all()) and bool((out[:, 3 + c:] == 0).all())
    for a, b in zip(sc.submconv_combine_backward(g[:, 1:], y, r.slots, r.rows, r.gates),
                    sc.submconv_combine_backward(g[:, 1:].contiguous(), y.contiguous(), r.slots, r.rows, r.gates)):
        assert torch.equal(a, b)
    note("combine empty")
    none = r.slots[:0]
    assert sc.submconv_combine(y, none, r.gates[:0]).shape == (0, c)
    dy, dgates = sc.submconv_combine_backward(g[:0, 1:], y, none, torch.full_like(r.rows, -1), r.gates[:0])
    assert bool((dy == 0).all()) and dy.shape == (n * k, c) and dgates.shape == (0, k)
    dy, dgates = sc.submconv_combine_backward(g[:, 1:], y[:0], r.slots, r.rows[:0], r.gates)
    assert dy.shape == (0, c) and bool((dgates == 0).all())
    assert bool((sc.submconv_combine(y[:0], r.slots, r.gates) == 0).all())


def test_combine_offsets_past_32_bits():
    n, k, ld, c = 150000, 2, 8192, 24
    wide = torch.empty((n * k, ld), dtype=torch.bfloat16, device=DEV)
    y0 = rows_of(n * k, c, "bf16", 10)
    y = wide[:, 8000:8000 + c]
    y.copy_(y0)
    r = plan(n, k, 6, 11)
    g = rows_of(n, c, "bf16", 12)
    note("combine offsets past 32 bits")
    assert torch.equal(sc.submconv_combine(y, r.slots, r.gates), sc.submconv_combine(y0, r.slots, r.gates))
    for a, b in zip(sc.submconv_combine_backward(g, y, r.slots, r.rows, r.gates), sc.submconv_combine_backward(g, y0, r.slots, r.rows, r.gates)):
        assert torch.equal(a, b)
    del wide, y
    torch.cuda.empty_cache()
