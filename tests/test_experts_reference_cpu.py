"""The 64-bit references of the operators with experts against differences of their forward parts and
hand-worked cases.  CPU only."""
import numpy as np
import pytest

import experts_reference as ex


def slope(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("many,q_heads", [(3, 0), (1, 0), (2, 2)])
def test_head_norm_gradient_against_differences(split, many, q_heads):
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((5, 3, 8)), rng.standard_normal((5, 3, 8))
    w = rng.standard_normal((many, 8)) + 1
    pos, freqs, sections = rng.integers(0, 9, (5, 3)), rng.random(3), (1, 1, 1)
    (dx, dw), _ = ex.head_norm_backward(g, x, w, q_heads, pos, freqs, sections, 1e-3, split, 0, 0)
    f = lambda a, b: float((ex.head_norm(a, b, q_heads, pos, freqs, sections, 1e-3, split, 0)[0] * g).sum())  # noqa: E731
    for _ in range(3):
        d, e = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        assert abs(slope(lambda a: f(a, w), x, d) - (dx * d).sum()) < 1e-6
        assert abs(slope(lambda b: f(x, b), w, e) - (dw * e).sum()) < 1e-6


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradient_against_differences(normalize):
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((6, 7)), rng.standard_normal((6, 3))
    x[1, 2] = x[3, :5] = -np.inf
    experts, gates = ex.route(x, 3, normalize)[:2]
    dx, _ = ex.route_backward(g, x, experts, gates, normalize, 0)
    f = lambda a: float((ex.route(a, 3, normalize)[1] * g).sum())  # noqa: E731
    for _ in range(3):
        d = rng.standard_normal(x.shape)
        assert abs(slope(f, x, d) - (dx * d).sum()) < 1e-6


def test_route_by_hand():
    inf = np.inf
    x = np.array([[1.0, 2.0, 2.0, 0.0], [-inf, -inf, 0.5, -inf], [-inf] * 4, [0.0, -0.0, 0.0, -1.0]])
    experts, gates, offsets, rows, slots, _ = ex.route(x, 2, True)
    assert experts.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 1]]
    assert np.allclose(gates, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]])
    assert offsets.tolist() == [0, 1, 3, 5, 5]
    assert rows.tolist() == [3, 0, 3, 0, 1, 1, 2, 2]
    assert slots.tolist() == [[1, 3], [4, 5], [6, 7], [0, 2]]


def test_products_and_combination_against_differences():
    rng = np.random.default_rng(3)
    x, w, b = rng.standard_normal((4, 5)), rng.standard_normal((3, 6, 5)), rng.standard_normal((3, 6))
    offsets, rows = [0, 3, 3, 7], np.array([3, 0, 1, 2, 2, 0, 1, 3])
    g = rng.standard_normal((8, 6))
    (dx, dw, db), _ = ex.grouped_linear_backward(g, x, w, offsets, rows, 0)
    f = lambda a, c, e: float((ex.grouped_linear(a, c, e, offsets, rows, 8, 0)[0] * g).sum())  # noqa: E731
    whole = np.zeros_like(x)
    np.add.at(whole, rows, dx)
    d, e, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), rng.standard_normal(b.shape)
    assert abs(slope(lambda a: f(a, w, b), x, d) - (whole * d).sum()) < 1e-6
    assert abs(slope(lambda a: f(x, a, b), w, e) - (dw * e).sum()) < 1e-6
    assert abs(slope(lambda a: f(x, w, a), b, h) - (db * h).sum()) < 1e-6
    y, slots, gates = rng.standard_normal((8, 5)), np.array([[1, 5], [2, 6], [3, 4], [0, 7]]), rng.random((4, 2))
    g = rng.standard_normal((4, 5))
    (dy, dgates), _ = ex.combine_backward(g, y, slots, rows, gates, 0)
    f = lambda a, c: float((ex.combine(a, slots, c, 0)[0] * g).sum())  # noqa: E731
    d, e = rng.standard_normal(y.shape), rng.standard_normal(gates.shape)
    assert abs(slope(lambda a: f(a, gates), y, d) - (dy * d).sum()) < 1e-6
    assert abs(slope(lambda a: f(y, a), gates, e) - (dgates * e).sum()) < 1e-6


def test_bad_offsets_count_as_the_largest_so_far():
    assert ex.bounds_of([-3, 5, 2, 90], 10).tolist() == [0, 5, 5, 10]
