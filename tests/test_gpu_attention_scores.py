"""Ragged attention on scores whose size, not their difference, is large: what a query's sums are
scaled by when a maximum moves, in one pass, between the runs of a split and between the pieces of a cut tile.

Scores are exact here (one or two products of small whole numbers and a power of two times one), so
the only errors left are the roundings of the weights, their sums and the result."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import block_reference as ref
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
KEYS, STEP, DIM = 2560, 32, 32

# (heads, queries) for which the keys are not split, are split between blocks, and are not split but the
# last round of tiles is cut along them: by the number of tiles next to the blocks that run at once
# (768 in fp32 and 1024 in bf16 at this width)
PATHS = {("f32", "whole"): (600, 3), ("bf16", "whole"): (700, 3), ("f32", "split"): (4, 3), ("bf16", "split"): (4, 3),
         ("f32", "cut"): (900, 3), ("bf16", "cut"): (600, 130)}


@pytest.mark.parametrize("size", [1000.0, 79 * 2.0 ** 8, 23 * 2.0 ** 16, 99 * 2.0 ** 21, -119 * 2.0 ** 22, 101 * 2.0 ** 25])
@pytest.mark.parametrize("path", ["whole", "split", "cut"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_large_scores_beside_a_rising_row(dtype, path, size):
    """Query 0 sees the score `size` at every key, query 1 a maximum that moves in every tile of 32 keys, query
    2 both: `size` and a slow rise.  Queries of one wave share nothing but its instructions."""
    h, nq = PATHS[dtype, path]
    slope = max(0.25, 2.0 ** (np.floor(np.log2(abs(size))) - 23))   # size + slope t is exact in fp32
    tile = np.arange(KEYS) // STEP
    pattern = np.array([[size, 0.0], [0.0, 16.0], [size, slope]])
    q, k, v = np.zeros((nq, 1, DIM)), np.zeros((KEYS, 1, DIM)), np.zeros((KEYS, 1, DIM))
    q[:, 0, :2] = pattern[np.arange(nq) % 3]
    k[:, 0, 0], k[:, 0, 1] = 1.0, tile
    v[np.arange(KEYS), 0, tile * DIM // (KEYS // STEP)] = 1.0       # element d marks its part of the keys
    tq, tk, tv = (torch.from_numpy(t.astype(np.float32)).to(DEV).to(TYPES[dtype]) for t in (q, k, v))
    assert np.array_equal(to_f64(tq), q) and np.array_equal(to_f64(tk), k)
    note("attention scores of size %g %s %s" % (size, dtype, path))
    many = lambda t: t.expand(t.shape[0], h, DIM)  # noqa: E731
    off = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    out, lse = sc.submconv_attention(many(tq), many(tk), many(tv), off(nq), off(KEYS), scale=1.0, return_lse=True)
    out, lse = to_f64(out), lse.cpu().numpy().astype(np.float64)

    relative = np.array([[0.0, 0.0], [0.0, 16.0], [0.0, slope]]) @ np.stack([np.ones(KEYS), tile])   # scores less `size`
    w = np.exp(relative - relative.max(axis=1, keepdims=True))
    expect = (w / w.sum(axis=1, keepdims=True)) @ v[:, 0]
    low = ref.UNIT[dtype] if dtype == "bf16" else 0.0
    # sums over the keys twice (values and weights); weights to a few roundings, an exponent's relative error of
    # two (scale log2 e) at differences that matter (up to 100), the weights' and the result's own rounding
    tol = (2 * KEYS + 500) * ref.U32 + 2 * low
    for i in range(min(nq, 3)):
        gap = np.abs(out[i::3] - expect[i]) - tol * expect[i] - 1e-30
        assert gap.max() <= 0, "query %d: worst %.3e of %.3e" % (i, gap.max(), expect[i].max())
        true = (size if i != 1 else 0.0) + relative[i].max() + np.log(w[i].sum())
        assert np.abs(lse[i::3] - true).max() <= 8 * ref.U32 * abs(true) + (KEYS + 64) * ref.U32


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_scores_around_the_change_of_form(sign):
    """A maximum that passes the size (2^30 / log2 e) where weights change from one form to the other."""
    d, n = 32, 200
    edge = 2.0 ** 30 / np.log2(np.e)
    low = np.float32(sign * edge) - np.float32(128.0)
    high = low + np.float32(256.0)
    assert abs(float(low)) * np.log2(np.e) > 2.0 ** 30 > abs(float(high)) * np.log2(np.e) if sign < 0 else \
        abs(float(low)) * np.log2(np.e) < 2.0 ** 30 < abs(float(high)) * np.log2(np.e)
    v = torch.from_numpy(np.random.default_rng(1).standard_normal((n, 1, d)).astype(np.float32)).to(DEV)
    q, k = torch.zeros((33, 1, d), device=DEV), torch.zeros((n, 1, d), device=DEV)
    q[..., 0] = 1.0
    k[:64, 0, 0], k[64:, 0, 0] = float(low), float(high)
    note("attention scores around the change of form %+d" % sign)
    off = lambda m: torch.tensor([0, m], dtype=torch.int32, device=DEV)  # noqa: E731
    out = to_f64(sc.submconv_attention(q, k, v, off(33), off(n), scale=1.0))
    expect = to_f64(v)[64:].mean(axis=0)
    assert np.abs(out - expect).max() <= 4 * n * ref.U32 * np.abs(to_f64(v)).max()


def test_attention_largest_scale():
    """The largest scale that is taken, on products of its inverse's size."""
    d, n, scale = 32, 100, 1e38
    v = torch.from_numpy(np.random.default_rng(2).standard_normal((n, 1, d)).astype(np.float32)).to(DEV)
    q, k = torch.zeros((5, 1, d), device=DEV), torch.zeros((n, 1, d), device=DEV)
    q[..., 0] = 2.0 ** -63
    k[:40, 0, 0], k[40:, 0, 0] = 2.0 ** -63, 2.0 ** -62
    off = lambda m: torch.tensor([0, m], dtype=torch.int32, device=DEV)  # noqa: E731
    note("attention largest scale")
    out, _, bound, _ = ref.attention(to_f64(q), to_f64(k), to_f64(v), np.array([0, 5]), np.array([0, n]), float(np.float32(scale)), ref.U32)
    got = to_f64(sc.submconv_attention(q, k, v, off(5), off(n), scale=scale))
    assert (np.abs(got - out) <= bound).all()
