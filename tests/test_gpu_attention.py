"""Ragged softmax attention and its gradients on the GPU against the 64-bit definition.

The bounds are worst cases of the kernels' roundings (block_reference.py): d products and
sums in a score, n additions in a sum over n keys, one rounding of each weight (and of each
weight's gradient) to bf16 where the tensors are bf16, and one rounding of the result."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

import block_reference as ref
from gpu_common import note, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def device_offsets(o):
    return torch.from_numpy(np.asarray(o, dtype=np.int32)).to(DEV)


def heads(n, h, d, dtype, rng, std=1.0):
    return torch.from_numpy((std * rng.standard_normal((n, h, d))).astype(np.float32)).to(DEV).to(TYPES[dtype])


def within(name, got, expect, bound):
    err = np.abs(to_f64(got) - expect)
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3e with bound %.3e" % (
        name, bad.sum(), bad.size, np.nanmax(np.where(bad, err, 0)), bound[bad][0])


def check(lq, lk, h, hk, d, dtype, seed=0, std=1.3, scale=None, backward=True):
    rng = np.random.default_rng([seed, sum(lq), h, d])
    qo = offsets(lq)
    ko = qo if lk is None else offsets(lk)
    q, k, v, g = (heads(n, m, d, dtype, rng, s) for n, m, s in ((qo[-1], h, std), (ko[-1], hk, std), (ko[-1], hk, 1.0), (qo[-1], h, 1.0)))
    scale = d ** -0.5 if scale is None else scale
    tq, tk = device_offsets(qo), device_offsets(ko)
    note("attention lq=%s lk=%s h=%d/%d d=%d %s" % (lq[:8], None if lk is None else lk[:8], h, hk, d, dtype))
    out, lse = sc.submconv_attention(q, k, v, tq, tk, scale=scale, return_lse=True)
    q64, k64, v64, g64 = (to_f64(t) for t in (q, k, v, g))
    expect, elos, bound, lse_err = ref.attention(q64, k64, v64, qo, ko, scale, ref.UNIT[dtype])
    within("out", out, expect, bound)
    got = lse.cpu().numpy().astype(np.float64)
    assert (np.isneginf(got) == np.isneginf(elos)).all()
    fine = np.isfinite(elos)
    assert (np.abs(got[fine] - elos[fine]) <= lse_err[fine]).all()
    assert torch.equal(sc.submconv_attention(q, k, v, tq, tk, scale=scale), out), "the same call gives the same bits"
    if not backward:
        return
    note("  backward")
    grads = sc.submconv_attention_backward(g, q, k, v, out, lse, tq, tk, scale=scale)
    expect, bounds = ref.attention_backward(g64, q64, k64, v64, qo, ko, scale, ref.UNIT[dtype])
    for name, a, b, c in zip(("dq", "dk", "dv"), grads, expect, bounds):
        within(name, a, b, c)
    again = sc.submconv_attention_backward(g, q, k, v, out, lse, tq, tk, scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(grads, again)), "the same call gives the same bits"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 64, 72, 88, 96, 104, 128])
def test_attention_head_widths(d, dtype):
    check([70, 1, 133], None, 2, 2, d, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 191, 257, 640])
def test_attention_lengths(n, dtype):
    check([n], None, 2, 1, 64, dtype)
    check([5], [n], 1, 1, 128, dtype)
    check([n], [7], 1, 1, 32, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("h,hk", [(1, 1), (3, 1), (6, 2), (8, 8), (12, 3), (20, 1)])
def test_attention_shared_heads(h, hk, dtype):
    check([45, 0, 150], [77, 13, 129], h, hk, 64, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_empty_rows(dtype):
    """Entries without keys, without queries, and without both, first, last and in between."""
    check([0, 40, 3, 0, 130, 0, 9], [5, 0, 200, 0, 0, 64, 0], 2, 2, 64, dtype)
    check([3, 4], [0, 0], 2, 1, 32, dtype)
    check([0, 0], [3, 70], 2, 1, 32, dtype)
    check([0], [0], 1, 1, 32, dtype)


@pytest.mark.parametrize("entries", [63, 64, 65, 200, 4500])
def test_attention_many_entries(entries):
    """More entries than one comparison of the tile lookup holds (64), and than two (4096)."""
    rng = np.random.default_rng(entries)
    check(list(rng.integers(0, 6, entries)), list(rng.integers(0, 9, entries)), 1, 1, 32, "f32", seed=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_few_queries_many_keys(dtype):
    """The keys of an entry are split between blocks and joined."""
    check([1], [20011], 2, 1, 64, dtype)
    check([1, 2, 0, 1], [9000, 21, 700, 15003], 4, 2, 128, dtype)
    check([3, 0, 5], [12000, 0, 0], 2, 2, 32, dtype)
    check([200], [8000], 1, 1, 96, dtype, backward=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_many_queries_few_keys(dtype):
    """The backward pass splits the queries between blocks for the keys' gradients."""
    check([20011], [3], 2, 1, 64, dtype)
    check([9000, 21, 0, 8003], [1, 5, 9, 140], 2, 2, 128, dtype)
    check([6000, 700], [0, 33], 3, 1, 32, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_sizes_of_scores(dtype):
    """Saturated, flat, far negative and very large scores."""
    check([100], [150], 2, 2, 64, dtype, std=6.0)
    check([100], [150], 2, 2, 64, dtype, scale=1e-6)
    check([65], [300], 1, 1, 32, dtype, scale=3.0)
    rng = np.random.default_rng(5)
    # every score near -400, and rising along the keys so that the running maximum moves in every tile
    q, k, v = (heads(n, 1, 32, dtype, rng) for n in (40, 500, 500))
    q[..., 0], k[..., 0] = 8.0, torch.linspace(-60, -40, 500, device=DEV)[:, None].to(k.dtype)
    qo, ko = offsets([40]), offsets([500])
    note("attention rising scores %s" % dtype)
    out, lse = sc.submconv_attention(q, k, v, device_offsets(qo), device_offsets(ko), scale=1.0, return_lse=True)
    expect, _, bound, _ = ref.attention(to_f64(q), to_f64(k), to_f64(v), qo, ko, 1.0, ref.UNIT[dtype])
    within("out", out, expect, bound)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_extreme_scores(dtype):
    """Scores of the type's lowest size weigh nothing beside others, all alike among themselves;
    scores of -inf weigh nothing at all, and a query that has no others gives zeros."""
    d, n = 32, 130
    v = heads(n, 1, d, dtype, np.random.default_rng(6))
    q = torch.zeros((33, 1, d), device=DEV).to(TYPES[dtype])
    q[..., 0] = 1.0
    k = torch.zeros((n, 1, d), device=DEV).to(TYPES[dtype])
    qo, ko = device_offsets([0, 33]), device_offsets([0, n])
    low = float(torch.finfo(TYPES[dtype]).min)
    tol = n * ref.U32 * 4 + ref.UNIT[dtype] * 4
    note("attention extreme scores %s" % dtype)
    k[:, 0, 0] = low
    out = to_f64(sc.submconv_attention(q, k, v, qo, ko, scale=1.0))
    assert np.abs(out - to_f64(v).mean(axis=0)).max() <= tol
    k[100:, 0, 0] = 1.0
    out = to_f64(sc.submconv_attention(q, k, v, qo, ko, scale=1.0))
    assert np.abs(out - to_f64(v)[100:].mean(axis=0)).max() <= tol
    k[:100, 0, 0] = -float("inf")
    out = to_f64(sc.submconv_attention(q, k, v, qo, ko, scale=1.0))
    assert np.abs(out - to_f64(v)[100:].mean(axis=0)).max() <= tol
    k[:, 0, 0] = -float("inf")
    out, lse = sc.submconv_attention(q, k, v, qo, ko, scale=1.0, return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("few", [False, True])
def test_attention_does_not_read_other_rows(dtype, few):
    """NaN and infinities in rows of other entries and outside every entry reach nothing."""
    rng = np.random.default_rng(7)
    lq, lk = ([2, 3], [9001, 8000]) if few else ([150, 33], [201, 70])
    h, hk, d = 2, 1, 64
    q, g = heads(sum(lq) + 9, h, d, dtype, rng), heads(sum(lq) + 9, h, d, dtype, rng)
    k, v = heads(sum(lk) + 11, hk, d, dtype, rng), heads(sum(lk) + 11, hk, d, dtype, rng)
    qo, ko = np.array([4, 4 + lq[0], 4 + sum(lq)]), np.array([6, 6 + lk[0], 6 + sum(lk)])
    for t, lo, hi in ((q, 4, 4 + lq[0]), (g, 4, 4 + lq[0]), (k, 6, 6 + lk[0]), (v, 6, 6 + lk[0])):
        t[:lo] = float("nan")
        t[hi:] = float("inf")
        t[-1] = float("nan")
    note("attention other rows %s few=%s" % (dtype, few))
    tq, tk = device_offsets(qo), device_offsets(ko)
    out, lse = sc.submconv_attention(q, k, v, tq, tk, return_lse=True)
    a, b = slice(4, 4 + lq[0]), slice(6, 6 + lk[0])
    args = [to_f64(t) for t in (q[a], k[b], v[b])]
    one_q, one_k = offsets(lq[:1]), offsets(lk[:1])
    expect, _, bound, _ = ref.attention(*args, one_q, one_k, d ** -0.5, ref.UNIT[dtype])
    within("out", out[a], expect, bound)
    assert bool((out[:4] == 0).all()) and bool((out[4 + sum(lq):] == 0).all()), "queries of no entry give zeros"
    assert bool(torch.isneginf(lse[:4]).all()) and bool(torch.isneginf(lse[4 + sum(lq):]).all())
    grads = sc.submconv_attention_backward(g, q, k, v, out, lse, tq, tk)
    expect, bounds = ref.attention_backward(to_f64(g[a]), *args, one_q, one_k, d ** -0.5, ref.UNIT[dtype])
    for name, x, at, e, w in zip(("dq", "dk", "dv"), grads, (a, b, b), expect, bounds):
        within(name, x[at], e, w)
    assert bool((grads[1][:6] == 0).all()) and bool((grads[2][6 + sum(lk):] == 0).all())
    assert bool((grads[0][:4] == 0).all()) and bool((grads[0][4 + sum(lq):] == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_views(dtype):
    """Parts of a packed projection, head-major tensors, odd element offsets, a shared (broadcast) value
    head, and gradients written into a packed tensor: the same bits as contiguous tensors."""
    rng = np.random.default_rng(8)
    n, h, d = 203, 4, 72
    qkv = heads(n, 3 * h, d, dtype, rng)
    q, k, v = qkv[:, :h], qkv[:, h:2 * h], qkv[:, 2 * h:]
    g = heads(n, h, d, dtype, rng)
    off = device_offsets([0, 80, 203])
    note("attention views %s" % dtype)
    qc, kc, vc = q.contiguous(), k.contiguous(), v.contiguous()
    plain, plse = sc.submconv_attention(qc, kc, vc, off, return_lse=True)
    out, lse = sc.submconv_attention(q, k, v, off, return_lse=True)
    assert torch.equal(out, plain) and torch.equal(lse, plse)
    odd = torch.zeros((n, h, d + 5), dtype=q.dtype, device=DEV)
    odd[..., 3:3 + d] = q
    major = kc.transpose(0, 1).contiguous().transpose(0, 1)
    held = torch.zeros((n, h, d + 1), dtype=q.dtype, device=DEV)
    assert torch.equal(sc.submconv_attention(odd[..., 3:3 + d], major, v, off, out=held[..., 1:]), plain)
    assert bool((held[..., 0] == 0).all())
    expect = sc.submconv_attention_backward(g, qc, kc, vc, plain, plse, off)
    packed = torch.zeros((n, 3 * h, d), dtype=q.dtype, device=DEV)
    sc.submconv_attention_backward(g, odd[..., 3:3 + d], major, v, held[..., 1:], lse, off,
                                   dq=packed[:, :h], dk=packed[:, h:2 * h], dv=packed[:, 2 * h:])
    assert all(torch.equal(packed[:, i * h:(i + 1) * h], expect[i]) for i in range(3))
    one = v[:, :1].expand(n, h, d)
    assert torch.equal(sc.submconv_attention(q, k, one, off), sc.submconv_attention(q, k, one.contiguous(), off))


def test_attention_offsets_past_32_bits():
    """Keys more than 2^32 bytes (and 2^31 elements) into the tensor."""
    n, ld, d = 270001, 8192, 32
    note("attention offsets past 32 bits")
    rng = np.random.default_rng(9)
    wide = torch.empty((n, ld), dtype=torch.bfloat16, device=DEV)
    k, v = wide[:, :d].unsqueeze(1), wide[:, d:2 * d].unsqueeze(1)
    k.copy_(heads(n, 1, d, "bf16", rng))
    v.copy_(heads(n, 1, d, "bf16", rng))
    q = heads(140, 2, d, "bf16", rng)
    qo, ko = device_offsets([0, 70, 140]), device_offsets([0, 1000, n])
    assert torch.equal(sc.submconv_attention(q, k, v, qo, ko), sc.submconv_attention(q, k.contiguous(), v.contiguous(), qo, ko))
    del wide, k, v
    torch.cuda.empty_cache()


def test_attention_offsets_outside_the_tensors():
    """Offsets are data on the device: values out of range or order are clamped there, so no call
    leaves the tensors.  Entries before the first bad one keep their results."""
    rng = np.random.default_rng(10)
    q, k, v = (heads(n, 1, 32, "f32", rng) for n in (64, 90, 90))
    good = sc.submconv_attention(q, k, v, device_offsets([0, 20, 64]), device_offsets([0, 30, 90]))
    note("attention clamped offsets")
    out = sc.submconv_attention(q, k, v, device_offsets([0, 20, 2000]), device_offsets([0, 30, 5000]))
    assert torch.equal(out, good)


@pytest.mark.parametrize("dtype", ["f32"])
@pytest.mark.parametrize("h,hk,d", [(2, 2, 32), (4, 1, 64)])
def test_attention_gradient_against_differences(h, hk, d, dtype):
    rng = np.random.default_rng([11, d])
    qo, ko = offsets([21, 0, 40]), offsets([33, 5, 17])
    q, k, v, g = (heads(n, m, d, dtype, rng) for n, m in ((61, h), (55, hk), (55, hk), (61, h)))
    tq, tk = device_offsets(qo), device_offsets(ko)
    note("attention differences h=%d/%d d=%d" % (h, hk, d))
    out, lse = sc.submconv_attention(q, k, v, tq, tk, return_lse=True)
    grads = [to_f64(t) for t in sc.submconv_attention_backward(g, q, k, v, out, lse, tq, tk)]
    args = [to_f64(t) for t in (q, k, v)]
    g64 = to_f64(g)
    loss = lambda a: float((ref.attention(*a, qo, ko, d ** -0.5, ref.U32)[0] * g64).sum())  # noqa: E731
    step = 1e-4
    for i in range(3):
        for _ in range(3):
            dirn = rng.standard_normal(args[i].shape)
            hi, lo = list(args), list(args)
            hi[i], lo[i] = args[i] + step * dirn, args[i] - step * dirn
            slope = (loss(hi) - loss(lo)) / (2 * step)
            # step^2 times a third derivative, and fp32 rounding of each gradient element
            assert abs(slope - float((grads[i] * dirn).sum())) <= 1e-4 * float(np.abs(grads[i] * dirn).sum()) + 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("h,hk,d,lens", [(13, 13, 32, [3900]), (14, 7, 64, [5003, 2000]), (8, 8, 128, [4200, 0, 3001])])
def test_attention_long_tiles(h, hk, d, lens, dtype):
    """Long entries, whose last round of tiles is cut into pieces and joined, against the same rows
    with hundreds of empty entries behind them (never cut), and 40 queries against 64 bits."""
    rng = np.random.default_rng([12, h, d])
    qo = offsets(lens)
    n = int(qo[-1])
    q, k, v, g = (heads(n, m, d, dtype, rng) for m in (h, hk, hk, h))
    t = device_offsets(qo)
    many = device_offsets(list(qo) + [n] * 300)
    note("attention long tiles h=%d/%d d=%d %s %s" % (h, hk, d, lens, dtype))
    out, lse = sc.submconv_attention(q, k, v, t, return_lse=True)
    grads = sc.submconv_attention_backward(g, q, k, v, out, lse, t)
    assert torch.equal(sc.submconv_attention(q, k, v, t), out)
    assert all(torch.equal(a, b) for a, b in zip(grads, sc.submconv_attention_backward(g, q, k, v, out, lse, t)))
    plain, plse = sc.submconv_attention(q, k, v, many, return_lse=True)
    pgrads = sc.submconv_attention_backward(g, q, k, v, plain, plse, many)
    # both sides are within max(lens) additions and a few roundings of the exact values
    tol = 4 * ref.UNIT[dtype] + 4 * max(lens) * ref.U32
    for name, a, b in (("out", out, plain), ("lse", lse, plse)) + tuple(zip(("dq", "dk", "dv"), grads, pgrads)):
        gap = float((a.float() - b.float()).abs().max())
        assert gap <= tol * float(b.float().abs().max()), "%s: %.3e apart" % (name, gap)
    pick = np.sort(rng.choice(n, 40, replace=False))
    for e in range(len(lens)):
        rows = pick[(pick >= qo[e]) & (pick < qo[e + 1])]
        if not len(rows):
            continue
        some, keys = [to_f64(x[rows]) for x in (q, g)], [to_f64(x[qo[e]:qo[e + 1]]) for x in (k, v)]
        one, all_ = np.array([0, len(rows)]), np.array([0, lens[e]])
        expect, _, bound, _ = ref.attention(some[0], *keys, one, all_, d ** -0.5, ref.UNIT[dtype])
        within("out", out[rows], expect, bound)
        expect, bounds = ref.attention_backward(some[1], some[0], *keys, one, all_, d ** -0.5, ref.UNIT[dtype])
        within("dq", grads[0][rows], expect[0], bounds[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_splits_among_many_entries(dtype):
    """Few rows on one side and more entries than lanes can count (254): the long side is split into runs
    numbered with gaps, also where one entry holds all of it."""
    none = [0] * 298
    check([2] + none + [1], [45011] + none + [0], 2, 1, 32, dtype)   # above 128 rows an entry on average
    check([1] + none + [2], [300] + none + [45001], 1, 1, 64, dtype)
    check([45011] + none + [0], [2] + none + [1], 2, 1, 32, dtype)
    check([2] + none[:200] + [1], [30000] + none[:200] + [5001], 2, 2, 32, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_splits_among_many_long_entries(dtype):
    """The same with more than 512 rows an entry on average, from where on bf16 is split too; and one entry on
    both sides of its limit of 768 rows."""
    none = [0] * 298
    check([2] + none + [1], [160011] + none + [0], 2, 1, 32, dtype)
    check([1] + none + [2], [300] + none + [160001], 1, 1, 64, dtype)
    check([160011] + none + [0], [2] + none + [1], 1, 1, 32, dtype)
    check([2] + none[:260] + [1], [130000] + none[:260] + [9001], 2, 2, 32, dtype)
    check([5], [767], 2, 1, 64, dtype)
    check([5], [768], 2, 1, 64, dtype)


def test_attention_heads_far_apart():
    """Query heads of a group more than 2^30 bytes apart (head-major memory of a very large set): the
    same bits as next to each other."""
    n, d, far = 150, 32, (1 << 28) + 64
    rng = np.random.default_rng(13)
    note("attention heads far apart")
    memory = torch.empty(2 * far, dtype=torch.bfloat16, device=DEV)
    q = memory.as_strided((n, 2, d), (d, far, 1))
    q.copy_(heads(n, 2, d, "bf16", rng))
    k, v, g = heads(n, 1, d, "bf16", rng), heads(n, 1, d, "bf16", rng), heads(n, 2, d, "bf16", rng)
    off = device_offsets([0, 60, n])
    near = q.contiguous()
    out, lse = sc.submconv_attention(q, k, v, off, return_lse=True)
    expect, elos = sc.submconv_attention(near, k, v, off, return_lse=True)
    assert torch.equal(out, expect) and torch.equal(lse, elos)
    got, want = sc.submconv_attention_backward(g, q, k, v, out, lse, off), sc.submconv_attention_backward(g, near, k, v, out, lse, off)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del memory, q
    torch.cuda.empty_cache()
