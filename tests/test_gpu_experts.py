"""The operators with experts as a program uses them: in a HIP graph, on another stream, at once on two, refused
by the binding, and together in the example block against 64 bits."""
import os
import sys

import numpy as np
import pytest
import torch

import synth
import submanifold_sparse_convolution_submconv3d_amd as sc

from gpu_common import note

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_block  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16


def randn(*shape, dtype=F32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def inputs(dtype, n, cin=256, cout=320, experts=6, k=2, heads=6, dim=32):
    """Everything that `all_operators` takes; widths and rows reach each of the products' kernels by `n`."""
    pos = torch.from_numpy(np.random.default_rng(1).integers(0, 64, (n, 3), dtype=np.int32)).to(DEV)
    return dict(x=randn(n, heads, dim, dtype=dtype, seed=1), gx=randn(n, heads, dim, dtype=dtype, seed=2), w=1 + 0.2 * randn(heads, dim, seed=3),
                pos=pos, freqs=sc.rotary_freqs((5, 5, 5), device=DEV), logits=randn(n, experts, dtype=dtype, seed=4), gg=randn(n, k, seed=5),
                rows=randn(n, cin, dtype=dtype, seed=6), weight=randn(experts, cout, cin, dtype=dtype, seed=7), bias=randn(experts, cout, seed=8),
                gy=randn(n * k, cout, dtype=dtype, seed=9), go=randn(n, cout, dtype=dtype, seed=10), k=k)


def all_operators(x, gx, w, pos, freqs, logits, gg, rows, weight, bias, gy, go, k):
    turn = (w, pos, freqs, (5, 5, 5))
    y, rstd = sc.submconv_head_norm_rotary(x, *turn, return_rstd=True)
    out = [y, rstd, *sc.submconv_head_norm_rotary_backward(gx, x, rstd, *turn)]
    for normalize in (True, False):
        r = sc.submconv_route(logits, k, normalize=normalize)
        out += [*r, sc.submconv_route_backward(gg, logits, r.experts, r.gates, normalize=normalize)]
    u = sc.submconv_grouped_linear(rows, weight, r.offsets, bias=bias, rows=r.rows)
    out += [u, *sc.submconv_grouped_linear_backward(gy, rows, weight, r.offsets, rows=r.rows, need_bias=True)]
    return out + [sc.submconv_combine(u, r.slots, r.gates), *sc.submconv_combine_backward(go, u, r.slots, r.rows, r.gates),
                  sc.submconv_combine(out[-3], r.slots)]


SIZES = [(F32, 5), (F32, 700), (F32, 9000), (BF16, 5), (BF16, 700), (BF16, 30000)]


@pytest.mark.parametrize("dtype,n", SIZES)
def test_operators_in_a_graph(dtype, n):
    """No call synchronises or clears memory: a capture replays, and follows its inputs."""
    args = inputs(dtype, n)
    note("expert operators graph %s n=%d" % (dtype, n))
    all_operators(**args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_operators(**args)
    for rep in range(3):
        if rep:
            for i, name in enumerate(("x", "gx", "logits", "gg", "rows", "weight", "gy", "go")):
                t = args[name]
                t.copy_(randn(*t.shape, dtype=t.dtype, seed=100 * rep + i))
        eager = all_operators(**args)
        for t in captured:
            t.zero_()
        torch.cuda.synchronize()
        note("expert operators replay %d" % rep)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), "replay %d differs" % rep
    graph.reset()


def test_two_graphs():
    """Two captures of different sizes, replayed in turn and around eager calls, do not share anything."""
    first, second = inputs(BF16, 3000), inputs(BF16, 800)
    graphs, captured = [], []
    note("expert operators two graphs")
    for args in (first, second):
        all_operators(**args)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            captured.append(all_operators(**args))
    expect = [all_operators(**first), all_operators(**second)]
    for _ in range(2):
        for g in graphs:
            g.replay()
        all_operators(**inputs(F32, 500))
        for g in reversed(graphs):
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, expect):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    for g in graphs:
        g.reset()


@pytest.mark.parametrize("dtype,n", SIZES)
def test_operators_on_other_streams(dtype, n):
    """Behind slow work on a stream of its own, while the same calls run on another."""
    args, other = inputs(dtype, n), inputs(dtype, n + 13)
    expect, expect_other = all_operators(**args), all_operators(**other)
    torch.cuda.synchronize()
    note("expert operators on other streams %s n=%d" % (dtype, n))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(one):
        slow = randn(2000, 2000, seed=1)
        late = {k: torch.empty_like(args[k]) for k in ("x", "logits", "rows")}
        for _ in range(20):
            slow = slow @ slow * 1e-3
        for k, t in late.items():
            t.copy_(args[k] + 0 * slow[0, 0].to(t.dtype))     # ready only when the work before it is
        got = all_operators(**{**args, **late})
    with torch.cuda.stream(two):
        got_other = [all_operators(**other) for _ in range(3)][-1]
    one.synchronize()
    two.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, expect))
    assert all(torch.equal(a, b) for a, b in zip(got_other, expect_other))


def test_equal_calls_give_equal_bits():
    for dtype, n in SIZES:
        args = inputs(dtype, n)
        note("expert operators twice %s n=%d" % (dtype, n))
        for a, b in zip(all_operators(**args), all_operators(**args)):
            assert torch.equal(a, b)


def test_binding_refusals():
    h, x = randn(6, 4, 16), randn(6, 16)
    w, pos, freqs = randn(4, 16), torch.zeros((6, 3), dtype=torch.int32, device=DEV), randn(6)
    weight, off = randn(2, 8, 16), torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV)
    rows = torch.zeros(6, dtype=torch.int32, device=DEV)
    note("expert binding refusals")
    y, rstd = sc.submconv_head_norm_rotary(h, w, pos, freqs, (2, 2, 2), return_rstd=True)
    r = sc.submconv_route(x, 2)
    u = randn(12, 8)
    for error, call in (
            (ValueError, lambda: sc.submconv_head_norm_rotary(x)),
            (TypeError, lambda: sc.submconv_head_norm_rotary(h.half())),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, randn(3, 16))),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, randn(2, 16))),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, w, q_heads=2)),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, q_heads=2)),
            (sc.SubmconvError, lambda: sc.submconv_head_norm_rotary(h, randn(2, 16), q_heads=5)),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, randn(4, 15))),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, w, pos, freqs, (2, 2))),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, w, pos, None, (2, 2, 2))),
            (ValueError, lambda: sc.submconv_head_norm_rotary(h, w, pos, freqs, (2, 2, 1))),
            (sc.SubmconvError, lambda: sc.submconv_head_norm_rotary(h, w, pos, randn(9), (3, 3, 3))),
            (TypeError, lambda: sc.submconv_head_norm_rotary(h, w, pos.long(), freqs, (2, 2, 2))),
            (sc.SubmconvError, lambda: sc.submconv_head_norm_rotary(h, w, eps=-1.0)),
            (sc.SubmconvError, lambda: sc.submconv_head_norm_rotary(h, w, out=h[:1].expand(6, 4, 16))),
            (ValueError, lambda: sc.submconv_head_norm_rotary_backward(h[:5], h, rstd, w)),
            (ValueError, lambda: sc.submconv_head_norm_rotary_backward(h, h, rstd[:5], w)),
            (sc.SubmconvError, lambda: sc.submconv_head_norm_rotary_backward(h, y, rstd, w, dx=y)),
            (ValueError, lambda: sc.submconv_route(x[0], 2)),
            (TypeError, lambda: sc.submconv_route(x.long(), 2)),
            (sc.SubmconvError, lambda: sc.submconv_route(x, 0)),
            (sc.SubmconvError, lambda: sc.submconv_route(x, 17)),
            (sc.SubmconvError, lambda: sc.submconv_route(x, -1)),
            (sc.SubmconvError, lambda: sc.submconv_route(randn(4, 600), 2)),
            (ValueError, lambda: sc.submconv_route(x.t(), 2)),
            (ValueError, lambda: sc.submconv_route_backward(r.gates[:5], x, r.experts, r.gates)),
            (TypeError, lambda: sc.submconv_route_backward(r.gates, x, r.experts.long(), r.gates)),
            (ValueError, lambda: sc.submconv_grouped_linear(x, weight[0], off)),
            (ValueError, lambda: sc.submconv_grouped_linear(x, randn(2, 8, 15), off)),
            (TypeError, lambda: sc.submconv_grouped_linear(x, weight.to(BF16), off)),
            (ValueError, lambda: sc.submconv_grouped_linear(x, weight.transpose(1, 2).contiguous().transpose(1, 2), off)),
            (ValueError, lambda: sc.submconv_grouped_linear(x, weight, off[:2])),
            (TypeError, lambda: sc.submconv_grouped_linear(x, weight, off.long())),
            (ValueError, lambda: sc.submconv_grouped_linear(x, weight, off, bias=randn(8))),
            (TypeError, lambda: sc.submconv_grouped_linear(x, weight, off, bias=randn(2, 8).to(BF16))),
            (TypeError, lambda: sc.submconv_grouped_linear(x, weight, off, rows=rows.long())),
            (ValueError, lambda: sc.submconv_grouped_linear(x, weight, off, out=randn(5, 8))),
            (sc.SubmconvError, lambda: sc.submconv_grouped_linear(x, randn(2, 16, 16), off, out=x)),
            (ValueError, lambda: sc.submconv_grouped_linear_backward(randn(5, 8), x, weight, off)),
            (ValueError, lambda: sc.submconv_combine(u, r.slots[0], r.gates)),
            (ValueError, lambda: sc.submconv_combine(u, r.slots, r.gates[:5])),
            (TypeError, lambda: sc.submconv_combine(u, r.slots.long(), r.gates)),
            (sc.SubmconvError, lambda: sc.submconv_combine(u, torch.zeros((6, 17), dtype=torch.int32, device=DEV))),
            (sc.SubmconvError, lambda: sc.submconv_combine(u, r.slots, r.gates, out=u[:6])),
            (ValueError, lambda: sc.submconv_combine_backward(randn(6, 7), u, r.slots, r.rows, r.gates)),
            (ValueError, lambda: sc.submconv_combine_backward(randn(6, 8), u, r.slots, r.rows[:5], r.gates))):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("dtype,rel", [(F32, 4e-5), (BF16, 5e-2)])
def test_example_block(dtype, rel):
    """The example's forward and gradients against the same block in 64 bits with autograd, each row's experts taken
    as the example chose them.  fp32: a chain of some ten operators with sums of up to a thousand terms, 2^-24 * 600;
    bf16: some fifteen roundings of 2^-8 in a row, of which those of one sign add up and the others' squares."""
    res, batch, c, heads, experts, k, hidden = 16, 3, 64, 2, 5, 2, 96
    coords = synth.random_coords(600, res, batch, 3)
    coords = coords[np.lexsort(coords.T[::-1])]
    tc = torch.from_numpy(np.ascontiguousarray(coords)).to(DEV)
    n, d = len(coords), c // heads
    block = expert_block.ExpertBlock(c, heads, experts, k, hidden, dtype=dtype)
    for i, name in enumerate(("gamma1", "beta1", "gamma2", "beta2", "w_heads", "up_bias", "down_bias")):
        getattr(block, name).add_(0.1 * randn(*getattr(block, name).shape, seed=20 + i))
    x, grad = randn(n, c, dtype=dtype, seed=13), randn(n, c, dtype=dtype, seed=14)
    note("example with experts %s n=%d" % (dtype, n))
    out, saved = block.forward(tc, x, batch)
    grads = block.backward(grad, saved)
    chosen = saved[-4].experts.long().cpu()

    leaf = {name: getattr(block, name) for name in ("gamma1", "beta1", "gamma2", "beta2", "w_heads", "w_qkv", "w_out", "w_route", "up", "up_bias",
                                                    "down", "down_bias")}
    leaf = {k_: v.detach().double().cpu().requires_grad_(True) for k_, v in {"x": x, **leaf}.items()}
    angle = torch.zeros(n, d // 2, dtype=torch.float64)
    freqs, s = block.freqs.double().cpu(), block.sections[0]
    for a in range(3):
        angle[:, a * s:(a + 1) * s] = torch.from_numpy(coords[:, 1 + a:2 + a].astype(np.float64)) * freqs[a * s:(a + 1) * s]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    rotate = lambda t: torch.view_as_real(torch.view_as_complex(t.reshape(*t.shape[:-1], d // 2, 2).contiguous()) * turn).flatten(-2)  # noqa: E731
    qkv = (torch.nn.functional.layer_norm(leaf["x"], (c,), leaf["gamma1"], leaf["beta1"], block.eps) @ leaf["w_qkv"]).view(n, 3 * heads, d)
    qk = qkv[:, :2 * heads]
    qk = rotate(qk / torch.sqrt((qk * qk).mean(-1, keepdim=True) + block.eps) * leaf["w_heads"])
    same = torch.from_numpy(coords[:, 0][:, None] == coords[:, 0][None])
    scores = (torch.einsum("ihd,jhd->hij", qk[:, :heads], qk[:, heads:]) * d ** -0.5).masked_fill(~same, -float("inf"))
    att = torch.einsum("hij,jhd->ihd", scores.softmax(-1), qkv[:, 2 * heads:]).reshape(n, c)
    mid = leaf["x"] + att @ leaf["w_out"]
    n2 = torch.nn.functional.layer_norm(mid, (c,), leaf["gamma2"], leaf["beta2"], block.eps)
    gates = (n2 @ leaf["w_route"]).gather(1, chosen).softmax(-1)
    expect = mid
    for j in range(k):
        u = torch.einsum("nc,nhc->nh", n2, leaf["up"][chosen[:, j]]) + leaf["up_bias"][chosen[:, j]]
        y = torch.einsum("nh,nch->nc", torch.nn.functional.gelu(u), leaf["down"][chosen[:, j]]) + leaf["down_bias"][chosen[:, j]]
        expect = expect + gates[:, j:j + 1] * y
    expect.backward(grad.double().cpu())
    assert set(grads) == set(leaf)
    for name, got, want in [("out", out, expect.detach())] + [(m, grads[m], leaf[m].grad) for m in leaf]:
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= rel, "%s: relative error %.2e" % (name, err)


def test_example_runs():
    note("example with experts, as a program")
    expert_block.main()
