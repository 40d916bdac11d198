"""Refusals of the heads' norm, the routing, the grouped products and the combination: every bad size, type,
pointer, distance or overlap comes back as a status before any HIP call.  CPU only; pointers are never read."""
import ctypes

import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

E_INVALID_ARG, E_UNSUPPORTED, E_ALIAS = -1, -4, -5
P = lambda i: ctypes.c_void_p(i << 36)  # noqa: E731  (addresses 64 GiB apart)
AT = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return sc.load_library()


def check(call, invalid=(), unsupported=(), alias=()):
    for code, cases in ((E_INVALID_ARG, invalid), (E_UNSUPPORTED, unsupported), (E_ALIAS, alias)):
        for bad in cases:
            assert call(**bad) == code, bad


def heads(lib, x=P(1), x_row=256, x_head=64, w=P(2), many=4, q_heads=0, pdtype=0, eps=1e-6, pos=P(3), pos_row=4, freqs=P(4),
          sections=(10, 10, 10), axes=3, n=10, heads=4, dim=64, dtype=0, split=0, out=P(5), out_row=256, out_head=64, rstd=P(6)):
    s = None if sections is None else (ctypes.c_int32 * max(1, len(sections)))(*sections)
    return lib.submconv_head_norm_rotary(x, x_row, x_head, w, many, q_heads, pdtype, eps, pos, pos_row, freqs, s, axes, n, heads, dim, dtype,
                                         split, out, out_row, out_head, rstd, None)


def test_head_norm_refusals(lib):
    assert heads(lib, n=0) == 0 and heads(lib, n=0, x=None, out=None) == 0
    check(lambda **k: heads(lib, **k),
          invalid=(dict(n=-1), dict(n=1 << 31), dict(x=None), dict(out=None), dict(pos=None), dict(freqs=None), dict(sections=None),
                   dict(split=2), dict(sections=(10, -1, 3)), dict(sections=(11, 11, 11)), dict(pos_row=-1), dict(x_row=-4),
                   dict(out_row=255), dict(out_head=63), dict(eps=-1.0), dict(eps=float("nan")), dict(many=2), dict(many=0), dict(many=5),
                   dict(q_heads=2), dict(q_heads=5, many=2), dict(q_heads=-1), dict(w=None), dict(w=None, many=2, q_heads=2),
                   dict(x=AT(0x1002)), dict(rstd=AT(0x1002)), dict(w=AT(0x1002))),
          unsupported=(dict(dim=63), dict(dim=0), dict(dim=514, x_head=514, out_head=514), dict(heads=0), dict(heads=1025), dict(axes=-1),
                       dict(axes=5, sections=(1,) * 5), dict(dtype=2), dict(pdtype=3)),
          alias=(dict(out=AT((1 << 36) + 16)), dict(out=P(1), out_row=512), dict(out=P(2)), dict(out=P(3)), dict(out=P(4)), dict(rstd=P(1)),
                 dict(rstd=P(5)), dict(rstd=P(2))))


def heads_bwd(lib, g=P(1), x=P(2), rstd=P(3), w=P(4), many=4, q_heads=0, pdtype=0, pos=P(5), pos_row=4, freqs=P(6), sections=(10, 10, 10), axes=3,
              strides=(256, 64) * 3, n=1000, heads=4, dim=64, dtype=1, split=0, dx=P(7), dw=P(8), ws=P(9), nbytes=1 << 30):
    s = None if sections is None else (ctypes.c_int32 * max(1, len(sections)))(*sections)
    st = None if strides is None else (ctypes.c_int64 * 6)(*strides)
    return lib.submconv_head_norm_rotary_backward(g, x, rstd, w, many, q_heads, pdtype, pos, pos_row, freqs, s, axes, st, n, heads, dim, dtype,
                                                  split, dx, dw, ws, nbytes, None)


def test_head_norm_backward_refusals(lib):
    need = lib.submconv_head_norm_rotary_backward_workspace(1000, 4, 64, 1, 4, 0)
    assert need > 0 and lib.submconv_head_norm_rotary_backward_workspace(1000, 4, 63, 1, 4, 0) == 0
    assert lib.submconv_head_norm_rotary_backward_workspace(1000, 4, 64, 1, 2, 0) == 0
    assert heads_bwd(lib, n=0, dw=None) == 0
    check(lambda **k: heads_bwd(lib, **k),
          invalid=(dict(n=-1), dict(g=None), dict(x=None), dict(rstd=None), dict(dx=None), dict(pos=None), dict(ws=None), dict(nbytes=need - 1),
                   dict(strides=None), dict(strides=(256, 64, 256, 64, 255, 64)), dict(strides=(-1, 64) + (256, 64) * 2), dict(many=3),
                   dict(ws=AT(0x1008)), dict(split=-1)),
          unsupported=(dict(dim=20000), dict(dtype=7), dict(pdtype=2)),
          alias=(dict(dx=P(2)), dict(dx=P(1), strides=(256, 64, 256, 64, 512, 64)), dict(dw=P(4)), dict(dw=P(7)), dict(ws=P(2)), dict(dx=P(3)),
                 dict(dx=P(5))))


def route(lib, logits=P(1), row=8, n=5000, experts=8, k=2, dtype=0, normalize=1, chosen=P(2), gates=P(3), offsets=P(4), rows=P(5), slots=P(6),
          ws=P(7), nbytes=1 << 30):
    return lib.submconv_route(logits, row, n, experts, k, dtype, normalize, chosen, gates, offsets, rows, slots, ws, nbytes, None)


def test_route_refusals(lib):
    need = lib.submconv_route_workspace(5000, 8, 2)
    assert need > 0 and lib.submconv_route_workspace(0, 8, 2) == 0 and lib.submconv_route_workspace(100, 8, 2) == 0 and lib.submconv_route_workspace(10, 8, 9) == 0
    check(lambda **k: route(lib, **k),
          invalid=(dict(n=-1), dict(n=1 << 30), dict(logits=None), dict(chosen=None), dict(gates=None), dict(offsets=None), dict(rows=None),
                   dict(slots=None), dict(ws=None), dict(nbytes=need - 1), dict(normalize=2), dict(row=-1), dict(row=(1 << 24) + 1),
                   dict(logits=AT(0x1002)), dict(rows=AT(0x1001)), dict(ws=AT(0x1004))),
          unsupported=(dict(experts=0), dict(experts=513), dict(k=0), dict(k=9), dict(k=17, experts=32), dict(dtype=2)),
          alias=(dict(gates=P(2)), dict(chosen=P(1)), dict(rows=P(6)), dict(offsets=P(3)), dict(ws=P(1))))


def route_bwd(lib, grad=P(1), logits=P(2), row=8, n=100, experts=8, k=2, dtype=0, normalize=0, chosen=P(3), gates=P(4), out=P(5), out_row=8):
    return lib.submconv_route_backward(grad, logits, row, n, experts, k, dtype, normalize, chosen, gates, out, out_row, None)


def test_route_backward_refusals(lib):
    assert route_bwd(lib, n=0) == 0
    check(lambda **k: route_bwd(lib, **k),
          invalid=(dict(n=-1), dict(grad=None), dict(logits=None), dict(chosen=None), dict(gates=None), dict(out=None), dict(out_row=7),
                   dict(normalize=-1), dict(out=AT(0x1002))),
          unsupported=(dict(k=0), dict(experts=600, out_row=600), dict(dtype=5)),
          alias=(dict(out=P(2)), dict(out=P(1)), dict(out=P(3)), dict(out=P(4))))


def linear(lib, x=P(1), x_row=64, nx=100, rows=P(2), w=P(3), bias=P(4), offsets=P(5), groups=4, n=200, cin=64, cout=32, dtype=1, out=P(6),
           out_row=32):
    return lib.submconv_grouped_linear(x, x_row, nx, rows, w, bias, offsets, groups, n, cin, cout, dtype, out, out_row, None)


def test_grouped_linear_refusals(lib):
    assert linear(lib, n=0) == 0
    check(lambda **k: linear(lib, **k),
          invalid=(dict(n=-1), dict(n=(1 << 31) - 1), dict(nx=-1), dict(nx=1 << 31), dict(x=None), dict(w=None), dict(offsets=None), dict(out=None),
                   dict(rows=None), dict(x_row=-1), dict(out_row=31), dict(groups=0), dict(groups=(1 << 16) + 1), dict(x=AT(0x1001)),
                   dict(bias=AT(0x1002)), dict(offsets=AT(0x1002))),
          unsupported=(dict(cin=0), dict(cin=(1 << 16) + 1), dict(cout=0, out_row=0), dict(dtype=2), dict(groups=1 << 16, cin=1 << 12, cout=1 << 12, out_row=1 << 12),
                       dict(n=1 << 30, cout=8192, out_row=8192)),
          alias=(dict(out=P(1)), dict(out=P(2)), dict(out=P(3)), dict(out=P(4)), dict(out=P(5))))


def linear_bwd(lib, g=P(1), g_row=32, x=P(2), x_row=64, nx=100, rows=P(3), w=P(4), offsets=P(5), groups=4, n=200, cin=64, cout=32, dtype=1,
               dx=P(6), dx_row=64, dw=P(7), db=P(8), ws=P(9), nbytes=1 << 34):
    return lib.submconv_grouped_linear_backward(g, g_row, x, x_row, nx, rows, w, offsets, groups, n, cin, cout, dtype, dx, dx_row, dw, db, ws,
                                                nbytes, None)


def test_grouped_linear_backward_refusals(lib):
    assert linear_bwd(lib, dx=None, dw=None, db=None) == 0
    need = lib.submconv_grouped_linear_backward_workspace(4, 200, 64, 32, 1)
    assert lib.submconv_grouped_linear_backward_workspace(0, 200, 64, 32, 1) == 0
    check(lambda **k: linear_bwd(lib, **k),
          invalid=(dict(n=-1), dict(g=None), dict(x=None), dict(w=None), dict(offsets=None), dict(rows=None), dict(dw=None), dict(dx_row=63),
                   dict(g_row=-1), dict(groups=0), dict(g=AT(0x1001)), dict(ws=AT(0x1008))) + ((dict(nbytes=need - 1), dict(ws=None)) if need else ()),
          unsupported=(dict(cin=0, dx_row=0), dict(dtype=3), dict(groups=1 << 16, cin=4096, cout=4096, dx_row=4096)),
          alias=(dict(dx=P(1)), dict(dx=P(4)), dict(dw=P(2)), dict(dw=P(6)), dict(db=P(7)), dict(dw=P(1)), dict(db=P(3)), dict(dx=P(5))))
    assert linear_bwd(lib, g=None, n=0, rows=P(3), x=None, dw=None, db=None) == 0


def combine(lib, y=P(1), y_row=64, np=200, slots=P(2), gates=P(3), n=100, k=2, c=64, dtype=0, out=P(4), out_row=64):
    return lib.submconv_combine(y, y_row, np, slots, gates, n, k, c, dtype, out, out_row, None)


def combine_bwd(lib, g=P(1), g_row=64, y=P(2), y_row=64, np=200, slots=P(3), rows=P(4), gates=P(5), n=100, k=2, c=64, dtype=0, dy=P(6), dy_row=64,
                dgates=P(7)):
    return lib.submconv_combine_backward(g, g_row, y, y_row, np, slots, rows, gates, n, k, c, dtype, dy, dy_row, dgates, None)


def test_combine_refusals(lib):
    assert combine(lib, n=0) == 0
    check(lambda **k: combine(lib, **k),
          invalid=(dict(n=-1), dict(np=-1), dict(np=1 << 31), dict(y=None), dict(slots=None), dict(out=None), dict(y_row=-1), dict(out_row=63),
                   dict(out=AT(0x1002)), dict(slots=AT(0x1002))),
          unsupported=(dict(k=0), dict(k=17), dict(c=0), dict(c=(1 << 16) + 1, out_row=1 << 17), dict(dtype=2)),
          alias=(dict(out=P(1)), dict(out=P(2)), dict(out=P(3))))
    assert combine_bwd(lib, dy=None, dgates=None) == 0 and combine_bwd(lib, n=0, np=0) == 0
    check(lambda **k: combine_bwd(lib, **k),
          invalid=(dict(n=-1), dict(g=None), dict(y=None), dict(slots=None), dict(rows=None), dict(g_row=-1), dict(dy_row=63), dict(dgates=AT(0x1002))),
          unsupported=(dict(k=0), dict(c=0, dy_row=0), dict(dtype=-1)),
          alias=(dict(dy=P(1)), dict(dy=P(2)), dict(dy=P(3)), dict(dy=P(4)), dict(dgates=P(5)), dict(dgates=P(6)), dict(dgates=P(2))))


def test_last_error_names_the_argument(lib):
    assert route(lib, k=17, experts=32) == E_UNSUPPORTED and b"k = 17" in lib.submconv_last_error()
    assert linear(lib, cin=0) == E_UNSUPPORTED and b"cin = 0" in lib.submconv_last_error()
    assert heads(lib, many=3) == E_INVALID_ARG and b"weight_rows = 3" in lib.submconv_last_error()
    assert combine(lib, out=P(1)) == E_ALIAS and b"out overlaps y" in lib.submconv_last_error() or b"y overlaps out" in lib.submconv_last_error()


def test_binding_refuses_host_tensors():
    x, h, i = torch.zeros((4, 8)), torch.zeros((4, 2, 8)), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sc.submconv_head_norm_rotary(h), lambda: sc.submconv_head_norm_rotary_backward(h, h, x),
                 lambda: sc.submconv_route(x, 2), lambda: sc.submconv_route_backward(x, x, i, x),
                 lambda: sc.submconv_grouped_linear(x, h, i), lambda: sc.submconv_grouped_linear_backward(x, x, h, i),
                 lambda: sc.submconv_combine(x, i), lambda: sc.submconv_combine_backward(x, x, i, i)):
        with pytest.raises((TypeError, ValueError)):
            call()
