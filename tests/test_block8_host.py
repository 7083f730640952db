"""8-bit blocks of 128 without a GPU: refusals of the C ABI come before any CUDA
call, and those of the torch front end."""

import os

import pytest
import torch
from torch.autograd import forward_ad

from reduce_scatter_gb300 import dg, layer, ops

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dg.LIB_PATH) or not os.path.exists(layer.EXT_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return layer.lib()


def _quantize(L, x=16, ld=64, xt=dg.TYPE_BF16, v=16, t=dg.TYPE_E4M3, s=16, br=1, rows=4, cols=64):
    return L.dg_layer_block8_quantize(x, ld, xt, v, t, s, 1, 4, br, 0, rows, cols, None)


def _values(L, v=16, t=dg.TYPE_E4M3, s=16, br=1, y=16, yt=dg.TYPE_BF16, rows=4, cols=64):
    return L.dg_layer_block8_dequantize(v, t, s, 1, 4, br, y, yt, rows, cols, None)


def _matmul(L, a=16, at=dg.TYPE_E4M3, sa=16, abr=1, ta=0, b=16, bt=dg.TYPE_E5M2, sb=16, bbr=128, tb=1, d=16, dt=dg.TYPE_BF16, m=4,
            n=64, k=64, ws=256, st=16):
    return L.dg_layer_block8_matmul(a, at, sa, 1, 1, abr, ta, b, bt, sb, 1, 1, bbr, tb, d, dt, m, n, k, ws, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), dg.ERR_ARG), (dict(rows=2**31), dg.ERR_ARG), (dict(cols=72), dg.ERR_SHAPE), (dict(t=dg.TYPE_BF16), dg.ERR_ARG),
    (dict(br=64), dg.ERR_ARG), (dict(x=None), dg.ERR_ARG), (dict(xt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(ld=60), dg.ERR_ARG),
    (dict(v=8), dg.ERR_ARG), (dict(s=None), dg.ERR_ARG), (dict(x=8), dg.ERR_ARG),
])
def test_quantize_refuses(L, kw, code):
    assert _quantize(L, **kw) == code and L.dg_layer_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), dg.ERR_ARG), (dict(cols=8), dg.ERR_SHAPE), (dict(t=dg.TYPE_F32), dg.ERR_ARG), (dict(yt=dg.TYPE_E4M3), dg.ERR_ARG),
    (dict(y=8), dg.ERR_ARG), (dict(v=None), dg.ERR_ARG), (dict(br=2), dg.ERR_ARG),
])
def test_values_refuse(L, kw, code):
    assert _values(L, **kw) == code and L.dg_layer_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), dg.ERR_ARG), (dict(k=2**31 - 255), dg.ERR_ARG), (dict(n=60), dg.ERR_SHAPE), (dict(k=72), dg.ERR_SHAPE),
    (dict(at=dg.TYPE_BF16), dg.ERR_ARG), (dict(dt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(abr=2), dg.ERR_ARG), (dict(ta=1), dg.ERR_ARG),
    (dict(tb=0, bbr=1), dg.ERR_ARG), (dict(ta=1, abr=128, m=24), dg.ERR_SHAPE), (dict(tb=0, n=72), dg.ERR_SHAPE),
    (dict(a=None), dg.ERR_ARG), (dict(sb=None), dg.ERR_ARG), (dict(d=None), dg.ERR_ARG), (dict(st=None), dg.ERR_ARG),
    (dict(ws=None), dg.ERR_ARG), (dict(ws=8), dg.ERR_ARG), (dict(b=8), dg.ERR_ARG), (dict(d=8), dg.ERR_ARG),
    (dict(m=2**31 - 256, n=2**31 - 256), dg.ERR_ARG),
])
def test_product_refuses(L, kw, code):
    assert _matmul(L, **kw) == code and L.dg_layer_last_error()


def test_nothing_to_do(L):
    assert _quantize(L, rows=0, x=None) == dg.OK and _quantize(L, cols=0, x=None) == dg.OK
    assert _values(L, rows=0, v=None) == dg.OK
    assert _matmul(L, m=0, a=None) == dg.OK and _matmul(L, n=0, b=None) == dg.OK


def _q(rows=4, cols=64, br=1, dtype=E4M3):
    return ops.Block8Tensor(torch.zeros(rows, cols).to(dtype), torch.ones(-(-rows // br), -(-cols // 128)), br)


def test_front_end_refuses(L):
    x = torch.ones(4, 64, dtype=BF16)
    for call, error in [
            (lambda: ops.quantize_block8(x.half()), TypeError), (lambda: ops.quantize_block8(x, dtype=BF16), ValueError),
            (lambda: ops.quantize_block8(x, block_rows=64), ValueError), (lambda: ops.quantize_block8(x, block_rows=1.5), TypeError),
            (lambda: ops.quantize_block8(torch.tensor(1.0)), ValueError), (lambda: ops.quantize_block8(x), ValueError),  # not CUDA
            (lambda: ops.dequantize_block8(x), TypeError), (lambda: ops.dequantize_block8(_q(), out_dtype=E4M3), ValueError),
            (lambda: ops.dequantize_block8(_q()._replace(block_rows=2)), ValueError),
            (lambda: ops.dequantize_block8(_q()._replace(scales=torch.ones(4, 2))), ValueError),
            (lambda: ops.dequantize_block8(_q()._replace(scales=torch.ones(4, 1, dtype=BF16))), ValueError),
            (lambda: ops.dequantize_block8(_q()._replace(values=x)), ValueError),
            (lambda: ops.dequantize_block8(_q(cols=72)), ValueError),
            (lambda: ops.dequantize_block8(_q()._replace(values=torch.zeros(64, 4).to(E4M3).t())), ValueError),
            (lambda: ops.block8_matmul(_q(), _q(cols=48)), ValueError), (lambda: ops.block8_matmul(_q(), x), TypeError),
            (lambda: ops.block8_matmul(_q(64, 64), _q(64, 64), trans_a=True), ValueError),
            (lambda: ops.block8_matmul(_q(64, 64), _q(64, 64), trans_b=False), ValueError)]:
        with pytest.raises(error):
            call()


def test_derivatives_are_refused(L):
    x = torch.ones(4, 64, dtype=BF16)
    with pytest.raises(ValueError, match="no gradient"):
        ops.quantize_block8(x.clone().requires_grad_())
    learned = _q()._replace(scales=torch.ones(4, 1, requires_grad=True))
    for call in (lambda: ops.block8_matmul(learned, _q()), lambda: ops.block8_matmul(_q(), learned), lambda: ops.dequantize_block8(learned)):
        with pytest.raises(ValueError, match="no gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="forward-mode"):
            ops.quantize_block8(dual)
        s = torch.ones(4, 1)
        with pytest.raises(ValueError, match="forward-mode"):
            ops.block8_matmul(_q()._replace(scales=forward_ad.make_dual(s, s)), _q())


# ---------------------------------------------------- layer norm, kept rows


def _norm(L, x=16, ld=64, xt=dg.TYPE_BF16, r=None, rt=0, w=16, wt=0, b=16, bt=0, y=16, yt=dg.TYPE_BF16, ys=None, s=None, kept=None,
          kt=dg.TYPE_E4M3, ks=None, rows=2, hidden=64, eps=1e-5):
    return L.dg_layer_layer_norm(x, ld, xt, r, ld, rt, w, wt, b, bt, y, yt, ys, 1, 2, s, ld, kept, kt, ks, 1, 2, None, None, rows, hidden,
                                 eps, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), dg.ERR_ARG), (dict(hidden=-1), dg.ERR_ARG), (dict(rows=2**31), dg.ERR_ARG), (dict(hidden=2**31 - 8), dg.ERR_ARG),
    (dict(xt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(r=16, s=16, rt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(wt=dg.TYPE_E4M3), dg.ERR_ARG),
    (dict(bt=dg.TYPE_E5M2), dg.ERR_ARG), (dict(yt=dg.TYPE_F32), dg.ERR_ARG), (dict(kept=16, kt=dg.TYPE_BF16, ks=16), dg.ERR_ARG),
    (dict(eps=-1.0), dg.ERR_ARG), (dict(eps=float("nan")), dg.ERR_ARG), (dict(x=None), dg.ERR_ARG), (dict(y=None), dg.ERR_ARG),
    (dict(r=16), dg.ERR_ARG), (dict(s=16), dg.ERR_ARG), (dict(yt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(kept=16), dg.ERR_ARG),
    (dict(yt=dg.TYPE_E4M3, ys=16, hidden=72), dg.ERR_SHAPE), (dict(kept=16, ks=16, hidden=40), dg.ERR_SHAPE),
])
def test_layer_norm_refuses(L, kw, code):
    assert _norm(L, **kw) == code and L.dg_layer_last_error()


def _norm_grad(L, dy=16, h=16, ht=dg.TYPE_BF16, hs=None, w=16, wt=0, mean=16, rstd=16, dh=None, dx=16, dw=16, db=16, bt=0, ws=256, rows=2,
               hidden=64):
    return L.dg_layer_layer_norm_backward(dy, 64, h, 64, ht, hs, 1, 2, w, wt, mean, rstd, dh, 64, dx, dw, db, bt, ws, rows, hidden, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), dg.ERR_ARG), (dict(hidden=2**31), dg.ERR_ARG), (dict(ht=99), dg.ERR_ARG), (dict(wt=dg.TYPE_E4M3), dg.ERR_ARG),
    (dict(bt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(ht=dg.TYPE_E4M3, hs=16, hidden=72), dg.ERR_SHAPE), (dict(ht=dg.TYPE_E4M3), dg.ERR_ARG),
    (dict(dy=None), dg.ERR_ARG), (dict(mean=None), dg.ERR_ARG), (dict(dx=None), dg.ERR_ARG), (dict(ws=None), dg.ERR_ARG),
    (dict(ws=8), dg.ERR_ARG), (dict(w=None, wt=dg.TYPE_E4M3), dg.ERR_ARG),
])
def test_layer_norm_gradient_refuses(L, kw, code):
    assert _norm_grad(L, **kw) == code and L.dg_layer_last_error()


def test_layer_norm_of_nothing(L):
    assert _norm(L, rows=0, x=None, y=None) == dg.OK and _norm(L, hidden=0, x=None, y=None) == dg.OK
    assert _norm_grad(L, hidden=0, dy=None) == dg.OK
    assert L.dg_layer_layer_norm_backward_workspace(0, 8) == 0
    assert L.dg_layer_layer_norm_backward_workspace(3, 8) == 2 * 3 * 8 * 4


def test_layer_norm_front_end_refuses(L):
    x, w = torch.ones(4, 64, dtype=BF16), torch.ones(64, dtype=BF16)
    rows = torch.ones(4)
    for call, error in [
            (lambda: ops.layer_norm(x.half()), TypeError), (lambda: ops.layer_norm(torch.tensor(1.0)), TypeError),
            (lambda: ops.layer_norm(x, w[:32]), ValueError), (lambda: ops.layer_norm(x, w.half()), TypeError),
            (lambda: ops.layer_norm(x, w, w.view(1, 64)), ValueError), (lambda: ops.layer_norm(x, residual=x[:2]), ValueError),
            (lambda: ops.layer_norm(x, residual=x.half()), TypeError), (lambda: ops.layer_norm(x, out_dtype=torch.float32), ValueError),
            (lambda: ops.layer_norm(x, keep_dtype=BF16), ValueError), (lambda: ops.layer_norm(x[:, :40], out_dtype=E4M3), ValueError),
            (lambda: ops.layer_norm(x, w, w), ValueError),  # not CUDA
            (lambda: ops.layer_norm(x.clone().requires_grad_(), out_dtype=E4M3), ValueError),
            (lambda: ops.layer_norm_backward(x.float(), x, w, rows, rows), TypeError),
            (lambda: ops.layer_norm_backward(x, x[:2], w, rows, rows), ValueError),
            (lambda: ops.layer_norm_backward(x, x, w, rows[:2], rows), ValueError),
            (lambda: ops.layer_norm_backward(x, x, w, rows, rows.half()), TypeError),
            (lambda: ops.layer_norm_backward(x, x, w, rows, rows, d_residual=x.float()), ValueError),
            (lambda: ops.layer_norm_backward(x, _q(br=128), w, rows, rows), ValueError),
            (lambda: ops.layer_norm_backward(x, _q(rows=3), w, rows, rows), ValueError),
            (lambda: ops.layer_norm_backward(x, x, w, rows, rows, bias_dtype=E4M3), ValueError),
            (lambda: ops.layer_norm_backward(x, x, w, rows, rows), ValueError)]:
        with pytest.raises(error):
            call()


def _kept_grad(L, d=16, ld=64, v=16, vt=dg.TYPE_E4M3, s=16, ends=16, e=2, out=16, dt=dg.TYPE_BF16, t=4, n=64, k=64, ws=256, pws=256,
               st=16):
    return L.dg_layer_grouped_weight_grad8(d, ld, v, vt, s, 1, 4, ends, e, out, 0, dt, t, n, k, ws, pws, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(t=-1), dg.ERR_ARG), (dict(e=0), dg.ERR_ARG), (dict(e=1025), dg.ERR_ARG), (dict(vt=dg.TYPE_BF16), dg.ERR_ARG),
    (dict(k=72), dg.ERR_SHAPE), (dict(n=60), dg.ERR_SHAPE), (dict(dt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(v=None), dg.ERR_ARG),
    (dict(s=None), dg.ERR_ARG), (dict(v=8), dg.ERR_ARG), (dict(ws=8), dg.ERR_ARG), (dict(ws=None), dg.ERR_ARG),
    (dict(d=None), dg.ERR_ARG), (dict(ends=None), dg.ERR_ARG), (dict(out=None), dg.ERR_ARG), (dict(st=None), dg.ERR_ARG),
    (dict(pws=None), dg.ERR_ARG), (dict(ld=60), dg.ERR_ARG),
])
def test_kept_gradient_refuses(L, kw, code):
    assert _kept_grad(L, **kw) == code and L.dg_layer_last_error()


def test_linear_refuses(L):
    x, w = torch.ones(4, 64, dtype=BF16), torch.ones(32, 64, dtype=BF16)
    for call, error in [(lambda: ops.block8_linear(x.float(), w), TypeError), (lambda: ops.block8_linear(x, w.float()), TypeError),
                        (lambda: ops.block8_linear(x, w[:, :32]), ValueError), (lambda: ops.block8_linear(x, w[:24]), ValueError),
                        (lambda: ops.block8_linear(x[:, :24], w[:, :24]), ValueError), (lambda: ops.block8_linear(x, w, dtype=BF16), ValueError),
                        (lambda: ops.block8_linear(x, w, grad_dtype=BF16), ValueError), (lambda: ops.block8_linear(x, w), ValueError),
                        (lambda: ops.grouped_matmul(x, w.view(2, 64, 16), torch.zeros(2, dtype=torch.int32), keep_dtype=BF16), ValueError)]:
        with pytest.raises(error):
            call()


def test_forward_mode_is_refused(L):
    x, w = torch.ones(4, 64, dtype=BF16), torch.ones(32, 64, dtype=BF16)
    rows = torch.ones(4)
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))

        for call in (lambda: ops.block8_linear(dual(x), w), lambda: ops.layer_norm(dual(x)),
                     lambda: ops.layer_norm(x, dual(w[0])), lambda: ops.layer_norm(x, w[0], dual(w[0])),
                     lambda: ops.layer_norm(x, residual=dual(x)), lambda: ops.layer_norm_backward(dual(x), x, None, rows, rows),
                     lambda: ops.layer_norm_backward(x, dual(x), None, rows, rows),
                     lambda: ops.layer_norm_backward(x, x, None, dual(rows), rows),
                     lambda: ops.layer_norm_backward(x, x, None, rows, rows, d_residual=dual(x))):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
