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
