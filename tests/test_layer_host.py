"""The operators of reduce_scatter_gb300.layer without a GPU: every declared
symbol is exported, argument errors come before any CUDA call, sizes of
workspaces and scale layouts, and the refusals of the torch front end."""

import os
import re

import pytest
import torch

from reduce_scatter_gb300 import dg, layer, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dg.LIB_PATH) or not os.path.exists(layer.EXT_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return layer.lib()


def test_every_declared_symbol_is_exported(L):
    with open(os.path.join(ROOT, "include", "dg_layer.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(dg_layer_[a-z_0-9]+)\s*\(", src))
    assert names == set(layer.EXPORTS)
    for name in names:
        assert hasattr(L, name), name


def _norm(L, x=16, ldx=8, res=None, rt=0, w=16, wt=0, y=16, yt=0, s=None, sc=None, sin=None, rows=2, hidden=8, eps=1e-5):
    return L.dg_layer_add_rms_norm(x, ldx, res, ldx, rt, w, wt, y, yt, s, ldx, sc, sin, None, rows, hidden, eps, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(hidden=-8), dict(yt=dg.TYPE_F32), dict(wt=dg.TYPE_E4M3), dict(eps=-1.0), dict(x=None),
    dict(w=None), dict(y=None), dict(res=16), dict(s=16), dict(yt=dg.TYPE_E4M3), dict(eps=float("nan")),
    dict(res=16, s=16, rt=dg.TYPE_E5M2), dict(rows=2**31),
])
def test_norm_refuses(L, kw):
    assert _norm(L, **kw) == dg.ERR_ARG and L.dg_layer_last_error()


def test_norm_of_nothing(L):
    assert _norm(L, rows=0, x=None, y=None, w=None) == dg.OK
    assert _norm(L, hidden=0, x=None, y=None, w=None) == dg.OK
    assert L.dg_layer_add_rms_norm_backward_workspace(0, 8) == 0
    assert L.dg_layer_add_rms_norm_backward_workspace(3, 8) == 3 * 8 * 4


def _grouped(L, a=16, lda=64, at=0, b=16, ldb=64, lde=64 * 64, bt=0, nm=0, ends=16, e=2, d=16, dt=0, t=4, n=64, k=64,
             ws=256, st=16):
    return L.dg_layer_grouped_matmul(a, lda, at, b, ldb, lde, bt, nm, ends, e, None, 0, None, 0, 0, d, dt, t, n, k,
                                     ws, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(t=-1), dg.ERR_ARG), (dict(e=0), dg.ERR_ARG), (dict(e=1025), dg.ERR_ARG), (dict(bt=dg.TYPE_E4M3), dg.ERR_ARG),
    (dict(at=dg.TYPE_F32, bt=dg.TYPE_F32), dg.ERR_ARG), (dict(dt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(n=60), dg.ERR_SHAPE),
    (dict(k=60), dg.ERR_SHAPE), (dict(k=72, at=dg.TYPE_E4M3, bt=dg.TYPE_E4M3), dg.ERR_SHAPE),
    (dict(nm=1, at=dg.TYPE_E4M3, bt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(a=8), dg.ERR_ARG), (dict(b=None), dg.ERR_ARG),
    (dict(d=None), dg.ERR_ARG), (dict(lda=68), dg.ERR_ARG), (dict(lda=56), dg.ERR_ARG), (dict(lde=0), dg.ERR_ARG),
    (dict(ends=None), dg.ERR_ARG), (dict(st=None), dg.ERR_ARG),
])
def test_grouped_refuses(L, kw, code):
    assert _grouped(L, **kw) == code and L.dg_layer_last_error()


def test_grouped_of_nothing(L):
    assert _grouped(L, t=0, a=None, d=None) == dg.OK
    assert _grouped(L, n=0, b=None, d=None) == dg.OK


@pytest.mark.parametrize("kw,code", [
    (dict(n=60), dg.ERR_SHAPE), (dict(k=36), dg.ERR_SHAPE), (dict(dt=dg.TYPE_E4M3), dg.ERR_ARG), (dict(d=None), dg.ERR_ARG),
    (dict(ld=60), dg.ERR_ARG), (dict(e=0), dg.ERR_ARG), (dict(ws=8), dg.ERR_ARG), (dict(a=None), dg.ERR_ARG),
])
def test_weight_grad_refuses(L, kw, code):
    v = dict(a=16, ld=64, e=2, d=16, dt=0, t=4, n=64, k=64, ws=256) | kw
    assert L.dg_layer_grouped_weight_grad(16, 64, v["a"], v["ld"], 16, v["e"], v["d"], v["dt"], v["t"], v["n"], v["k"],
                                          v["ws"], 256, 16, None) == code


def test_mx4_refuses(L):
    q = L.dg_layer_mx4_quantize
    assert q(16, 48, 0, 16, 16, 2, 48, None) == dg.ERR_SHAPE
    assert q(16, 64, dg.TYPE_E4M3, 16, 16, 2, 64, None) == dg.ERR_ARG
    assert q(8, 64, 0, 16, 16, 2, 64, None) == dg.ERR_ARG
    assert q(16, 68, 0, 16, 16, 2, 64, None) == dg.ERR_ARG
    assert q(None, 64, 0, 16, 16, 0, 64, None) == dg.OK
    assert L.dg_layer_mx4_dequantize(16, 16, 16, dg.TYPE_E5M2, 2, 64, None) == dg.ERR_ARG
    m = L.dg_layer_mx4_matmul
    assert m(16, 16, 16, 16, 16, 0, 4, 60, 64, 256, 16, None) == dg.ERR_SHAPE
    assert m(16, 16, 16, 16, 16, 0, 4, 64, 48, 256, 16, None) == dg.ERR_SHAPE
    assert m(16, 16, 16, 16, 16, dg.TYPE_E4M3, 4, 64, 64, 256, 16, None) == dg.ERR_ARG
    assert m(16, None, 16, 16, 16, 0, 4, 64, 64, 256, 16, None) == dg.ERR_ARG
    assert m(24, 16, 16, 16, 16, 0, 4, 64, 64, 256, 16, None) == dg.ERR_ARG
    assert m(None, None, None, None, None, 0, 0, 64, 64, None, None, None) == dg.OK
    assert L.dg_layer_mx4_scale_bytes(129, 288) == 2 * 2 * 1024
    assert L.dg_layer_mx4_scale_bytes(0, 288) == 0


def test_front_end_refuses_on_cpu(L):
    x, w = torch.zeros(4, 64, dtype=BF16), torch.ones(64, dtype=BF16)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w)                                    # not CUDA tensors
    with pytest.raises(TypeError):
        ops.add_rms_norm(x.float(), w)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w[:32])
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w, residual=x[:2])
    with pytest.raises(TypeError):
        ops.add_rms_norm(x, w, residual=x.half())
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w, out_dtype=torch.float32)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w, scale=1.0)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w, inplace=True)
    with pytest.raises(ValueError):
        ops.add_rms_norm_backward(x, x, w, torch.ones(3))
    ends = torch.tensor([2, 4], dtype=torch.int32)
    b = torch.zeros(2, 64, 32, dtype=BF16)
    with pytest.raises(ValueError):
        ops.grouped_matmul(x, b, ends)                            # not CUDA tensors
    with pytest.raises(ValueError):
        ops.grouped_matmul(x, b[:, :32], ends)
    with pytest.raises(ValueError):
        ops.grouped_matmul(x, b, ends.long())
    with pytest.raises(ValueError):
        ops.grouped_matmul(x, b, ends[:1])
    with pytest.raises(ValueError):
        ops.grouped_matmul_backward(x, x, b, ends)
    with pytest.raises(TypeError):
        ops.quantize_mx4(x.half())
    with pytest.raises(ValueError):
        ops.quantize_mx4(x)                                       # not a CUDA tensor
    with pytest.raises(TypeError):
        ops.mx4_matmul(x, x)
    q = ops.MX4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 2, 512, dtype=torch.uint8), 4, 64)
    with pytest.raises(ValueError):
        ops.mx4_matmul(q, q._replace(scales=q.scales[:, :1]))
    with pytest.raises(ValueError):
        ops.dequantize_mx4(q._replace(codes=q.codes[:, :8]))
