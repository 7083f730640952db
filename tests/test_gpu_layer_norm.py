"""Residual add + RMS norm on the GPU, element by element against the 64-bit
form: every output type, residual type and access path; rows that are zero, not
finite or strided; the gradient against the formula and against differences."""

import pytest
import torch

from reduce_scatter_gb300 import dg, ops
from tests import layer_common as lc
from tests.layer_common import U16, U32, assert_within, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
FP8 = {E4M3: (448.0, 3, -6), E5M2: (57344.0, 2, -14)}  # largest finite, mantissa bits, least exponent

# one warp per row, register kernels of 1, 2, 4 and 8 vectors, the looping
# kernel; odd sizes take the element-wise kernels of 4, 16 and many values
SIZES = [(1, 8), (5, 128), (1, 1), (3, 33), (7, 1000), (2, 1001), (700, 2048), (3, 4099), (2, 8192), (700, 8200),
         (1, 16384), (400, 16384), (2, 24576), (1, 32776), (1, 16387), (1, 40001)]


def check8(q, scale, y, hidden, dtype):
    """q * scale within half a step of y: the step is 2^-mantissa relative to
    the value, at least the subnormal step; the division adds 2 roundings."""
    top, mant, emin = FP8[dtype]
    rel = lc.norm_rel(hidden) + 4 * U32
    want = y / scale.double()[..., None]
    step = torch.maximum(want.abs() * 2.0 ** -mant, torch.full_like(want, 2.0 ** (emin - mant)))
    assert_within(q.float(), want, step / 2 * (1 + rel) + want.abs() * rel, "q")
    assert q.float().abs().max() <= top


@pytest.mark.parametrize("rows,hidden", SIZES)
@pytest.mark.parametrize("res", [None, BF16, F32])
def test_bf16_output(rows, hidden, res):
    x, w = rand((rows, hidden), 1), rand((hidden,), 2, dtype=BF16 if res != F32 else F32)
    r = None if res is None else rand((rows, hidden), 3, 2.0, res)
    got = ops.add_rms_norm(x, w, residual=r, keep_rstd=True)
    h, rstd, y = lc.norm(x, w, r)
    assert got.scale is None and torch.equal(got.residual, h)
    rel = lc.norm_rel(hidden)
    assert_within(got.rstd, rstd, rel * rstd, "rstd")
    assert_within(got.y, y, (U16 * (1 + rel) + rel) * y.abs(), "y")


@pytest.mark.parametrize("rows,hidden", SIZES)
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_8bit_output(rows, hidden, dtype):
    x, w = rand((rows, hidden), 4), rand((hidden,), 5)
    r = rand((rows, hidden), 6, 2.0) if rows % 2 else None
    got = ops.add_rms_norm(x, w, residual=r, out_dtype=dtype)
    h, _, y = lc.norm(x, w, r)
    assert got.y.dtype == dtype and got.scale.shape == (rows,) and torch.equal(got.residual, h)
    want = y.abs().amax(-1) / FP8[dtype][0]
    assert_within(got.scale, want, (lc.norm_rel(hidden) + 2 * U32) * want, "scale")
    check8(got.y, got.scale, y, hidden, dtype)


@pytest.mark.parametrize("as_tensor", [False, True])
@pytest.mark.parametrize("hidden", [512, 515])
def test_given_scale(hidden, as_tensor):
    x, w = rand((9, hidden), 7), rand((hidden,), 8)
    s = 2.0 ** -7  # values up to ~4 become up to ~500: some saturate
    got = ops.add_rms_norm(x, w, out_dtype=E4M3, scale=torch.tensor([s], device="cuda") if as_tensor else s)
    assert got.scale is None and got.residual is x
    _, _, y = lc.norm(x, w)
    check8(got.y, torch.full((9,), s, device="cuda"), y.clamp(-448 * s, 448 * s), hidden, E4M3)


def test_rows_of_zeros_and_not_finite():
    for hidden in (256, 259, 40000, 40001):
        x, w = rand((5, hidden), 9), rand((hidden,), 10)
        x[0] = 0
        x[1, 3] = float("nan")
        x[2, 3] = float("inf")
        clean = ops.add_rms_norm(x[3:], w, out_dtype=E4M3)
        got = ops.add_rms_norm(x, w, out_dtype=E4M3)
        q = got.y.float()
        assert got.scale[0] == 1 and not q[0].any()
        assert torch.isnan(q[1]).all() and got.scale[1] == 1
        assert torch.isnan(q[2, 3]) and torch.isfinite(got.scale[2])   # inf * 0; the others become 0
        assert not q[2, 4:].any()
        assert torch.equal(got.y[3:].view(torch.uint8), clean.y.view(torch.uint8))
        assert torch.equal(got.scale[3:], clean.scale)
        y = ops.add_rms_norm(x, w).y
        assert not y[0].any() and torch.isnan(y[1]).all() and torch.isfinite(y[3:]).all()


def test_strides_shapes_in_place_and_streams():
    big = rand((2, 6, 300), 11)
    x, w = big[:, 1:4, 8:264], rand((256,), 12)          # rows 600 bytes apart, aligned start: odd pitch in vectors
    r = rand((2, 3, 256), 13)
    h, _, y = lc.norm(x, w, r)
    got = ops.add_rms_norm(x, w, residual=r)
    assert got.y.shape == x.shape and torch.equal(got.residual, h)
    tol = (U16 * (1 + lc.norm_rel(256)) + lc.norm_rel(256)) * y.abs()
    assert_within(got.y, y, tol, "y")
    two = big.view(12, 300)[:, :256]                      # a matrix with a row pitch
    assert torch.equal(ops.add_rms_norm(two, w).y, ops.add_rms_norm(two.contiguous(), w).y)
    off = rand((4, 257), 14)[:, 1:]                       # rows that start off a 16-byte boundary
    assert torch.equal(ops.add_rms_norm(off, w).y, ops.add_rms_norm(off.clone(), w).y)
    keep = r.clone()
    got2 = ops.add_rms_norm(x, w, residual=keep, inplace=True)
    assert got2.residual is keep and torch.equal(keep, h) and torch.equal(got2.y, got.y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2 = ops.add_rms_norm(x, w, residual=r).y
    s.synchronize()
    assert torch.equal(y2, got.y)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x.transpose(0, 1), w, residual=r.transpose(0, 1).transpose(1, 2).contiguous().transpose(1, 2),
                         inplace=True)
    assert ops.add_rms_norm(x[:0], w).y.shape == (0, 3, 256)


def test_graph_replay():
    x, w, r = rand((33, 1024), 15), rand((1024,), 16), rand((33, 1024), 17)
    ops.add_rms_norm(x, w, residual=r, out_dtype=E4M3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ops.add_rms_norm(x, w, residual=r, out_dtype=E4M3)
    x.copy_(rand((33, 1024), 18))
    g.replay()
    want = ops.add_rms_norm(x, w, residual=r, out_dtype=E4M3)
    torch.cuda.synchronize()
    assert torch.equal(got.y.view(torch.uint8), want.y.view(torch.uint8)) and torch.equal(got.scale, want.scale)


def grad(dy, h, w, dh, eps=1e-5):
    """(dx, dw, dx bound, dw bound) in fp64."""
    hidden, rows = h.shape[-1], h.shape[0]
    hd, dyd = h.double(), dy.double()
    rstd = 1.0 / torch.sqrt(hd.pow(2).mean(-1, keepdim=True) + eps)
    xh, g = hd * rstd, dyd * w.double()
    dot, mag = (g * xh).mean(-1, keepdim=True), (g * xh).abs().mean(-1, keepdim=True)
    dx = rstd * (g - xh * dot)
    rel = lc.norm_rel(hidden) + lc.norm_rel(hidden)     # of xh, and of the sum of products
    bx = 3 * rel * rstd * (g.abs() + xh.abs() * mag)
    if dh is not None:
        dx = dx + dh.double()
        bx = bx + 4 * U32 * dh.double().abs()
    dw, mw = (dyd * xh).sum(0), (dyd * xh).abs().sum(0)
    return dx, dw, bx, (rel + (rows + 64) * U32) * mw


@pytest.mark.parametrize("rows,hidden", [(1, 8), (3, 100), (5, 1001), (700, 256), (331, 4096), (37, 8192), (3, 8200),
                                         (9, 16384), (2, 16392), (4, 5000), (3, 8191), (2, 20001)])
@pytest.mark.parametrize("f32,with_dh", [(False, True), (False, False), (True, True)])
def test_gradient(rows, hidden, f32, with_dh):
    t = F32 if f32 else BF16
    h, w, dy = rand((rows, hidden), 21, 2.0, t), rand((hidden,), 22, dtype=t), rand((rows, hidden), 23)
    dh = rand((rows, hidden), 24, 0.5, t) if with_dh else None
    rstd = (1.0 / torch.sqrt(h.double().pow(2).mean(-1) + 1e-5)).float()
    dx, dw = ops.add_rms_norm_backward(dy, h, w, rstd, d_residual=dh)
    wx, ww, bx, bw = grad(dy, h, w, dh)
    out = 0.0 if f32 else U16
    assert dx.dtype == t and dw.dtype == t
    assert_within(dx, wx, bx * (1 + out) + out * wx.abs(), "dx")
    assert_within(dw, ww, bw * (1 + out) + out * ww.abs(), "dw")
    again = ops.add_rms_norm_backward(dy, h, w, rstd, d_residual=dh)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_gradient_against_differences():
    rows, hidden, eps = 6, 96, 1e-5
    h, w, dy, dh = rand((rows, hidden), 31, dtype=F32), rand((hidden,), 32, dtype=F32), rand((rows, hidden), 33), rand(
        (rows, hidden), 34, dtype=F32)
    rstd = (1.0 / torch.sqrt(h.double().pow(2).mean(-1) + eps)).float()
    dx, dw = ops.add_rms_norm_backward(dy, h, w, rstd, d_residual=dh)

    def f(hd, wd):
        y = hd / torch.sqrt(hd.pow(2).mean(-1, keepdim=True) + eps) * wd
        return ((y * dy.double()).sum() + (hd * dh.double()).sum())

    _, _, bx, bw = grad(dy, h, w, dh)
    step = 1e-5
    for seed in range(3):
        vh, vw = rand((rows, hidden), 40 + seed, dtype=F32).double(), rand((hidden,), 50 + seed, dtype=F32).double()
        hd, wd = h.double(), w.double()
        diff = (f(hd + step * vh, wd + step * vw) - f(hd - step * vh, wd - step * vw)) / (2 * step)
        got = (dx.double() * vh).sum() + (dw.double() * vw).sum()
        # the kernel's bound, and the difference's own error: step^2 times the third derivative (here of order 1 to
        # 100 per row) and fp64 rounding over the step
        tol = (bx * vh.abs()).sum() + (bw * vw.abs()).sum() + 1e-6 * (1 + diff.abs())
        assert (got - diff).abs() <= tol, (float(got), float(diff), float(tol))


@pytest.mark.parametrize("res", [None, BF16, F32])
def test_autograd(res):
    rows, hidden = 12, 264
    x, w = rand((rows, hidden), 61).requires_grad_(), rand((hidden,), 62).requires_grad_()
    r = None if res is None else rand((rows, hidden), 63, dtype=res).requires_grad_()
    dy = rand((rows, hidden), 64)
    out = ops.add_rms_norm(x, w, residual=r)
    if res is None:
        out.y.backward(dy)
        dh = None
    else:
        dh = rand((rows, hidden), 65, dtype=res)
        torch.autograd.backward([out.y, out.residual], [dy, dh])
    h, _, _ = lc.norm(x.detach(), w.detach(), None if r is None else r.detach())
    wx, ww, bx, bw = grad(dy, h, w.detach(), dh)
    assert_within(x.grad, wx, 2 * bx + 2 * U16 * wx.abs(), "x.grad")
    assert_within(w.grad, ww, 2 * bw + U16 * ww.abs(), "w.grad")
    if r is not None:
        out_u = U16 if res == BF16 else 0.0
        assert r.grad.dtype == res
        assert_within(r.grad, wx, 2 * bx + out_u * wx.abs(), "r.grad")
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w, out_dtype=E4M3)
    with torch.no_grad():
        assert ops.add_rms_norm(x, w, out_dtype=E4M3).y.dtype == E4M3


def test_feeds_the_scaled_all_gather_product():
    # rows in 8 bits with a given scale, as fused_all_gather_scaled_matmul takes them
    x, w = rand((256, 512), 71), rand((512,), 72)
    W = rand((128, 512), 73, 0.05).to(E4M3)
    s = 2.0 ** -5
    q = ops.add_rms_norm(x, w, out_dtype=E4M3, scale=s).y
    _, (D,) = ops.fused_all_gather_scaled_matmul(q, [W.t()], s, [1.0], 0, 2, out_dtypes=[F32])
    v, m = lc.product(q.float() * s, W.float())
    assert_within(D, v, lc.product_bound(v, m, 512, out16=False), "D")


def test_refusals():
    x, w = rand((4, 64), 81), rand((64,), 82)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w.cpu())
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, w, out_dtype=E4M3, scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, rand((128,), 83)[::2])
    with pytest.raises(dg.DGError) as e:
        ops.add_rms_norm(x, w, eps=-1.0)
    assert e.value.code == dg.ERR_ARG
    with pytest.raises(ValueError):
        ops.add_rms_norm_backward(x, x, w, torch.ones(4, device="cuda"), d_residual=x.float())
    with pytest.raises(TypeError):
        ops.add_rms_norm_backward(x.float(), x, w, torch.ones(4, device="cuda"))
