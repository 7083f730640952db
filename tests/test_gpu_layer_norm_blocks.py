"""Layer norm on the GPU against the 64-bit form: every type of input, residual
and output, 8-bit blocks, rows kept in 8 bits, the gradient against the formula
and against differences; rows that are constant, not finite, strided.

Bounds (U32 per fp32 operation, sums of H values H + 8 of them): the mean is
corrected by the sum of the differences from it where that is above 2^-21 of the
deviation, so its error is that of a sum of small numbers, (H + 8) U32 mean|h -
mu|, 2^-21 of the deviation, and two roundings."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests.layer_common import U16, U32, assert_within, rand
from tests.test_gpu_block8 import FP8, quantized, spread

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
EPS = 1e-5

# one warp per row; register kernels of 1, 2 and 8 vectors; streamed rows; the looping kernel; odd sizes element-wise
SIZES = [(1, 8), (5, 128), (1, 1), (3, 33), (7, 1000), (2, 1001), (700, 2048), (3, 4099), (2, 8192), (700, 8208), (1, 16384),
         (400, 16384), (2, 24576), (1, 32784), (1, 16387), (1, 40001), (330, 2064)]
# many rows that start and end inside vectors: streamed
ODD = [(700, 1001), (331, 4099), (500, 777), (310, 16369), (320, 8190), (400, 502)]


def inputs(rows, hidden, seed, xt=BF16, rt=None, wt=BF16):
    x = (rand((rows, hidden), seed, dtype=F32) + 3 * rand((rows, 1), seed + 1, dtype=F32)).to(xt)
    r = None if rt is None else rand((rows, hidden), seed + 2, 2.0, rt)
    w = (1 + rand((hidden,), seed + 3, 0.2, F32)).to(wt)
    b = rand((hidden,), seed + 4, 0.3, wt)
    return x, r, w, b


def norm64(x, r, w, b, eps=EPS):
    """h as it is stored; mean, rstd, y in 64 bits; the bounds of the mean, of rstd and of y before its last rounding."""
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    f = h.double()
    H = f.shape[-1]
    mu = f.mean(-1, keepdim=True)
    c = f - mu
    rstd = 1.0 / torch.sqrt(c.pow(2).mean(-1, keepdim=True) + eps)
    wd = 1.0 if w is None else w.double()
    y = c * rstd * wd + (0.0 if b is None else b.double())
    e_mu = (H + 8) * U32 * c.abs().mean(-1, keepdim=True) + 2.0 ** -21 * c.pow(2).mean(-1, keepdim=True).sqrt() + 2 * U32 * mu.abs()
    e_rstd = ((H + 16) * U32 + (e_mu * rstd) ** 2) * rstd
    scaled = (c * rstd * wd).abs()
    e_y = (e_mu + 2 * U32 * c.abs()) * rstd * (w.double().abs() if w is not None else 1.0) + scaled * (e_rstd / rstd + 4 * U32) + 2 * U32 * y.abs()
    return h, mu[..., 0], rstd[..., 0], y, e_mu[..., 0], e_rstd[..., 0], e_y


def check_stats(got, mu, rstd, e_mu, e_rstd):
    assert_within(got.mean, mu, e_mu, "mean")
    assert_within(got.rstd, rstd, e_rstd, "rstd")


def check_blocks(q, y, e_y, dtype):
    """q against the rows y, known to e_y: within half a step of the 8 bits and y's bound, in units of the scale."""
    top, mant, emin = FP8[dtype]
    rows, cols = y.shape
    amax = torch.nn.functional.pad(y.abs(), (0, -cols % 128)).view(rows, -1, 128).amax(-1)
    e_max = torch.nn.functional.pad(e_y, (0, -cols % 128)).view(rows, -1, 128).amax(-1)
    c = torch.where(amax > 0, amax / top, 1.0)
    assert_within(q.scales, c, e_max / top + 2 * U32 * c, "scales")
    s = spread(q.scales.double(), 1, rows, cols)
    v = y / s
    step = torch.maximum(v.abs() * 2.0 ** -mant, torch.full_like(v, 2.0 ** (emin - mant)))
    slack = (e_y + spread(e_max, 1, rows, cols)) / s + 4 * U32 * v.abs()
    assert_within(q.values.float(), v, step / 2 * (1 + 4 * U32) + slack * 1.25, "values")  # (a step may grow within the slack)


@pytest.mark.parametrize("rows,hidden", SIZES + ODD)
@pytest.mark.parametrize("xt,rt", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, F32), (F32, BF16)])
def test_16_bit_output(rows, hidden, xt, rt):
    x, r, w, b = inputs(rows, hidden, 1, xt, rt, F32 if rows == 7 or hidden == 8208 else BF16)
    got = ops.layer_norm(x, w, b, residual=r, keep_stats=True)
    h, mu, rstd, y, e_mu, e_rstd, e_y = norm64(x, r, w, b)
    assert torch.equal(got.residual, h) and got.kept is None and got.y.dtype == BF16
    check_stats(got, mu, rstd, e_mu, e_rstd)
    assert_within(got.y, y, e_y + U16 * (y.abs() + e_y), "y")


@pytest.mark.parametrize("rows,hidden", [s for s in SIZES if s[1] % 16 == 0])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("keep", [None, E4M3, E5M2])
def test_blocks(rows, hidden, dtype, keep):
    x, r, w, b = inputs(rows, hidden, 10, F32 if rows == 5 else BF16, BF16 if rows % 2 else None)
    got = ops.layer_norm(x, w, b, residual=r, out_dtype=dtype, keep_dtype=keep, keep_stats=keep is not None)
    h, mu, rstd, y, e_mu, e_rstd, e_y = norm64(x, r, w, b)
    assert torch.equal(got.residual, h) and got.y.values.dtype == dtype and got.y.block_rows == 1
    check_blocks(got.y, y, e_y, dtype)
    if keep is None:
        assert got.mean is None and got.kept is None
        return
    check_stats(got, mu, rstd, e_mu, e_rstd)
    v, c = quantized(h, 1, keep, True)
    assert torch.equal(got.kept.scales.double(), c) and torch.equal(got.kept.values.float().double(), v)
    plain = ops.quantize_block8(h, dtype=keep, pow2=True)
    assert torch.equal(plain.values.view(torch.uint8), got.kept.values.view(torch.uint8))
    same = ops.layer_norm(x, w, b, residual=r, keep_dtype=keep)   # a 16-bit output beside the kept rows
    assert torch.equal(same.kept.values.view(torch.uint8), got.kept.values.view(torch.uint8))
    assert torch.equal(same.y, ops.layer_norm(x, w, b, residual=r).y)


def test_weight_and_bias_may_be_missing():
    for hidden in (512, 515, 16384):
        x, _, w, b = inputs(320, hidden, 20)
        for ww, bb in ((None, None), (w, None), (None, b)):
            _, _, _, y, _, _, e_y = norm64(x, None, ww, bb)
            got = ops.layer_norm(x, ww, bb)
            assert_within(got.y, y, e_y + U16 * (y.abs() + e_y), "y")


def test_rows_of_one_value_and_not_finite():
    for hidden in (1, 256, 259, 2048, 40000, 40001):
        x, _, w, b = inputs(330 if hidden == 2048 else 6, hidden, 30)
        x[0] = 2.5
        if hidden > 1:
            x[1, 3 % hidden], x[2, 3 % hidden] = float("nan"), float("inf")
        got = ops.layer_norm(x, w, b, keep_stats=True)
        assert torch.equal(got.y[0], b) and got.mean[0] == 2.5
        assert_within(got.rstd[:1], torch.full((1,), EPS ** -0.5, dtype=torch.float64, device="cuda"), 4 * U32 * EPS ** -0.5, "rstd")
        if hidden > 1:
            assert torch.isnan(got.y[1:3]).all() and torch.isnan(got.rstd[1:3]).all()
        rest = ops.layer_norm(x[3:], w, b)
        assert torch.equal(got.y[3:], rest.y)
        if hidden % 16 == 0:
            q = ops.layer_norm(x, w, b, out_dtype=E4M3, keep_dtype=E4M3)
            assert torch.isnan(q.y.values[1:3].float()).all() and torch.isfinite(q.y.scales).all()
            assert torch.isfinite(q.y.values[3:].float()).all()
            kept = q.kept.values.float()
            assert torch.isnan(kept[1]).sum() == 1 and torch.isnan(kept[2]).sum() == 1 and torch.isfinite(q.kept.scales).all()


def test_a_mean_far_above_the_deviation():
    x = rand((4, 4096), 40, dtype=F32) + 3000.0
    got = ops.layer_norm(x, keep_stats=True)
    _, mu, rstd, y, e_mu, e_rstd, e_y = norm64(x, None, None, None)
    check_stats(got, mu, rstd, e_mu, e_rstd)
    assert_within(got.y, y, e_y + U16 * (y.abs() + e_y), "y")
    assert e_y.max() < 0.1


def test_strides_shapes_and_streams():
    big = rand((2, 6, 304), 41)
    w, b = rand((256,), 42), rand((256,), 43)
    for x in (big[:, 1:4, 8:264], big[:, 1:4, 1:257], big[:, ::2, 48:], rand((256, 10), 44).t(), rand((1, 256), 45).expand(5, 256)):
        plain = x.contiguous()
        r = rand(x.shape, 46)
        got, want = ops.layer_norm(x, w, b, residual=r, keep_stats=True), ops.layer_norm(plain, w, b, residual=r, keep_stats=True)
        assert got.y.shape == x.shape and got.mean.shape == x.shape[:-1]
        assert torch.equal(got.y, want.y) and torch.equal(got.residual, want.residual)
        q, p = ops.layer_norm(x, w, b, out_dtype=E5M2, keep_dtype=E4M3), ops.layer_norm(plain, w, b, out_dtype=E5M2, keep_dtype=E4M3)
        for one, two in ((q.y, p.y), (q.kept, p.kept)):
            assert torch.equal(one.values.view(torch.uint8), two.values.view(torch.uint8)) and torch.equal(one.scales, two.scales)
    off = rand((257,), 47)[1:]
    assert torch.equal(ops.layer_norm(plain, off, off).y, ops.layer_norm(plain, off.clone(), off.clone()).y)
    a, c = ops.layer_norm(plain, off, off, out_dtype=E4M3).y, ops.layer_norm(plain, off.clone(), off.clone(), out_dtype=E4M3).y
    assert torch.equal(a.values.view(torch.uint8), c.values.view(torch.uint8))
    want = ops.layer_norm(plain, w, b).y
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = ops.layer_norm(plain, w, b).y
    s.synchronize()
    assert torch.equal(y, want)
    assert ops.layer_norm(big[:0, :, :256], w, b).y.shape == (0, 6, 256)
    none = ops.layer_norm(big[:, :, :0], keep_stats=True)
    assert none.y.shape == (2, 6, 0) and torch.isnan(none.rstd).all()


def test_odd_rows_in_wider_ones():
    # rows that start where densely packed ones would, in a wider matrix; neighbours that are not finite stay out
    wide = torch.full((400, 1009), float("nan"), device="cuda", dtype=BF16)
    x = wide[:, :1001]
    x.copy_(rand((400, 1001), 48))
    w, b, r = rand((1001,), 49), rand((1001,), 50), rand((400, 1001), 51)
    got, want = ops.layer_norm(x, w, b, residual=r, keep_stats=True), ops.layer_norm(x.contiguous(), w, b, residual=r, keep_stats=True)
    assert torch.equal(got.y, want.y) and torch.equal(got.residual, want.residual) and torch.equal(got.mean, want.mean)
    f = ops.layer_norm(x, w, b, keep_stats=True)
    dwide = torch.full((400, 1009), float("inf"), device="cuda", dtype=BF16)
    dy = dwide[:, :1001]
    dy.copy_(rand((400, 1001), 52))
    for one, two in zip(ops.layer_norm_backward(dy, x, w, f.mean, f.rstd), ops.layer_norm_backward(dy.contiguous(), x.contiguous(), w, f.mean, f.rstd)):
        assert torch.equal(one, two) and torch.isfinite(one).all()
    off = rand((400 * 1001 + 1,), 53)[1:].view(400, 1001)  # (a start off 16 bytes)
    _, _, _, y, _, _, e_y = norm64(off, None, w, b)
    assert_within(ops.layer_norm(off, w, b).y, y, e_y + U16 * (y.abs() + e_y), "y")


# ----------------------------------------------------------------- gradient


def grad64(dy, f, mean, rstd, w, dh, out16):
    """dx, dw, db in 64 bits from the values f, and their bounds."""
    H, rows = f.shape[-1], f.shape[0]
    m, s = mean.double()[..., None], rstd.double()[..., None]
    d = dy.double()
    xh = (f - m) * s
    g = d * (1.0 if w is None else w.double())
    m1, m2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dx = s * (g - m1 - xh * m2)
    n = 2 * (H + 16) * U32
    err = s * (4 * U32 * (g.abs() + m1.abs()) + n * g.abs().mean(-1, keepdim=True)
               + xh.abs() * (n * (g * xh).abs().mean(-1, keepdim=True) + 6 * U32 * m2.abs())) + 4 * U32 * dx.abs()
    if dh is not None:
        dx = dx + dh.double()
        err = err + 2 * U32 * dx.abs()
    if out16:
        err = err + U16 * (dx.abs() + err)
    k = 2 * (rows + 8) * U32
    return dx, err, (d * xh).sum(0), k * (d * xh).abs().sum(0), d.sum(0), k * d.abs().sum(0)


def check_grad(got, want, w16, b16):
    dx, e_dx, dw, e_dw, db, e_db = want
    assert_within(got[0], dx, e_dx, "dx")
    if got[1] is not None:
        assert_within(got[1], dw, e_dw + (U16 * (dw.abs() + e_dw) if w16 else U32 * dw.abs()), "dw")
    if got[2] is not None:
        assert_within(got[2], db, e_db + (U16 * (db.abs() + e_db) if b16 else U32 * db.abs()), "db")


@pytest.mark.parametrize("rows,hidden", SIZES + ODD + [(1300, 512), (20, 8195), (9, 16390), (8, 510), (1500, 1023)])
@pytest.mark.parametrize("ht", [BF16, F32])
@pytest.mark.parametrize("has_dh", [False, True])
def test_gradient(rows, hidden, ht, has_dh):
    x, _, w, _ = inputs(rows, hidden, 50, ht, None, F32 if has_dh and rows > 5 else BF16)
    dy = rand((rows, hidden), 55)
    dh = rand((rows, hidden), 56, 1.0, ht) if has_dh else None
    f = ops.layer_norm(x, w, keep_stats=True)
    got = ops.layer_norm_backward(dy, x, w, f.mean, f.rstd, d_residual=dh, bias_dtype=F32 if rows == 2 else None)
    assert got[0].dtype == ht and got[1].dtype == w.dtype
    check_grad(got, grad64(dy, x.double(), f.mean, f.rstd, w, dh, ht == BF16), w.dtype == BF16, got[2].dtype == BF16)


@pytest.mark.parametrize("rows,hidden", [s for s in SIZES if s[1] % 16 == 0])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("has_dh", [False, True])
def test_gradient_from_kept_rows(rows, hidden, dtype, has_dh):
    x, _, w, b = inputs(rows, hidden, 60)
    dy = rand((rows, hidden), 65)
    dh = rand((rows, hidden), 66) if has_dh else None
    f = ops.layer_norm(x, w, b, keep_stats=True, keep_dtype=dtype)
    got = ops.layer_norm_backward(dy, f.kept, w, f.mean, f.rstd, d_residual=dh)
    values = ops.dequantize_block8(f.kept, out_dtype=F32)
    check_grad(got, grad64(dy, values.double(), f.mean, f.rstd, w, dh, True), True, True)
    scaled = ops.quantize_block8(x, dtype=dtype)            # scales that are no powers of two, rows next to each other or not
    for scales in (scaled.scales, scaled.scales.t().contiguous().t()):
        q = ops.Block8Tensor(scaled.values, scales, 1)
        got = ops.layer_norm_backward(dy, q, w, f.mean, f.rstd, d_residual=dh)
        want = grad64(dy, q.values.float().double() * spread(scales.double(), 1, rows, hidden), f.mean, f.rstd, w, dh, True)
        extra = U32 * ops.dequantize_block8(q, out_dtype=F32).double().abs() * f.rstd.double()[:, None]  # the product with the scale
        d = dy.double().abs()
        dx, e_dx, dw, e_dw, db, e_db = want
        m2 = (d * w.double().abs() * (q.values.float().double() * spread(scales.double(), 1, rows, hidden) - f.mean.double()[:, None]).abs()
              * f.rstd.double()[:, None]).mean(-1, keepdim=True)
        m3 = (d * w.double().abs() * extra).mean(-1, keepdim=True)
        xh = (q.values.float().double() * spread(scales.double(), 1, rows, hidden) - f.mean.double()[:, None]).abs() * f.rstd.double()[:, None]
        e_dx = e_dx + 2 * f.rstd.double()[:, None] * (extra * m2 + xh * m3)
        check_grad(got, (dx, e_dx, dw, e_dw + 2 * (d * extra).sum(0), db, e_db), True, True)


def test_gradient_against_differences():
    x, r, w, b = inputs(12, 96, 70, BF16, F32)
    dy = rand((12, 96), 75)
    h = (x.float() + r).double()
    f = ops.layer_norm(x, w, b, residual=r, keep_stats=True)
    dx, dw, db = ops.layer_norm_backward(dy, f.residual, w, f.mean, f.rstd)

    def loss(h, w, b):
        c = h - h.mean(-1, keepdim=True)
        return ((c / torch.sqrt(c.pow(2).mean(-1, keepdim=True) + EPS) * w + b) * dy.double()).sum()

    at = [h, w.double(), b.double()]
    for i, grad in enumerate((dx, dw, db)):
        v = rand(at[i].shape, 76 + i, dtype=F32).double()
        lo, hi = list(at), list(at)
        t = 1e-4
        lo[i], hi[i] = at[i] - t * v, at[i] + t * v
        want = (loss(*hi) - loss(*lo)) / (2 * t)
        got = (grad.double() * v).sum()
        # the gradients' rounding, and the differences' error of order t^2
        tol = (U16 if grad.dtype == BF16 else 300 * U32) * (grad.double() * v).abs().sum() + 1e-5 * (1 + want.abs())
        assert (got - want).abs() <= tol, (i, float(got), float(want))


@pytest.mark.parametrize("keep", [None, E4M3])
@pytest.mark.parametrize("xt,rt", [(BF16, None), (BF16, F32), (F32, BF16)])
def test_autograd(keep, xt, rt):
    x, r, w, b = inputs(40, 256, 80, xt, rt)
    b = b.float()
    leaves = [t.requires_grad_() for t in (x, w, b)] + ([r.requires_grad_()] if r is not None else [])
    got = ops.layer_norm(x, w, b, residual=r, keep_dtype=keep, keep_stats=True)
    dy, dh = rand((40, 256), 85), rand((40, 256), 86)
    loss = (got.y.float() * dy.float()).sum()
    if r is not None:
        loss = loss + (got.residual.float() * dh.float()).sum()
    loss.backward()
    with torch.no_grad():
        h = got.kept if keep else got.residual.detach()
        ht = BF16 if keep else got.residual.dtype
        dx, dw, db = ops.layer_norm_backward(dy, h, w.detach(), got.mean, got.rstd, d_residual=dh.to(ht) if r is not None else None,
                                             bias_dtype=F32)
    assert torch.equal(x.grad, dx.to(xt)) and torch.equal(w.grad, dw) and torch.equal(b.grad, db) and b.grad.dtype == F32
    if r is not None:
        assert torch.equal(r.grad, dx.to(rt))
    # parts of the graph: only the sum, a missing bias, a frozen weight
    if r is not None:
        for t in leaves:
            t.grad = None
        ops.layer_norm(x, w, b, residual=r, keep_dtype=keep).residual.backward(dh.to(rt))
        assert torch.equal(r.grad, dh.to(rt)) and torch.equal(x.grad, dh.to(rt).to(xt)) and w.grad is None
    x.grad = None
    ops.layer_norm(x, w.detach(), None, keep_dtype=keep).y.backward(dy)
    assert x.grad is not None and x.grad.dtype == xt


def test_gradient_shapes_and_graph():
    x, _, w, b = inputs(330, 2048, 90)
    x3, dy3 = x.view(3, 110, 2048), rand((3, 110, 2048), 95)
    f = ops.layer_norm(x3, w, b, keep_stats=True)
    dx, dw, db = ops.layer_norm_backward(dy3, x3, w, f.mean, f.rstd)
    flat = ops.layer_norm_backward(dy3.view(330, 2048), x, w, f.mean.view(-1), f.rstd.view(-1))
    assert torch.equal(dx.view(330, 2048), flat[0]) and torch.equal(dw, flat[1]) and torch.equal(db, flat[2])
    t = dy3.transpose(0, 1).contiguous().transpose(0, 1)                   # the same values in another order of memory
    assert torch.equal(ops.layer_norm_backward(t, x3, w, f.mean, f.rstd)[0], dx)
    assert ops.layer_norm_backward(dy3, x3, None, f.mean, f.rstd)[1:] == (None, None)
    only = ops.layer_norm_backward(dy3, x3, None, f.mean, f.rstd, bias_dtype=F32)
    assert only[1] is None and only[2].dtype == F32
    none = ops.layer_norm_backward(dy3[:0], x3[:0], w, f.mean[:0], f.rstd[:0])
    assert none[0].shape == (0, 110, 2048) and not none[1].any() and not none[2].any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = ops.layer_norm(x, w, b, keep_stats=True, keep_dtype=E4M3)
        out = ops.layer_norm_backward(flat[0], g.kept, w, g.mean, g.rstd)
    x.copy_(rand(x.shape, 96))
    graph.replay()
    g2 = ops.layer_norm(x, w, b, keep_stats=True, keep_dtype=E4M3)
    for one, two in zip(out, ops.layer_norm_backward(flat[0], g2.kept, w, g2.mean, g2.rstd)):
        assert torch.equal(one, two)


# ----------------------------- rows that leave an SM one at a time, with few threads

WIDE = [(310, 8200), (320, 9216), (330, 10256), (310, 12288), (400, 12280), (1000, 8208)]


@pytest.mark.parametrize("rows,hidden", WIDE)
@pytest.mark.parametrize("xt,rt,wt", [(BF16, None, BF16), (BF16, BF16, F32), (BF16, F32, BF16)])
def test_wide_rows(rows, hidden, xt, rt, wt):
    x, r, w, b = inputs(rows, hidden, 101, xt, rt, wt)
    got = ops.layer_norm(x, w, b, residual=r, keep_stats=True)
    h, mu, rstd, y, e_mu, e_rstd, e_y = norm64(x, r, w, b)
    assert torch.equal(got.residual, h)
    check_stats(got, mu, rstd, e_mu, e_rstd)
    assert_within(got.y, y, e_y + U16 * (y.abs() + e_y), "y")
    if hidden % 16:
        return
    got = ops.layer_norm(x, w, b, residual=r, out_dtype=E4M3, keep_dtype=E5M2, keep_stats=True)
    check_blocks(got.y, y, e_y, E4M3)
    check_stats(got, mu, rstd, e_mu, e_rstd)
    v, c = quantized(h, 1, E5M2, True)
    assert torch.equal(got.residual, h) and torch.equal(got.kept.scales.double(), c) and torch.equal(got.kept.values.float().double(), v)
    x[3, hidden - 1], x[4, 0] = float("inf"), float("nan")
    bad = ops.layer_norm(x, w, b, residual=r, out_dtype=E4M3, keep_dtype=E5M2)
    others = torch.arange(rows, device="cuda") // 2 != 1
    others[4] = False
    assert torch.equal(bad.y.values.view(torch.uint8)[others], got.y.values.view(torch.uint8)[others])
    assert torch.isnan(bad.y.values[3:5].float()).all() and not torch.isnan(bad.kept.values[3, :-1].float()).any()
