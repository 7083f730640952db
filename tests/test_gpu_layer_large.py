"""The layer operators where element offsets pass 32 bits: rows (or experts) at
the start, beside the 2^31 and 2^32 marks and at the end against the 64-bit form."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests import layer_common as lc
from tests.layer_common import U16, assert_within, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn


def big(*shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda", dtype=BF16).normal_(0.0, std, generator=g)


def marks(rows, pitch):
    """Rows at both ends and around the multiples of 2^31 elements."""
    at = {0, 1, rows - 1}
    for m in range(2 ** 31, rows * pitch, 2 ** 31):
        at |= {m // pitch - 1, m // pitch, m // pitch + 1}
    return torch.tensor(sorted(r for r in at if 0 <= r < rows), device="cuda")


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def test_norm_and_gradient():
    rows, hidden = 270000, 16384                       # 4.4e9 values
    x, r, w = big(rows, hidden, seed=1), big(rows, hidden, seed=2), rand((hidden,), 3)
    at = marks(rows, hidden)
    got = ops.add_rms_norm(x, w, residual=r, out_dtype=E4M3, keep_rstd=True)
    h, rstd, y = lc.norm(x[at], w, r[at])
    assert torch.equal(got.residual[at], h)
    step = (y.abs() / got.scale[at].double()[:, None] * 2.0 ** -3).clamp(min=2.0 ** -9) * got.scale[at].double()[:, None]
    assert_within(got.y.view(torch.uint8)[at].view(E4M3).double() * got.scale[at].double()[:, None], y, step / 2 * 1.01, "y")
    dx, dw = ops.add_rms_norm_backward(x, got.residual, w, got.rstd, d_residual=r)
    hd, dy = h.double(), x[at].double()
    xh, g = hd * rstd[:, None], dy * w.double()
    want = rstd[:, None] * (g - xh * (g * xh).mean(-1, keepdim=True)) + r[at].double()
    rel = 2 * lc.norm_rel(hidden)
    mag = rstd[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True)) + r[at].double().abs()
    assert_within(dx[at], want, 3 * rel * mag + U16 * (want.abs() + 3 * rel * mag), "dx")
    assert torch.isfinite(dw.float()).all()


def test_grouped_rows_and_output():
    for T, K, N in ((540000, 8192, 64), (540000, 64, 8192)):   # A, then D, of 4.4e9 values
        a, b = big(T, K, seed=4), big(2, N, K, seed=5, std=0.1).transpose(1, 2)
        ends = torch.tensor([T - 300, T], dtype=torch.int32, device="cuda")
        d = ops.grouped_matmul(a, b, ends)
        at = marks(T, max(K, N))
        for e in range(2):
            rows = at[(at >= T - 300) == bool(e)]
            v, m = lc.product(a[rows], b[e].t())
            assert_within(d[rows], v, lc.product_bound(v, m, K), "D")
        dd = big(T, N, seed=6, std=0.1)
        _, db = ops.grouped_matmul_backward(dd, a, b, ends, need=(False, True))
        v, m = lc.product(a[T - 300:].t(), dd[T - 300:].t())
        assert_within(db[1], v, lc.product_bound(v, m, 300), "dB")
        ops.check_products()
        del a, b, d, dd, db


def test_grouped_experts():
    E, N, K = 600, 1024, 8192                            # 5e9 weights
    w = big(E, N, K, seed=7, std=0.1)
    b = w.transpose(1, 2)
    a, dd = big(2 * E, K, seed=8), big(2 * E, N, seed=9)
    ends = torch.arange(2, 2 * E + 1, 2, dtype=torch.int32, device="cuda")
    d = ops.grouped_matmul(a, b, ends)
    da, db = ops.grouped_matmul_backward(dd, a, b, ends)
    for e in (0, 255, 256, 511, 512, 599):
        rows = slice(2 * e, 2 * e + 2)
        v, m = lc.product(a[rows], w[e])
        assert_within(d[rows], v, lc.product_bound(v, m, K), "D")
        v, m = lc.product(dd[rows], w[e].t())
        assert_within(da[rows], v, lc.product_bound(v, m, N), "dA")
        v, m = lc.product(a[rows].t(), dd[rows].t())
        assert_within(db[e], v, lc.product_bound(v, m, 2), "dB")
    ops.check_products()


def test_mx4():
    rows, cols = 270000, 16384
    x = big(rows, cols, seed=10)
    q = ops.quantize_mx4(x)
    at = marks(rows, cols)
    y = ops.dequantize_mx4(q)
    for r in at.tolist():                                # a band of 128 rows as a matrix of its own
        r0 = r // 128 * 128
        band = ops.quantize_mx4(x[r0:r0 + 128])
        assert torch.equal(band.codes, q.codes[r0:r0 + 128]) and torch.equal(band.scales[0], q.scales[r0 // 128])
        assert torch.equal(ops.dequantize_mx4(band), y[r0:r0 + 128])
    w = ops.quantize_mx4(rand((64, cols), 11))
    d = ops.mx4_matmul(q, w)
    v, m = lc.product(y[at], ops.dequantize_mx4(w))
    assert_within(d[at], v, lc.product_bound(v, m, cols), "D")
    del x, q, y, d
    a, w = ops.quantize_mx4(rand((rows, 32), 12)), ops.quantize_mx4(rand((cols, 32), 13))
    d = ops.mx4_matmul(a, w)                             # 4.4e9 outputs
    v, m = lc.product(ops.dequantize_mx4(a)[at], ops.dequantize_mx4(w))
    assert_within(d[at], v, lc.product_bound(v, m, 32), "D")
    ops.check_products()
