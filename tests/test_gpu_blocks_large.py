"""8-bit blocks, layer norm and kept rows where element offsets pass 32 bits:
rows at the start, beside the multiples of 2^31 and at the end against the
64-bit form."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests import layer_common as lc
from tests.layer_common import U16, U32, assert_within, rand
from tests.test_gpu_block8 import quantized, spread, values64
from tests.test_gpu_layer_large import big, marks
from tests.test_gpu_layer_norm_blocks import check_blocks, norm64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def rows_of(values, at):
    """Rows of an 8-bit matrix (indexed as bytes)."""
    return values.view(torch.uint8)[at].view(values.dtype)


def test_quantise_and_values():
    rows, cols = 270000, 16384                          # 4.4e9 values
    x = big(rows, cols, seed=1)
    at = marks(rows, cols)
    q = ops.quantize_block8(x)
    v, c = quantized(x[at], 1, E4M3, False)
    assert torch.equal(rows_of(q.values, at).float().double(), v)
    assert_within(q.scales[at], c, U32 * c, "scales")
    y = ops.dequantize_block8(q)
    f = v * spread(q.scales[at].double(), 1, len(at), cols)
    assert_within(y[at], f, (U16 * (1 + U32) + U32) * f.abs(), "y")
    del q, y
    q = ops.quantize_block8(x, block_rows=128, pow2=True)
    y = ops.dequantize_block8(q)
    for b in sorted({int(r) // 128 for r in at}):
        part = slice(b * 128, min(b * 128 + 128, rows))
        v, c = quantized(x[part], 128, E4M3, True)
        assert torch.equal(rows_of(q.values, part).float().double(), v) and torch.equal(q.scales[b].double(), c[0])
        assert torch.equal(y[part].double(), v * spread(c, 128, *v.shape))


def check_gradient_rows(dx, dy, f, mean, rstd, w, dh, at):
    H = f.shape[-1]
    m, s, d = mean[at].double()[:, None], rstd[at].double()[:, None], dy[at].double()
    xh, g = (f - m) * s, d * w.double()
    m1, m2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    want = s * (g - m1 - xh * m2) + dh[at].double()
    n = 2 * (H + 16) * U32
    err = s * (4 * U32 * (g.abs() + m1.abs()) + n * g.abs().mean(-1, keepdim=True)
               + xh.abs() * (n * (g * xh).abs().mean(-1, keepdim=True) + 6 * U32 * m2.abs())) + 8 * U32 * (want.abs() + dh[at].double().abs())
    assert_within(dx[at], want, err + U16 * (want.abs() + err), "dx")


def test_layer_norm_to_blocks_and_its_gradient():
    rows, hidden = 270000, 16384
    x, r, w, b = big(rows, hidden, seed=2), big(rows, hidden, seed=3), rand((hidden,), 4), rand((hidden,), 5)
    at = marks(rows, hidden)
    got = ops.layer_norm(x, w, b, residual=r, out_dtype=E4M3, keep_stats=True, keep_dtype=E5M2)
    h, mu, rstd, y, e_mu, e_rstd, e_y = norm64(x[at], r[at], w, b)
    assert torch.equal(got.residual[at], h)
    check_blocks(ops.Block8Tensor(rows_of(got.y.values, at), got.y.scales[at], 1), y, e_y, E4M3)
    assert_within(got.mean[at], mu, e_mu, "mean")
    assert_within(got.rstd[at], rstd, e_rstd, "rstd")
    v, c = quantized(h, 1, E5M2, True)
    assert torch.equal(rows_of(got.kept.values, at).float().double(), v) and torch.equal(got.kept.scales[at].double(), c)
    dx, dw, db = ops.layer_norm_backward(x, got.kept, w, got.mean, got.rstd, d_residual=r)
    check_gradient_rows(dx, x, v * spread(c, 1, len(at), hidden), got.mean, got.rstd, w, r, at)
    assert torch.isfinite(dw.float()).all() and torch.isfinite(db.float()).all()


def test_layer_norm_of_odd_rows_and_its_gradient():
    rows, hidden = 270000, 16001                         # 4.3e9 values in rows that start inside vectors
    x, r, w, b = big(rows, hidden, seed=6), big(rows, hidden, seed=7), rand((hidden,), 8), rand((hidden,), 9)
    at = marks(rows, hidden)
    got = ops.layer_norm(x, w, b, residual=r, keep_stats=True)
    h, mu, rstd, y, e_mu, e_rstd, e_y = norm64(x[at], r[at], w, b)
    assert torch.equal(got.residual[at], h)
    assert_within(got.y[at], y, e_y + U16 * (y.abs() + e_y), "y")
    dx, dw, db = ops.layer_norm_backward(x, got.residual, w, got.mean, got.rstd, d_residual=r)
    check_gradient_rows(dx, x, h.double(), got.mean, got.rstd, w, r, at)
    assert torch.isfinite(dw.float()).all() and torch.isfinite(db.float()).all()


def check_rows(D, a, y, at, k):
    """Rows `at` of D against those of the values a (64 bits) times y.T."""
    want, mag = lc.product(a, y)
    assert_within(D[at], want, lc.product_bound(want, mag, k), "D")


def some_blocks(rows, cols, block_rows, seed):
    """A large matrix in 8-bit blocks without its 16-bit form: finite bytes, scales around 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    values = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    for part in values.split(1 << 16):
        part.random_(0, 112, generator=g)                # e4m3 up to 1.75 * 2^6
    scales = torch.empty((-(-rows // block_rows), cols // 128), device="cuda").uniform_(0.5, 2.0, generator=g)
    return ops.Block8Tensor(values.view(E4M3), scales, block_rows)


def test_products():
    rows, k = 270000, 16384
    a, w = some_blocks(rows, k, 1, 10), ops.quantize_block8(rand((64, k), 11), block_rows=128)
    at = marks(rows, k)
    part = rows_of(a.values, at).float().double() * spread(a.scales[at].double(), 1, len(at), k)
    check_rows(ops.block8_matmul(a, w), part, values64(w), at, k)        # values past 2^32
    few = ops.quantize_block8(rand((5, k), 12))
    D = ops.block8_matmul(few, a)                                            # as the weights of few rows
    check_rows(D.t(), part, values64(few), at, k)
    del a, D
    tall = some_blocks(rows, k, 128, 13)                                     # summed over its rows
    left = ops.quantize_block8(rand((rows, 16), 14), block_rows=128)
    cols = torch.tensor([0, 127, 128, k - 1], device="cuda")
    y = torch.stack([tall.values.view(torch.uint8)[:, int(c)].contiguous().view(E4M3).float().double()
                     * tall.scales[:, int(c) // 128].double().repeat_interleave(128)[:rows] for c in cols])
    for few_rows in (False, True):
        if few_rows:                                                         # 16 rows, not transposed: K = rows
            a16 = ops.quantize_block8(rand((16, rows), 15))
            D, x = ops.block8_matmul(a16, tall, trans_b=False), values64(a16)
        else:
            D, x = ops.block8_matmul(left, tall, trans_a=True, trans_b=False), values64(left).t()
        want, mag = lc.product(x, y)
        assert_within(D[:, cols], want, lc.product_bound(want, mag, rows), "D")
    del tall, left, D
    a, b = ops.quantize_block8(rand((rows, 128), 16)), ops.quantize_block8(rand((k, 128), 17), block_rows=128)
    check_rows(ops.block8_matmul(a, b), values64(a)[at], values64(b), at, 128)   # a result past 2^32
    ops.check_products()


def test_kept_rows():
    T, K, N = 540000, 8192, 64
    kept = some_blocks(T, K, 1, 18)
    dd = big(T, N, seed=19, std=0.1)
    B = torch.empty((2, N, K), dtype=BF16, device="cuda").transpose(1, 2)
    ends = torch.tensor([T - 300, T], dtype=torch.int32, device="cuda")
    dB = ops.grouped_matmul_backward(dd, kept, B, ends, need=(False, True))[1]
    tail = slice(T - 300, T)
    # the values as they enter: rounded to bf16
    v = (rows_of(kept.values, tail).float() * spread(kept.scales[tail], 1, 300, K)).to(BF16)
    want, mag = lc.product(v.t(), dd[tail].t())
    assert_within(dB[1], want, lc.product_bound(want, mag, 300), "dB")
    head = torch.tensor([0, 1, 4095, K - 1], device="cuda")
    cols = [(kept.values.view(torch.uint8)[: T - 300, int(c)].contiguous().view(E4M3).float()
             * kept.scales[: T - 300, int(c) // 128]).to(BF16) for c in head]
    want, mag = lc.product(torch.stack(cols), dd[: T - 300].t())
    assert_within(dB[0][head], want, lc.product_bound(want, mag, T - 300), "dB of the long group")
    ops.check_products()
