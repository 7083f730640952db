"""8-bit tensors with a scale for each block of 128 on the GPU, against the
definition in 64 bits: quantisation bit by bit, values, products in every
orientation; edges, special values, streams, graphs."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests import layer_common as lc
from tests.layer_common import U16, U32, assert_within, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
FP8 = {E4M3: (448.0, 3, -6), E5M2: (57344.0, 2, -14)}  # largest finite, mantissa bits, least exponent


def spread(scales, block_rows, rows, cols):
    """A block's scale at each of its values."""
    s = scales.repeat_interleave(128, 1)[:, :cols]
    return s if block_rows == 1 else s.repeat_interleave(block_rows, 0)[:rows]


def pow2(e):
    """2^e in 64 bits, exactly (torch.ldexp goes through pow, which is not exact on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def nearest8(v, dtype):
    """64-bit values on the type's grid, ties to even, saturating."""
    top, mant, emin = FP8[dtype]
    _, ex = torch.frexp(v)
    step = pow2((ex - 1).clamp(min=emin) - mant)
    return (torch.round(v / step) * step).clamp(-top, top)


def quantized(x, block_rows, dtype, powers):
    """(values, scales) of the definition, in 64 bits."""
    top = FP8[dtype][0]
    f = x.double()
    fin = torch.where(torch.isfinite(f), f.abs(), torch.zeros_like(f))
    rows, cols = f.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    amax = torch.nn.functional.pad(fin, (0, bc * 128 - cols, 0, br * block_rows - rows)).view(br, block_rows, bc, 128).amax((1, 3))
    c = amax / top
    if powers:
        m, e = torch.frexp(c)
        c = pow2(torch.where(m == 0.5, e - 1, e))
    low = c <= 2.0 ** -126
    c = torch.where(amax == 0, 1.0, torch.where(low, 2.0 ** -126, c))
    each = spread(c, block_rows, rows, cols)
    v = f / each
    if not powers:
        a = spread(torch.where(low, top * 2.0 ** -126, amax), block_rows, rows, cols)
        v = torch.where(spread(amax == 0, block_rows, rows, cols), v, f * top / a)
    return torch.where(torch.isfinite(f), nearest8(v, dtype), torch.nan), c


QSIZES = [(1, 16), (3, 128), (130, 144), (128, 256), (257, 1040), (33, 8192), (1, 28672), (640, 4112)]


@pytest.mark.parametrize("rows,cols", QSIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("xt,powers", [(BF16, False), (BF16, True), (F32, False), (F32, True)])
def test_quantize(rows, cols, block_rows, dtype, xt, powers):
    # magnitudes that differ from row to row and from block to block; a block of zeros
    x = rand((rows, cols), 1, dtype=F32) * torch.exp(2 * rand((rows, 1), 2, dtype=F32)) * torch.exp(2 * rand((1, cols), 3, dtype=F32))
    x = x.to(xt)
    x[:128, :128] *= 0 if rows > 128 else 1
    q = ops.quantize_block8(x, block_rows=block_rows, dtype=dtype, pow2=powers)
    want, c = quantized(x, block_rows, dtype, powers)
    assert q.values.dtype == dtype and q.values.shape == x.shape and q.scales.shape == c.shape and q.block_rows == block_rows
    if powers:
        assert torch.equal(q.scales.double(), c)
    else:
        assert_within(q.scales, c, U32 * c, "scales")
    got = q.values.float().double()
    if xt == BF16 or powers:
        assert torch.equal(got, want)
    else:  # x top is rounded to fp32 first: a value that close to halfway may go either way
        step = torch.maximum(want.abs() * 2.0 ** -FP8[dtype][1], torch.full_like(want, 2.0 ** (FP8[dtype][2] - FP8[dtype][1])))
        v = x.double() / spread(c, block_rows, rows, cols)
        assert_within(got, v, step / 2 * (1 + 4 * U32) + v.abs() * 4 * U32, "values")
        assert (got != want).double().mean() < 1e-4


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("powers", [False, True])
def test_quantize_special_values(block_rows, dtype, powers):
    x = rand((256, 272), 4, dtype=F32)
    x[0, 0], x[1, 1], x[2, 130] = float("nan"), float("inf"), -float("inf")
    x[128:, :128] = float("nan")
    x[128:, 128:256] *= 2.0 ** -140          # below the least scale
    x[:128, 256:] *= 2.0 ** 124 / x[:128, 256:].abs().max()
    x[:128, 128:256] *= 2.0 ** 120
    q = ops.quantize_block8(x, block_rows=block_rows, dtype=dtype, pow2=powers)
    want, c = quantized(x, block_rows, dtype, powers)
    got = q.values.float().double()
    assert torch.equal(torch.isnan(got), ~torch.isfinite(x))
    assert_within(q.scales, c, U32 * c, "scales")
    ok = torch.isfinite(x)
    assert (got[ok] != want[ok]).double().mean() < 1e-4
    assert (q.scales[-1, 0] == 1) and (q.scales[-1, 1] == 2.0 ** -126)


@pytest.mark.parametrize("rows,cols", QSIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("out", [BF16, F32])
def test_dequantize(rows, cols, block_rows, out):
    for dtype, powers in ((E4M3, False), (E5M2, True)):
        q = ops.quantize_block8(rand((rows, cols), 5), block_rows=block_rows, dtype=dtype, pow2=powers)
        want = q.values.float().double() * spread(q.scales.double(), block_rows, rows, cols)
        got = ops.dequantize_block8(q, out_dtype=out)
        if powers:
            assert torch.equal(got.double(), want)
        else:
            assert_within(got, want, ((U16 * (1 + U32) if out == BF16 else 0) + U32) * want.abs(), "y")


def values64(q):
    return q.values.float().double() * spread(q.scales.double(), q.block_rows, *q.values.shape)


def check_product(a, b, ta, tb, out):
    got = ops.block8_matmul(a, b, trans_a=ta, trans_b=tb, out_dtype=out)
    x, y = values64(a), values64(b)
    x, y = x.t() if ta else x, y if tb else y.t()
    want, mag = lc.product(x, y)
    assert got.dtype == out and got.shape == want.shape
    assert_within(got, want, lc.product_bound(want, mag, x.shape[1], out == BF16), "D")
    return got


SIZES = [(1, 8, 16), (5, 16, 128), (129, 264, 144), (256, 256, 128), (300, 520, 1040), (8, 2048, 8192), (1000, 3328, 8208),
         (513, 1032, 2048), (64, 256, 4096), (2049, 776, 528)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("abr,bbr", [(1, 128), (128, 128), (1, 1), (128, 1)])
def test_product(m, n, k, abr, bbr):
    a = ops.quantize_block8(rand((m, k), 6) * torch.exp(rand((m, 1), 7)), block_rows=abr)
    b = ops.quantize_block8(rand((n, k), 8) * torch.exp(rand((n, 1), 9)), block_rows=bbr, dtype=E5M2 if m == 300 else E4M3)
    check_product(a, b, False, True, BF16 if m % 2 else F32)
    ops.check_products()


@pytest.mark.parametrize("m,n,k", [(1, 256, 4096), (16, 8, 128), (17, 264, 272), (33, 520, 8192), (48, 2048, 1040), (65, 13312, 2064),
                                   (96, 128, 28672), (127, 3328, 4112), (128, 1032, 128), (128, 20000, 512)])
@pytest.mark.parametrize("abr,bbr,tb", [(1, 128, True), (1, 1, True), (128, 128, False), (128, 1, True), (1, 128, False)])
def test_product_of_few_rows(m, n, k, abr, bbr, tb):
    if not tb:
        n = (n + 15) // 16 * 16
    a = ops.quantize_block8(rand((m, k), 30) * torch.exp(rand((m, 1), 31)), block_rows=abr, dtype=E5M2 if m == 33 else E4M3)
    b = ops.quantize_block8(rand((n, k) if tb else (k, n), 32) * torch.exp(rand((n if tb else k, 1), 33)), block_rows=bbr)
    first = check_product(a, b, False, tb, BF16)
    check_product(a, b, False, tb, F32)
    assert torch.equal(first, ops.block8_matmul(a, b, trans_b=tb))
    ops.check_products()


@pytest.mark.parametrize("m,n,k", [(16, 16, 16), (128, 256, 128), (272, 528, 1000), (1024, 304, 130), (400, 2048, 8192), (2064, 784, 528)])
@pytest.mark.parametrize("ta,tb", [(True, True), (False, False), (True, False)])
def test_product_of_transposes(m, n, k, ta, tb):
    k = (k + 15) // 16 * 16 if not ta or tb else k
    a = ops.quantize_block8(rand((k, m) if ta else (m, k), 10) * torch.exp(rand((k if ta else m, 1), 11)), block_rows=128, dtype=E5M2)
    b = ops.quantize_block8(rand((n, k) if tb else (k, n), 12) * torch.exp(rand((n if tb else k, 1), 13)), block_rows=128)
    check_product(a, b, ta, tb, BF16)
    check_product(a, b, ta, tb, F32)
    ops.check_products()


def test_product_of_special_values():
    x, w = rand((40, 512), 14), rand((64, 512), 15)
    x[3, 7] = float("nan")
    x[9] = 0
    a, b = ops.quantize_block8(x), ops.quantize_block8(w, block_rows=128)
    d = ops.block8_matmul(a, b)
    assert torch.isnan(d[3]).all() and not d[9].any()
    rest = torch.arange(40, device="cuda") != 3
    clean = ops.block8_matmul(ops.quantize_block8(x.nan_to_num()), b)
    assert torch.equal(d[rest], clean[rest])
    # scales far from 1: their product is formed first
    big = ops.Block8Tensor(a.values, a.scales * 2.0 ** 90, 1)
    small = ops.Block8Tensor(b.values, b.scales * 2.0 ** -90, 128)
    assert torch.equal(ops.block8_matmul(big, small)[rest], d[rest])


def test_scales_of_any_strides_and_views():
    a, b = ops.quantize_block8(rand((70, 400), 16)), ops.quantize_block8(rand((136, 400), 17), block_rows=128)
    want = ops.block8_matmul(a, b)
    rows = ops.Block8Tensor(a.values, a.scales.t().contiguous().t(), 1)
    wide = torch.full((4, 9), float("nan"), device="cuda")
    wide[::2, 1::2] = b.scales
    assert torch.equal(ops.block8_matmul(rows, ops.Block8Tensor(b.values, wide[::2, 1::2], 128)), want)
    shared = ops.Block8Tensor(a.values, torch.ones((), device="cuda").expand(70, 4), 1)
    check_product(shared, b, False, True, F32)
    off = torch.empty(70 * 400 + 8, dtype=torch.uint8, device="cuda")[8:].view(70, 400).copy_(a.values.view(torch.uint8)).view(E4M3)
    assert torch.equal(ops.block8_matmul(ops.Block8Tensor(off, a.scales, 1), b), want)
    assert torch.equal(ops.dequantize_block8(ops.Block8Tensor(off, a.scales, 1)), ops.dequantize_block8(a))
    x = rand((12, 6, 300), 18)
    part = x[:, 1:4, 8:264]                               # rows that start and step off 16-byte boundaries, two row pitches
    q, r = ops.quantize_block8(part), ops.quantize_block8(part.contiguous().view(36, 256))
    assert torch.equal(q.values.view(torch.uint8), r.values.view(torch.uint8)) and torch.equal(q.scales, r.scales)


def test_nothing():
    a, b = ops.quantize_block8(rand((0, 256), 19)), ops.quantize_block8(rand((24, 256), 20), block_rows=128)
    assert ops.block8_matmul(a, b).shape == (0, 24)
    assert ops.dequantize_block8(a).shape == (0, 256)
    none = ops.quantize_block8(rand((5, 0), 21))
    assert none.scales.shape == (5, 0)
    d = ops.block8_matmul(none, ops.quantize_block8(rand((24, 0), 22)))
    assert d.shape == (5, 24) and not d.any()
    tall = ops.quantize_block8(rand((0, 32), 23), block_rows=128)
    assert not ops.block8_matmul(tall, tall, trans_a=True, trans_b=False).any()


def test_streams_graphs_and_repetition():
    x, w = rand((200, 4096), 24), rand((512, 4096), 25)
    b = ops.quantize_block8(w, block_rows=128)
    want = ops.block8_matmul(ops.quantize_block8(x), b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = [ops.block8_matmul(ops.quantize_block8(x), b) for _ in range(3)]
    here = [ops.block8_matmul(ops.quantize_block8(x), b) for _ in range(3)]  # at the same time, in another workspace
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs + here)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.block8_matmul(ops.quantize_block8(x), b)
    for seed in (26, 27):
        x.copy_(rand(x.shape, seed))
        graph.replay()
        also = ops.block8_matmul(ops.quantize_block8(x), b)
        assert torch.equal(got, also)
    ops.check_products()


@pytest.mark.parametrize("m", [5, 128, 300])
def test_scales_whose_product_alone_is_in_range(m):
    # 2^120 and 2^-120: the scales are multiplied with each other first, whichever blocks they belong to
    for a_rows, b_rows in ((1, 1), (128, 1), (1, 128), (128, 128)):
        a = ops.quantize_block8(rand((m, 512), 60), block_rows=a_rows, pow2=True)
        b = ops.quantize_block8(rand((272, 512), 61), block_rows=b_rows, pow2=True)
        want = check_product(a, b, False, True, F32)
        for e in (120, -120):
            far = ops.Block8Tensor(a.values, a.scales * 2.0 ** e, a_rows)
            assert torch.equal(ops.block8_matmul(far, ops.Block8Tensor(b.values, b.scales * 2.0 ** -e, b_rows), out_dtype=F32), want)
    ops.check_products()


@pytest.mark.parametrize("m,n,k", [(129, 128, 512), (600, 1000, 1040), (2048, 8, 4096)])
def test_column_scales_of_any_strides(m, n, k):
    a, b = ops.quantize_block8(rand((m, k), 62)), ops.quantize_block8(rand((n, k), 63) * torch.exp(rand((n, 1), 64)))
    want = check_product(a, b, False, True, BF16)
    blocks = b.scales.shape[1]
    for scales in (b.scales.contiguous(), torch.full((n, 2 * blocks + 1), float("nan"), device="cuda")[:, 1::2].copy_(b.scales),
                   torch.empty(blocks * (n + 1) + 1, device="cuda")[1:].view(blocks, n + 1)[:, :n].t().copy_(b.scales)):
        assert torch.equal(ops.block8_matmul(a, ops.Block8Tensor(b.values, scales, 1)), want)
    ops.check_products()
