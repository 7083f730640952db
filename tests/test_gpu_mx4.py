"""Microscaled 4 bits on the GPU: codes and scales bit for bit against an
independent encoder, the way back, and the block-scaled product element by
element against the 64-bit form."""

import numpy as np
import pytest
import torch

from reduce_scatter_gb300 import dg, ops
from tests import layer_common as lc
from tests.layer_common import assert_within, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def unpack(codes):
    c = codes.cpu().numpy()
    out = np.empty((c.shape[0], c.shape[1] * 2), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = c & 15, c >> 4
    return out


def check_codes(x, q):
    want, byte = lc.mx4_encode(x.double().cpu().numpy())
    assert (q.rows, q.cols) == tuple(x.shape)
    assert np.array_equal(q.scales.cpu().numpy(), lc.mx4_tiled(byte))
    assert np.array_equal(unpack(q.codes), want)
    return want, byte


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (127, 256), (128, 288), (129, 96), (300, 1056), (1, 8192),
                                       (1000, 1024), (4200, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_scales_and_back(rows, cols, dtype):
    x = rand((rows, cols), 1, dtype=dtype) * torch.exp(rand((cols,), 2, 3.0, F32)).to(dtype)
    q = ops.quantize_mx4(x)
    code, byte = check_codes(x, q)
    v = lc.mx4_values(code, byte)
    for out in (BF16, F32):
        got = ops.dequantize_mx4(q, out_dtype=out)
        assert got.dtype == out and np.array_equal(got.double().cpu().numpy(), v)


def test_every_tie_saturation_and_extreme():
    # every bf16 magnitude of two octaves beside a maximum that fixes the scale: all the ties, both signs
    m = torch.arange(0x3e00, 0x4100, dtype=torch.int32).to(torch.int16).view(BF16)
    rows = []
    for part in m.split(31):
        for sign in (1.0, -1.0):
            r = torch.full((32,), 7.0, dtype=BF16)   # scale 1; 7 saturates to 6
            r[: part.numel()] = part * sign
            rows.append(r)
    x = torch.stack(rows).cuda()
    check_codes(x, ops.quantize_mx4(x))
    tiny = torch.finfo(BF16).tiny
    y = torch.zeros((8, 64), dtype=BF16)
    y[0, 0], y[1, 5] = torch.finfo(BF16).max, -torch.finfo(BF16).max
    y[2, 1], y[2, 2] = tiny, tiny / 4                # the smallest normal value, a subnormal
    y[3, 33] = tiny * 8
    y[4, 0], y[4, 40] = float("nan"), 1.0
    y[5, 31], y[5, 32] = float("inf"), -2.0
    y[6, 7] = -0.0
    y[7] = 2.0 ** -120
    y = y.cuda()
    q = ops.quantize_mx4(y)
    code, byte = check_codes(y, q)
    got = ops.dequantize_mx4(q, out_dtype=F32).double().cpu().numpy()
    assert np.array_equal(got, lc.mx4_values(code, byte), equal_nan=True)
    assert np.isnan(got[4, :32]).all() and got[4, 40] == 1 and np.isnan(got[5, :32]).all() and got[5, 32] == -2
    z = torch.zeros((2, 32), device="cuda")
    z[0, 0], z[1, 0] = 1e-40, 3e38                   # an fp32 subnormal, nearly the largest
    check_codes(z, ops.quantize_mx4(z))


def test_strides_shapes_streams_and_refusals():
    big = rand((2, 5, 320), 3)
    x = big[:, 1:4, 32:288]
    q = ops.quantize_mx4(x)
    check_codes(x.reshape(6, 256), q)
    off = rand((4, 65), 4)[:, 1:]                    # misaligned rows
    check_codes(off, ops.quantize_mx4(off))
    pitched = rand((6, 96), 5)[:, :64]
    check_codes(pitched, ops.quantize_mx4(pitched))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q2 = ops.quantize_mx4(x)
    s.synchronize()
    assert torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)
    e = ops.quantize_mx4(x[:0])
    assert e.rows == 0 and ops.dequantize_mx4(e).shape == (0, 256)
    with pytest.raises(ValueError):
        ops.quantize_mx4(rand((2, 48), 6))
    with pytest.raises(ValueError):
        ops.dequantize_mx4(q, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        ops.mx4_matmul(q, ops.quantize_mx4(rand((8, 64), 7)))
    with pytest.raises(dg.DGError) as err:
        ops.mx4_matmul(ops.quantize_mx4(rand((4, 64), 8)), ops.quantize_mx4(rand((12, 64), 9)))
    assert err.value.code == dg.ERR_SHAPE


# (M, N, K): tiles of 192 (even and odd) x 256, K blocks of 256 with ragged ends
SHAPES = [(1, 8, 32), (8, 256, 256), (33, 264, 288), (192, 256, 512), (193, 520, 96), (400, 136, 1056), (577, 768, 2048),
          (64, 1000, 4096), (1000, 1304, 320), (2, 512, 28672)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", [BF16, F32])
def test_product(M, N, K, out):
    a = rand((M, K), 11) * torch.exp(rand((K,), 12, 1.5, F32)).to(BF16)
    b = rand((N, K), 13, 0.02)
    qa, qb = ops.quantize_mx4(a), ops.quantize_mx4(b)
    d = ops.mx4_matmul(qa, qb, out_dtype=out)
    ops.check_products()
    v, m = lc.product(ops.dequantize_mx4(qa, out_dtype=F32), ops.dequantize_mx4(qb, out_dtype=F32))
    assert d.dtype == out
    assert_within(d, v, lc.product_bound(v, m, K, out == BF16), "D")


def test_scales_reach_their_rows_and_blocks():
    # codes of 1 with scales that name the row and block: exact sums show any misplaced scale
    M, N, K = 200, 300 // 8 * 8, 1024
    for which in range(2):
        a, b = torch.ones((M, K), device="cuda"), torch.ones((N, K), device="cuda")
        t = a if which == 0 else b
        r = torch.arange(t.shape[0], device="cuda")[:, None]
        j = torch.arange(K // 32, device="cuda")[None, :]
        e = (r * 7 + j * 5) % 13 - 6
        t.view(t.shape[0], -1, 32).mul_(torch.exp2(e.double()).float()[..., None])
        qa, qb = ops.quantize_mx4(a), ops.quantize_mx4(b)
        d = ops.mx4_matmul(qa, qb, out_dtype=F32)
        assert torch.equal(d.double(), a.double() @ b.double().t()), which


def test_nan_blocks_and_empty():
    a, b = rand((5, 256), 14), rand((16, 256), 15)
    a[2, 40], b[3, 200] = float("nan"), float("inf")
    d = ops.mx4_matmul(ops.quantize_mx4(a), ops.quantize_mx4(b)).float()
    bad = torch.zeros((5, 16), dtype=torch.bool, device="cuda")
    bad[2], bad[:, 3] = True, True
    assert torch.equal(torch.isnan(d), bad)
    assert ops.mx4_matmul(ops.quantize_mx4(a[:0]), ops.quantize_mx4(b)).shape == (0, 16)


def test_cut_tiles_same_bits():
    # a long K over few tiles is cut among the SM pairs and joined in the order of K
    a, w = ops.quantize_mx4(rand((3, 16384), 18)), ops.quantize_mx4(rand((520, 16384), 19))
    want = ops.mx4_matmul(a, w, out_dtype=F32)
    v, m = lc.product(ops.dequantize_mx4(a, out_dtype=F32), ops.dequantize_mx4(w, out_dtype=F32))
    assert_within(want, v, lc.product_bound(v, m, 16384, False), "D")
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for turn in range(12):
        with torch.cuda.stream(streams[turn % 3]):
            got.append(ops.mx4_matmul(a, w, out_dtype=F32))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    ops.check_products()


def test_graph_and_stream():
    a, w = rand((50, 512), 16), ops.quantize_mx4(rand((264, 512), 17))
    want = ops.mx4_matmul(ops.quantize_mx4(a), w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ops.mx4_matmul(ops.quantize_mx4(a), w)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d2 = ops.mx4_matmul(ops.quantize_mx4(a), w)
    s.synchronize()
    assert torch.equal(d2, want)
