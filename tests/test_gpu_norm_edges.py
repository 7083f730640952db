"""Residual add + RMS norm on the GPU at the edges: values near the ends of
fp32's range, in-place sums and the tensors they touch, host threads, rows of
no values, special rows among streamed ones."""

import threading

import pytest
import torch

from reduce_scatter_gb300 import dg, layer, ops
from tests import layer_common as lc
from tests.layer_common import U16, U32, assert_within, rand
from tests.test_gpu_layer_norm import FP8

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LEAST = 2.0 ** -126                                   # the least row scale

# rows x hidden of every forward kernel: registers (one warp, 1, 2 and 8 vectors), element-wise (4 and 16 values),
# looping (vectors and elements), streamed
PATHS = [(5, 256), (3, 8192), (2, 16384), (2, 24576), (4, 259), (3, 4099), (2, 40000), (2, 40001), (700, 2048), (400, 16384)]


def check_q(q, scale, y, hidden, dtype):
    """q * scale within half a step of y (the step: 2^-mantissa of the value, at least the subnormal one), beside the
    relative errors of rstd and four more roundings, and 2^-22: the products before the last factor (at most 2^127)
    may be subnormal, off by 2^-150."""
    top, mant, emin = FP8[dtype]
    rel = lc.norm_rel(hidden) + 4 * U32
    want = (y / scale.double()[..., None]).clamp(-top, top)
    step = torch.maximum(want.abs() * 2.0 ** -mant, torch.full_like(want, 2.0 ** (emin - mant)))
    assert_within(q.float(), want, step / 2 * (1 + rel) + want.abs() * rel + 2.0 ** -22, "q")


def patterned(rows, hidden, size):
    """Rows of 0, 1/4, 1/2 and 1 with both signs, times `size` of each row's turn."""
    at = torch.arange(hidden, device="cuda")
    row = torch.tensor([0.0, 0.25, 0.5, 1.0], device="cuda")[at % 4] * torch.where(at % 8 < 4, 1.0, -1.0)
    sizes = torch.tensor([size[i % len(size)] for i in range(rows)], dtype=torch.float64, device="cuda")
    return sizes[:, None] * row


@pytest.mark.parametrize("rows,hidden", PATHS)
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_values_near_the_ends_of_the_range(rows, hidden, dtype):
    # products h w far below 1 and above fp32's range: the values that they stand for are finite, zeros stay zeros
    for size, w in (([1e-38, 1e-40, 1e-37, 1e-36, 1e-34], 1.0), ([1e-35, 1e-33, 1e-30], 0.75), ([1e-18, 1e-20], 1e-19),
                    ([1e12, 3e18 / hidden ** 0.5, 1.0], 1e30)):
        x = patterned(rows, hidden, size).to(BF16)
        weight = torch.full((hidden,), w, device="cuda")
        for r in (None, torch.zeros_like(x), torch.zeros((rows, hidden), device="cuda")):
            got = ops.add_rms_norm(x, weight, residual=r, out_dtype=dtype)
            _, _, y = lc.norm(x, weight, r)
            want = (y.abs().amax(-1) / FP8[dtype][0]).clamp(min=LEAST)
            assert_within(got.scale, want, (lc.norm_rel(hidden) + 2 * U32) * want, "scale")
            check_q(got.y, got.scale, y, hidden, dtype)
            assert not got.y.float()[y == 0].any()


@pytest.mark.parametrize("rows,hidden", PATHS)
def test_given_scales_near_the_ends_of_the_range(rows, hidden):
    # (1e-38 and 1e-40 are subnormal)
    for s, size in ((1e-37, [1e-37, 3e-38]), (1e-38, [1e-38]), (1e-40, [1.2e-40]), (1e30, [1.0]), (1e-3, [1e-3, 1.0, 50.0])):
        x = patterned(rows, hidden, size).to(BF16)
        weight = torch.full((hidden,), 1.0 if s < 1 else 1e32, device="cuda")
        scale = torch.tensor([s], dtype=F32, device="cuda")
        got = ops.add_rms_norm(x, weight, out_dtype=E4M3, scale=scale)
        _, _, y = lc.norm(x, weight)
        check_q(got.y, scale.expand(rows), y, hidden, E4M3)
        assert not got.y.float()[y == 0].any()


def test_ordinary_rows_keep_their_bits():
    # a power of two in the row changes the scale by it and nothing else, where eps does not count
    x, w = rand((700, 2048), 101), rand((2048,), 102)
    want = ops.add_rms_norm(x, w, eps=0.0, out_dtype=E4M3)
    for e in (-30, -6, 1, 8, 40):
        got = ops.add_rms_norm(x * 2.0 ** e, w, eps=0.0, out_dtype=E4M3)
        assert torch.equal(got.y.view(torch.uint8), want.y.view(torch.uint8)) and torch.equal(got.scale, want.scale), e


def test_in_place_sum_is_seen_by_autograd():
    x, w = rand((6, 64), 111), rand((64,), 112)
    r = rand((6, 64), 113)
    weight = rand((32, 64), 114).requires_grad_()
    out = torch.nn.functional.linear(r, weight)           # saves r
    before = r._version
    with torch.no_grad():
        ops.add_rms_norm(x, w, residual=r, inplace=True)
    assert r._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    # the norm's own saved sum
    xs = x.clone().requires_grad_()
    n = ops.add_rms_norm(xs, w, residual=r)
    with torch.no_grad():
        ops.add_rms_norm(x, w, residual=n.residual, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        n.y.sum().backward()
    with torch.inference_mode():                           # tensors without a version
        t = r.clone()
        assert ops.add_rms_norm(x, w, residual=t, inplace=True).residual is t
    keep = t.clone()
    with torch.no_grad(), pytest.raises(RuntimeError):
        ops.add_rms_norm(x, w, residual=t, inplace=True)   # as torch's own in-place operations
    assert torch.equal(t, keep)


def test_in_place_sum_refuses_shared_memory():
    x, w = rand((4, 64), 121), rand((64,), 122)
    buf = rand((5, 64), 123)
    keep = buf.clone()
    for r, xx, ww in ((buf[:1].expand(4, 64), x, w),                    # one row for all
                      (buf.view(-1).as_strided((4, 64), (32, 1)), x, w),  # rows that overlap
                      (buf[1:], buf[:4], w),                            # the sum of a row is the next row's x
                      (buf[1:], x, buf[2])):                            # a row of it is the weight
        with pytest.raises(ValueError):
            ops.add_rms_norm(xx, ww, residual=r, inplace=True)
    torch.cuda.synchronize()
    assert torch.equal(buf, keep)
    # the same tensor twice, and columns of one matrix, do not overlap
    h, _, _ = lc.norm(buf, w, buf)
    ops.add_rms_norm(buf, w, residual=buf, inplace=True)
    assert torch.equal(buf, h)
    both = rand((4, 128), 124)
    h, _, _ = lc.norm(both[:, :64], w, both[:, 64:])
    ops.add_rms_norm(both[:, :64], w, residual=both[:, 64:], inplace=True)
    assert torch.equal(both[:, 64:], h)
    one = rand((1, 64), 125)
    row = one.as_strided((1, 64), (3, 1))                               # a single row has no pitch
    h, _, _ = lc.norm(x[:1], w, row)
    ops.add_rms_norm(x[:1], w, residual=row, inplace=True)
    assert torch.equal(one, h)


def test_long_and_short_rows_from_two_threads():
    # the streamed kernels' shared memory depends on the row; the limit on it is the process's
    L = layer.lib()
    rows, failed = 400, []

    def calls(hidden):
        x, r, dy = (rand((rows, hidden), 130 + i) for i in range(3))
        w = rand((hidden,), 133)
        y, h, dx, dw = (torch.empty_like(t) for t in (x, x, x, w))
        rstd = torch.empty((rows,), device="cuda")
        ws = torch.empty((L.dg_layer_add_rms_norm_backward_workspace(rows, hidden),), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        stream = torch.cuda.Stream().cuda_stream

        def go():
            for _ in range(2000):
                rc = L.dg_layer_add_rms_norm(x.data_ptr(), hidden, r.data_ptr(), hidden, 0, w.data_ptr(), 0, y.data_ptr(), 0,
                                             h.data_ptr(), hidden, None, None, rstd.data_ptr(), rows, hidden, 1e-5, stream)
                if rc == dg.OK:
                    rc = L.dg_layer_add_rms_norm_backward(dy.data_ptr(), hidden, h.data_ptr(), hidden, 0, w.data_ptr(), 0,
                                                          rstd.data_ptr(), None, 0, dx.data_ptr(), dw.data_ptr(),
                                                          ws.data_ptr(), rows, hidden, stream)
                if rc != dg.OK:
                    failed.append((hidden, rc, L.dg_layer_last_error()))
                    return

        return go

    threads = [threading.Thread(target=calls(hidden)) for hidden in (16384, 2048)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_rows_of_no_values():
    for shape in ((3, 0), (2, 3, 0), (0,)):
        x, w = torch.zeros(shape, dtype=BF16, device="cuda"), torch.zeros((0,), dtype=BF16, device="cuda")
        dirty = torch.full((4096,), 7.0, device="cuda")    # what a fresh allocation may hold
        del dirty
        got = ops.add_rms_norm(x, w, out_dtype=E4M3, keep_rstd=True)
        assert got.y.shape == shape and got.scale.shape == shape[:-1]
        assert (got.scale == 1).all()                      # as of a row of zeros
        assert torch.isnan(got.rstd).all()                 # the mean of nothing
        dx, dw = ops.add_rms_norm_backward(x, x, w, got.rstd)
        assert dx.shape == shape and dw.shape == (0,)
    q = ops.quantize_mx4(torch.zeros((2, 3, 0), dtype=BF16, device="cuda"))
    assert q.rows == 6 and ops.dequantize_mx4(q).shape == (6, 0)
    d = ops.mx4_matmul(q, ops.quantize_mx4(torch.zeros((8, 0), dtype=BF16, device="cuda")))
    assert d.shape == (6, 8) and not d.any()


@pytest.mark.parametrize("rows,hidden", [(700, 2048), (400, 8200)])
@pytest.mark.parametrize("res", [None, BF16, F32])
def test_special_rows_among_streamed_ones(rows, hidden, res):
    # the same rows a few at a time take another kernel, whose results are known
    x, w = rand((rows, hidden), 141), rand((hidden,), 142, dtype=F32)
    r = None if res is None else rand((rows, hidden), 143, 2.0, res)
    x[0] = x[rows // 2] = 0
    x[1, 3] = x[rows - 1, hidden - 1] = float("nan")
    x[2, 3], x[rows - 2, 5] = float("inf"), -float("inf")
    w[7] = 3e38                                            # products beyond fp32 where the row's value is above 1
    if r is not None:
        r[0] = r[rows // 2] = 0
    at = [0, 1, 2, 3, 4, rows // 2, rows - 3, rows - 2, rows - 1]
    for kw in (dict(), dict(scale=0.01)):
        got = ops.add_rms_norm(x, w, residual=r, out_dtype=E4M3, keep_rstd=True, **kw)
        few = ops.add_rms_norm(x[at], w, residual=None if r is None else r[at], out_dtype=E4M3, keep_rstd=True, **kw)
        assert torch.equal(got.residual[at].view(torch.uint8), few.residual.view(torch.uint8))
        # sums of squares are added in another order
        rel = 2 * lc.norm_rel(hidden)
        ok = torch.isfinite(few.rstd)
        assert torch.equal(torch.isfinite(got.rstd[at]), ok)
        assert_within(got.rstd[at][ok], few.rstd[ok].double(), rel * few.rstd[ok].double(), "rstd")
        a, b = got.y.view(torch.uint8)[at].view(E4M3).float(), few.y.float()
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        a, b = torch.nan_to_num(a).double(), torch.nan_to_num(b).double()
        assert_within(a, b, torch.maximum(b.abs() * 2.0 ** -3, torch.full_like(b, 2.0 ** -9)), "q")
        if not kw:
            assert got.scale[0] == 1 and got.scale[1] == 1 and torch.isfinite(got.scale).all()
            assert_within(got.scale[at], few.scale.double(), (rel + 4 * U32) * few.scale.double(), "scale")


@pytest.mark.parametrize("res", [BF16, F32])
def test_streamed_in_place_and_given_scale(res):
    rows, hidden = 700, 2048
    x, w, r = rand((rows, hidden), 151), rand((hidden,), 152), rand((rows, hidden), 153, 2.0, res)
    h, _, y = lc.norm(x, w, r)
    apart = ops.add_rms_norm(x, w, residual=r, out_dtype=E4M3, scale=2.0 ** -6)
    got = ops.add_rms_norm(x, w, residual=r, out_dtype=E4M3, scale=2.0 ** -6, inplace=True)
    assert got.residual is r and torch.equal(r, h) and torch.equal(apart.residual, h)
    assert torch.equal(got.y.view(torch.uint8), apart.y.view(torch.uint8))
    check_q(got.y, torch.full((rows,), 2.0 ** -6, device="cuda"), y, hidden, E4M3)
