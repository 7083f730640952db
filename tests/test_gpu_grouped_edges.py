"""Products grouped by expert on the GPU at the edges: a single expert's
strides, scales of every shape and size, gradients whose tiles are drawn, the
32-bit weight gradient of the C ABI."""

import pytest
import torch

from reduce_scatter_gb300 import dg, layer, ops
from tests import layer_common as lc
from tests.layer_common import assert_within, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def ends_of(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("stride", [1, 0, 64 * 72 + 3])
def test_a_single_expert_has_no_pitch(stride):
    # the stride of a dimension of one is anything
    a, w = rand((20, 64), 1), rand((64 * 72,), 2)
    for b in (w.as_strided((1, 64, 72), (stride, 1, 64)), w.as_strided((1, 64, 72), (stride, 72, 1))):
        d = ops.grouped_matmul(a, b, ends_of([13]))
        want, bound = lc.grouped(a, b, [13])
        assert_within(d, want, bound, "D")
        dd = rand((20, 72), 3)
        da, db = ops.grouped_matmul_backward(dd, a, b, ends_of([13]))
        want, bound = lc.grouped(dd, b.transpose(1, 2), [13])
        assert_within(da, want, bound, "dA")
        want, bound = lc.grouped_weight_grad(dd, a, [13])
        assert_within(db, want, bound, "dB")


def test_a_vector_of_column_scales_is_one_for_each_expert():
    a = rand((9, 64), 11).to(E4M3)
    ends = ends_of([4, 9])
    for n in (8, 16):
        b = rand((2, n, 64), 12).to(E4M3).transpose(1, 2)
        per_expert = torch.tensor([0.5, 2.0], device="cuda")
        d = ops.grouped_matmul(a, b, ends, scale_b=per_expert)
        want, bound = lc.grouped(a, b, [4, 9], sb=per_expert[:, None].expand(2, n))
        assert_within(d, want, bound, "D")
        one = ops.grouped_matmul(a, b, ends, scale_b=torch.tensor(0.5, device="cuda"))
        assert torch.equal(one, ops.grouped_matmul(a, b, ends, scale_b=torch.tensor([0.5], device="cuda")))
        row = torch.rand((1, n), device="cuda")
        assert torch.equal(ops.grouped_matmul(a, b, ends, scale_b=row), ops.grouped_matmul(a, b, ends, scale_b=row.expand(2, n)))
        with pytest.raises(ValueError):
            ops.grouped_matmul(a, b, ends, scale_b=torch.ones(n, device="cuda"))   # (as many as columns)


@pytest.mark.parametrize("a_scale,b_scale", [(2.0 ** -120, 2.0 ** -20), (2.0 ** -126, 2.0 ** -30), (2.0 ** 90, 2.0 ** 50),
                                             (2.0 ** 50, 2.0 ** 90), (2.0 ** -126, 2.0 ** 100), (2.0 ** -70, 1.0), (0.01, 0.003)])
@pytest.mark.parametrize("T,ends", [(7, [1, 5]), (5, [5, 5]), (303, [300, 301])])
def test_products_of_scales_beyond_the_range(T, ends, a_scale, b_scale):
    # scale_a scale_b may underflow or overflow where D does not
    K, N = 64, 40
    if a_scale * b_scale > 1e30:                          # sums of one product 2^-18 keep D in range
        a, b = torch.zeros((T, K), device="cuda"), torch.zeros((2, N, K), device="cuda")
        a[:, 5], b[:, :, 5] = 2.0 ** -9, -2.0 ** -9
    else:
        a, b = (rand(s, 21 + i, 100.0, F32).clamp(-448, 448) for i, s in enumerate(((T, K), (2, N, K))))
    a, b = a.to(E4M3), b.to(E4M3).transpose(1, 2)
    g = torch.Generator(device="cuda").manual_seed(23)
    sa = (1 + torch.rand((T,), device="cuda", generator=g)) * a_scale
    sb = (1 + torch.rand((2, N), device="cuda", generator=g)) * b_scale
    sa[0], sb[0, 3] = 0.0, 0.0
    d = ops.grouped_matmul(a, b, ends_of(ends), scale_a=sa, scale_b=sb, out_dtype=F32)
    want, bound = lc.grouped(a, b, ends, sa, sb, out16=False)
    # beside the sum's and the factors' bound two roundings to the subnormal step, 2^-149
    assert_within(d, want, bound + 2.0 ** -148, "D")
    same = ops.grouped_matmul(a, b, ends_of(ends), scale_a=sa, scale_b=sb)
    assert torch.equal(same, d.to(BF16))


def workspace():
    """A products' workspace of the test's own."""
    return torch.zeros(layer.lib().dg_layer_products_workspace(), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("ends", [[2100, 2100, 4096], [1400, 2800, 4000]])
@pytest.mark.parametrize("f32", [False, True])
def test_weight_gradient_with_drawn_tiles(ends, f32):
    # 192 tiles of 16 and more K blocks over the SM pairs, an empty group's without any; through the C ABI, in both types
    T, N, K, E = 4096, 2048, 2048, len(ends)
    a, dd, e = rand((T, K), 31), rand((T, N), 32), ends_of(ends)
    L = layer.lib()
    ws, status = workspace(), torch.zeros(1, dtype=torch.int64, device="cuda")
    tails = torch.empty(L.dg_layer_grouped_grad_workspace(E, N, K), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    db = [torch.full((E, N, K), 7.0, dtype=F32 if f32 else BF16, device="cuda") for _ in range(3)]
    for out in db:
        assert L.dg_layer_grouped_weight_grad(dd.data_ptr(), N, a.data_ptr(), K, e.data_ptr(), E, out.data_ptr(),
                                              dg.TYPE_F32 if f32 else dg.TYPE_BF16, T, N, K, tails.data_ptr(),
                                              ws.data_ptr(), status.data_ptr(), stream) == dg.OK
    assert L.dg_layer_check(status.data_ptr(), stream) == dg.OK
    start = 0
    for k, end in enumerate(ends):
        v, m = lc.product(dd[start:end].t(), a[start:end].t())
        assert_within(db[0][k], v, lc.product_bound(v, m, end - start, not f32), k)
        start = end
    assert torch.equal(db[0], db[1]) and torch.equal(db[0], db[2])
    assert not ws[:2048].any()
    if not f32:
        got = ops.grouped_matmul_backward(dd, a, torch.empty((E, N, K), dtype=BF16, device="cuda").transpose(1, 2), e,
                                          need=(False, True))[1]
        assert torch.equal(got.transpose(1, 2), db[0])


@pytest.mark.parametrize("T,N,K,ends", [(65, 64, 72, [64, 65]), (300, 264, 200, [0, 100, 100, 131, 300]), (63, 40, 72, [16, 32, 63])])
def test_weight_gradient_in_32_bits(T, N, K, ends):
    a, dd, e, E = rand((T, K), 33), rand((T, N), 34), ends_of(ends), len(ends)
    L = layer.lib()
    ws, status = workspace(), torch.zeros(1, dtype=torch.int64, device="cuda")
    tails = torch.empty(L.dg_layer_grouped_grad_workspace(E, N, K), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    db = torch.full((E, N, K), 7.0, device="cuda")
    assert L.dg_layer_grouped_weight_grad(dd.data_ptr(), N, a.data_ptr(), K, e.data_ptr(), E, db.data_ptr(), dg.TYPE_F32, T,
                                          N, K, tails.data_ptr(), ws.data_ptr(), status.data_ptr(), stream) == dg.OK
    assert L.dg_layer_check(status.data_ptr(), stream) == dg.OK
    want, _ = lc.grouped_weight_grad(dd, a, ends)
    start = 0
    for k, end in enumerate(ends):
        _, m = lc.product(dd[start:end].t(), a[start:end].t())
        assert_within(db[k], want[k].t(), lc.product_bound(want[k].t(), m, end - start, False), k)
        start = end


def test_8bit_rows_with_drawn_tiles():
    # 16 K blocks and more, 11 x 11 tiles and more: drawn; twice on one workspace, whose counters end at zero
    T, N, K, ends = 2400, 2816, 2048, [700, 700, 1500, 2300]
    a, b = rand((T, K), 41, 60.0).to(E4M3), rand((4, N, K), 42, 60.0).to(E4M3)
    L, e = layer.lib(), ends_of(ends)
    ws, status = workspace(), torch.zeros(1, dtype=torch.int64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    want, bound = lc.grouped(a, b.transpose(1, 2), ends)
    for _ in range(2):
        d = torch.full((T, N), 7.0, dtype=BF16, device="cuda")
        assert L.dg_layer_grouped_matmul(a.data_ptr(), K, dg.TYPE_E4M3, b.data_ptr(), K, N * K, dg.TYPE_E4M3, 0, e.data_ptr(),
                                         4, None, 0, None, 0, 0, d.data_ptr(), dg.TYPE_BF16, T, N, K, ws.data_ptr(),
                                         status.data_ptr(), stream) == dg.OK
        assert_within(d, want, bound, "D")
        assert not ws[:2048].any()
    assert L.dg_layer_check(status.data_ptr(), stream) == dg.OK
