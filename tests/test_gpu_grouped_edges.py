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
