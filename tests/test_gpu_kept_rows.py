"""Weight gradients from rows kept in 8 bits, and linear layers in 8-bit blocks
with their gradients, on the GPU against the 64-bit forms."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests import layer_common as lc
from tests.layer_common import U16, U32, assert_within, rand
from tests.test_gpu_block8 import check_product, values64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def cuda_ends(ends):
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


# (rows, K, N, ends): one group, empty groups, groups of one row, ends that do not reach the rows, tails of every kind
CASES = [(1, 16, 8, [1]), (64, 128, 128, [64]), (63, 144, 264, [63]), (200, 272, 72, [0, 65, 65, 66, 130, 200]),
         (777, 512, 768, [100, 101, 400, 400, 777]), (300, 1040, 328, [10, 250]), (1000, 256, 2048, [999, 1000]),
         (2048, 2048, 1024, [2048]), (130, 16, 512, [0, 0, 0]), (129, 4112, 16, [128, 129])]


@pytest.mark.parametrize("t,k,n,ends", CASES)
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("n_major", [False, True])
def test_weight_gradient(t, k, n, ends, dtype, pow2, n_major):
    E = len(ends)
    a = rand((t, k), 1) * torch.exp(2 * rand((t, 1), 2))
    dd = rand((t, n), 3)
    kept = ops.quantize_block8(a, dtype=dtype, pow2=pow2)
    B = torch.empty((E, k, n), dtype=BF16, device="cuda") if n_major else torch.empty((E, n, k), dtype=BF16, device="cuda").transpose(1, 2)
    dA, dB = ops.grouped_matmul_backward(dd, kept, B, cuda_ends(ends), need=(False, True))
    assert dA is None and dB.shape == B.shape and dB.stride() == B.stride()
    value = values64(kept)
    want, bound = lc.grouped_weight_grad(dd, value, ends)
    if not pow2:  # the product with the scale, and its rounding to bf16
        _, mag = lc.grouped_weight_grad(dd.abs(), value.abs(), ends)
        total, _ = lc.grouped_weight_grad(dd.abs(), value.abs(), ends)
        bound = bound + (U16 + 2 * U32) * total * (1 + U16)
    assert_within(dB, want, bound, "dB")
    ops.check_products()


def test_other_rows_do_not_enter():
    # rows past the last end, and those of other groups, may be anything
    t, k, n, ends = 300, 256, 264, [70, 70, 201]
    a, dd = rand((t, k), 10), rand((t, n), 11)
    kept = ops.quantize_block8(a, pow2=True)
    B = torch.empty((3, n, k), dtype=BF16, device="cuda").transpose(1, 2)
    want = ops.grouped_matmul_backward(dd, kept, B, cuda_ends(ends), need=(False, True))[1]
    values, scales, dd2 = kept.values.clone(), kept.scales.clone(), dd.clone()
    values.view(torch.uint8)[201:] = 0x7f
    scales[201:] = float("inf")
    dd2[201:] = float("nan")
    got = ops.grouped_matmul_backward(dd2, ops.Block8Tensor(values, scales, 1), B, cuda_ends(ends), need=(False, True))[1]
    assert torch.equal(got, want) and not want[1].any()
    values, dd2 = kept.values.clone(), dd.clone()
    values.view(torch.uint8)[69] = 0x7f                      # the first group's last row
    dd2[70] = float("inf")                                   # the third's first
    got = ops.grouped_matmul_backward(dd2, ops.Block8Tensor(values, kept.scales, 1), B, cuda_ends(ends), need=(False, True))[1]
    assert torch.isnan(got[0]).all() and not got[1].any() and not torch.isfinite(got[2]).any()


def test_strides_and_both_gradients():
    t, k, n, ends = 140, 272, 136, [30, 140]
    kept = ops.quantize_block8(rand((t, k), 20), pow2=True)
    W = rand((2, n, k), 21, 0.1)
    dd = rand((t, n + 24), 22)[:, 8:-16]
    dA, dB = ops.grouped_matmul_backward(dd, kept, W.transpose(1, 2), cuda_ends(ends))
    plain = ops.dequantize_block8(kept)
    wA, wB = ops.grouped_matmul_backward(dd, plain, W.transpose(1, 2), cuda_ends(ends))
    assert torch.equal(dA, wA) and torch.equal(dB, wB)
    rows = ops.Block8Tensor(kept.values, kept.scales.t().contiguous().t(), 1)
    assert torch.equal(ops.grouped_matmul_backward(dd, rows, W.transpose(1, 2), cuda_ends(ends), need=(False, True))[1], wB)
    only, none = ops.grouped_matmul_backward(dd, None, W.transpose(1, 2), cuda_ends(ends), need=(True, False))
    assert torch.equal(only, wA) and none is None
    with pytest.raises(TypeError):
        ops.grouped_matmul_backward(dd, None, W.transpose(1, 2), cuda_ends(ends))
    for bad in (ops.quantize_block8(plain, block_rows=128), ops.quantize_block8(plain[:100]), ops.quantize_block8(plain[:, :256])):
        with pytest.raises(ValueError):
            ops.grouped_matmul_backward(dd, bad, W.transpose(1, 2), cuda_ends(ends))


def test_nothing():
    W = rand((2, 24, 32), 23)
    kept = ops.quantize_block8(rand((0, 32), 24))
    dA, dB = ops.grouped_matmul_backward(rand((0, 24), 25), kept, W.transpose(1, 2), cuda_ends([0, 0]))
    assert dA.shape == (0, 32) and dB.shape == (2, 32, 24) and not dB.any()


@pytest.mark.parametrize("keep", [E4M3, E5M2])
def test_autograd_of_kept_rows(keep):
    t, k, n, ends = 200, 256, 136, cuda_ends([70, 200])
    A, W = rand((t, k), 30), rand((2, n, k), 31, 0.1)
    dd = rand((t, n), 32)
    a, w = A.clone().requires_grad_(), W.clone().requires_grad_()
    out = ops.grouped_matmul(a, w.transpose(1, 2), ends, keep_dtype=keep)
    assert torch.equal(out, ops.grouped_matmul(A, W.transpose(1, 2), ends))
    out.backward(dd)
    dA, dB = ops.grouped_matmul_backward(dd, ops.quantize_block8(A, dtype=keep, pow2=True), W.transpose(1, 2), ends)
    assert torch.equal(a.grad, dA) and torch.equal(w.grad, dB.transpose(1, 2))
    # frozen weights keep nothing of A; a frozen input asks for dB alone
    a2 = A.clone().requires_grad_()
    ops.grouped_matmul(a2, W.transpose(1, 2), ends, keep_dtype=keep).backward(dd)
    assert torch.equal(a2.grad, dA)
    w2 = W.clone().requires_grad_()
    ops.grouped_matmul(A, w2.transpose(1, 2), ends, keep_dtype=keep).backward(dd)
    assert torch.equal(w2.grad, w.grad)


# ------------------------------------------------------------ linear layers


@pytest.mark.parametrize("lead,n,k", [((1,), 16, 16), ((130,), 144, 272), ((3, 50), 512, 1040), ((257,), 2048, 512)])
@pytest.mark.parametrize("dtype,grad", [(E4M3, E5M2), (E4M3, E4M3), (E5M2, E5M2)])
def test_linear(lead, n, k, dtype, grad):
    x, w, dy = rand((*lead, k), 40), rand((n, k), 41, 0.1), rand((*lead, n), 42)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = ops.block8_linear(a, b, dtype=dtype, grad_dtype=grad)
    y.backward(dy)
    xq, wq = ops.quantize_block8(x, block_rows=128, dtype=dtype), ops.quantize_block8(w, block_rows=128, dtype=dtype)
    dq = ops.quantize_block8(dy, block_rows=128, dtype=grad)
    assert y.shape == (*lead, n) and torch.equal(y.view(-1, n), check_product(xq, wq, False, True, BF16))
    assert torch.equal(a.grad.view(-1, k), check_product(dq, wq, False, False, BF16)) and a.grad.shape == x.shape
    assert torch.equal(b.grad, check_product(dq, xq, True, False, BF16))
    ops.check_products()
    b.grad = None
    ops.block8_linear(x, b, dtype=dtype, grad_dtype=grad).backward(dy)
    assert b.grad is not None
    with torch.no_grad():
        assert torch.equal(ops.block8_linear(a, b, dtype=dtype), y)


def test_linear_gradient_against_differences():
    # of the product of the 8-bit values, which is linear in each
    x, w, dy = rand((48, 64), 50), rand((32, 64), 51), rand((48, 32), 52)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    ops.block8_linear(a, b, grad_dtype=E4M3).backward(dy)
    xq, wq, dq = (values64(ops.quantize_block8(t, block_rows=128)) for t in (x, w, dy))
    for grad, at, other in ((a.grad, xq, wq), (b.grad, wq, xq)):
        v = rand(at.shape, 53).double()

        def loss(t):
            return ((t @ other.t() if at is xq else other @ t.t()) * dq).sum()

        want = loss(at + 0.5 * v) - loss(at - 0.5 * v)
        got = (grad.double() * v).sum()
        assert (got - want).abs() <= 2 * U16 * (grad.double() * v).abs().sum() + 1e-9


# ------------------------------------------------------------- all together


def test_a_training_step_in_8_bits():
    """Norm to kept rows and a linear layer: the gradients of the whole chain
    against the 64-bit chain over the same kept values."""
    t, k, n = 300, 512, 384
    x, g, c, w, dy = rand((t, k), 60), rand((k,), 61, 0.2) + 1, rand((k,), 62, 0.1), rand((n, k), 63, 0.1), rand((t, n), 64)
    leaves = [v.clone().requires_grad_() for v in (x, g, c, w)]
    r = ops.layer_norm(*leaves[:3], keep_dtype=E4M3, keep_stats=True)
    ops.block8_linear(r.y, leaves[3], grad_dtype=E4M3).backward(dy)
    yq, wq, dq = (ops.quantize_block8(v.detach(), block_rows=128) for v in (r.y, w, dy))
    dyn = ops.block8_matmul(dq, wq, trans_b=False)
    dx, dg, dc = ops.layer_norm_backward(dyn, r.kept, g, r.mean, r.rstd)
    for got, want in zip(leaves, (dx, dg, dc, ops.block8_matmul(dq, yq, trans_a=True, trans_b=False))):
        assert torch.equal(got.grad, want)
    # serving: rows of the norm as 8-bit blocks straight into the product
    with torch.no_grad():
        q = ops.layer_norm(x, g, c, out_dtype=E4M3).y
        check_product(q, wq, False, True, BF16)
        ops.check_products()


def test_graph_of_a_step():
    t, k, n, ends = 300, 512, 384, cuda_ends([100, 300])
    x, g, c, dy = rand((t, k), 70), rand((k,), 71, 0.2) + 1, rand((k,), 72, 0.1), rand((t, n), 73)
    B = rand((2, n, k), 74, 0.1).transpose(1, 2)

    def step():
        r = ops.layer_norm(x, g, c, keep_stats=True, keep_dtype=E4M3)
        kept = ops.quantize_block8(r.y, pow2=True)
        d = ops.grouped_matmul(r.y, B, ends)
        da, db = ops.grouped_matmul_backward(dy, kept, B, ends)
        return (d, db, *ops.layer_norm_backward(da, r.kept, g, r.mean, r.rstd))

    step()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    x.copy_(rand(x.shape, 75))
    graph.replay()
    for got, want in zip(out, step()):
        assert torch.equal(got, want)
    ops.check_products()
