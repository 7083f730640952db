"""Products of 8-bit blocks whose CTA pairs walk many tiles with a K of one block,
so that a tile's output leaves while the next one's is written beside it; the
columns end where a warp stores an odd number of boxes of 128 bytes."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests.layer_common import rand
from tests.test_gpu_block8 import check_product

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def check_repeated(a, b, ta, tb, out):
    """All of D within the bound, and the same bits from calls that follow one another."""
    first = check_product(a, b, ta, tb, out)
    for D in [ops.block8_matmul(a, b, trans_a=ta, trans_b=tb, out_dtype=out) for _ in range(6)]:
        assert torch.equal(D, first)
    ops.check_products()


# N % 128 in 1..64 in 16 bits, in 1..32 or 65..96 in 32 bits; the last two: whole and even numbers of boxes
@pytest.mark.parametrize("m,n,k,out", [(100000, 64, 16, BF16), (100000, 16, 128, BF16), (100000, 16, 128, F32), (100000, 200, 128, F32),
                                       (20000, 576, 16, BF16), (20000, 2880, 128, BF16), (50000, 784, 16, BF16), (50000, 784, 16, F32),
                                       (20000, 8288, 128, F32), (50000, 512, 128, F32), (50000, 128, 128, BF16)])
@pytest.mark.parametrize("abr,bbr", [(1, 128), (128, 128), (1, 1)])
def test_many_tiles_of_one_block(m, n, k, out, abr, bbr):
    a = ops.quantize_block8(rand((m, k), 1) * torch.exp(rand((m, 1), 2)), block_rows=abr)
    b = ops.quantize_block8(rand((n, k), 3) * torch.exp(rand((n, 1), 4)), block_rows=bbr)
    check_repeated(a, b, False, True, out)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("ta,tb,m,n,k", [(True, False, 8192, 2880, 64),       # the weight's gradient of 64 tokens
                                         (True, False, 8192, 2880, 120), (True, False, 16384, 592, 1), (True, True, 16384, 576, 128),
                                         (False, False, 20000, 576, 128), (False, False, 50000, 80, 112)])  # the input's gradient
def test_many_tiles_of_transposes(ta, tb, m, n, k, out):
    a = ops.quantize_block8(rand((k, m) if ta else (m, k), 5), block_rows=128, dtype=torch.float8_e5m2)
    b = ops.quantize_block8(rand((n, k) if tb else (k, n), 6), block_rows=128)
    check_repeated(a, b, ta, tb, out)
