"""Where the roundings of 8-bit blocks fall: the norm's blocks of values that lie
halfway between two 8-bit ones, values brought back with any scale."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests.layer_common import U32, assert_within, rand
from tests.test_gpu_block8 import FP8, pow2, quantized, spread

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def halfway(hidden, dtype):
    """bf16 values that are 3/256 times midpoints of the type's positive numbers, each block's largest one 3/256 times its top."""
    top, mant, _ = FP8[dtype]
    g = torch.Generator(device="cuda").manual_seed(1)
    odd = torch.randint(0, 2 ** mant, (hidden,), device="cuda", generator=g).double() * 2 + 1 + 2 ** (mant + 1)  # (mant + 2 bits)
    v = odd * pow2(torch.randint(-6, 4, (hidden,), device="cuda", generator=g))
    v *= torch.randint(0, 2, (hidden,), device="cuda", generator=g).double() * 2 - 1
    v[::128] = top
    b = (v * 3 / 256).to(BF16)
    assert torch.equal(b.double() * 256 / 3, v)
    return b


# register kernels of one and of 8 vectors, streamed rows with and without whole threads, the looping kernel
@pytest.mark.parametrize("rows,hidden", [(5, 512), (2, 24576), (400, 4096), (400, 2064), (2, 32784)])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("ties", [True, False])
def test_norm_blocks_of_values_halfway(rows, hidden, dtype, ties):
    # With weights of zero a row is the bias, in 16 bits.  A block's values go through one multiplier top / max|y|, off by
    # at most one fp32 unit (2 U32), and a product (U32): so what is farther than 3 U32 of itself from halfway goes to the
    # nearest 8-bit value, and the rest to one of the two that are as near.
    top, mant, emin = FP8[dtype]
    b = halfway(hidden, dtype) if ties else rand((hidden,), 2)
    got = ops.layer_norm(rand((rows, hidden), 3), torch.zeros_like(b), b, out_dtype=dtype).y
    plain = ops.quantize_block8(b.expand(rows, hidden).contiguous(), dtype=dtype)
    want, c = quantized(b.expand(rows, hidden), 1, dtype, False)
    assert torch.equal(got.scales, plain.scales) and torch.equal(plain.values.float().double(), want)
    peak = torch.nn.functional.pad(b.double().abs(), (0, -hidden % 128)).view(-1, 128).amax(1).repeat_interleave(128)[:hidden]
    v = (b.double() * top / peak).expand(rows, hidden)
    _, e = torch.frexp(v)
    step = pow2((e - 1).clamp(min=emin) - mant)
    q = got.values.float().double()
    off = 3 * U32 * (1 + 2 * U32) * v.abs()
    assert_within(q, v, step / 2 + off, "values")
    far = ((v.abs() / step % 1) - 0.5).abs() * step > off
    assert torch.equal(q[far], want[far])
    assert not ties or (~far).double().mean() > 0.9


@pytest.mark.parametrize("rows,cols,block_rows", [(3, 128, 1), (200, 272, 128), (257, 1040, 1), (1000, 4112, 128)])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_values_are_the_rounded_products(rows, cols, block_rows, dtype):
    # value times scale in fp32, then bf16; exact for powers of two from 2^-117 on
    q = ops.quantize_block8(rand((rows, cols), 4) * torch.exp(rand((rows, 1), 5)), block_rows=block_rows, dtype=dtype)
    for s in (1.0, 2.0 ** -100, 2.0 ** -126 / float(q.scales.min())):
        p = ops.Block8Tensor(q.values, q.scales * s, block_rows)
        product = q.values.float() * spread(p.scales, block_rows, rows, cols)
        assert torch.equal(ops.dequantize_block8(p), product.to(BF16)) and torch.equal(ops.dequantize_block8(p, out_dtype=F32), product)
    g = torch.Generator(device="cuda").manual_seed(6)
    powers = pow2(torch.randint(-117, 100, q.scales.shape, device="cuda", generator=g))
    p = ops.Block8Tensor(q.values, powers.float(), block_rows)
    assert torch.equal(ops.dequantize_block8(p).double(), q.values.float().double() * spread(powers, block_rows, rows, cols))
