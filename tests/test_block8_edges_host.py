"""8-bit blocks and layer norm without a GPU: refusals at the ends of what is
allowed."""

import os

import pytest
import torch

from reduce_scatter_gb300 import dg, layer, ops

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(dg.LIB_PATH) or not os.path.exists(layer.EXT_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return layer.lib()


@pytest.mark.parametrize("start", range(16))
def test_a_host_tensor_is_refused_wherever_it_starts(start):
    x, rows = torch.ones(4, 64, dtype=BF16), torch.ones(4)
    values = torch.zeros(start + 4 * 64, dtype=torch.uint8)[start:].view(4, 64).view(E4M3)
    kept = ops.Block8Tensor(values, torch.ones(4, 1), 1)
    B, ends = torch.ones(1, 64, 8, dtype=BF16), torch.tensor([4], dtype=torch.int32)
    for call in (lambda: ops.layer_norm_backward(x, kept, None, rows, rows), lambda: ops.dequantize_block8(kept),
                 lambda: ops.block8_matmul(kept, kept._replace(block_rows=1)),
                 lambda: ops.grouped_matmul_backward(x[:, :8], kept, B, ends)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("hidden", [2**31 - 8191, 2**31 - 31, 2**31 - 8, 2**31 - 1])
def test_rows_longer_than_the_norm_takes(L, hidden):
    # (the last ones' columns, rounded up to whole blocks of threads, are beyond 32 bits)
    grad = L.dg_layer_layer_norm_backward(16, hidden, 16, hidden, dg.TYPE_BF16, None, 1, 1, None, 0, 16, 16, None, hidden, 16, 16, 16,
                                          dg.TYPE_BF16, 256, 1, hidden, None)
    norm = L.dg_layer_layer_norm(16, hidden, dg.TYPE_BF16, None, 0, 0, None, 0, None, 0, 16, dg.TYPE_BF16, None, 1, 1, None, 0, None,
                                 dg.TYPE_E4M3, None, 1, 1, None, None, 1, hidden, 1e-5, None)
    assert grad == norm == dg.ERR_ARG and b"out of range" in L.dg_layer_last_error()
