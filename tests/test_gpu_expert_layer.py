"""The layer operators together (examples/expert_layer.py): each stage of the
serving path against the 64-bit form of that stage on the values that reached
it, and the gradients of the training step against a 64-bit autograd of the
same layer."""

import importlib.util
import os

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests import layer_common as lc
from tests.layer_common import U16, assert_within, rand

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_serving_path(tokens):
    hidden, ffn, experts = 512, 256, 6
    layer = example().ExpertLayer(hidden, ffn, experts)
    x, residual = rand((tokens, hidden), 1), rand((tokens, hidden), 2)
    t = {}
    out, new_residual = layer.forward(x, residual, t)
    ops.check_products()
    h, _, y = lc.norm(x, layer.norm, residual)
    assert torch.equal(new_residual, h)
    # an e4m3 value is within half a step, 2^-4 of itself or 2^-10 of the scale, of the norm's
    got = t["n"].y.double() * t["n"].scale.double()[:, None]
    assert_within(got, y, y.abs() * (2.0 ** -4 + 1e-3) + t["n"].scale.double()[:, None] * 2.0 ** -10, "norm")
    assert int(t["ends"][-1]) == 2 * tokens and (t["rows"].bincount(minlength=tokens) == 2).all()
    ends = t["ends"].tolist()
    want, bound = lc.grouped(t["a"], layer.up8.transpose(1, 2), ends, t["sa"], layer.up_scale)
    assert_within(t["up"], want, bound, "up")
    want, bound = lc.grouped(t["act"], layer.down.transpose(1, 2), ends)
    assert_within(t["down"], want, bound, "down")
    for a, w, d in ((t["normed"], layer.shared_up, t["s_up"]), (t["s_act"], layer.shared_down, t["shared"])):
        v, m = lc.product(ops.dequantize_mx4(ops.quantize_mx4(a), out_dtype=torch.float32),
                          ops.dequantize_mx4(w, out_dtype=torch.float32))
        assert_within(d, v, lc.product_bound(v, m, a.shape[1]), "shared")
    assert torch.isfinite(out.float()).all()


def test_training_step():
    tokens, hidden, ffn, experts = 96, 256, 128, 4
    layer = example().ExpertLayer(hidden, ffn, experts, seed=3)
    x, residual, d_out = rand((tokens, hidden), 4), rand((tokens, hidden), 5), rand((tokens, hidden), 6)
    got = layer.train_step(x, residual, d_out)
    ops.check_products()
    # the same layer in 64 bits, with the routing that the bf16 norm gave
    h = (x.float() + residual.float()).to(torch.bfloat16)
    p = {k: v.detach().double().requires_grad_() for k, v in dict(h=h, norm=layer.norm, up=layer.up, down=layer.down).items()}
    n = p["h"] / torch.sqrt(p["h"].pow(2).mean(-1, keepdim=True) + 1e-5) * p["norm"]
    y16 = ops.add_rms_norm(x, layer.norm, residual=residual).y
    rows, weight, ends = example().route(y16 @ layer.router.t(), layer.top_k)
    starts = [0] + ends.tolist()
    parts = []
    for e in range(experts):
        a = n[rows[starts[e]:starts[e + 1]]]
        up = a @ p["up"][e].t()
        gate, value = up.chunk(2, dim=-1)
        parts.append((torch.nn.functional.silu(gate) * value) @ p["down"][e].t())
    routed = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda").index_add(0, rows, torch.cat(parts) * weight.double()[:, None])
    (routed + p["h"]).backward(d_out.double())
    # every value on the way is rounded to bf16 a handful of times (norm, up, activation, down and their gradients: at
    # most 16 roundings of U16 each), with errors that are independent of one another, so in the 2-norm of a whole
    # gradient they stay below 16 U16
    want = dict(x=p["h"].grad, residual=p["h"].grad, norm=p["norm"].grad, up=p["up"].grad, down=p["down"].grad)
    for k, w in want.items():
        rel = (got[k].double() - w).norm() / w.norm()
        assert rel <= 16 * U16, (k, float(rel))
