"""An expert layer on the layer operators: residual add and RMS norm, routed
experts as grouped products, a shared expert in microscaled 4 bits.

    python examples/expert_layer.py [--tokens 4096] [--hidden 8192] [--experts 8]

``ExpertLayer.forward`` is the serving path (8-bit rows and routed weights,
4-bit shared weights); ``train_step`` runs the norm and the routed experts in
bf16 with gradients.  Routing (softmax, top-k, sort by expert) is plain torch;
the rows of each expert stay on the device, so nothing waits for the host.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from reduce_scatter_gb300 import ops  # noqa: E402

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


def route(logits: torch.Tensor, top_k: int):
    """``(rows, weights, ends)``: the token of each routed row in the order of
    the experts, its weight, and the experts' ends (int32, on the device)."""
    weight, expert = torch.softmax(logits.float(), -1).topk(top_k, dim=-1)
    weight = weight / weight.sum(-1, keepdim=True)
    order = torch.argsort(expert.flatten(), stable=True)
    counts = torch.zeros(logits.shape[-1], dtype=torch.int32, device=logits.device)
    counts.scatter_add_(0, expert.flatten(), torch.ones_like(order, dtype=torch.int32))
    return order // top_k, weight.flatten()[order], counts.cumsum(0, dtype=torch.int32)


def glu(up: torch.Tensor) -> torch.Tensor:
    gate, value = up.chunk(2, dim=-1)
    return F.silu(gate) * value


def quantize_columns(w: torch.Tensor):
    """bf16 (experts, N, K) weights as e4m3 with a scale for each expert's row N."""
    scale = w.abs().amax(-1).float().clamp(min=1e-12) / E4M3_MAX
    return (w / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


class ExpertLayer:
    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int = 2, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, std):
            return torch.randn(shape, device=device, generator=g, dtype=torch.float32).mul_(std).to(torch.bfloat16)

        self.top_k = top_k
        self.norm = 1 + rand(hidden, std=0.1)
        self.router = rand(experts, hidden, std=hidden ** -0.5)
        self.up = rand(experts, 2 * ffn, hidden, std=hidden ** -0.5)
        self.down = rand(experts, hidden, ffn, std=ffn ** -0.5)
        # laid out once for serving
        self.up8, self.up_scale = quantize_columns(self.up)
        self.shared_up = ops.quantize_mx4(rand(2 * ffn, hidden, std=hidden ** -0.5))
        self.shared_down = ops.quantize_mx4(rand(hidden, ffn, std=ffn ** -0.5))

    @torch.no_grad()
    def forward(self, x: torch.Tensor, residual: torch.Tensor, trace: dict | None = None):
        """(tokens, hidden) output of the layer, and the new residual stream."""
        n = ops.add_rms_norm(x, self.norm, residual=residual, out_dtype=E4M3)
        normed = (n.y.float() * n.scale[:, None]).to(torch.bfloat16)
        rows, weight, ends = route(normed @ self.router.t(), self.top_k)
        a, sa = n.y.view(torch.uint8)[rows].view(E4M3), n.scale[rows]
        up = ops.grouped_matmul(a, self.up8.transpose(1, 2), ends, scale_a=sa, scale_b=self.up_scale)
        act = glu(up)
        down = ops.grouped_matmul(act, self.down.transpose(1, 2), ends)
        routed = torch.zeros(x.shape, dtype=torch.float32, device=x.device).index_add_(0, rows, down.float() * weight[:, None])
        s_up = ops.mx4_matmul(ops.quantize_mx4(normed), self.shared_up)
        s_act = glu(s_up)
        shared = ops.mx4_matmul(ops.quantize_mx4(s_act), self.shared_down)
        out = (routed + shared.float()).to(torch.bfloat16)
        if trace is not None:
            trace.update(n=n, normed=normed, rows=rows, weight=weight, ends=ends, a=a, sa=sa, up=up, act=act, down=down,
                         s_up=s_up, s_act=s_act, shared=shared, out=out)
        return out, n.residual

    def train_step(self, x: torch.Tensor, residual: torch.Tensor, d_out: torch.Tensor) -> dict:
        """Gradients of sum(out * d_out) of the routed experts in bf16, with the
        residual stream added to the output."""
        leaves = dict(x=x, residual=residual, norm=self.norm, up=self.up, down=self.down)
        p = {k: v.detach().requires_grad_() for k, v in leaves.items()}
        n = ops.add_rms_norm(p["x"], p["norm"], residual=p["residual"])
        rows, weight, ends = route(n.y.detach() @ self.router.t(), self.top_k)
        up = ops.grouped_matmul(n.y[rows], p["up"].transpose(1, 2), ends)
        down = ops.grouped_matmul(glu(up), p["down"].transpose(1, 2), ends)
        routed = torch.zeros(x.shape, dtype=torch.float32, device=x.device).index_add(0, rows, down.float() * weight[:, None])
        (routed.to(torch.bfloat16) + n.residual).backward(d_out)
        return {k: v.grad for k, v in p.items()}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--ffn", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--iterations", type=int, default=20)
    a = ap.parse_args()
    layer = ExpertLayer(a.hidden, a.ffn, a.experts)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    residual, d_out = torch.randn_like(x), torch.randn_like(x)
    for name, step in (("serving", lambda: layer.forward(x, residual)), ("training", lambda: layer.train_step(x, residual, d_out))):
        for _ in range(3):
            step()
        ops.check_products()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.iterations):
            step()
        end.record()
        end.synchronize()
        ms = start.elapsed_time(end) / a.iterations
        print(f"{name}: {a.tokens} tokens, hidden {a.hidden}, {a.experts} experts of {a.ffn}: {ms:.3f} ms")


if __name__ == "__main__":
    main()
