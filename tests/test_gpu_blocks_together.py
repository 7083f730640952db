"""Several operators of 8-bit blocks, layer norm and kept rows at once: two
streams, graphs that replay side by side, inputs that repeat rows or share
memory, gradients that arrive in unusual layouts."""

import pytest
import torch

from reduce_scatter_gb300 import ops
from tests.layer_common import rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def flat(out):
    """Tensors of nested results; 8-bit ones as bytes."""
    if isinstance(out, torch.Tensor):
        return [out.view(torch.uint8) if out.element_size() == 1 else out]
    return [t for o in out if isinstance(o, (torch.Tensor, tuple)) for t in flat(o)]


def same(a, b):
    a, b = flat(a), flat(b)
    return len(a) == len(b) and all(torch.equal(x.nan_to_num(), y.nan_to_num()) if x.is_floating_point() else torch.equal(x, y)
                                    for x, y in zip(a, b))


class Work:
    """Every operator over inputs of its own; the products are cut along K, so that they use their workspace."""

    def __init__(self, seed, rows=300):
        self.x, self.r, self.few = rand((rows, 2048), seed), rand((rows, 2048), seed + 1), rand((7, 2048), seed + 2)
        self.odd, self.w3 = rand((rows, 1001), seed + 3), rand((1001,), seed + 4)
        self.g, self.b = rand((2048,), seed + 5), rand((2048,), seed + 6)
        self.w = ops.quantize_block8(rand((512, 2048), seed + 7, 0.1), block_rows=128)
        self.B = rand((3, 512, 2048), seed + 8, 0.1).transpose(1, 2)
        self.dy = rand((rows, 512), seed + 9)
        self.ends = torch.tensor([rows // 3, rows // 3, rows - 1], dtype=torch.int32, device="cuda")

    def run(self):
        n = ops.layer_norm(self.x, self.g, self.b, residual=self.r, out_dtype=E4M3, keep_stats=True, keep_dtype=E5M2)
        few = ops.layer_norm(self.few, self.g, self.b, out_dtype=E4M3)
        dq = ops.quantize_block8(self.dy, block_rows=128, dtype=E5M2)
        xq = ops.quantize_block8(self.x, block_rows=128)
        o = ops.layer_norm(self.odd, self.w3, keep_stats=True)
        return (n, few, ops.block8_matmul(n.y, self.w), ops.block8_matmul(few.y, self.w, out_dtype=F32),
                ops.block8_matmul(dq, xq, trans_a=True, trans_b=False), ops.block8_matmul(dq, self.w, trans_b=False),
                ops.grouped_matmul_backward(self.dy, n.kept, self.B, self.ends),
                ops.layer_norm_backward(self.x, n.kept, self.g, n.mean, n.rstd, d_residual=self.r),
                ops.layer_norm_backward(self.odd, self.odd, self.w3, o.mean, o.rstd), o)


def test_two_streams_at_once():
    work = [Work(1), Work(100, 331)]
    want = [w.run() for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work[i].run())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(g, want[i]) for g in got[i])
    ops.check_products()


def test_two_graphs_side_by_side_and_calls_beside_them():
    work = [Work(200), Work(300, 331)]
    want = [w.run() for w in work]
    torch.cuda.synchronize()
    graphs, outs = [], []
    capture = torch.cuda.Stream()                        # both graphs come from the same stream
    for w in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=capture):
            outs.append(w.run())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(capture):
            here = work[0].run()
    torch.cuda.synchronize()
    assert same(outs[0], want[0]) and same(outs[1], want[1]) and same(here, want[0])
    ops.check_products()


def test_inputs_that_repeat_rows_or_share_memory():
    row, g, b = rand((1, 1024), 10), rand((1024,), 11), rand((1024,), 12)
    many, each = row.expand(400, 1024), row.expand(400, 1024).contiguous()
    assert same(ops.layer_norm(many, g, b, residual=many, out_dtype=E4M3, keep_dtype=E4M3),
                ops.layer_norm(each, g, b, residual=each, out_dtype=E4M3, keep_dtype=E4M3))
    assert same(ops.layer_norm(many, g, b, residual=many).y, ops.layer_norm(each, g, b, residual=each).y)
    assert same(ops.quantize_block8(many), ops.quantize_block8(each))
    f = ops.layer_norm(each, g, b, keep_stats=True)
    one = torch.ones((), dtype=BF16, device="cuda").expand(400, 1024)        # (as the gradient of a sum arrives)
    want = ops.layer_norm_backward(one.contiguous(), each, g, f.mean, f.rstd)
    assert same(ops.layer_norm_backward(one, many, g, f.mean, f.rstd), want)
    windows = rand((3000,), 13).unfold(0, 1025, 1)[:400]                      # rows that overlap, a value apart
    assert same(ops.layer_norm(windows).y, ops.layer_norm(windows.contiguous()).y)
    q = ops.quantize_block8(rand((64, 256), 14))
    a, w = q, ops.Block8Tensor(q.values, q.scales, 1)                         # a product with itself
    d = ops.block8_matmul(a, w)
    assert torch.equal(d, d.t())


def test_gradients_of_sums_and_of_transposed_results():
    x, w, g = rand((150, 512), 20), rand((256, 512), 21, 0.1), rand((512,), 22)
    for through in (lambda y: y.sum(), lambda y: y.t()[:, ::2].float().pow(2).sum()):
        grads = []
        for same_layout in (False, True):
            a, b, c = (t.clone().requires_grad_() for t in (x, w, g))
            y = ops.block8_linear(ops.layer_norm(a, c, keep_dtype=E4M3).y, b)
            if same_layout:
                y.register_hook(lambda d: d.contiguous())
            through(y).backward()
            grads.append((a.grad, b.grad, c.grad))
        assert same(*grads)
    ops.check_products()


def test_one_leaf_used_twice():
    x, w = rand((130, 256), 30), rand((256, 256), 31, 0.1)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    out = ops.layer_norm(a, residual=a)                   # the same tensor as both addends
    out.y.backward(x)
    f = ops.layer_norm(x, residual=x, keep_stats=True)
    dx = ops.layer_norm_backward(x, f.residual, None, f.mean, f.rstd)[0]
    assert torch.equal(a.grad, dx + dx)
    ops.block8_linear(ops.block8_linear(x, b), b).backward(x)
    first = b.grad.clone()
    b.grad = None
    ops.block8_linear(ops.block8_linear(x, b), b).backward(x)
    assert torch.equal(b.grad, first)


def test_a_weight_with_a_tangent_is_refused():
    x, w = rand((16, 64), 40), rand((32, 64), 41)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(w, torch.ones_like(w))
        with pytest.raises(ValueError, match="forward-mode"):
            ops.block8_linear(x, dual)


def test_a_captured_step_with_autograd():
    # forward and backward of norm, 8-bit linear and experts with kept rows in one graph, as torch's own recipe captures them
    x, r, g, b = rand((200, 512), 50), rand((200, 512), 51), rand((512,), 52, 0.2) + 1, rand((512,), 53, 0.1)
    w, W = rand((256, 512), 54, 0.1), rand((3, 64, 256), 55, 0.1)
    ends = torch.tensor([50, 50, 199], dtype=torch.int32, device="cuda")
    leaves = [t.requires_grad_() for t in (g, b, w, W)]

    def step():
        n = ops.layer_norm(x, g, b, residual=r, keep_dtype=E4M3)
        y = ops.grouped_matmul(ops.block8_linear(n.y, w), W.transpose(1, 2), ends, keep_dtype=E5M2)
        (y.float().pow(2).sum() + n.residual.float().sum()).backward()

    def clear():
        for t in leaves:
            t.grad = None

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
            clear()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = [t.grad for t in leaves]
    for seed in (56, 57):
        x.copy_(rand(x.shape, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        clear()
        step()
        assert all(torch.equal(a, t.grad) for a, t in zip(got, leaves))
        clear()
    ops.check_products()
