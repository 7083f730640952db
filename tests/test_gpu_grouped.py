"""Products grouped by expert on the GPU, element by element against the 64-bit
form: ragged, empty and single-row groups, ends that are out of order or short
of the rows, both weight layouts, 8 bits with scales, gradients."""

import pytest
import torch

from reduce_scatter_gb300 import dg, ops
from tests import layer_common as lc
from tests.layer_common import U16, assert_within, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def ends_of(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# (T, K, N, ends): tiles of 256 x 256 met from both sides, K blocks of 64 and
# their ragged ends, groups of one row, empty groups first, last and between
CASES = [
    (1, 8, 8, [1]),
    (1, 64, 256, [0, 1, 1]),
    (31, 72, 264, [31]),
    (33, 64, 128, [1, 33]),
    (256, 128, 256, [256]),
    (257, 136, 520, [257]),
    (300, 200, 248, [0, 100, 100, 131, 300]),
    (1000, 512, 768, [3, 260, 261, 900, 900, 1000]),
    (77, 1032, 40, [16, 32, 48, 64, 77]),
    (2500, 64, 256, [2100, 2500]),
    (130, 4096, 136, [65, 130]),
]


@pytest.mark.parametrize("T,K,N,ends", CASES)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("n_major", [False, True])
def test_bf16(T, K, N, ends, out, n_major):
    a, E = rand((T, K), 1), len(ends)
    b = rand((E, K, N), 2, 0.1) if n_major else rand((E, N, K), 2, 0.1).transpose(1, 2)
    d = ops.grouped_matmul(a, b, ends_of(ends), out_dtype=out)
    ops.check_products()
    want, bound = lc.grouped(a, b, ends, out16=out == BF16)
    assert d.dtype == out
    assert_within(d, want, bound, "D")


@pytest.mark.parametrize("T,K,N,ends", [c for c in CASES if c[1] % 16 == 0])
@pytest.mark.parametrize("types", [(E4M3, E4M3), (E5M2, E4M3)])
def test_8bit_with_scales(T, K, N, ends, types):
    E = len(ends)
    a = rand((T, K), 3, 4.0).float().to(types[0])
    b = rand((E, N, K), 4, 4.0).float().to(types[1]).transpose(1, 2)
    g = torch.Generator(device="cuda").manual_seed(5)
    sa = torch.rand((T,), device="cuda", generator=g) + 0.1
    sb = torch.rand((E, N), device="cuda", generator=g) + 0.1
    for s1, s2 in ((sa, sb), (None, None), (sa[:1], sb[:, 0]), (sa, None)):
        d = ops.grouped_matmul(a, b, ends_of(ends), scale_a=s1, scale_b=s2)
        w1 = None if s1 is None else s1.expand(T)
        w2 = None if s2 is None else (s2 if s2.dim() == 2 else s2[:, None].expand(E, N))
        want, bound = lc.grouped(a, b, ends, w1, w2)
        assert_within(d, want, bound, "D")
    ops.check_products()


@pytest.mark.parametrize("ends", [[0, 0, 0], [10, 5, 40], [-3, 20, 90], [100, 200, 300], [50, 50, 20]])
def test_ends_out_of_order_or_range(ends):
    # clamped to [previous end, T]; rows past the last group are 0
    T = 64
    a, b = rand((T, 64), 6), rand((3, 48, 64), 7).transpose(1, 2)
    d = ops.grouped_matmul(a, b, ends_of(ends))
    want, bound = lc.grouped(a, b, ends)
    assert_within(d, want, bound, "D")
    dd = rand((T, 48), 8)
    da, db = ops.grouped_matmul_backward(dd, a, b, ends_of(ends))
    want, bound = lc.grouped(dd, b.transpose(1, 2), ends)
    assert_within(da, want, bound, "dA")
    want, bound = lc.grouped_weight_grad(dd, a, ends)
    assert_within(db, want, bound, "dB")


def test_not_finite_rows_stay_in_their_group():
    T, ends = 200, [70, 133]                     # rows past 133 belong to no group
    a, b, dd = rand((T, 64), 9), rand((2, 72, 64), 10).transpose(1, 2), rand((T, 72), 11)
    want, bound = lc.grouped(a, b, ends)
    wg, bg = lc.grouped_weight_grad(dd, a, ends)
    a[133:], dd[133:] = float("nan"), float("inf")
    a[70], dd[71] = float("inf"), float("nan")
    d = ops.grouped_matmul(a, b, ends_of(ends))
    keep = [i for i in range(T) if i != 70]
    assert_within(d[keep], want[keep], bound[keep], "D")
    assert not torch.isfinite(d[70].float()).any()
    da, db = ops.grouped_matmul_backward(dd, a, b, ends_of(ends))
    assert_within(db[0], wg[0], bg[0], "dB of the first group")
    assert not torch.isfinite(db[1].float()).any()
    assert not da[133:].any() and torch.isfinite(da[:70].float()).all() and not torch.isfinite(da[71].float()).any()


GRAD_CASES = [(1, 8, 8, [1]), (65, 64, 256, [64, 65]), (300, 200, 264, [0, 100, 100, 131, 300]),
              (1000, 512, 768, [3, 260, 261, 900, 900, 1000]), (63, 72, 40, [16, 32, 63]), (640, 320, 136, [128, 640]),
              (513, 1032, 520, [513])]


@pytest.mark.parametrize("T,K,N,ends", GRAD_CASES)
@pytest.mark.parametrize("n_major", [False, True])
def test_gradients(T, K, N, ends, n_major):
    E = len(ends)
    a, dd = rand((T, K), 12), rand((T, N), 13)
    b = rand((E, K, N), 14, 0.1) if n_major else rand((E, N, K), 14, 0.1).transpose(1, 2)
    da, db = ops.grouped_matmul_backward(dd, a, b, ends_of(ends))
    ops.check_products()
    want, bound = lc.grouped(dd, b.transpose(1, 2), ends)
    assert_within(da, want, bound, "dA")
    want, bound = lc.grouped_weight_grad(dd, a, ends)
    assert db.shape == b.shape and db.stride() == b.stride()
    assert_within(db, want, bound, "dB")
    # a fixed order of additions
    again = ops.grouped_matmul_backward(dd, a, b, ends_of(ends))
    assert torch.equal(again[0], da) and torch.equal(again[1], db)
    only = ops.grouped_matmul_backward(dd, a, b, ends_of(ends), need=(False, True))
    assert only[0] is None and torch.equal(only[1], db)


def test_gradient_against_differences():
    # D is linear in A and in B, so differences of the 64-bit form are exact up to rounding
    T, K, N, ends = 90, 64, 48, [20, 20, 77]
    a, b, dd = rand((T, K), 15), rand((3, N, K), 16).transpose(1, 2), rand((T, N), 17)
    da, db = ops.grouped_matmul_backward(dd, a, b, ends_of(ends))
    va, vb = rand((T, K), 18).double(), rand((3, K, N), 19).double()

    def f(x, w):
        return (lc.grouped(x, w, ends)[0] * dd.double()).sum()

    ad, bd, step = a.double(), b.double(), 0.5
    diff_a = (f(ad + step * va, bd) - f(ad - step * va, bd)) / (2 * step)
    diff_b = (f(ad, bd + step * vb) - f(ad, bd - step * vb)) / (2 * step)
    _, ba = lc.grouped(dd, b.transpose(1, 2), ends)
    _, bb = lc.grouped_weight_grad(dd, a, ends)
    assert ((da.double() * va).sum() - diff_a).abs() <= (ba * va.abs()).sum() + 1e-9
    assert ((db.double() * vb).sum() - diff_b).abs() <= (bb * vb.abs()).sum() + 1e-9


def test_autograd_and_strided_gradient():
    T, K, N, ends = 50, 64, 40, [13, 50]
    a, w = rand((T, K), 21).requires_grad_(), rand((2, N, K), 22).requires_grad_()
    out = ops.grouped_matmul(a, w.transpose(1, 2), ends_of(ends))
    out.sum().backward()                          # the incoming gradient is a broadcast
    dd = torch.ones((T, N), dtype=BF16, device="cuda")
    want, bound = lc.grouped(dd, w.detach(), ends)
    assert_within(a.grad, want, bound, "dA")
    want, bound = lc.grouped_weight_grad(dd, a.detach(), ends)
    assert w.grad.shape == w.shape
    assert_within(w.grad.transpose(1, 2), want, bound, "dB")
    with pytest.raises(ValueError):
        ops.grouped_matmul(a, w.transpose(1, 2), ends_of(ends), scale_a=torch.ones(1, device="cuda"))


def test_strides_streams_and_graph():
    T, K, N, ends = 150, 128, 96, [40, 41, 150]
    big = rand((T, 200), 23)
    a = big[:, 8:136]                             # a row pitch
    wide = rand((N, 3, K), 24)
    b = wide.permute(1, 2, 0)                     # experts interleaved: rows along K with another pitch
    e = ends_of(ends)
    want, bound = lc.grouped(a, b, ends)
    d = ops.grouped_matmul(a, b, e)
    assert_within(d, want, bound, "D")
    same = ops.grouped_matmul(big[:, 7:135], b, e)   # misaligned rows are copied
    w2, b2 = lc.grouped(big[:, 7:135], b, ends)
    assert_within(same, w2, b2, "D")
    three = big[:, 1:129]                         # misaligned rows in another place
    w3, b3 = lc.grouped(three, b, ends)
    assert_within(ops.grouped_matmul(three, b, e), w3, b3, "D")
    rows = rand((1, K), 26).expand(T, K)          # a broadcast row
    w4, b4 = lc.grouped(rows, b, ends)
    assert_within(ops.grouped_matmul(rows, b, e), w4, b4, "D")
    one = rand((1, N, K), 25).transpose(1, 2)
    d1 = ops.grouped_matmul(a, one.expand(3, K, N), e)   # a broadcast expert
    w1, b1 = lc.grouped(a, one.expand(3, K, N), ends)
    assert_within(d1, w1, b1, "D")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d2 = ops.grouped_matmul(a, b, e)
    s.synchronize()
    assert torch.equal(d2, d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg_out = ops.grouped_matmul(a, b, e)
        db_out = ops.grouped_matmul_backward(d, a, b, e)[1]
    e.copy_(ends_of([100, 100, 120]))             # the groups are read on the device at replay time
    g.replay()
    torch.cuda.synchronize()
    want, bound = lc.grouped(a, b, [100, 100, 120])
    assert_within(dg_out, want, bound, "D replayed")
    want, bound = lc.grouped_weight_grad(d, a, [100, 100, 120])
    assert_within(db_out, want, bound, "dB replayed")


def test_many_experts_and_empty_problems():
    E, K, N = 1024, 64, 64
    counts = torch.randint(0, 3, (E,), generator=torch.Generator().manual_seed(26))
    ends = counts.cumsum(0).to(torch.int32)
    T = int(ends[-1])
    a, b = rand((T, K), 27), rand((E, N, K), 28).transpose(1, 2)
    want, bound = lc.grouped(a, b, ends.tolist())
    assert_within(ops.grouped_matmul(a, b, ends.cuda()), want, bound, "D")
    dd = rand((T, N), 29)
    want, bound = lc.grouped_weight_grad(dd, a, ends.tolist())
    assert_within(ops.grouped_matmul_backward(dd, a, b, ends.cuda())[1], want, bound, "dB")
    z = ops.grouped_matmul(a[:0], b, torch.zeros_like(ends).cuda())
    assert z.shape == (0, N)
    da, db = ops.grouped_matmul_backward(z, a[:0], b, torch.zeros_like(ends).cuda())
    assert da.shape == (0, K) and not db.any()
    assert ops.grouped_matmul(a, b[:, :, :0], ends.cuda()).shape == (T, 0)
    ops.check_products()


def test_check_reports_and_clears_a_wait_that_ran_out():
    # the word as a kernel would leave it (launch 5 gave up wait 0x101)
    from reduce_scatter_gb300 import layer

    word = torch.tensor([(5 << 32) | 0x101], dtype=torch.int64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert layer.lib().dg_layer_check(word.data_ptr(), stream) == dg.ERR_HANG
    assert b"0x101" in layer.lib().dg_layer_last_error()
    assert layer.lib().dg_layer_check(word.data_ptr(), stream) == dg.OK
    assert layer.lib().dg_layer_check(None, stream) == dg.ERR_ARG


def test_same_bits_every_time_and_side_by_side():
    # tiles are drawn in any order and cut tiles are joined by whichever pair comes last
    cases = [(1000, 1024, 768, [3, 260, 261, 900, 1000]), (20, 8192, 512, [7, 20]), (5000, 1024, 1024, [900, 1800, 5000])]
    made = [(rand((T, K), 34), rand((len(e), N, K), 35).transpose(1, 2), ends_of(e), rand((T, N), 36)) for T, K, N, e in cases]
    want = [(ops.grouped_matmul(a, b, e), *ops.grouped_matmul_backward(d, a, b, e)) for a, b, e, d in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for turn in range(4):
        for k, (a, b, e, d) in enumerate(made):
            with torch.cuda.stream(streams[(turn + k) % 3]):
                got.append((k, ops.grouped_matmul(a, b, e), *ops.grouped_matmul_backward(d, a, b, e)))
    torch.cuda.synchronize()
    for k, *r in got:
        assert all(torch.equal(x, y) for x, y in zip(r, want[k])), k
    ops.check_products()


def test_refusals():
    a, b, e = rand((8, 64), 30), rand((2, 32, 64), 31).transpose(1, 2), ends_of([4, 8])
    with pytest.raises(TypeError):
        ops.grouped_matmul(a.to(E4M3), b, e)
    with pytest.raises(TypeError):
        ops.grouped_matmul(a.float(), b.float(), e)
    with pytest.raises(ValueError):
        ops.grouped_matmul(a, b, e, out_dtype=E4M3)
    with pytest.raises(ValueError):
        ops.grouped_matmul(a, b, e, scale_a=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError):
        ops.grouped_matmul(a, b, e, scale_a=2.0)
    with pytest.raises(ValueError):
        ops.grouped_matmul(a, b, e.cpu())
    with pytest.raises(dg.DGError) as err:
        ops.grouped_matmul(rand((8, 60), 32), rand((2, 32, 60), 33).transpose(1, 2), e)
    assert err.value.code == dg.ERR_SHAPE
    with pytest.raises(dg.DGError) as err:
        ops.grouped_matmul(a, rand((2, 36, 64), 33).transpose(1, 2), e)
    assert err.value.code == dg.ERR_SHAPE
