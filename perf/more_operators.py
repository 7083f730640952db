"""Measured cases of the operators of an 8-bit training step: layer norm (to 16
bits, to 8-bit blocks of 128, and its gradient, also from rows kept in 8 bits),
products of 8-bit tensors with a scale for each block of 128, weight gradients
from activations kept in 8 bits.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits) or, with ``own`` set, through ``reduce_scatter_gb300.ops``.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
MIN_SCALE = 2.0 ** -126

# ------------------------------------------------------------------- cases


def listed():
    return [
        # the rows of four sequences that each decode one token, as 8-bit blocks for the next product
        dict(name="norm_token_blocks", op="norm", rows=4, hidden=8192, residual=True, out="e4m3"),
        # a prefill's activations at the hidden size of the TP=8 all-gather workload
        dict(name="norm_prefill_blocks", op="norm", rows=8192, hidden=16384, residual=True, out="e4m3"),
        # a training step of the norm, an odd number of rows: output, new residual and all gradients
        dict(name="norm_train", op="norm_train", rows=4099, hidden=8192, residual=True, keep=None),
        # rows whose length is no multiple of anything
        dict(name="norm_train_odd", op="norm_train", rows=2047, hidden=5003, residual=False, keep=None),
        # a training step that keeps the norm's input in 8 bits for the way back
        dict(name="norm_train_kept", op="norm_train", rows=8192, hidden=8192, residual=False, keep="e4m3"),
        # decoding through a weight in 8-bit blocks: activations quantised on the way
        dict(name="blocks_linear_token", op="linear", rows=8, n=8192, k=28672, out="bf16"),
        # one rank's slab of the TP=8 all-gather workload in 8-bit blocks
        dict(name="blocks_linear_prefill", op="linear", rows=16384, n=13312, k=16384, out="bf16"),
        # an odd number of rows, and a last block of 16 columns
        dict(name="blocks_linear_ragged", op="linear", rows=1003, n=3328, k=8208, out="f32"),
        # one training step of a linear layer in 8 bits: output and both gradients, operands quantised on the way
        dict(name="blocks_train", op="train", rows=8192, n=8192, k=8192, grad="e5m2"),
        # a training step of experts whose rows are kept in 8 bits until the weight's gradient
        dict(name="kept_experts", op="kept", tokens=8192, experts=8, k=8192, n=2048, empty=0),
        # the same of one large weight
        dict(name="kept_dense", op="kept", tokens=16384, experts=1, k=8192, n=8192, empty=0),
        # a small training step: short odd groups, one of them empty
        dict(name="kept_small", op="kept", tokens=777, experts=5, k=512, n=768, empty=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "linear", "train", "kept"])
    if op == "norm":
        return dict(op=op, rows=_log_int(rng, 1, 8192), hidden=_log_int(rng, 8, 1024) * 16, residual=rng.random() < 0.5,
                    out=rng.choice(["e4m3", "e5m2", "bf16"]))
    if op == "norm_train":
        keep = rng.choice([None, "e4m3", "e5m2"])
        hidden = _log_int(rng, 128, 16384)
        if keep is not None:
            hidden = (hidden + 15) // 16 * 16
        elif rng.random() < 0.6:
            hidden = (hidden + 7) // 8 * 8
        return dict(op=op, rows=_log_int(rng, 1, 8192), hidden=hidden, residual=keep is None and rng.random() < 0.5, keep=keep)
    if op == "linear":
        return dict(op=op, rows=_log_int(rng, 1, 8192), n=_log_int(rng, 16, 1664) * 8, k=_log_int(rng, 4, 1024) * 16,
                    out=rng.choice(["bf16", "f32"]))
    if op == "train":
        return dict(op=op, rows=_log_int(rng, 1, 512) * 16, n=_log_int(rng, 4, 512) * 16, k=_log_int(rng, 4, 512) * 16,
                    grad=rng.choice(["e4m3", "e5m2"]))
    k = _log_int(rng, 4, 512) * 16
    n = _log_int(rng, 4, 512) * 16
    experts = _log_int(rng, 1, 64)
    while experts * k * n > 8 * 8192 * 2048:
        experts = max(1, experts // 2)
        if experts == 1:
            break
    return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, k=k, n=n, empty=rng.randrange(0, experts + 1) // 2)


# ------------------------------------------------------------------ inputs


def _counts(case, seed):
    """Rows of each expert: uneven popularity, ``empty`` experts that nobody chose."""
    r = np.random.RandomState((seed * 9973 + case["tokens"] * 31 + case["experts"]) % (2**32 - 1))
    p = np.exp(0.7 * r.randn(case["experts"]))
    p[r.permutation(case["experts"])[: case["empty"]]] = 0.0
    return r.multinomial(case["tokens"], p / p.sum())


def _randn(g, shape, std=1.0, dtype=torch.bfloat16):
    """Normal values, made in bands so that a large input needs no large fp32 copy."""
    rows = shape[0]
    band = max(1, (1 << 25) // max(1, math.prod(shape[1:])))
    parts = [torch.randn((min(band, rows - r), *shape[1:]), device="cuda", generator=g).mul_(std).to(dtype)
             for r in range(0, rows, band)]
    return parts[0] if len(parts) == 1 else torch.cat(parts)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    op = case["op"]
    st = dict(case)
    if op in ("norm", "norm_train"):
        rows, hidden = case["rows"], case["hidden"]
        # channels of different offset and magnitude, as a layer's activations have
        offset = torch.randn(hidden, device="cuda", generator=g) * 0.5
        st["x"] = (_randn(g, (rows, hidden), dtype=torch.float32) + offset).to(torch.bfloat16)
        st["r"] = _randn(g, (rows, hidden), 2.0) if case["residual"] else None
        st["w"] = (1.0 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).to(torch.bfloat16)
        st["b"] = (0.1 * torch.randn(hidden, device="cuda", generator=g)).to(torch.bfloat16)
        if op == "norm_train":
            st["dy"] = _randn(g, (rows, hidden), 0.1)
            st["dh"] = _randn(g, (rows, hidden), 0.1) if case["residual"] else None
        return st
    if op == "linear":
        st["x"] = _randn(g, (case["rows"], case["k"]))
        # the weight as a program keeps it: 8-bit values and a scale for each 128 x 128, made once at loading
        st["w8"], st["sw"] = _plain_blocks(_randn(g, (case["n"], case["k"]), 0.02), "e4m3", 128)
        return st
    if op == "train":
        st["x"] = _randn(g, (case["rows"], case["k"]))
        st["w"] = _randn(g, (case["n"], case["k"]), 0.02)
        st["dy"] = _randn(g, (case["rows"], case["n"]), 0.1)
        return st
    ends = np.cumsum(_counts(case, seed)).astype(np.int32)
    st["ends"], st["bounds"] = torch.from_numpy(ends).cuda(), [0] + [int(v) for v in ends]
    st["a"] = _randn(g, (case["tokens"], case["k"]))
    st["w"] = _randn(g, (case["experts"], case["n"], case["k"]), 0.02)
    st["dd"] = _randn(g, (case["tokens"], case["n"]), 0.1)
    return st


# -------------------------------------------------------------- plain forms


def _plain_blocks(x, kind, block_rows, pow2=False):
    """(8-bit values, fp32 scales) of a matrix: one scale for each ``block_rows`` x 128."""
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    f = x.float()
    if br * block_rows != rows or bc * 128 != cols:
        f = torch.nn.functional.pad(f, (0, bc * 128 - cols, 0, br * block_rows - rows))
    f = f.view(br, block_rows, bc, 128)
    amax = f.abs().amax((1, 3))
    top = TOP[kind]
    # values are x top / amax: the product is exact for 16-bit x, so what lies halfway between two 8-bit values stays there
    scale, num, den = amax / top, torch.full_like(amax, top), amax
    if pow2:
        m, e = torch.frexp(amax)  # top = 0.875 * 2^9 or 2^16
        e = e - (9 if kind == "e4m3" else 16) + (m > 0.875).to(e.dtype)
        scale = ((e.clamp(min=-126) + 127) << 23).view(torch.float32)  # (exp2 is not exact on the GPU)
        num, den = 1.0 / scale, torch.ones_like(amax)
    least, one = scale <= MIN_SCALE, torch.ones_like(amax)
    scale, num, den = torch.where(least, MIN_SCALE * one, scale), torch.where(least, one / MIN_SCALE, num), torch.where(least, one, den)
    scale, num = torch.where(amax > 0, scale, one), torch.where(amax > 0, num, one)
    q = (f * num[:, None, :, None]).div_(den[:, None, :, None]).clamp_(-top, top).to(FLOAT8[kind])
    return q.view(br * block_rows, bc * 128)[:rows, :cols].contiguous(), scale


def _plain_values(q, scale, block_rows):
    """fp32 values of 8-bit blocks."""
    s = scale.repeat_interleave(128, 1)[:, : q.shape[1]]
    if block_rows != 1:
        s = s.repeat_interleave(block_rows, 0)[: q.shape[0]]
    return q.float() * s


def _plain_stats(st):
    h = st["x"] if st["r"] is None else (st["x"].float() + st["r"].float()).to(torch.bfloat16)
    f = h.float()
    mean = f.mean(-1, keepdim=True)
    rstd = torch.rsqrt((f - mean).pow(2).mean(-1, keepdim=True) + EPS)
    return h, mean, rstd, (f - mean) * rstd * st["w"].float() + st["b"].float()


def _plain_norm(st):
    h, _, _, y = _plain_stats(st)
    if st["out"] == "bf16":
        return y.to(torch.bfloat16), h
    return (*_plain_blocks(y, st["out"], 1), h)


def _plain_norm_train(st):
    h, mean, rstd, y = _plain_stats(st)
    kept = None
    f = h.float()
    if st["keep"]:
        kept = _plain_blocks(h, st["keep"], 1, pow2=True)
        f = _plain_values(*kept, 1)
    dy, xh = st["dy"].float(), (f - mean) * rstd
    g = dy * st["w"].float()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    dw, db = (dy * xh).sum(0), dy.sum(0)
    out = [y.to(torch.bfloat16), mean[:, 0], rstd[:, 0], dx.to(torch.bfloat16), dw.to(torch.bfloat16), db.to(torch.bfloat16)]
    return out + (list(kept) if kept else [h])


def _plain_linear(st):
    a = _plain_values(*_plain_blocks(st["x"], "e4m3", 1), 1)
    d = a @ _plain_values(st["w8"], st["sw"], 128).t()
    return d.to(torch.bfloat16) if st["out"] == "bf16" else d


def _plain_train(st):
    x = _plain_values(*_plain_blocks(st["x"], "e4m3", 128), 128)
    w = _plain_values(*_plain_blocks(st["w"], "e4m3", 128), 128)
    dy = _plain_values(*_plain_blocks(st["dy"], st["grad"], 128), 128)
    return [t.to(torch.bfloat16) for t in (x @ w.t(), dy @ w, dy.t() @ x)]


def _plain_kept(st):
    kept = _plain_blocks(st["a"], "e4m3", 1, pow2=True)
    a, dd, b = _plain_values(*kept, 1), st["dd"].float(), st["bounds"]
    dw = torch.zeros_like(st["w"])
    for e in range(st["experts"]):
        if b[e + 1] > b[e]:
            dw[e] = (dd[b[e]:b[e + 1]].t() @ a[b[e]:b[e + 1]]).to(torch.bfloat16)
    return [*kept, dw]


_PLAIN = {"norm": _plain_norm, "norm_train": _plain_norm_train, "linear": _plain_linear, "train": _plain_train,
          "kept": _plain_kept}

# ------------------------------------------------------- the framework's own


def _own(st):
    from reduce_scatter_gb300 import ops

    op = st["op"]
    if op == "norm":
        out = torch.bfloat16 if st["out"] == "bf16" else FLOAT8[st["out"]]
        r = ops.layer_norm(st["x"], st["w"], st["b"], residual=st["r"], eps=EPS, out_dtype=out)
        return (r.y, r.residual) if st["out"] == "bf16" else (r.y.values, r.y.scales, r.residual)
    if op == "norm_train":
        r = ops.layer_norm(st["x"], st["w"], st["b"], residual=st["r"], eps=EPS, keep_stats=True,
                           keep_dtype=FLOAT8[st["keep"]] if st["keep"] else None)
        dx, dw, db = ops.layer_norm_backward(st["dy"], r.kept if st["keep"] else r.residual, st["w"], r.mean, r.rstd,
                                             d_residual=st["dh"])
        out = [r.y, r.mean, r.rstd, dx, dw, db]
        return out + ([r.kept.values, r.kept.scales] if st["keep"] else [r.residual])
    if op == "linear":
        return ops.block8_matmul(ops.quantize_block8(st["x"]), ops.Block8Tensor(st["w8"], st["sw"], 128),
                                 out_dtype=torch.bfloat16 if st["out"] == "bf16" else torch.float32)
    if op == "train":
        x = ops.quantize_block8(st["x"], block_rows=128)
        w = ops.quantize_block8(st["w"], block_rows=128)
        dy = ops.quantize_block8(st["dy"], block_rows=128, dtype=FLOAT8[st["grad"]])
        return [ops.block8_matmul(x, w), ops.block8_matmul(dy, w, trans_b=False),
                ops.block8_matmul(dy, x, trans_a=True, trans_b=False)]
    kept = ops.quantize_block8(st["a"], pow2=True)
    _, dw = ops.grouped_matmul_backward(st["dd"], kept, st["w"].transpose(1, 2), st["ends"], need=(False, True))
    return [kept.values, kept.scales, dw.transpose(1, 2)]


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ----------------------------------------------------------- least work


def work(case):
    op = case["op"]
    if op in ("norm", "norm_train"):
        e = case["rows"] * case["hidden"]
        if op == "norm":
            out = 2 if case["out"] == "bf16" else 1
            return {"bytes": e * (2 + out + (4 if case["residual"] else 0)) + 4 * case["hidden"], "flops": 12 * e}
        # forward: x (and the residual) in, y out (and the sum, or 8-bit rows); backward: dy, the sum (and dh) in, dx out
        each = 10 if case["keep"] else (10 + (6 if case["residual"] else 0))
        return {"bytes": e * each + 8 * case["hidden"], "flops": 28 * e}
    if op == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k + (2 if case["out"] == "bf16" else 4) * m * n, "flops": 2 * m * n * k}
    if op == "train":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": 4 * (m * n + m * k + n * k), "flops": 6 * m * n * k}
    t, n, k = case["tokens"], case["n"], case["k"]
    return {"bytes": 3 * t * k + 2 * t * n + 2 * case["experts"] * n * k, "flops": 2 * t * n * k}


# ---------------------------------------------------- definition in 64 bits

_MANTISSA, _LEAST = {"e4m3": 3, "e5m2": 2}, {"e4m3": -6, "e5m2": -14}


def _pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_blocks(x, kind, rows_each, pow2=False):
    """(values of the 8 bits, scales, what they stand for) of a matrix in 64 bits."""
    top, out, vals, rows = TOP[kind], [], [], x.shape[0]
    scales = torch.empty((-(-rows // rows_each), -(-x.shape[1] // 128)), dtype=torch.float64, device=x.device)
    for j, part in enumerate(x.double().split(128, 1)):
        peak = torch.stack([p.abs().amax() for p in part.split(rows_each)]) if rows_each > 1 else part.abs().amax(1)
        c = peak / top
        if pow2:
            m, e = torch.frexp(c)
            c = _pow2(torch.where(m == 0.5, e - 1, e))
        # what each value is multiplied by and then divided by (c itself is rounded: halfway values would move)
        up, down = torch.full_like(c, top), peak
        plain = (peak > 0) & (c > MIN_SCALE) & (not pow2)
        c = torch.where(peak > 0, c.clamp(min=MIN_SCALE), torch.ones_like(c))
        up, down = torch.where(plain, up, torch.ones_like(c)), torch.where(plain, down, c)
        scales[:, j] = c
        each, up, down = ((t.repeat_interleave(rows_each)[:rows] if rows_each > 1 else t)[:, None] for t in (c, up, down))
        v = part * up / down
        _, ex = torch.frexp(v)
        step = _pow2((ex - 1).clamp(min=_LEAST[kind]) - _MANTISSA[kind])
        v = torch.clamp(torch.round(v / step) * step, -top, top)
        out.append(v)
        vals.append(v * each)
    return torch.cat(out, 1), scales, torch.cat(vals, 1)


def _exact_norm(case, st):
    h = st["x"].double()
    if st["r"] is not None:
        h = (h + st["r"].double()).float().bfloat16().double()
    n = h.shape[1]
    mu = h.sum(1, keepdim=True) / n
    c = h - mu
    s = 1.0 / torch.sqrt((c * c).sum(1, keepdim=True) / n + EPS)
    w = st["w"].double()
    y = c * s * w + st["b"].double()
    if case["op"] == "norm":
        if case["out"] == "bf16":
            return y, h
        v, scale, _ = _exact_blocks(y, case["out"], 1)
        return v, scale, h
    tail = [h]
    if case["keep"]:
        v, scale, f = _exact_blocks(h, case["keep"], 1, pow2=True)
        c, tail = f - mu, [v, scale]
    dy, xh = st["dy"].double(), c * s
    g = dy * w
    dx = s * (g - g.sum(1, keepdim=True) / n - xh * ((g * xh).sum(1, keepdim=True) / n))
    if st["dh"] is not None:
        dx = dx + st["dh"].double()
    return [y, mu[:, 0], s[:, 0], dx, torch.einsum("th,th->h", dy, xh), dy.sum(0), *tail]


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12 or w["bytes"] > 3e9:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_train"):
        return _exact_norm(case, st)
    if op == "linear":
        a = _exact_blocks(st["x"], "e4m3", 1)[2]
        i = torch.arange(case["n"], device="cuda")[:, None] // 128
        j = torch.arange(case["k"], device="cuda")[None, :] // 128
        return torch.einsum("mk,nk->mn", a, st["w8"].double() * st["sw"].double()[i, j])
    if op == "train":
        x, wt, dy = (_exact_blocks(st[n], k, 128)[2] for n, k in (("x", "e4m3"), ("w", "e4m3"), ("dy", case["grad"])))
        return [torch.einsum("tk,nk->tn", x, wt), torch.einsum("tn,nk->tk", dy, wt), torch.einsum("tn,tk->nk", dy, x)]
    v, scale, a = _exact_blocks(st["a"], "e4m3", 1, pow2=True)
    b, dd = st["bounds"], st["dd"].double()
    parts = [torch.einsum("tn,tk->nk", dd[b[e]:b[e + 1]], a[b[e]:b[e + 1]]) for e in range(case["experts"])]
    return [v, scale, torch.stack(parts)]
