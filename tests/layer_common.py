"""Plain 64-bit forms of the layer operators, and the error bounds that their
tests hold the kernels to.

Bounds (U16 = 2^-8 and U32 = 2^-24, the unit roundoffs of bf16 and fp32):

* a sum of n products accumulated in fp32, in any order, each addition off by
  at most one unit in the last place of the running sum (2 * U32, which also
  covers truncation), is off by at most 2 * U32 * (n + 8) * sum |a b|; the 8
  covers the scale factors;
* one rounding to bf16 adds U16 times the value's magnitude.
"""

from __future__ import annotations

import numpy as np
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def rand(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def assert_within(got, want, bound, what=""):
    """|got - want| <= bound, element by element (fp64), nothing NaN."""
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert not torch.isnan(got).any(), what
    over = (got - want).abs() - bound
    worst = int(over.argmax()) if over.numel() else 0
    assert over.numel() == 0 or over.max() <= 0, (what, float(got.flatten()[worst]), float(want.flatten()[worst]),
                                                  float(bound.flatten()[worst]))


def product(a, b):
    """(a @ b.T, |a| @ |b|.T) in fp64."""
    a, b = a.double(), b.double()
    return a @ b.t(), a.abs() @ b.abs().t()


def product_bound(value, mag, n, out16=True):
    return 2 * U32 * (n + 8) * mag + (U16 * (value.abs() + 2 * U32 * (n + 8) * mag) if out16 else 0.0)


def grouped(a, b, ends, sa=None, sb=None, out16=True):
    """fp64 grouped product of a (T, K) with b (E, K, N), and its error bound."""
    T, N = a.shape[0], b.shape[2]
    d = torch.zeros(T, N, dtype=torch.float64, device=a.device)
    bound = torch.zeros_like(d)
    start = 0
    for e, end in enumerate(ends):
        end = min(max(int(end), start), T)
        v, m = product(a[start:end], b[e].t())
        if sa is not None:
            v, m = v * sa.double()[start:end, None], m * sa.double()[start:end, None].abs()
        if sb is not None:
            v, m = v * sb.double()[e], m * sb.double()[e].abs()
        d[start:end] = v
        bound[start:end] = product_bound(v, m, a.shape[1], out16)
        start = end
    return d, bound


def grouped_weight_grad(dd, a, ends):
    """fp64 sum over each group of a[t, :, None] * dd[t, None, :] (E, K, N), and its bound."""
    out, bounds, start = [], [], 0
    for end in ends:
        end = min(max(int(end), start), a.shape[0])
        v, m = product(a[start:end].t(), dd[start:end].t())
        out.append(v)
        bounds.append(product_bound(v, m, end - start))
        start = end
    return torch.stack(out), torch.stack(bounds)


def norm(x, w, residual=None, eps=1e-5):
    """(h, rstd, y) in fp64; h is rounded to the residual's type, as stored."""
    if residual is not None:
        h = x.float() + residual.float()
        h = h.to(residual.dtype)
    else:
        h = x
    hd = h.double()
    rstd = 1.0 / torch.sqrt(hd.pow(2).mean(-1) + eps)
    return h, rstd, hd * rstd[..., None] * w.double()


def norm_rel(hidden):
    """Relative error of rstd and of each y before its last rounding: the sum of
    squares (hidden additions), the division, rsqrt (2 units) and two products."""
    return (hidden + 16) * U32


def mx4_encode(x):
    """(codes 0..15, scale bytes) of an (rows, cols) array, by nearest value with ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    f = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(f).all(-1)
    f = np.where(bad[..., None], 0.0, f)
    top = np.abs(f).max(-1)
    _, ex = np.frexp(top)
    e = np.where(top > 0, np.maximum(ex - 1 - 2, -127), -127)
    v = np.abs(f) / np.ldexp(1.0, e)[..., None]
    dist = np.abs(v[..., None] - E2M1)
    # among equally near codes the even one
    code = np.argmin(dist * 4 + (np.arange(8) % 2) * 1e-9, axis=-1)
    code = code + 8 * np.signbit(f)
    code[bad] = 0
    return code.reshape(rows, cols).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx4_values(code, byte):
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return (v.reshape(*byte.shape, 32) * scale[..., None]).reshape(code.shape)


def mx4_tiled(byte):
    """Scale bytes (rows, cols / 32) in the tiled layout, element by element."""
    rows, blocks = byte.shape
    ct = -(-blocks // 8) * 2
    out = np.zeros((-(-rows // 128), ct, 512), dtype=np.uint8)
    r, s = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    out[r // 128, s // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + s % 4] = byte
    return out
