"""The attention operators in 64 bits on the CPU, with the error bounds that the kernels'
roundings allow, for the GPU tests.

Bounds count roundings (u16 = 2^-8 is bf16's half step, u32 = 2^-24 fp32's):
  - a score is a sum of D exact products in fp32, then a few fp32 operations and exp2:
    its error is at most `ds` = (D + 8) u32 scale sum|q k| + 4 u32 (1 + max |s|) in the exponent;
  - softmax weights (and score gradients) are rounded to bf16 as operands: u16 each;
  - fp32 sums of n terms add n u32 of the sum of magnitudes;
  - each output is rounded once: u16 of its value.
"""

import math

import torch

U16, U32, U8 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4


def rows_of(cu):
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def prompt(q, k, v, cu, scale):
    """q [T, H, D], k, v [T, G, D] float64 -> out, lse, tol_out, tol_lse (rows of no sequence: 0,
    -inf, 0, 0)."""
    T, H, D = q.shape
    group = H // k.shape[1]
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    tol_lse = torch.zeros((H, T), dtype=torch.float64)
    for a, b in rows_of(cu):
        for h in range(H if b > a else 0):
            x, y, z = q[a:b, h], k[a:b, h // group], v[a:b, h // group]
            o, l, t, tl = one(x, y, z, scale, torch.ones(b - a, b - a, dtype=torch.bool).tril())
            out[a:b, h], lse[h, a:b], tol[a:b, h], tol_lse[h, a:b] = o, l, t, tl
    return out, lse, tol, tol_lse


def one(x, y, z, scale, mask):
    """Attention of rows x over keys y and values z where mask, with its bounds."""
    s = (x @ y.t() * scale).masked_fill(~mask, -math.inf)
    l = s.logsumexp(1)
    p = (s - l[:, None]).exp()
    o = p @ z
    d = score_error(x, y, s, scale, mask)
    n = y.shape[0]
    t = U16 * o.abs() + (U16 + 2 * d[:, None] + n * U32) * (p @ z.abs()) * (1 + U16)
    return o, l, t, 2 * d + (n + 4) * U32 + 2 * U32 * l.abs()


def score_error(x, y, s, scale, mask):
    """Per row, the largest error of a score (absolute, so relative in its exponential)."""
    mag = (x.abs() @ y.abs().t() * scale).masked_fill(~mask, 0.0).amax(1)
    return (x.shape[1] + 8) * U32 * mag + 4 * U32 * (1 + mag)


def prompt_bwd(do, q, k, v, cu, scale):
    """dq, dk, dv and their bounds; the kernel's delta uses the bf16 output."""
    T, H, D = q.shape
    group = H // k.shape[1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    tq, tk, tv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, b in rows_of(cu):
        for h in range(H if b > a else 0):
            g = h // group
            x, y, z, w = q[a:b, h], k[a:b, g], v[a:b, g], do[a:b, h]
            n = b - a
            mask = torch.ones(n, n, dtype=torch.bool).tril()
            o, l, to, tl = one(x, y, z, scale, mask)
            s = (x @ y.t() * scale).masked_fill(~mask, -math.inf)
            p = (s - l[:, None]).exp()
            delta = (w * o).sum(1, keepdim=True)
            e = p * (w @ z.t() - delta)
            d = (score_error(x, y, s, scale, mask) + tl)[:, None]
            e_dp = (D + 2) * U32 * (w.abs() @ z.abs().t())
            e_delta = (w.abs() * to).sum(1, keepdim=True) + D * U32 * (w * o).abs().sum(1, keepdim=True)
            ee = (U16 + 2 * d) * e.abs() + p * (1 + 2 * d) * (e_dp + e_delta) * (1 + U16)
            dq[a:b, h] = scale * (e @ y)
            tq[a:b, h] = scale * ((ee + n * U32 * e.abs()) @ y.abs())
            dk[a:b, g] += scale * (e.t() @ x)
            tk[a:b, g] += scale * ((ee + n * group * U32 * e.abs()).t() @ x.abs())
            dv[a:b, g] += p.t() @ w
            tv[a:b, g] += (U16 + 2 * d + n * group * U32).mul(p).t() @ w.abs()
    for x, t in ((dq, tq), (dk, tk), (dv, tv)):
        t.mul_(1 + U16).add_(U16 * x.abs())
    return (dq, dk, dv), (tq, tk, tv)


def rotate(x, pos, inv_freq, interleaved, rotary):
    """x [T, heads, D] float64 at positions pos -> rotated, and the bound before its rounding."""
    half = rotary // 2
    ang = pos.double()[:, None] * inv_freq.double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    one_, two = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
    y, t = x.clone(), torch.zeros_like(x)
    a, b = x[..., one_], x[..., two]
    y[..., one_], y[..., two] = a * c - b * s, b * c + a * s
    # the reduced angle, sine and cosine to 4 u32 each, two products and their sum
    t[..., one_] = t[..., two] = (a.abs() + b.abs()) * 8 * U32
    return y, t


def check(got, want, tol, what):
    """|got - want| <= tol element by element, finite throughout."""
    got = got.double().cpu()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite"
    err = (got - want).abs() - tol
    worst = err.max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: {int((err > 0).sum())} of {err.numel()} beyond the bound, worst by {worst:.3g}"
