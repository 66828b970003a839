"""Attention under a sliding window with first tokens that stay visible, in 64 bits on the CPU,
with the bounds of attn_ref.py."""

import math

import torch

from tests import attn_ref as ref

U16, U32 = ref.U16, ref.U32


def seen(n, window, sinks):
    """[n, n]: whether row t sees key u."""
    t, u = torch.arange(n)[:, None], torch.arange(n)[None]
    return (u <= t) & ((t - u < window) | (u < sinks))


def prompt(q, k, v, cu, scale, window, sinks):
    T, H, D = q.shape
    group = H // k.shape[1]
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    tol_lse = torch.zeros((H, T), dtype=torch.float64)
    for a, b in ref.rows_of(cu):
        for h in range(H if b > a else 0):
            x, y, z = q[a:b, h], k[a:b, h // group], v[a:b, h // group]
            out[a:b, h], lse[h, a:b], tol[a:b, h], tol_lse[h, a:b] = ref.one(x, y, z, scale, seen(b - a, window, sinks))
    return out, lse, tol, tol_lse


def prompt_bwd(do, q, k, v, cu, scale, window, sinks):
    """dq, dk, dv and their bounds (as in attn_ref.prompt_bwd; the sums over slots add fp32
    roundings of at most as many terms as there are rows).  In a row of up to 8 keys delta is
    summed from them in fp32, not from the bf16 output, and dS (of tiles next to the diagonal) is used
    as two bf16 numbers."""
    T, H, D = q.shape
    group = H // k.shape[1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    tq, tk, tv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, b in ref.rows_of(cu):
        for h in range(H if b > a else 0):
            g = h // group
            x, y, z, w = q[a:b, h], k[a:b, g], v[a:b, g], do[a:b, h]
            n = b - a
            mask = seen(n, window, sinks)
            o, l, to, tl = ref.one(x, y, z, scale, mask)
            s = (x @ y.t() * scale).masked_fill(~mask, -math.inf)
            p = (s - l[:, None]).exp()
            delta = (w * o).sum(1, keepdim=True)
            e = p * (w @ z.t() - delta)
            d = (ref.score_error(x, y, s, scale, mask) + tl)[:, None]
            e_dp = (D + 2) * U32 * (w.abs() @ z.abs().t())
            e_delta = (w.abs() * to).sum(1, keepdim=True) + D * U32 * (w * o).abs().sum(1, keepdim=True)
            few = mask.sum(1, keepdim=True) <= 8
            pdp = p * (w @ z.t()).abs()
            e_delta = torch.where(few, ((2 * d + (n + 4) * U32) * pdp + p * e_dp).sum(1, keepdim=True), e_delta)
            u_ds = torch.where(few, U16 * U16, U16)
            ee = (u_ds + 2 * d) * e.abs() + p * (1 + 2 * d) * (e_dp + e_delta) * (1 + U16)
            dq[a:b, h] = scale * (e @ y)
            tq[a:b, h] = scale * ((ee + n * U32 * e.abs()) @ y.abs())
            dk[a:b, g] += scale * (e.t() @ x)
            tk[a:b, g] += scale * ((ee + n * group * U32 * e.abs()).t() @ x.abs())
            dv[a:b, g] += p.t() @ w
            tv[a:b, g] += (U16 + 2 * d + n * group * U32).mul(p).t() @ w.abs()
    for x, t in ((dq, tq), (dk, tk), (dv, tv)):
        t.mul_(1 + U16).add_(U16 * x.abs())
    return (dq, dk, dv), (tq, tk, tv)
