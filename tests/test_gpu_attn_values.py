"""GPU tests of keys with infinite elements that a query sees: a score of -inf is weight 0, whatever
the sequence's length and the head's size are.  The reference takes a finite element in its place
whose weight, below exp(-100), is 0 in fp32 as well."""

import math

import pytest
import torch

from tests import attn_ref as ref
from tests.test_gpu_attn import BF16, Rank, cu_of, i32, normal, split, ub, workspace  # noqa: F401  (ub: a fixture)

pytestmark = pytest.mark.gpu
FAR = -256.0  # with queries of 4 and a scale of 1/8 or more, a score of -128


@pytest.mark.parametrize("H,G,D,lens", [
    (2, 1, 64, [70, 33]),              # four groups of waves
    (4, 2, 40, [100]),
    (2, 2, 64, [96, 31, 65]),
    (72, 72, 64, [520, 131]),          # one group
    (96, 12, 64, [500]),               # heads of a group in parts
])
def test_gradient_of_keys_without_weight(ub, H, G, D, lens):
    T, cu = sum(lens), cu_of(lens)
    x = normal(21, (T, (H + 2 * G) * D))
    q, k, _ = split(x, (H, G, D))  # views of copies: written back below
    q[..., 0] = 4.0
    k[..., 0] = 0.0
    at = [cu[i] + n // 2 for i, n in enumerate(lens)] + [cu[i] + n - 1 for i, n in enumerate(lens)]
    k[at, :, 0] = FAR
    x[:, : H * D], x[:, H * D:(H + G) * D] = q.reshape(T, -1), k.reshape(T, -1)
    do = normal(22, (T, H * D))
    scale = 0.125
    args = [t.double() for t in split(x, (H, G, D))]
    o, l, to, tl = ref.prompt(*args, cu, scale)
    grads, tols = ref.prompt_bwd(do.double().reshape(T, H, D), *args, cu, scale)
    y = x.clone()
    y.view(T, -1, D)[at, H: H + G, 0] = -math.inf
    yd, dod = y.cuda(), do.cuda()
    out, lse = torch.empty((T, H * D), dtype=BF16, device="cuda"), torch.empty((H, T), device="cuda")
    dx = torch.full_like(yd, math.nan)
    cfg = ub.make_attn_cfg(H, G, D, softmax_scale=scale)
    ws = workspace(ub, ub.UB_ATTN_PROMPT_BWD, cfg, T, len(lens))
    hs = [ub.heads(yd, c) for c in (0, H * D, (H + G) * D)]
    with Rank(ub, T) as h:
        ub.ub_attn_prompt(h, *hs, ub.heads(out), lse, i32(cu), len(lens), cfg)
        ub.ub_attn_prompt_bwd(h, ub.heads(dod), *hs, ub.heads(out), lse,
                              *[ub.heads(dx, c) for c in (0, H * D, (H + G) * D)], i32(cu), len(lens), cfg, ws)
        torch.cuda.synchronize()
    ref.check(out.reshape(T, H, D), o, to, "out")
    ref.check(lse, l, tl, "lse")
    dq, dk, dv = split(dx, (H, G, D))
    seen = torch.zeros(T, dtype=torch.bool)  # rows that see such a key: dq takes 0 times its element
    for i, n in enumerate(lens):
        seen[cu[i] + n // 2: cu[i + 1]] = True
    ref.check(dq.cpu()[~seen], grads[0][~seen], tols[0][~seen], "dq")
    for name, got, want, tol in (("dk", dk, grads[1], tols[1]), ("dv", dv, grads[2], tols[2])):
        want[at] = 0.0  # weight 0, where the finite element's is not quite
        ref.check(got, want, tol, name)
        assert bool((got[at] == 0).all()), name


@pytest.mark.parametrize("page", [16, 24])  # a block of tokens in one page, and token by token
@pytest.mark.parametrize("H,G,D", [(2, 1, 8), (4, 2, 40), (6, 3, 80), (2, 2, 72), (3, 1, 104), (4, 2, 64), (2, 1, 128)])
def test_decode_of_keys_without_weight(ub, H, G, D, page):
    lens = [1 + page, 300]
    n, per = len(lens), -(-max(lens) // page)
    scale = 0.125
    q = normal(31, (n, H, D))
    q[..., 0] = 4.0
    k, v = normal(32, (n * per, G, page, D)), normal(33, (n * per, G, page, D))
    k[..., 0] = 0.0
    table = torch.arange(n * per, dtype=torch.int32).view(n, per)
    where = [(i, u) for i, m in enumerate(lens) for u in (0, m // 2, m - 1)]
    for i, u in where:
        k[i * per + u // page, :, u % page, 0] = FAR
    y = k.clone()
    for i, u in where:
        y[i * per + u // page, :, u % page, 0] = -math.inf
    cfg = ub.make_attn_cfg(H, G, D, softmax_scale=scale)
    qd, kd, vd = q.reshape(n, -1).cuda(), y.cuda(), v.cuda()
    out, lse = torch.empty((n, H * D), dtype=BF16, device="cuda"), torch.empty((H, n), device="cuda")
    ws = workspace(ub, ub.UB_ATTN_DECODE, cfg, n, n)
    with Rank(ub, n) as h:
        ub.ub_attn_decode(h, ub.heads(qd), ub.make_kv_cache(kd, vd), table.cuda(), i32(lens), n, ub.heads(out), lse, cfg, ws)
        torch.cuda.synchronize()
    for i, m in enumerate(lens):
        u = torch.arange(m)
        pg, off = i * per + u // page, u % page
        for g in range(G):
            hs = slice(g * (H // G), (g + 1) * (H // G))
            o, l, to, tl = ref.one(q[i, hs].double(), k[pg, g, off].double(), v[pg, g, off].double(), scale,
                                   torch.ones(H // G, m, dtype=torch.bool))
            ref.check(out[i].reshape(H, D)[hs], o, to, f"out {i} {g}")
            ref.check(lse[hs, i], l, tl, f"lse {i} {g}")
