"""GPU tests of attention under a sliding window (prompts, gradient, decode) against 64 bits
(tests/window_ref.py): windows of one token to more than there are, first tokens that stay
visible, long sequences whose first keys' gradient comes from several workgroups, hidden places
that hold anything, pages that the window left behind."""

import math

import pytest
import torch

from tests import attn_ref as ref
from tests import window_ref as wref
from tests.test_gpu_attn import (BF16, F8, Rank, cu_of, decode_case, i32, make, normal, split, ub, values,  # noqa: F401
                                 workspace)

pytestmark = pytest.mark.gpu


def run(ub, x, do, lens, shape, window, sinks, times=1):
    """out, lse and the gradient's matrix of documents x, each run's the same bits."""
    H, G, D = shape
    T, n = x.shape[0], len(lens)
    cfg, win = ub.make_attn_cfg(H, G, D), ub.make_attn_window(window, sinks)
    xd, dod = x.cuda(), do.cuda()
    out = torch.full((T, H * D + 8), math.nan, dtype=BF16, device="cuda")
    lse = torch.full((H, T), math.nan, device="cuda")
    dx = torch.full_like(xd, math.nan)
    cols = (0, H * D, (H + G) * D)
    hs, ds, cu = [ub.heads(xd, c) for c in cols], [ub.heads(dx, c) for c in cols], i32(cu_of(lens))
    ws = workspace(ub, ub.UB_ATTN_PROMPT_WINDOW_BWD, cfg, T, n)
    ws.fill_(0xFF)  # needs no preparation
    first = None
    with Rank(ub, T) as h:
        for _ in range(times):
            ub.ub_attn_prompt_window(h, *hs, ub.heads(out), lse, cu, n, win, cfg)
            ub.ub_attn_prompt_window_bwd(h, ub.heads(dod), *hs, ub.heads(out), lse, *ds, cu, n, win, cfg, ws)
            got = out.clone(), lse.clone(), dx.clone()
            first = first or got
        torch.cuda.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return got


def check(ub, shape, lens, pad, window, sinks, times=2):
    H, G, D = shape
    x, T = make(shape, lens, pad, seed=sum(lens) + D)
    cu, used, scale = cu_of(lens), sum(lens), D ** -0.5
    do = torch.full((T, H * D), math.nan, dtype=BF16)
    do[:used] = normal(7, (used, H * D))
    out, lse, dx = run(ub, x, do, lens, shape, window, sinks, times)
    q, k, v = (t[:used].double() for t in split(x, shape))
    o, l, to, tl = wref.prompt(q, k, v, cu, scale, window, sinks)
    assert bool(torch.isnan(out[:, H * D:]).all())  # nothing past the heads
    ref.check(out[:used, : H * D].reshape(used, H, D), o, to, "out")
    ref.check(lse[:, :used], l, tl, "lse")
    assert bool((out[used:, : H * D] == 0).all()) and bool((lse[:, used:] == -math.inf).all())
    want, tol = wref.prompt_bwd(do[:used].double().reshape(used, H, D), q, k, v, cu, scale, window, sinks)
    for name, g, w, t in zip(("dq", "dk", "dv"), split(dx, shape), want, tol):
        ref.check(g[:used], w, t, name)
        assert bool((g[used:] == 0).all()), name
    assert bool(torch.isnan(dx[:, (H + 2 * G) * D:]).all())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (3, 5), (8, 0), (9, 0), (2, 64), (31, 0), (33, 5), (64, 0), (100, 33), (129, 4),
                                          (1 << 31, 0), (200, 64)])
@pytest.mark.parametrize("shape,lens,pad", [
    ((1, 1, 8), [1], 0),
    ((2, 2, 64), [1, 0, 2, 127, 128, 129], 1),
    ((8, 2, 128), [64, 63, 400], 7),
    ((6, 3, 80), [350, 31], 2),
    ((2, 2, 24), [3] * 70 + [0] * 5 + [300] + [1] * 60, 4),  # more sequences than lanes
])
def test_prompt_and_gradient(ub, shape, lens, pad, window, sinks):  # noqa: F811
    check(ub, shape, lens, pad, window, sinks)


@pytest.mark.parametrize("shape,lens,pad,window,sinks", [
    ((2, 1, 64), [1800, 30, 900], 3, 40, 4),          # slots of two sequences; the second's rest is short
    ((4, 4, 128), [0, 1400], 0, 100, 64),
    ((3, 1, 96), [641, 640, 1, 1700], 1, 1, 1),
    ((8, 1, 40), [1900], 0, 600, 16),                 # heads of a group in several parts
    ((64, 64, 24), [1300, 0, 100], 2, 70, 4),         # one group of waves
    ((72, 8, 64), [1, 300, 1100], 0, 130, 33),
    ((66, 22, 80), [1000], 1, 64, 2),
])
def test_long_sequences(ub, shape, lens, pad, window, sinks):  # noqa: F811
    """First keys whose later rows go to other workgroups."""
    check(ub, shape, lens, pad, window, sinks)


@pytest.mark.parametrize("H,T", [(2, 700), (128, 530)])
@pytest.mark.parametrize("low,high", [(0.0, 60.0), (-300.0, 300.0), (100.0, -100.0)])
@pytest.mark.parametrize("window,sinks", [(150, 0), (150, 3)])
def test_scores_that_leave_the_first_tile(ub, H, T, low, high, window, sinks):  # noqa: F811
    D = 16
    x = torch.zeros((T, 3, H, D), dtype=BF16)
    x[:, 0, :, 0] = 4.0
    x[:, 0, :, 1:] = normal(1, (T, H, D - 1))
    x[:, 1, :, 0] = (torch.linspace(low, high, T) / 4)[:, None].to(BF16)
    x[:, 1, :, 1:] = normal(2, (T, H, D - 1))
    x[:, 2] = normal(3, (T, H, D))
    x = x.reshape(T, -1)
    cu = [0, 65, 66, T]
    out, lse = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda"), torch.full((H, T), math.nan, device="cuda")
    xd = x.cuda()
    with Rank(ub, T) as h:
        ub.ub_attn_prompt_window(h, ub.heads(xd), ub.heads(xd, H * D), ub.heads(xd, 2 * H * D), ub.heads(out), lse, i32(cu),
                                 3, ub.make_attn_window(window, sinks), ub.make_attn_cfg(H, H, D, softmax_scale=1.0))
        torch.cuda.synchronize()
    q, k, v = (t.double() for t in split(x, (H, H, D)))
    w, l, tw, tl = wref.prompt(q, k, v, cu, 1.0, window, sinks)
    ref.check(out.reshape(T, H, D), w, tw, "out")
    ref.check(lse, l, tl, "lse")


@pytest.mark.parametrize("H,G,D,lens", [(2, 1, 64, [30, 333, 70]), (4, 2, 128, [500]), (96, 48, 40, [100, 590])])
@pytest.mark.parametrize("r", [0, 1, 63, 100, 200])
@pytest.mark.parametrize("window,sinks", [(50, 0), (50, 2), (130, 1)])
def test_values_that_are_hidden(ub, H, G, D, lens, r, window, sinks):  # noqa: F811
    """NaN and inf in row r of a sequence: rows that do not see it (before it, or past the window
    and it no first token) are as without it, and so are keys that its query does not see."""
    x, T = make((H, G, D), lens, 0, 11)
    cu, scale = cu_of(lens), D ** -0.5
    long = max(range(len(lens)), key=lambda i: lens[i])
    at, n = cu[long] + r, lens[long]
    do = normal(12, (T, H * D))
    q, k, v = (t.double() for t in split(x, (H, G, D)))
    o, l, to, tl = wref.prompt(q, k, v, cu, scale, window, sinks)
    grads, tols = wref.prompt_bwd(do.double().reshape(T, H, D), q, k, v, cu, scale, window, sinks)
    see = wref.seen(n, window, sinks)
    others = torch.ones(T, dtype=torch.bool)
    others[cu[long]: cu[long + 1]] = False
    blind, unseen, not_it = others.clone(), others.clone(), torch.ones(T, dtype=torch.bool)
    blind[cu[long]: cu[long + 1]] = ~see[:, r]    # rows that do not see key r
    unseen[cu[long]: cu[long + 1]] = ~see[r]      # keys that row r does not see
    not_it[at] = False
    for which in ("keys", "queries"):
        y, dy = x.clone(), do.clone()
        if which == "keys":
            y[at, H * D:(H + G) * D: 2] = math.inf
            y[at, (H + G) * D:] = math.nan
            y[at, -1] = -math.inf
        else:
            y[at, : H * D] = math.nan
            dy[at] = math.nan
            dy[at, ::3] = math.inf
        out, lse, dx = run(ub, y, dy, lens, (H, G, D), window, sinks)
        out = out[:, : H * D]
        dq, dk, dv = split(dx, (H, G, D))
        if which == "keys":
            checks = [(out.reshape(T, H, D), o, to, blind), (dq, grads[0], tols[0], blind)]
        else:
            checks = [(out.reshape(T, H, D), o, to, not_it), (dq, grads[0], tols[0], not_it),
                      (dk, grads[1], tols[1], unseen), (dv, grads[2], tols[2], unseen)]
        for i, (got, want, tol, rows) in enumerate(checks):
            ref.check(got.cpu()[rows], want[rows], tol[rows], f"{which} {i}")
        rows = blind if which == "keys" else not_it
        ref.check(lse.cpu()[:, rows], l[:, rows], tl[:, rows], f"{which} lse")


def test_keys_without_scores(ub):  # noqa: F811
    """Scores of -inf at all keys of a window: rows that see nothing else get 0 and -inf."""
    H, D, T, window = 2, 64, 500, 70
    x = normal(5, (T, 3, H, D))
    x[:, 0, :, 0] = -3e38
    x[:, 1, :, 0] = 0.0
    x[100:300, 1, :, 0] = 3e38
    x = x.reshape(T, -1)
    out, lse = torch.empty((T, H * D), dtype=BF16, device="cuda"), torch.empty((H, T), device="cuda")
    xd = x.cuda()
    with Rank(ub, T) as h:
        ub.ub_attn_prompt_window(h, ub.heads(xd), ub.heads(xd, H * D), ub.heads(xd, 2 * H * D), ub.heads(out), lse,
                                 i32([0, T]), 1, ub.make_attn_window(window), ub.make_attn_cfg(H, H, D))
        torch.cuda.synchronize()
    none = torch.arange(T).ge(100 + window - 1) & torch.arange(T).lt(300)
    assert bool((out.cpu()[none] == 0).all()) and bool((lse.cpu()[:, none] == -math.inf).all())
    q, k, v = (t.double() for t in split(x, (H, H, D)))
    q[..., 0] = 0.0
    for g in range(H):
        mask = wref.seen(T, window, 0)
        mask[:, 100:300] = False
        o, l, t, tl = ref.one(q[~none, g], k[:, g], v[:, g], D ** -0.5, mask[~none])
        ref.check(out.cpu()[~none].reshape(-1, H, D)[:, g], o, t, "out")
        ref.check(lse.cpu()[g, ~none], l, tl, "lse")


def test_no_sequences(ub):  # noqa: F811
    H, G, D, T = 2, 1, 64, 5
    x = torch.full((T, (H + 2 * G) * D), math.nan, dtype=BF16)
    for lens in ([], [0, 0]):
        out, lse, dx = run(ub, x, x[:, : H * D], lens, (H, G, D), 3, 1)
        assert bool((out[:, : H * D] == 0).all()) and bool((lse == -math.inf).all()) and bool((dx == 0).all())


def test_gradient_against_differences(ub):  # noqa: F811
    """The directional derivative of sum(out * dout) against central differences of the 64-bit
    forward pass at the same bf16 point."""
    shape, lens, window, sinks = (4, 2, 64), [50, 1, 700], 20, 2
    H, G, D = shape
    T, cu = sum(lens), cu_of(lens)
    x, _ = make(shape, lens, 0, 11)
    x = x[:, : (H + 2 * G) * D].contiguous()
    do = normal(12, (T, H * D))
    dx = run(ub, x, do, lens, shape, window, sinks)[2]
    f = lambda y: (wref.prompt(*split(y, shape), cu, D ** -0.5, window, sinks)[0].reshape(T, -1) * do.double()).sum()
    _, tol = wref.prompt_bwd(do.double().reshape(T, H, D), *(t.double() for t in split(x, shape)), cu, D ** -0.5, window, sinks)
    tol = torch.cat([t.reshape(T, -1) for t in tol], 1)
    for seed in (1, 2, 3):
        e = torch.randn(x.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        step = 1e-4  # the difference's own error is of the order step^2
        want = (f(x.double() + step * e) - f(x.double() - step * e)) / (2 * step)
        got = (dx.double().cpu() * e).sum()
        bound = (tol * e.abs()).sum() + 1e-5 * abs(want) + 1e-4
        assert abs(got - want) <= bound, (seed, float(got), float(want), float(bound))


@pytest.mark.parametrize("H,G,D,lens,page,f8,token_major,pad", [
    (1, 1, 8, [1], 1, False, False, 0),
    (8, 1, 128, [1000], 64, False, False, 0),
    (4, 4, 128, [1, 0, 37, 300, 128, 129], 16, False, True, 2),
    (8, 1, 128, [5, 0, 700], 64, True, False, 1),
    (8, 2, 128, [100, 250], 24, True, True, 0),
    (6, 3, 80, [33, 1, 260], 1, True, False, 0),
    (40, 2, 64, [150, 3], 16, False, False, 0),
    (4, 2, 96, [0, 1, 31, 32, 33, 500, 2000] * 20, 16, False, True, 1),
    (2, 1, 128, [20000, 9000], 48, False, False, 0),
    (3, 3, 72, [0, 257, 4100] * 25, 24, False, True, 0),
])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 1), (40, 0), (100, 33), (256, 4), (5000, 64), (1 << 31, 0)])
def test_decode(ub, H, G, D, lens, page, f8, token_major, pad, window, sinks):  # noqa: F811
    """Pages that hold no visible token have no id, and hidden places of the others hold NaN."""
    n, T, kc, vc, table, q = decode_case(H, G, D, lens, page, f8, token_major, pad)
    ks, vs = (40.0, 60.0) if f8 else (1.0, 1.0)
    kv, vv = values(kc) / ks, values(vc) / vs
    shown = table.clone()
    for i, m in enumerate(lens):
        for e in range(-(-m // page)):
            t = torch.arange(e * page, (e + 1) * page)
            see = (t < m) & ((t >= m - window) | (t < sinks))
            if not bool(see.any()):
                shown[i, e] = -1
                continue
            for c in (kc, vc):
                c.view(torch.uint8)[int(table[i, e]), :, torch.arange(page)[~see]] = 0x7F if f8 else 0xFF
    cfg, win = ub.make_attn_cfg(H, G, D), ub.make_attn_window(window, sinks)
    out = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda")
    lse = torch.full((H, T), math.nan, device="cuda")
    ws = workspace(ub, ub.UB_ATTN_DECODE_WINDOW, cfg, T, n)
    qd, td, ld, cache = q.cuda(), shown.cuda(), i32(lens), ub.make_kv_cache(kc, vc, ks, vs)
    with Rank(ub, T) as h:
        for _ in range(3):
            out.fill_(math.nan)
            ub.ub_attn_decode_window(h, ub.heads(qd), cache, td, ld, n, win, ub.heads(out), lse, cfg, ws)
        torch.cuda.synchronize()
    for i, m in enumerate(lens):
        got = out[i].reshape(H, D)
        if m == 0:
            assert bool((got == 0).all()) and bool((lse[:, i] == -math.inf).all())
            continue
        at = torch.arange(m)
        at = at[(at >= m - window) | (at < sinks)]
        pg, off = table[i].long()[at // page], at % page
        for g in range(G):
            x = q[i].double().reshape(H, D)[g * (H // G):(g + 1) * (H // G)]
            mask = torch.ones(H // G, len(at), dtype=torch.bool)
            o, l, to, tl = ref.one(x, kv[pg, g, off], vv[pg, g, off], D ** -0.5, mask)
            ref.check(got[g * (H // G):(g + 1) * (H // G)], o, to, f"out {i} {g}")
            ref.check(lse[g * (H // G):(g + 1) * (H // G), i], l, tl, f"lse {i} {g}")
    assert bool((out[n:] == 0).all()) and bool((lse[:, n:] == -math.inf).all())


def test_decode_bad_tables(ub):  # noqa: F811
    """A length past the table, a bad id of a page with visible tokens: NaN for that sequence."""
    H, G, D, page = 4, 2, 64, 16
    lens = [100, 20, 33, 40, 200]
    n, T, kc, vc, table, q = decode_case(H, G, D, lens, page, False, False, 0)
    cfg, win = ub.make_attn_cfg(H, G, D), ub.make_attn_window(30, 2)
    t, l = table.clone(), list(lens)
    t[0, 5] = -5          # positions 80 to 95, of which 70 and on are visible
    t[2, 0] = 1 << 30     # the first tokens'
    l[3], l[1] = 1 << 30, -7
    t[4, 5] = -1          # hidden
    out, lse = torch.zeros((T, H * D), dtype=BF16, device="cuda"), torch.zeros((H, T), device="cuda")
    ws = workspace(ub, ub.UB_ATTN_DECODE_WINDOW, cfg, T, n)
    qd = q.cuda()
    with Rank(ub, T) as h:
        ub.ub_attn_decode_window(h, ub.heads(qd), ub.make_kv_cache(kc, vc), t.cuda(), i32(l), n, win, ub.heads(out), lse, cfg, ws)
        torch.cuda.synchronize()
    for i in (0, 2, 3):
        assert bool(torch.isnan(out[i]).all()) and bool(torch.isnan(lse[:, i]).all())
    assert bool((out[1] == 0).all()) and bool((lse[:, 1] == -math.inf).all())
    assert bool(torch.isfinite(out[4]).all()) and bool(torch.isfinite(lse[:, 4]).all())
