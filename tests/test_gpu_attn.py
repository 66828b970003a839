"""GPU tests of the attention calls against their definitions in 64 bits (tests/attn_ref.py):
causal attention over packed sequences, its gradient, position rotation with the append to a
paged cache, and decode over the cache; lengths of zero and one, ragged tiles, head layouts,
strides, padding rows, garbage in places that no result may depend on, and bad page tables."""

import math

import pytest
import torch

from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ub():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import chunked_tp_overlap_amd.ub as m
    return m


class Rank:
    """A handle whose active shape is T rows."""

    def __init__(self, ub, T, hidden=64):
        self.ub = ub
        self.buf = torch.empty(T * hidden, dtype=BF16, device="cuda")
        self.h = ub.ub_init(T, hidden, 1, ub.UB_DTYPE_BF16, self.buf, T * hidden * 2)

    def __enter__(self):
        return self.h

    def __exit__(self, *exc):
        torch.cuda.synchronize()
        self.ub.ub_destroy(self.h)


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(seed, shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(BF16)


def workspace(ub, op, cfg, rows, n):
    b = ub.ub_attn_required_bytes(op, cfg, rows, n)
    return torch.zeros(max(b, 16), dtype=torch.uint8, device="cuda")


# H, G, D; lens; padding rows
PROMPTS = [
    ((1, 1, 8), [1], 0),
    ((2, 2, 64), [1, 0, 2, 127, 128, 129], 1),
    ((4, 4, 128), [300, 0, 1, 65], 3),
    ((8, 1, 128), [257], 0),
    ((8, 2, 128), [64, 63, 200], 7),
    ((6, 3, 80), [150, 31], 2),
    ((5, 1, 64), [33, 1, 1, 70], 5),
    ((16, 1, 128), [90], 0),
    ((2, 1, 24), [40, 300], 1),
    ((2, 2, 96), [0, 0, 130], 1),
    ((1, 1, 120), [513], 0),
    ((2, 2, 64), [3] * 70 + [0] * 5 + [100] + [1] * 60, 4),  # more sequences than lanes
]


def make(shape, lens, pad, seed):
    """The QKV matrix of a rank: pad rows and the columns after it hold NaN."""
    H, G, D = shape
    T = sum(lens) + pad
    W = (H + 2 * G) * D
    x = torch.full((T, W + 8), math.nan, dtype=BF16)
    x[: sum(lens), :W] = normal(seed, (sum(lens), W), 1.0)
    x[: sum(lens), : H * D] *= 1.5
    return x, T


def split(x, shape):
    H, G, D = shape
    T = x.shape[0]
    return (x[:, : H * D].reshape(T, H, D), x[:, H * D:(H + G) * D].reshape(T, G, D),
            x[:, (H + G) * D:(H + 2 * G) * D].reshape(T, G, D))


@pytest.mark.parametrize("shape,lens,pad", PROMPTS)
def test_prompt_and_gradient(ub, shape, lens, pad):
    H, G, D = shape
    x, T = make(shape, lens, pad, seed=sum(lens) + D)
    cu, used = cu_of(lens), sum(lens)
    cfg = ub.make_attn_cfg(H, G, D)
    scale = D ** -0.5
    xd = x.cuda()
    out = torch.full((T, H * D + 8), math.nan, dtype=BF16, device="cuda")
    lse = torch.full((H, T), math.nan, device="cuda")
    do = torch.full((T, H * D), math.nan, dtype=BF16)
    do[:used] = normal(7, (used, H * D))
    dod = do.cuda()
    dx = torch.full_like(xd, math.nan)
    hq, hk, hv = (ub.heads(xd, c) for c in (0, H * D, (H + G) * D))
    dq, dk, dv = (ub.heads(dx, c) for c in (0, H * D, (H + G) * D))
    ws = workspace(ub, ub.UB_ATTN_PROMPT_BWD, cfg, T, len(lens))
    ws.fill_(0xFF)  # needs no preparation
    with Rank(ub, T) as h:
        ub.ub_attn_prompt(h, hq, hk, hv, ub.heads(out), lse, i32(cu), len(lens), cfg)
        ub.ub_attn_prompt_bwd(h, ub.heads(dod), hq, hk, hv, ub.heads(out), lse, dq, dk, dv, i32(cu), len(lens),
                              cfg, ws)
        first = (out.clone(), lse.clone(), dx.clone())
        ub.ub_attn_prompt(h, hq, hk, hv, ub.heads(out), lse, i32(cu), len(lens), cfg)
        ub.ub_attn_prompt_bwd(h, ub.heads(dod), hq, hk, hv, ub.heads(out), lse, dq, dk, dv, i32(cu), len(lens),
                              cfg, ws)
        torch.cuda.synchronize()
    for a, b in zip(first, (out, lse, dx)):  # the same bits on every run
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    q, k, v = (t[:used].double() for t in split(x, shape))
    o, l, to, tl = ref.prompt(q, k, v, cu, scale)
    assert bool(torch.isnan(out[:, H * D:]).all())  # nothing past the heads
    ref.check(out[:used, : H * D].reshape(used, H, D), o, to, "out")
    ref.check(lse[:, :used], l, tl, "lse")
    assert bool((out[used:, : H * D] == 0).all()) and bool((lse[:, used:] == -math.inf).all())
    want, tol = ref.prompt_bwd(do[:used].double().reshape(used, H, D), q, k, v, cu, scale)
    for name, g, w, t in zip(("dq", "dk", "dv"), split(dx, shape), want, tol):
        ref.check(g[:used], w, t, name)
        assert bool((g[used:] == 0).all()), name
    assert bool(torch.isnan(dx[:, (H + 2 * G) * D:]).all())



@pytest.mark.parametrize("shape,lens,pad", [
    ((64, 64, 24), [700, 0, 330], 2),
    ((72, 8, 128), [1, 300, 613], 0),
    ((66, 22, 80), [1000], 1),
    ((70, 70, 64), [129, 500, 64, 63, 255], 7),
])
def test_prompt_and_gradient_many_heads(ub, shape, lens, pad):
    """Enough rows times heads for the kernels of one group of waves per workgroup."""
    assert (sum(lens) + pad) * shape[0] >= 64 * 1024
    test_prompt_and_gradient(ub, shape, lens, pad)


@pytest.mark.parametrize("H,T", [(2, 700), (128, 530)])
@pytest.mark.parametrize("low,high", [(0.0, 60.0), (-300.0, 300.0), (100.0, -100.0)])
def test_prompt_scores_that_leave_the_first_tile(ub, H, T, low, high):
    """Scores that rise (fall) along the keys by up to 600: beyond what the first tile's maximum
    can stand for, so that the pass is repeated with the running one."""
    D = 16
    x = torch.zeros((T, 3, H, D), dtype=BF16)
    x[:, 0, :, 0] = 4.0
    x[:, 0, :, 1:] = normal(1, (T, H, D - 1))
    x[:, 1, :, 0] = (torch.linspace(low, high, T) / 4)[:, None].to(BF16)
    x[:, 1, :, 1:] = normal(2, (T, H, D - 1))
    x[:, 2] = normal(3, (T, H, D))
    x = x.reshape(T, -1)
    cu = [0, 65, 66, T]
    out = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda")
    lse = torch.full((H, T), math.nan, device="cuda")
    xd = x.cuda()
    with Rank(ub, T) as h:
        ub.ub_attn_prompt(h, ub.heads(xd), ub.heads(xd, H * D), ub.heads(xd, 2 * H * D), ub.heads(out), lse, i32(cu), 3,
                          ub.make_attn_cfg(H, H, D, softmax_scale=1.0))
        torch.cuda.synchronize()
    q, k, v = (t.double() for t in split(x, (H, H, D)))
    w, l, tw, tl = ref.prompt(q, k, v, cu, 1.0)
    ref.check(out.reshape(T, H, D), w, tw, "out")
    ref.check(lse, l, tl, "lse")


def test_prompt_first_tile_without_scores(ub):
    """Scores of -inf at all keys of the first tiles, and finite ones after them."""
    H, D, T = 2, 64, 400
    x = normal(5, (T, 3, H, D))
    x[:, 0, :, 0] = -3e38
    x[:, 1, :, 0] = 0.0
    x[:140, 1, :, 0] = 3e38
    x = x.reshape(T, -1)
    out = torch.empty((T, H * D), dtype=BF16, device="cuda")
    lse = torch.empty((H, T), device="cuda")
    xd = x.cuda()
    with Rank(ub, T) as h:
        ub.ub_attn_prompt(h, ub.heads(xd), ub.heads(xd, H * D), ub.heads(xd, 2 * H * D), ub.heads(out), lse,
                          i32([0, T]), 1, ub.make_attn_cfg(H, H, D))
        torch.cuda.synchronize()
    assert bool((out[:140] == 0).all()) and bool((lse[:, :140] == -math.inf).all())
    q, k, v = (t.double() for t in split(x, (H, H, D)))
    q[..., 0] = 0.0
    for g in range(H):
        mask = torch.ones(T, T, dtype=torch.bool).tril()
        mask[:, :140] = False
        o, l, t, tl = ref.one(q[140:, g], k[:, g], v[:, g], D ** -0.5, mask[140:])
        ref.check(out[140:].reshape(-1, H, D)[:, g], o, t, "out")
        ref.check(lse[g, 140:], l, tl, "lse")



@pytest.mark.parametrize("H,G,D,lens", [(2, 1, 64, [30, 333, 70]), (4, 2, 128, [500]), (96, 48, 40, [100, 590]),
                                        (72, 72, 128, [940])])
@pytest.mark.parametrize("r", [1, 17, 63, 64, 200])
def test_prompt_values_that_the_mask_leaves_out(ub, H, G, D, lens, r):
    """NaN and inf in row r of a sequence: no row before it sees its key and value, and no key
    after it its query."""
    x, T = make((H, G, D), lens, 0, 11)
    cu, scale = cu_of(lens), D ** -0.5
    cfg = ub.make_attn_cfg(H, G, D)
    long = max(range(len(lens)), key=lambda i: lens[i])
    at = cu[long] + r  # other sequences and the rows named below are as without it
    do = normal(12, (T, H * D))
    q, k, v = (t.double() for t in split(x, (H, G, D)))
    o, l, to, tl = ref.prompt(q, k, v, cu, scale)
    grads, tols = ref.prompt_bwd(do.double().reshape(T, H, D), q, k, v, cu, scale)
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
        yd, dyd = y.cuda(), dy.cuda()
        out, lse = torch.empty((T, H * D), dtype=BF16, device="cuda"), torch.empty((H, T), device="cuda")
        dx = torch.empty_like(yd)
        ws = workspace(ub, ub.UB_ATTN_PROMPT_BWD, cfg, T, len(lens))
        hs = [ub.heads(yd, c) for c in (0, H * D, (H + G) * D)]
        with Rank(ub, T) as h:
            ub.ub_attn_prompt(h, *hs, ub.heads(out), lse, i32(cu), len(lens), cfg)
            ub.ub_attn_prompt_bwd(h, ub.heads(dyd), *hs, ub.heads(out), lse,
                                  *[ub.heads(dx, c) for c in (0, H * D, (H + G) * D)], i32(cu), len(lens), cfg, ws)
            torch.cuda.synchronize()
        dq, dk, dv = split(dx, (H, G, D))
        others = torch.ones(T, dtype=torch.bool)
        others[cu[long]: cu[long + 1]] = False
        before, after, not_it = others.clone(), others.clone(), torch.ones(T, dtype=torch.bool)
        before[cu[long]: at] = True
        after[at + 1: cu[long + 1]] = True
        not_it[at] = False
        if which == "keys":
            checks = [(out.reshape(T, H, D), o, to, before), (dq, grads[0], tols[0], before)]
        else:
            checks = [(out.reshape(T, H, D), o, to, not_it), (dq, grads[0], tols[0], not_it),
                      (dk, grads[1], tols[1], after), (dv, grads[2], tols[2], after)]
        for n, (got, want, tol, rows) in enumerate(checks):
            ref.check(got.cpu()[rows], want[rows], tol[rows], f"{which} {n}")
        rows = before if which == "keys" else not_it
        ref.check(lse.cpu()[:, rows], l[:, rows], tl[:, rows], f"{which} lse")


@pytest.mark.parametrize("scale,std", [(1.0, 2.0), (0.01, 1.0), (0.125, 8.0)])
def test_prompt_large_and_small_scores(ub, scale, std):
    """Scores far apart (one key takes the whole row) and nearly equal."""
    shape, lens = (2, 1, 64), [200]
    H, G, D = shape
    x = normal(5, (200, (H + 2 * G) * D), std)
    cfg = ub.make_attn_cfg(H, G, D, softmax_scale=scale)
    xd, out = x.cuda(), torch.empty((200, H * D), dtype=BF16, device="cuda")
    lse = torch.empty((H, 200), device="cuda")
    with Rank(ub, 200) as h:
        ub.ub_attn_prompt(h, ub.heads(xd), ub.heads(xd, H * D), ub.heads(xd, (H + G) * D), ub.heads(out), lse,
                          i32([0, 200]), 1, cfg)
        torch.cuda.synchronize()
    o, l, to, tl = ref.prompt(*(t.double() for t in split(x, shape)), [0, 200], scale)
    ref.check(out.reshape(200, H, D), o, to, "out")
    ref.check(lse, l, tl, "lse")


def test_prompt_strides_and_no_lse(ub):
    """Token-major and head-major views, other strides for each operand, no lse."""
    H, G, D, T = 4, 2, 64, 140
    q = normal(1, (H, T, D)).cuda().transpose(0, 1)       # head-major
    k = normal(2, (T, G, D + 16)).cuda()[..., :D]          # gaps between heads
    v = normal(3, (T, 3, G, D)).cuda()[:, 1]               # a slice of a wider matrix
    out = torch.full((H, T, D), math.nan, dtype=BF16, device="cuda").transpose(0, 1)
    cfg = ub.make_attn_cfg(H, G, D)
    with Rank(ub, T) as h:
        ub.ub_attn_prompt(h, ub.heads(q), ub.heads(k), ub.heads(v), ub.heads(out), None, i32([0, 60, T]), 2, cfg)
        torch.cuda.synchronize()
    o, _, to, _ = ref.prompt(q.double().cpu(), k.double().cpu(), v.double().cpu(), [0, 60, T], D ** -0.5)
    ref.check(out, o, to, "out")


def test_no_sequences(ub):
    """No sequence, and only empty ones: zeros everywhere."""
    H, G, D, T = 2, 1, 64, 5
    x = torch.full((T, (H + 2 * G) * D), math.nan, dtype=BF16, device="cuda")
    cfg = ub.make_attn_cfg(H, G, D)
    for cu in ([0], [0, 0, 0]):
        n = len(cu) - 1
        out, lse = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda"), torch.zeros((H, T), device="cuda")
        dx = torch.full_like(x, math.nan)
        ws = workspace(ub, ub.UB_ATTN_PROMPT_BWD, cfg, T, n)
        args = [ub.heads(x, c) for c in (0, H * D, (H + G) * D)]
        with Rank(ub, T) as h:
            ub.ub_attn_prompt(h, *args, ub.heads(out), lse, i32(cu), n, cfg)
            ub.ub_attn_prompt_bwd(h, ub.heads(out), *args, ub.heads(out), lse,
                                  *[ub.heads(dx, c) for c in (0, H * D, (H + G) * D)], i32(cu), n, cfg, ws)
            torch.cuda.synchronize()
        assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and bool((dx == 0).all())


def test_gradient_against_differences(ub):
    """The directional derivative of sum(out * dout) from the kernel's gradient against central
    differences of the 64-bit forward pass at the same bf16 point."""
    shape, lens = (4, 2, 64), [50, 1, 30]
    H, G, D = shape
    T, cu = sum(lens), cu_of(lens)
    x, _ = make(shape, lens, 0, 11)
    x = x[:, : (H + 2 * G) * D].contiguous()
    do = normal(12, (T, H * D))
    cfg = ub.make_attn_cfg(H, G, D)
    xd, dod = x.cuda(), do.cuda()
    out, lse = torch.empty((T, H * D), dtype=BF16, device="cuda"), torch.empty((H, T), device="cuda")
    dx = torch.empty_like(xd)
    ws = workspace(ub, ub.UB_ATTN_PROMPT_BWD, cfg, T, len(lens))
    args = [ub.heads(xd, c) for c in (0, H * D, (H + G) * D)]
    with Rank(ub, T) as h:
        ub.ub_attn_prompt(h, *args, ub.heads(out), lse, i32(cu), len(lens), cfg)
        ub.ub_attn_prompt_bwd(h, ub.heads(dod), *args, ub.heads(out), lse,
                              *[ub.heads(dx, c) for c in (0, H * D, (H + G) * D)], i32(cu), len(lens), cfg, ws)
        torch.cuda.synchronize()
    f = lambda y: (ref.prompt(*split(y, shape), cu, D ** -0.5)[0].reshape(T, -1) * do.double()).sum()
    _, tol = ref.prompt_bwd(do.double().reshape(T, H, D), *(t.double() for t in split(x, shape)), cu, D ** -0.5)
    tol = torch.cat([t.reshape(T, -1) for t in tol], 1)
    for seed in (1, 2, 3):
        e = torch.randn(x.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        step = 1e-4  # the difference's own error is of the order step^2
        want = (f(x.double() + step * e) - f(x.double() - step * e)) / (2 * step)
        got = (dx.double().cpu() * e).sum()
        bound = (tol * e.abs()).sum() + 1e-5 * abs(want) + 1e-4
        assert abs(got - want) <= bound, (seed, float(got), float(want), float(bound))


# ---- the cache ------------------------------------------------------------------------------
def make_cache(G, D, page, n_pages, f8, token_major, seed):
    shape = (n_pages, page, G, D) if token_major else (n_pages, G, page, D)
    xs = []
    for s in (seed, seed + 1):
        x = normal(s, shape)
        x = (x.float() * 40).to(F8) if f8 else x
        x = x.cuda()
        xs.append(x.transpose(1, 2) if token_major else x)
    return xs


def values(x):
    return (x.contiguous().view(torch.uint8).cpu().view(F8) if x.dtype == F8 else x.cpu()).double()


def raw(x):
    return x.contiguous().view(torch.uint8).clone()


APPENDS = [
    # H, G, D, rotary, interleaved, lens, past, page, e4m3, token_major, pad
    (8, 1, 128, 128, False, [1] * 16, 4096, 16, False, False, 0),
    (4, 4, 128, 128, False, [100, 0, 1, 37], 50, 64, False, True, 3),
    (8, 2, 128, 64, True, [70, 3], 2000, 24, True, False, 0),
    (6, 3, 80, 80, False, [33, 1], 7, 1, True, True, 1),
    (2, 1, 40, 32, True, [5, 90], 0, 128, False, False, 7),
    (2, 2, 64, 0, False, [20], 9, 16, False, False, 0),
    (5, 1, 64, 64, True, [9] * 90, 1000000, 16, False, False, 2),
]


@pytest.mark.parametrize("H,G,D,rotary,inter,lens,past,page,f8,token_major,pad", APPENDS)
def test_append(ub, H, G, D, rotary, inter, lens, past, page, f8, token_major, pad):
    n, used = len(lens), sum(lens)
    x, T = make((H, G, D), lens, pad, 3)
    pasts = [max(past - 3 * i, 0) for i in range(n)]
    first = [p // page for p in pasts]  # the table's earlier entries are never used: -1
    need = [-(-(p + m) // page) if m else f for p, m, f in zip(pasts, lens, first)]
    n_pages = max(sum(b - a for a, b in zip(first, need)), 1)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table, at = torch.full((n, max(max(need), 1)), -1, dtype=torch.int32), 0
    for i in range(n):
        table[i, first[i]: need[i]] = perm[at: at + need[i] - first[i]]
        at += need[i] - first[i]
    kc, vc = make_cache(G, D, page, n_pages, f8, token_major, 20)
    want = {"k": values(kc), "v": values(vc)}
    tols = {name: torch.zeros_like(w) for name, w in want.items()}
    ks, vs = 40.0, 60.0
    cfg = ub.make_attn_cfg(H, G, D, rotary_dim=rotary, rope_interleaved=inter)
    inv = (500000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1))).float()
    xd = x.cuda()
    q_out = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda")
    k_out = torch.full((T, G * D + 8), math.nan, dtype=BF16, device="cuda")
    with Rank(ub, T) as h:
        ub.ub_kv_append(h, ub.heads(xd), ub.heads(xd, H * D), ub.heads(xd, (H + G) * D), ub.heads(q_out),
                        ub.heads(k_out), inv.cuda() if rotary else None, i32(cu_of(lens)), i32(pasts), n,
                        ub.make_kv_cache(kc, vc, ks, vs), table.cuda(), cfg)
        torch.cuda.synchronize()
    pos = torch.tensor([p + j for p, m in zip(pasts, lens) for j in range(m)])
    seq = [i for i, m in enumerate(lens) for _ in range(m)]
    q, k, v = (t[:used].double() for t in split(x, (H, G, D)))
    yq, tq = ref.rotate(q, pos, inv, inter, rotary)
    yk, tk = ref.rotate(k, pos, inv, inter, rotary)
    ref.check(q_out[:used].reshape(used, H, D), yq, tq * (1 + ref.U16) + ref.U16 * yq.abs(), "q_out")
    ref.check(k_out[:used, : G * D].reshape(used, G, D), yk, tk * (1 + ref.U16) + ref.U16 * yk.abs(), "k_out")
    assert bool((q_out[used:] == 0).all()) and bool((k_out[used:, : G * D] == 0).all())
    assert bool(torch.isnan(k_out[:, G * D:]).all())
    for t in range(used):
        p = int(pos[t])
        pg, off = int(table[seq[t], p // page]), p % page
        for name, y, e, sc in (("k", yk, tk, ks), ("v", v, torch.zeros_like(v), vs)):
            if f8:  # one fp32 product, then E4M3: half a step, or 2^-10 among the subnormals
                w = (y[t] * sc).clamp(-448, 448)
                tols[name][pg, :, off] = (e[t] * sc + 2 * ref.U32 * w.abs()) * (1 + ref.U8) \
                    + torch.maximum(ref.U8 * w.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64))
            else:
                w = y[t]
                tols[name][pg, :, off] = e[t] * (1 + ref.U16) + ref.U16 * w.abs()
            want[name][pg, :, off] = w
    for name, c in (("k", kc), ("v", vc)):  # and every other slot as it was
        ref.check(values(c), want[name], tols[name], name + " cache")


def test_append_in_place_and_back(ub):
    """In place, and undone by the negated frequencies (two roundings to bf16)."""
    H, G, D, T = 4, 2, 64, 33
    x = normal(4, (T, (H + 2 * G) * D))
    xd = x.cuda()
    cfg = ub.make_attn_cfg(H, G, D)
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    q, k = ub.heads(xd), ub.heads(xd, H * D)
    with Rank(ub, T) as h:
        for f in (inv, -inv):
            ub.ub_kv_append(h, q, k, None, q, k, f, i32([0, 10, T]), None, 2, None, None, cfg)
        torch.cuda.synchronize()
    got, want = xd.double().cpu(), x.double()
    # a pair's norm bounds each rounding: u16 of it forth, u16 of it back
    y, w = got[:, : (H + G) * D].reshape(T, H + G, D), want[:, : (H + G) * D].reshape(T, H + G, D)
    norm = (w[..., : D // 2] ** 2 + w[..., D // 2:] ** 2).sqrt().repeat(1, 1, 2)
    assert bool(((y - w).abs() <= 3 * ref.U16 * norm).all())
    assert torch.equal(got[:, (H + G) * D:], want[:, (H + G) * D:])


@pytest.mark.parametrize("scale", [1.0, 0.37, 6e4])
def test_append_every_code(ub, scale):
    """Every bf16 value through an E4M3 cache: the codes ub_quantize_e4m3 gives, NaN's among them."""
    D, T = 64, 1024
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16).reshape(T, D).cuda()
    kc, vc = make_cache(1, D, 16, T // 16, True, False, 5)
    want = torch.empty((T, D), dtype=torch.uint8, device="cuda")
    table = torch.arange(T // 16, dtype=torch.int32, device="cuda")[None]
    with Rank(ub, T) as h:
        ub.ub_kv_append(h, None, ub.heads(x), ub.heads(x), None, None, None, i32([0, T]), None, 1,
                        ub.make_kv_cache(kc, vc, scale, scale), table, ub.make_attn_cfg(1, 1, D, rotary_dim=0))
        ub.ub_quantize_e4m3(x, D, want, D, T, D, scale)
        torch.cuda.synchronize()
    for c in (kc, vc):
        got = raw(c).reshape(T, D)
        bad = (got != want).flatten().nonzero().flatten()
        assert not len(bad), [(hex(i), int(got.flatten()[i]), int(want.flatten()[i])) for i in bad[:20].tolist()] + [len(bad)]


@pytest.mark.parametrize("T,H,G,D,rotary,inter,f8", [(2500, 6, 3, 80, 48, False, True), (5001, 5, 5, 64, 64, True, False),
                                                    (34001, 9, 1, 128, 112, True, True)])
def test_append_many_tokens(ub, T, H, G, D, rotary, inter, f8):
    """Several tokens to a workgroup, items of every section."""
    page, past = 64, 100
    x = normal(7, (T, (H + 2 * G) * D)).cuda()
    n_pages = -(-(T - 1 + past) // page)
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()[None]
    kc, vc = make_cache(G, D, page, n_pages, f8, True, 20)
    inv = (500000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)).float().cuda()
    q_out, k_out = torch.empty((T, H * D), dtype=BF16, device="cuda"), torch.empty((T, G * D), dtype=BF16, device="cuda")
    with Rank(ub, T) as h:
        ub.ub_kv_append(h, ub.heads(x), ub.heads(x, H * D), ub.heads(x, (H + G) * D), ub.heads(q_out), ub.heads(k_out),
                        inv, i32([0, T - 1]), i32([past]), 1, ub.make_kv_cache(kc, vc, 40.0, 60.0), table,
                        ub.make_attn_cfg(H, G, D, rotary_dim=rotary, rope_interleaved=inter))
        torch.cuda.synchronize()
    pos = past + torch.arange(T - 1, device="cuda")
    y, e = ref.rotate(x[:-1, : (H + G) * D].double().reshape(T - 1, H + G, D), pos, inv, inter, rotary)
    v = x[:-1, (H + G) * D:].double().reshape(T - 1, G, D)
    check = lambda got, w, e, what: ref.check(got, w.cpu(), (e * (1 + ref.U16) + ref.U16 * w.abs()).cpu(), what)
    check(q_out[:-1].reshape(T - 1, H, D), y[:, :H], e[:, :H], "q_out")
    check(k_out[:-1].reshape(T - 1, G, D), y[:, H:], e[:, H:], "k_out")
    assert bool((q_out[-1] == 0).all()) and bool((k_out[-1] == 0).all())
    at = table[0].long()[pos // page], pos % page
    for c, w, e, sc, what in ((kc, y[:, H:], e[:, H:], 40.0, "k"), (vc, v, torch.zeros_like(v), 60.0, "v")):
        got = (c.view(torch.uint8) if f8 else c)[at[0], :, at[1]]
        if f8:
            w = (w * sc).clamp(-448, 448)
            tol = (e * sc + 2 * ref.U32 * w.abs()) * (1 + ref.U8) + torch.maximum(ref.U8 * w.abs(), torch.full_like(w, 2.0 ** -10))
            ref.check(got.cpu().view(F8), w.cpu(), tol.cpu(), what)
        else:
            check(got, w, e, what)


def test_append_bad_pages(ub):
    """Tokens whose page is missing (negative position, past the table, a bad id) are not
    stored; the others are."""
    H, G, D, page = 2, 1, 64, 4
    lens, pasts = [6, 3, 2], [0, -2, 100]
    T, n_pages = sum(lens), 4
    x = normal(8, (T, (H + 2 * G) * D)).cuda()
    kc, vc = make_cache(G, D, page, n_pages, False, False, 30)
    before = raw(kc), raw(vc)
    table = i32([[2, n_pages], [1, -1], [0, 3]])
    cfg = ub.make_attn_cfg(H, G, D, rotary_dim=0)
    with Rank(ub, T) as h:
        ub.ub_kv_append(h, None, ub.heads(x, H * D), ub.heads(x, (H + G) * D), None, None, None, i32(cu_of(lens)),
                        i32(pasts), 3, ub.make_kv_cache(kc, vc), table, cfg)
        torch.cuda.synchronize()
    k, v = x[:, H * D:(H + G) * D], x[:, (H + G) * D:]
    for c, old, rows in ((kc, before[0], k), (vc, before[1], v)):
        old = old.view(BF16).view(n_pages, G, page, D)
        assert torch.equal(c[2, 0, :4], rows[0:4])          # sequence 0: page 2 holds, the next id is bad
        assert torch.equal(c[1, 0, 0], rows[8])             # sequence 1: positions -2, -1, 0
        assert torch.equal(c[1, 0, 1:], old[1, 0, 1:])
        assert torch.equal(c[0], old[0]) and torch.equal(c[3], old[3])


DECODES = [
    # H, G, D, lens, page, e4m3, token_major, pad
    (1, 1, 8, [1], 1, False, False, 0),
    (8, 1, 128, [1000], 64, False, False, 0),
    (4, 4, 128, [1, 0, 37, 300, 128, 129], 16, False, True, 2),
    (8, 1, 128, [5, 0, 700], 64, True, False, 1),
    (8, 2, 128, [100, 250], 24, True, True, 0),
    (6, 3, 80, [33, 1, 260], 1, True, False, 0),
    (6, 3, 80, [33, 1, 260], 128, False, False, 3),
    (5, 1, 64, [90] * 3, 16, False, False, 0),
    (16, 1, 128, [400], 16, False, False, 0),
    (40, 2, 64, [150, 3], 16, False, False, 0),  # a group of more than 16
    (2, 2, 64, [7, 0, 1] * 30, 24, True, False, 0),
    (2, 1, 96, [40000], 64, False, False, 0),
]


def decode_case(H, G, D, lens, page, f8, token_major, pad):
    n, T = len(lens), len(lens) + pad
    need = [-(-m // page) for m in lens]
    n_pages, most = max(sum(need), 1) + 1, max(max(need), 1)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    table, at = torch.full((n, most + 1), -1, dtype=torch.int32), 0
    kc, vc = make_cache(G, D, page, n_pages, f8, token_major, 40)
    for i, m in enumerate(need):
        table[i, :m] = perm[at: at + m]
        at += m
        if m and lens[i] % page:  # what the last page holds past the length is not looked at
            for c in (kc, vc):
                c.view(torch.uint8)[int(table[i, m - 1]), :, lens[i] % page:] = 0x7F if f8 else 0xFF
    q = torch.full((T, H * D), math.nan, dtype=BF16)
    q[:n] = normal(50, (n, H * D), 1.5)
    return n, T, kc, vc, table, q


@pytest.mark.parametrize("H,G,D,lens,page,f8,token_major,pad", DECODES)
def test_decode(ub, H, G, D, lens, page, f8, token_major, pad):
    n, T, kc, vc, table, q = decode_case(H, G, D, lens, page, f8, token_major, pad)
    ks, vs = (40.0, 60.0) if f8 else (1.0, 1.0)
    cfg = ub.make_attn_cfg(H, G, D)
    out = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda")
    lse = torch.full((H, T), math.nan, device="cuda")
    ws = workspace(ub, ub.UB_ATTN_DECODE, cfg, T, n)
    qd, td, ld = q.cuda(), table.cuda(), i32(lens)
    cache = ub.make_kv_cache(kc, vc, ks, vs)
    with Rank(ub, T) as h:
        ub.ub_attn_decode(h, ub.heads(qd), cache, td, ld, n, ub.heads(out), lse, cfg, ws)
        first = out.clone(), lse.clone()
        for _ in range(3):
            out.fill_(math.nan)
            ub.ub_attn_decode(h, ub.heads(qd), cache, td, ld, n, ub.heads(out), lse, cfg, ws)
        torch.cuda.synchronize()
    assert torch.equal(first[0].view(torch.int16), out.view(torch.int16)) and torch.equal(first[1], lse)
    kv, vv = values(kc) / ks, values(vc) / vs
    for i, m in enumerate(lens):
        got = out[i].reshape(H, D)
        if m == 0:
            assert bool((got == 0).all()) and bool((lse[:, i] == -math.inf).all())
            continue
        at = torch.arange(m)
        pg, off = table[i].long()[at // page], at % page
        for g in range(G):
            x = q[i].double().reshape(H, D)[g * (H // G):(g + 1) * (H // G)]
            mask = torch.ones(H // G, m, dtype=torch.bool)
            o, l, to, tl = ref.one(x, kv[pg, g, off], vv[pg, g, off], D ** -0.5, mask)
            ref.check(got[g * (H // G):(g + 1) * (H // G)], o, to, f"out {i} {g}")
            ref.check(lse[g * (H // G):(g + 1) * (H // G), i], l, tl, f"lse {i} {g}")
    assert bool((out[n:] == 0).all()) and bool((lse[:, n:] == -math.inf).all())



@pytest.mark.parametrize("H,G,D,lens,page,f8,token_major,pad", [
    (4, 2, 128, [0, 1, 31, 32, 33, 500, 2000] * 30, 16, True, True, 1),   # parts within and across ranges
    (4, 2, 128, [700, 0, 64, 5000] * 20, 48, False, False, 0),
    (3, 3, 72, [0, 257, 4100] * 25, 24, False, True, 0),                   # pages that a block of tokens leaves
    (2, 2, 48, [9000, 40, 17000], 32, True, False, 0),                    # over 32 steps of a wave
    (1, 1, 128, [70000], 16, False, False, 0),
    (600, 600, 16, [40, 90], 16, False, False, 0),                        # more heads than workgroups at once
])
def test_decode_ranges(ub, H, G, D, lens, page, f8, token_major, pad):
    test_decode(ub, H, G, D, lens, page, f8, token_major, pad)


def test_decode_bad_tables(ub):
    """A length past the table, a bad page id: NaN for that sequence, the others as ever."""
    H, G, D, page = 4, 2, 64, 16
    lens = [100, 20, 33, 40]
    n, T, kc, vc, table, q = decode_case(H, G, D, lens, page, False, False, 0)
    cfg = ub.make_attn_cfg(H, G, D)
    cache, qd = ub.make_kv_cache(kc, vc), q.cuda()
    outs = []
    for bad in (False, True):
        t, l = table.clone(), list(lens)
        if bad:
            t[0, 3] = -5
            t[2, 1] = 1 << 30
            l[3], l[1] = 1 << 30, -7
        out, lse = torch.zeros((T, H * D), dtype=BF16, device="cuda"), torch.zeros((H, T), device="cuda")
        ws = workspace(ub, ub.UB_ATTN_DECODE, cfg, T, n)
        with Rank(ub, T) as h:
            ub.ub_attn_decode(h, ub.heads(qd), cache, t.cuda(), i32(l), n, ub.heads(out), lse, cfg, ws)
            torch.cuda.synchronize()
        outs.append((out, lse))
    out, lse = outs[1]
    for i in (0, 2, 3):
        assert bool(torch.isnan(out[i]).all()) and bool(torch.isnan(lse[:, i]).all())
    assert bool((out[1] == 0).all()) and bool((lse[:, 1] == -math.inf).all())
    assert bool(torch.isfinite(outs[0][0]).all())
