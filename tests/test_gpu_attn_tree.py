"""GPU tests of drafted trees against 64 bits: attention over a paged cache, the append with
rotations by depth, and the move of accepted tokens."""

import math

import pytest
import torch

from tests import attn_ref as ref
from tests.test_gpu_attn import (BF16, F8, Rank, cu_of, i32, make, make_cache, normal, raw, split, ub, values,  # noqa: F401
                                 workspace)

pytestmark = pytest.mark.gpu


def tree(m, kind, seed):
    """Parents of m nodes: a chain, all of them roots, or any node before."""
    g = torch.Generator().manual_seed(seed)
    if kind == "chain":
        return list(range(-1, m - 1))
    if kind == "roots":
        return [-1] * m
    return [int(torch.randint(-1, j, (1,), generator=g)) if j else -1 for j in range(m)]


def seen_of(parents):
    m = len(parents)
    see = torch.zeros((m, m), dtype=torch.bool)
    for j, p in enumerate(parents):
        if 0 <= p < j:
            see[j] = see[p]
        see[j, j] = True
    return see


def make_case(H, G, D, trees, past, page, f8, token_major, pad):
    n, lens = len(trees), [len(t) for t in trees]
    T, full = sum(lens) + pad, [p + m for p, m in zip(past, lens)]
    need = [-(-m // page) for m in full]
    n_pages = sum(need) + 1
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    table, at = torch.full((n, max(need + [1]) + 1), -1, dtype=torch.int32), 0
    kc, vc = make_cache(G, D, page, n_pages, f8, token_major, 40)
    for i, m in enumerate(need):
        table[i, :m] = perm[at: at + m]
        at += m
        if m and full[i] % page:  # what the last page holds past the length is not looked at
            for c in (kc, vc):
                c.view(torch.uint8)[int(table[i, m - 1]), :, full[i] % page:] = 0x7F if f8 else 0xFF
    q = torch.full((T, H * D), math.nan, dtype=BF16)
    q[: sum(lens)] = normal(50, (sum(lens), H * D), 1.5)
    parents = torch.full((T,), 12345, dtype=torch.int32)
    parents[: sum(lens)] = torch.tensor([p for t in trees for p in t], dtype=torch.int32)
    return lens, T, full, kc, vc, table, q, parents


def attend(ub, q, cache, table, full, parents, lens, shape, T, times=2):  # noqa: F811
    H, G, D = shape
    cfg = ub.make_attn_cfg(H, G, D)
    out = torch.full((T, H * D + 8), math.nan, dtype=BF16, device="cuda")
    lse = torch.full((H, T), math.nan, device="cuda")
    ws = workspace(ub, ub.UB_ATTN_TREE, cfg, T, len(lens))
    ws.fill_(0xFF)
    qd, td, fd, pd, cu = q.cuda(), table.cuda(), i32(full), parents.cuda(), i32(cu_of(lens))
    first = None
    with Rank(ub, T) as h:
        for _ in range(times):
            ub.ub_attn_tree(h, ub.heads(qd), cache, td, fd, pd, cu, len(lens), ub.heads(out), lse, cfg, ws)
            got = out.clone(), lse.clone()
            first = first or got
            out.fill_(math.nan)
        torch.cuda.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert bool(torch.isnan(got[0][:, H * D:]).all())
    return got[0][:, : H * D], got[1]


def check_rows(out, lse, q, kv, vv, table, trees, full, page, shape, skip=()):
    H, G, D = shape
    row = 0
    for i, t in enumerate(trees):
        m = len(t)
        at = torch.arange(full[i])
        pg, off = table[i].long()[at // page], at % page
        see = torch.cat((torch.ones((m, full[i] - m), dtype=torch.bool), seen_of(t)), 1)
        for h in range(H if m and i not in skip else 0):
            x = q[row: row + m, h * D: (h + 1) * D].double()
            k, v = kv[pg, h // (H // G), off], vv[pg, h // (H // G), off]
            o, l, to, tl = ref.one(x, k, v, D ** -0.5, see)
            ref.check(out[row: row + m, h * D: (h + 1) * D], o, to, f"out {i} {h}")
            ref.check(lse[h, row: row + m], l, tl, f"lse {i} {h}")
        row += m
    assert bool((out[row:] == 0).all()) and bool((lse[:, row:] == -math.inf).all())


TREES = [
    # H, G, D, nodes, past, page, e4m3, token_major, pad
    (1, 1, 8, [1], [0], 1, False, False, 0),
    (8, 1, 128, [24], [1000], 64, False, False, 0),
    (4, 4, 128, [1, 0, 7, 60, 64, 65], [1, 0, 37, 300, 128, 129], 16, False, True, 2),
    (8, 1, 128, [5, 0, 30], [5, 3, 700], 64, True, False, 1),
    (8, 2, 128, [10, 25], [100, 250], 24, True, True, 0),
    (6, 3, 80, [33, 1, 20], [33, 0, 260], 1, True, False, 0),
    (6, 3, 80, [3, 1, 2], [33, 1, 260], 128, False, False, 3),
    (5, 1, 64, [9] * 3, [90] * 3, 16, False, False, 0),
    (16, 1, 128, [256], [400], 16, False, False, 0),
    (16, 1, 96, [256, 3], [0, 70], 16, True, False, 0),
    (40, 2, 64, [15, 3], [150, 3], 16, False, False, 0),
    (2, 2, 64, [7, 0, 1] * 30, [0, 5, 64] * 30, 24, True, False, 0),
    (2, 1, 96, [1], [20000], 64, False, False, 0),
    (2, 1, 40, [100, 256, 17], [3000, 64, 4000], 48, False, False, 0),
    (8, 1, 128, [60, 31, 50, 44] * 3, [2000, 30, 900, 5] * 3, 64, True, False, 0),
    # 17 to 32 columns, and few, of each type and size
    (4, 1, 128, [6, 8, 5], [700, 64, 3], 16, False, False, 0),
    (4, 1, 128, [6, 8, 5], [700, 64, 3], 16, True, True, 0),
    (3, 1, 96, [9, 8], [128, 1000], 40, True, False, 1),
    (3, 1, 80, [9, 8], [128, 1000], 40, False, True, 1),
    (8, 8, 128, [3, 9], [5000, 100], 64, True, False, 0),
    (2, 1, 48, [30, 25], [300, 77], 16, True, True, 3),
]


@pytest.mark.parametrize("H,G,D,nodes,past,page,f8,token_major,pad", TREES)
@pytest.mark.parametrize("kind", ["any", "chain", "roots"])
def test_tree(ub, H, G, D, nodes, past, page, f8, token_major, pad, kind):  # noqa: F811
    trees = [tree(m, kind, i) for i, m in enumerate(nodes)]
    lens, T, full, kc, vc, table, q, parents = make_case(H, G, D, trees, past, page, f8, token_major, pad)
    ks, vs = (40.0, 60.0) if f8 else (1.0, 1.0)
    out, lse = attend(ub, q, ub.make_kv_cache(kc, vc, ks, vs), table, full, parents, lens, (H, G, D), T)
    check_rows(out.cpu(), lse.cpu(), q, values(kc) / ks, values(vc) / vs, table, trees, full, page, (H, G, D))


def test_tree_many_sequences(ub):  # noqa: F811
    """More sequences than lanes, lengths of many sizes, parts within and across ranges."""
    H, G, D = 4, 2, 64
    nodes = [3, 0, 17, 40, 1, 8, 30] * 12
    past = [0, 4, 65, 3000, 31, 640, 12] * 12
    trees = [tree(m, "any", i) for i, m in enumerate(nodes)]
    lens, T, full, kc, vc, table, q, parents = make_case(H, G, D, trees, past, 16, False, True, 3)
    out, lse = attend(ub, q, ub.make_kv_cache(kc, vc), table, full, parents, lens, (H, G, D), T)
    check_rows(out.cpu(), lse.cpu(), q, values(kc), values(vc), table, trees, full, 16, (H, G, D))


@pytest.mark.parametrize("f8", [False, True])
def test_tree_two_rounds_of_parts(ub, f8):  # noqa: F811
    """So much work that parts are cut for two rounds of workgroups."""
    H, G, D = 16, 1, 16
    nodes, past = [30, 9] * 24, [9000, 14000] * 24
    trees = [tree(m, "any", i) for i, m in enumerate(nodes)]
    lens, T, full, kc, vc, table, q, parents = make_case(H, G, D, trees, past, 64, f8, False, 1)
    ks, vs = (40.0, 60.0) if f8 else (1.0, 1.0)
    out, lse = attend(ub, q, ub.make_kv_cache(kc, vc, ks, vs), table, full, parents, lens, (H, G, D), T)
    check_rows(out.cpu(), lse.cpu(), q, values(kc) / ks, values(vc) / vs, table, trees, full, 64, (H, G, D))


@pytest.mark.parametrize("low,high", [(0.0, 60.0), (-300.0, 300.0), (100.0, -100.0)])
@pytest.mark.parametrize("H,m", [(1, 4), (2, 200), (8, 30)])
def test_scores_that_rise_and_fall(ub, low, high, H, m):  # noqa: F811
    D, L, page = 16, 700, 16
    trees = [tree(m, "any", 1)]
    lens, T, full, kc, vc, table, q, parents = make_case(H, 1, D, trees, [L - m], page, False, False, 0)
    at = torch.arange(L)
    q[:, ::D] = 4.0
    pages = table[0].long()[at // page].cuda(), (at % page).cuda()
    kc[pages[0], 0, pages[1], 0] = (torch.linspace(low, high, L) / 4 / D ** -0.5).to(BF16).cuda()
    out, lse = attend(ub, q, ub.make_kv_cache(kc, vc), table, full, parents, lens, (H, 1, D), T)
    check_rows(out.cpu(), lse.cpu(), q, values(kc), values(vc), table, trees, full, page, (H, 1, D))


@pytest.mark.parametrize("H,G,D,m", [(2, 1, 64, 9), (8, 1, 128, 60), (4, 4, 96, 40), (16, 1, 128, 30)])
def test_values_on_other_paths(ub, H, G, D, m):  # noqa: F811
    """NaN and inf in a node's key and value: rows whose path does not hold it are as without."""
    page = 16
    trees = [tree(m, "any", 3), tree(m, "any", 4)]
    lens, T, full, kc, vc, table, q, parents = make_case(H, G, D, trees, [150, 31], page, False, False, 0)
    kv, vv = values(kc), values(vc)
    bad = m // 3
    for i in range(2):
        pos = full[i] - m + bad
        kc[int(table[i, pos // page]), :, pos % page, ::2] = math.inf
        vc[int(table[i, pos // page]), :, pos % page] = math.nan
        vc[int(table[i, pos // page]), :, pos % page, -1] = -math.inf
    out, lse = (x.cpu() for x in attend(ub, q, ub.make_kv_cache(kc, vc), table, full, parents, lens, (H, G, D), T))
    for i, t in enumerate(trees):
        rows = (~seen_of(t)[:, bad]).nonzero().flatten()
        assert len(rows) > 2
        at = torch.arange(full[i])
        pg, off = table[i].long()[at // page], at % page
        see = torch.cat((torch.ones((m, full[i] - m), dtype=torch.bool), seen_of(t)), 1)[rows]
        for h in range(H):
            x = q[i * m: (i + 1) * m, h * D: (h + 1) * D].double()[rows]
            o, l, to, tl = ref.one(x, kv[pg, h // (H // G), off], vv[pg, h // (H // G), off], D ** -0.5, see)
            ref.check(out[i * m: (i + 1) * m, h * D: (h + 1) * D][rows], o, to, f"out {i} {h}")
            ref.check(lse[h, i * m: (i + 1) * m][rows], l, tl, f"lse {i} {h}")


def test_bad_lengths_tables_and_parents(ub):  # noqa: F811
    """NaN for a sequence whose length, rows or pages are not there; parents that are no earlier
    node count as none; the other sequences as ever."""
    H, G, D, page = 4, 2, 64, 16
    nodes, past = [5, 4, 6, 300, 7, 3], [100, 20, 33, 40, 10, 50]
    trees = [tree(m, "any", i) for i, m in enumerate(nodes)]
    lens, T, full, kc, vc, table, q, parents = make_case(H, G, D, trees, past, page, False, False, 2)
    l, t = list(full), table.clone()
    l[1] = 3                      # fewer tokens than nodes
    t[2, 1] = 1 << 30             # a bad page
    l[4] = 1 << 30                # past the table; sequence 3 has too many nodes
    parents[0], parents[2], parents[3] = 5, 2, -77
    trees[0][0], trees[0][2], trees[0][3] = -1, -1, -1
    out, lse = (x.cpu() for x in attend(ub, q, ub.make_kv_cache(kc, vc), t, l, parents, lens, (H, G, D), T))
    row = 0
    for i, m in enumerate(nodes):
        if i in (1, 2, 3, 4):
            assert bool(torch.isnan(out[row: row + m]).all()) and bool(torch.isnan(lse[:, row: row + m]).all()), i
        row += m
    check_rows(out, lse, q, values(kc), values(vc), table, trees, full, page, (H, G, D), skip=(1, 2, 3, 4))


def test_no_sequences(ub):  # noqa: F811
    H, G, D, T = 2, 1, 64, 5
    kc, vc = make_cache(G, D, 16, 2, False, False, 1)
    q, parents = torch.full((T, H * D), math.nan, dtype=BF16), torch.zeros(T, dtype=torch.int32)
    for n in (0, 2):
        out, lse = attend(ub, q, ub.make_kv_cache(kc, vc), torch.zeros((max(n, 1), 1), dtype=torch.int32), [3] * n, parents,
                          [0] * n, (H, G, D), T)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


# ---- the append and the move of accepted tokens ----------------------------------------------
APPENDS = [
    # H, G, D, rotary, interleaved, nodes, past, page, e4m3, token_major, pad
    (8, 1, 128, 128, False, [24] * 4, [4000, 1, 77, 63], 16, False, False, 0),
    (4, 4, 128, 128, False, [30, 0, 1, 37], [50, 3, 0, 9], 64, False, True, 3),
    (8, 2, 128, 64, True, [40, 3], [2000, 17], 24, True, False, 0),
    (6, 3, 80, 80, False, [33, 1], [7, 1], 1, True, True, 1),
]


@pytest.mark.parametrize("H,G,D,rotary,inter,nodes,past,page,f8,token_major,pad", APPENDS)
def test_append_at(ub, H, G, D, rotary, inter, nodes, past, page, f8, token_major, pad):  # noqa: F811
    trees = [tree(m, "any", i) for i, m in enumerate(nodes)]
    lens, T, full, kc, vc, table, _, _ = make_case(H, G, D, trees, past, page, f8, token_major, pad)
    x, _ = make((H, G, D), nodes, pad, 3)
    used = sum(nodes)
    offsets = torch.full((T,), -(1 << 31), dtype=torch.int64)
    offsets[:used] = torch.randint(-3, 50, (used,), generator=torch.Generator().manual_seed(6))
    kc2, vc2 = kc.clone(), vc.clone()
    ks, vs = 40.0, 60.0
    cfg = ub.make_attn_cfg(H, G, D, rotary_dim=rotary, rope_interleaved=inter)
    inv = (500000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)).float()
    xd = x.cuda()
    q_out = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda")
    k_out = torch.full((T, G * D + 8), math.nan, dtype=BF16, device="cuda")
    rest = (ub.heads(xd), ub.heads(xd, H * D), ub.heads(xd, (H + G) * D), ub.heads(q_out), ub.heads(k_out), inv.cuda())
    place = torch.tensor([j for m in nodes for j in range(m)] + [0] * pad, dtype=torch.int32).cuda()
    with Rank(ub, T) as h:
        ub.ub_kv_append_at(h, *rest, offsets.to(torch.int32).cuda(), i32(cu_of(nodes)), i32(past), len(nodes),
                           ub.make_kv_cache(kc, vc, ks, vs), table.cuda(), cfg)
        torch.cuda.synchronize()
        got = q_out.clone(), k_out.clone()
        # offsets that say a row's own place: the same bits as without
        ub.ub_kv_append_at(h, *rest, place, i32(cu_of(nodes)), i32(past), len(nodes), ub.make_kv_cache(kc2, vc2, ks, vs),
                           table.cuda(), cfg)
        same = q_out.clone(), raw(kc2), raw(vc2)
        ub.ub_kv_append(h, *rest, i32(cu_of(nodes)), i32(past), len(nodes), ub.make_kv_cache(kc2, vc2, ks, vs),
                        table.cuda(), cfg)
        torch.cuda.synchronize()
    assert torch.equal(same[0].view(torch.int16), q_out.view(torch.int16))
    assert torch.equal(same[1], raw(kc2)) and torch.equal(same[2], raw(vc2))
    seq = torch.tensor([i for i, m in enumerate(nodes) for _ in range(m)])
    pos = torch.tensor(past)[seq] + offsets[:used]
    q, k, v = (t[:used].double() for t in split(x, (H, G, D)))
    yq, tq = ref.rotate(q, pos, inv, inter, rotary)
    yk, tk = ref.rotate(k, pos, inv, inter, rotary)
    ref.check(got[0][:used].reshape(used, H, D), yq, tq * (1 + ref.U16) + ref.U16 * yq.abs(), "q_out")
    ref.check(got[1][:used, : G * D].reshape(used, G, D), yk, tk * (1 + ref.U16) + ref.U16 * yk.abs(), "k_out")
    assert bool((got[0][used:] == 0).all())
    at = torch.tensor([p + j for p, m in zip(past, nodes) for j in range(m)])
    pg, off = table.long()[seq, at // page], at % page
    for c, y, e, sc, what in ((kc, yk, tk, ks, "k"), (vc, v, torch.zeros_like(v), vs, "v")):
        g = values(c)[pg, :, off]
        if f8:
            w = (y * sc).clamp(-448, 448)
            tol = (e * sc + 2 * ref.U32 * w.abs()) * (1 + ref.U8) + torch.maximum(ref.U8 * w.abs(), torch.full_like(w, 2.0 ** -10))
            ref.check(g, w, tol, what)
        else:
            ref.check(g, y, e * (1 + ref.U16) + ref.U16 * y.abs(), what)


COMPACTS = [
    # G, D, page, e4m3, token_major, lens, kept
    (1, 128, 16, False, False, [100, 0, 31], [[0, 3, 4, 9], [], [2, 3]]),
    (4, 128, 64, False, True, [63, 64, 1], [[0, 1, 2], [1, 2, 3, 7, 63, 64, 65, 130], [5]]),
    (3, 80, 1, True, False, [5, 7], [list(range(1, 40)), list(range(0, 80, 3))]),
    (2, 8, 24, False, False, [0], [list(range(1, 1500, 2))]),          # an eviction
    (1, 128, 48, True, True, [0, 11], [list(range(700, 1400)), list(range(3, 900, 2))]),
]


@pytest.mark.parametrize("G,D,page,f8,token_major,lens,kept", COMPACTS)
def test_compact(ub, G, D, page, f8, token_major, lens, kept):  # noqa: F811
    n, per = len(lens), -(-1600 // page)
    kc, vc = make_cache(G, D, page, n * per, f8, token_major, 9)
    table = torch.randperm(n * per, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(n, per)
    most = max(len(x) for x in kept) + 1
    lists = torch.full((n, most + 3), -1, dtype=torch.int32)
    for i, x in enumerate(kept):
        lists[i, : len(x)] = torch.tensor(x, dtype=torch.int32)
    want = {}
    for name, c in (("k", kc), ("v", vc)):
        w = raw(c).view(n * per, G, page, -1).clone()
        old = w.clone()
        for i, x in enumerate(kept):
            for d, j in enumerate(x):
                a, b = lens[i] + j, lens[i] + d
                w[int(table[i, b // page]), :, b % page] = old[int(table[i, a // page]), :, a % page]
        want[name] = w
    out = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    with Rank(ub, 8) as h:
        ub.ub_kv_compact(h, ub.make_kv_cache(kc, vc, 1.0, 1.0), table.cuda(), i32(lens), lists.cuda()[:, :most],
                         i32([len(x) for x in kept]), n, out, ub.make_attn_cfg(G, G, D, rotary_dim=0))
        torch.cuda.synchronize()
    assert out.tolist() == [a + len(x) for a, x in zip(lens, kept)]
    for name, c in (("k", kc), ("v", vc)):
        assert torch.equal(raw(c).view(n * per, G, page, -1), want[name]), name


def test_compact_bad_lists(ub):  # noqa: F811
    """A list ends before an entry that does not rise, is negative or lies past the table; counts
    beyond the rows' entries, bad pages."""
    G, D, page, per = 1, 64, 4, 5
    lens = [3, 2, 0, 15, -4, 1, 2]
    kept = [[1, 2, 2, 5], [-1, 3, 4, 5], [0, 4, 3, 9], [2, 4, 5, 6], [1, 2, 3, 4], [1, 3, 5, 7], [2, 3, 9, 10]]
    counts = [4, 4, 4, 4, 99, -3, 4]
    n = len(lens)
    kc, vc = make_cache(G, D, page, n * per, False, False, 9)
    old = raw(kc).view(n * per, page, -1)
    table = torch.arange(n * per, dtype=torch.int32).view(n, per)
    table[6, 1] = n * per  # tokens 4 to 7: neither read nor written
    out = torch.zeros(n, dtype=torch.int32, device="cuda")
    with Rank(ub, 8) as h:
        ub.ub_kv_compact(h, ub.make_kv_cache(kc, vc), table.cuda(), i32(lens), i32(kept), i32(counts), n, out,
                         ub.make_attn_cfg(1, 1, D, rotary_dim=0))
        torch.cuda.synchronize()
    valid = [[1, 2], [], [0, 4], [2, 4], [1, 2, 3, 4], [], [2, 3, 9, 10]]
    base = [max(x, 0) for x in lens]
    assert out.tolist() == [a + len(x) for a, x in zip(base, valid)]
    want = old.clone()
    for i, x in enumerate(valid):
        for d, j in enumerate(x):
            a, b = base[i] + j, base[i] + d
            if max(int(table[i, a // page]), int(table[i, b // page])) < n * per:
                want[int(table[i, b // page]), b % page] = old[int(table[i, a // page]), a % page]
    assert torch.equal(raw(kc).view(n * per, page, -1), want)


def far_cache(seed, n_pages=3, G=2, page=16, D=64):
    """Pages 2^31 elements apart, each offset past 32 bits but the first's."""
    caches = []
    for s in (seed, seed + 1):
        flat = torch.empty((n_pages - 1) * (1 << 31) + G * page * D, dtype=BF16, device="cuda")
        c = flat.as_strided((n_pages, G, page, D), (1 << 31, page * D, D, 1))
        c.copy_(normal(s, (n_pages, G, page, D)).cuda())
        caches.append(c)
    return caches


def test_offsets_past_32_bits(ub):  # noqa: F811
    """Trees, windowed decode, accepted tokens, copies and the append over pages far apart."""
    H, G, D, page = 4, 2, 64, 16
    kc, vc = far_cache(5)
    trees = [[-1, 0, 0, 1, -1]]
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    q = normal(50, (5, H * D), 1.5)
    cache = ub.make_kv_cache(kc, vc)
    kv, vv = kc.double().cpu(), vc.double().cpu()
    out, lse = attend(ub, q, cache, table, [45], torch.tensor(trees[0], dtype=torch.int32), [5], (H, G, D), 5)
    check_rows(out.cpu(), lse.cpu(), q, kv, vv, table, trees, [45], page, (H, G, D))
    cfg = ub.make_attn_cfg(H, G, D, rotary_dim=0)
    dec, dl = torch.zeros((5, H * D), dtype=BF16, device="cuda"), torch.zeros((H, 5), device="cuda")
    ws = workspace(ub, ub.UB_ATTN_DECODE_WINDOW, cfg, 5, 1)
    x = normal(60, (5, 2 * G * D)).cuda()
    td, qd = table.cuda(), q.cuda()
    with Rank(ub, 5) as h:
        ub.ub_attn_decode_window(h, ub.heads(qd), cache, td, i32([45]), 1, ub.make_attn_window(20, 3), ub.heads(dec), dl, cfg, ws)
        ub.ub_kv_append_at(h, None, ub.heads(x), ub.heads(x, G * D), None, None, None, i32([0] * 5), i32([0, 5]), i32([40]), 1,
                           cache, td, cfg)
        ub.ub_kv_compact(h, cache, td, i32([10]), i32([[2, 8, 30, 33]]), i32([4]), 1, i32([0]), cfg)
        ub.ub_kv_copy_pages(h, cache, i32([[2, 1, 7]]), 1, cfg)
        torch.cuda.synchronize()
    at = torch.tensor([0, 1, 2] + list(range(25, 45)))
    pg, off = table[0].long()[at // page], at % page
    for hh in range(H):
        o, l, to, tl = ref.one(q[:1, hh * D: (hh + 1) * D].double(), kv[pg, hh // 2, off], vv[pg, hh // 2, off], D ** -0.5,
                               torch.ones((1, len(at)), dtype=torch.bool))
        ref.check(dec[:1, hh * D: (hh + 1) * D], o, to, "decode")
        ref.check(dl[hh, :1], l, tl, "decode lse")
    for c, want, col in ((kc, kv, 0), (vc, vv, G * D)):
        for j in range(5):
            want[1, :, 8 + j] = x[j, col: col + G * D].double().cpu().view(G, D)
        old = want.clone()
        for d, j in enumerate((2, 8, 30, 33)):
            a, b = 10 + j, 10 + d
            want[int(table[0, b // page]), :, b % page] = old[int(table[0, a // page]), :, a % page]
        want[1, :, :7] = want[2, :, :7]
        assert torch.equal(c.double().cpu(), want)


@pytest.mark.parametrize("shape", [(4, 4, 128), (2, 1, 64), (4, 2, 96)])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("kind", ["roots", "chain", "any"])
def test_short_pasts(ub, shape, f8, kind):  # noqa: F811
    """Trees that begin in a group's first tile, after no token or a few: nodes that see none of a group's keys,
    but some of another's."""
    H, G, D = shape
    nodes, past = [24, 30, 17, 1, 24, 16, 9, 30], [0, 0, 5, 0, 33, 40, 50, 63]
    trees = [tree(m, kind, i) for i, m in enumerate(nodes)]
    lens, T, full, kc, vc, table, q, parents = make_case(H, G, D, trees, past, 16, f8, False, 1)
    ks, vs = (40.0, 60.0) if f8 else (1.0, 1.0)
    out, lse = attend(ub, q, ub.make_kv_cache(kc, vc, ks, vs), table, full, parents, lens, shape, T)
    check_rows(out.cpu(), lse.cpu(), q, values(kc) / ks, values(vc) / vs, table, trees, full, 16, shape)
