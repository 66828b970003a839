"""GPU tests of the attention block with a pool of pages: forks, drafted trees and their accepted
paths against the same tokens decoded one by one, a windowed block, and the calls together on
another stream and in a replayed graph."""

import math

import pytest
import torch

from tests import attn_ref as ref
from tests import window_ref as wref

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cached(b, i, n, page):
    """The bytes of sequence i's first n cached keys and values."""
    at = torch.arange(n)
    pg, off = b.pages[i].long().cpu()[at // page], at % page
    return [c.view(torch.uint8).cpu()[pg, :, off] for c in (b.k_cache, b.v_cache)]


def counted(b, page):
    """The counts that the table and the held lengths say."""
    want = torch.zeros(b.refs.shape[0], dtype=torch.int32)
    for row, n in zip(b.pages.tolist(), b.held.tolist()):
        for p in row[: -(-n // page)]:
            if p >= 0:
                want[p] += 1
    assert torch.equal(b.refs.cpu(), want)
    return int((want == 0).sum())


@pytest.mark.parametrize("cache,tp", [(BF16, 1), (F8, 4)])
def test_forks_and_drafts(cache, tp):
    """Two prompts, forked; trees of drafts, of which paths are accepted; more decoded tokens: the
    cache holds the bits that the same tokens leave when a block decodes them one by one, and
    each node's attention is that of its path."""
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    H, G, D, hidden, page = 4, 2, 64, 256, 16
    ks, vs = (30.0, 50.0) if cache is F8 else (1.0, 1.0)
    wqkv, wo = normal(1, hidden, (H + 2 * G) * D) / 16, normal(2, H * D, hidden) / 16
    make = lambda **kw: AttentionBlock(wqkv, wo, H, G, D, capacity=512, max_seqs=5, max_len=300, page=page, tp=tp, cache=cache,
                                       k_scale=ks, v_scale=vs, **kw)
    b = make(n_pages=60)
    lens = [100, 33]
    x = normal(3, sum(lens), hidden)
    b.prefill(x, lens)
    assert counted(b, page) == 60 - 7 - 3
    b.fork(i32([0, 1, 0, 1, 0]))
    assert counted(b, page) == 60 - 7 - 3 and b.lens.tolist() == [100, 33, 100, 33, 100]
    source = [0, 1, 0, 1, 0]
    trees = [[-1, 0, 1, 0, 3, -1], [-1], [-1, -1, 1, 2], [-1, 0, 0, 1], [-1, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13]]
    paths = [[0, 3, 4], [], [1, 2], [0, 1, 3], list(range(13))]
    nodes = normal(4, sum(len(t) for t in trees), hidden)
    b.draft(nodes, trees)
    rows = nodes.shape[0]
    kc, vc = ((c.view(torch.uint8).cpu().view(F8).double() if cache is F8 else c.double().cpu()) for c in (b.k_cache, b.v_cache))
    first = 0
    for i, t in enumerate(trees):
        see = torch.zeros((len(t), len(t)), dtype=torch.bool)
        for j, p in enumerate(t):
            if p >= 0:
                see[j] = see[p]
            see[j, j] = True
        n = int(b.lens[i])
        at = torch.arange(n + len(t))
        pg, off = b.pages[i].long().cpu()[at // page], at % page
        mask = torch.cat((torch.ones((len(t), n), dtype=torch.bool), see), 1)
        for h in range(H):
            q = b.q[first: first + len(t), h * D: (h + 1) * D].double().cpu()
            o, _, tol, _ = ref.one(q, kc[pg, h // 2, off] / ks, vc[pg, h // 2, off] / vs, D ** -0.5, mask)
            ref.check(b.attn[first: first + len(t), h * D: (h + 1) * D], o, tol, f"draft {i} {h}")
        first += len(t)
    assert first == rows
    kept = torch.full((5, 16), -1, dtype=torch.int32)
    for i, p in enumerate(paths):
        kept[i, : len(p)] = torch.tensor(p, dtype=torch.int32)
    b.accept(kept.cuda(), i32([len(p) for p in paths]))
    want_lens = [lens[s] + len(p) for s, p in zip(source, paths)]
    assert b.lens.tolist() == want_lens
    counted(b, page)
    more = [normal(20 + s, 5, hidden) for s in range(3)]
    for t in more:
        b.decode(t)
    free = counted(b, page)

    # the same tokens, one by one, in a block whose sequences have their own pages
    plain = make()
    full = [torch.cat((x[:100] if s == 0 else x[100:],)) for s in source]
    plain.prefill(torch.cat(full), [len(f) for f in full])
    starts = [0]
    for t in trees:
        starts.append(starts[-1] + len(t))
    for step in range(max(len(p) for p in paths)):
        rows_ = torch.stack([nodes[starts[i] + p[step]] if step < len(p) else nodes[0] for i, p in enumerate(paths)])
        before = plain.lens.clone()
        plain.decode(rows_)
        done = i32([step < len(p) for p in paths])
        plain.lens.copy_(before + done)  # a token past a path's end is written over by the next one
    for t in more:
        plain.decode(t)
    assert plain.lens.tolist() == b.lens.tolist() == [n + 3 for n in want_lens]
    for i, n in enumerate(b.lens.tolist()):
        for got, w, what in zip(cached(b, i, n, page), cached(plain, i, n, page), "kv"):
            assert torch.equal(got, w), (i, what)
    # and the last step's rows, which read the same bits
    assert torch.equal(b.q[:5], plain.q[:5])
    assert torch.equal(b.attn[:5].view(torch.int16), plain.attn[:5].view(torch.int16))
    b.prefill(x, lens)  # everything before is given back
    assert counted(b, page) == 60 - 7 - 3 and free < 60 - 10
    torch.cuda.synchronize()
    b.close()
    plain.close()


def test_draft_refusals():
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    w = normal(1, 128, 256), normal(2, 128, 128)
    b = AttentionBlock(*w, 2, 1, 64, capacity=300, max_seqs=2, max_len=64)
    x = normal(3, 4, 128)
    for trees in ([[-1, 1, 0, 0]], [[-1, -2, 0, 0]], [[-1, 0, 3, 0]], [[-1, 0]], [[-1] * 300]):
        with pytest.raises(ValueError, match="draft"):
            b.draft(x, trees)
    with pytest.raises(ValueError, match="fork"):
        b.fork(i32([0]))
    b.close()
    b = AttentionBlock(*w, 2, 1, 64, capacity=300, max_seqs=2, max_len=64, window=8)
    with pytest.raises(ValueError, match="window"):
        b.draft(x, [[-1, 0, 1, 2]])
    b.close()


@pytest.mark.parametrize("pool", [False, True])
def test_windowed_block(pool):
    """Prompts, decode steps and a training step under a window; a pool takes back what it hides."""
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    H, G, D, hidden, page, W, S = 4, 1, 64, 128, 16, 50, 3
    wqkv, wo = normal(1, hidden, (H + 2 * G) * D) / 11, normal(2, H * D, hidden) / 16
    b = AttentionBlock(wqkv, wo, H, G, D, capacity=512, max_seqs=2, max_len=300, page=page, tp=2, window=W, sinks=S,
                       n_pages=30 if pool else None)
    lens = [200, 41]
    x = normal(3, 241, hidden)
    b.prefill(x, lens)
    q, k = b.q[:241].view(241, H, D).double().cpu(), b.k[:241].view(241, G, D).double().cpu()
    v = b.qkv[:241, (H + G) * D:].reshape(241, G, D).double().cpu()
    cu = [0, 200, 241]
    o, _, t, _ = wref.prompt(q, k, v, cu, D ** -0.5, W, S)
    ref.check(b.attn[:241].view(241, H, D), o, t, "prompt")
    for s in range(20):
        b.decode(normal(10 + s, 2, hidden))
    assert b.lens.tolist() == [220, 61]
    for i, n in enumerate(b.lens.tolist()):
        at = torch.arange(n)
        at = at[(at >= n - W) | (at < S)]
        pg, off = b.pages[i].long().cpu()[at // page], at % page
        assert bool((pg >= 0).all())
        for h in range(H):
            o, _, t, _ = ref.one(b.q[i: i + 1, h * D: (h + 1) * D].double().cpu(), b.k_cache.double().cpu()[pg, 0, off],
                                 b.v_cache.double().cpu()[pg, 0, off], D ** -0.5, torch.ones((1, len(at)), dtype=torch.bool))
            ref.check(b.attn[i: i + 1, h * D: (h + 1) * D], o, t, f"decode {i} {h}")
    if pool:  # pages 0 and 10 to 13 of the first sequence, 0 to 3 of the second: 11 is its first visible token
        assert counted(b, page) == 30 - 5 - 4
        assert [e for e, p in enumerate(b.pages[0].tolist()) if p >= 0] == [0, 10, 11, 12, 13]
    d = normal(4, 241, H * D)
    _, dqkv = b.train(x, lens, d)
    q, k = b.q[:241].view(241, H, D).double().cpu(), b.k[:241].view(241, G, D).double().cpu()
    v = b.qkv[:241, (H + G) * D:].reshape(241, G, D).double().cpu()
    (_, _, dv), (_, _, tv) = wref.prompt_bwd(d.double().cpu().view(241, H, D), q, k, v, cu, D ** -0.5, W, S)
    ref.check(dqkv[:, (H + G) * D:].reshape(241, G, D), dv, tv, "dv")
    torch.cuda.synchronize()
    b.close()


def calls(seed):
    """A windowed training step, a windowed decode step, and a step of drafts from fork to the accepted
    tokens, on fixed buffers; `reset` puts back what the calls change."""
    import chunked_tp_overlap_amd.ub as ub

    H, G, D, T, page, n = 8, 2, 128, 700, 16, 4
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = dict(dtype=BF16, device="cuda")
    x = torch.randn((T, (H + 2 * G) * D), generator=g, device="cuda").to(BF16)
    d = torch.randn((T, H * D), generator=g, device="cuda").to(BF16)
    buf = torch.empty(T * 64, **bf)
    s = dict(x=x, d=d, ub=ub)
    s["h"] = ub.ub_init(T, 64, 1, ub.UB_DTYPE_BF16, buf, T * 64 * 2)
    cfg, win = ub.make_attn_cfg(H, G, D), ub.make_attn_window(60, 4)
    cu = i32([0, 301, 301, 302, 692])
    held = i32([301, 0, 1, 390])
    per, n_pages = 30, 120
    table = torch.full((n, per), -1, dtype=torch.int32, device="cuda")
    at = 0
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    for i, m in enumerate(held.tolist()):
        k = -(-m // page)
        table[i, :k] = torch.arange(at, at + k, dtype=torch.int32, device="cuda")
        refs[at: at + k] = 1
        at += k
    trees = [[-1, 0, 0, 2], [-1], [-1, 0, 1], [-1, -1, 1, 2, 3]] * 2
    parents = i32([p for t in trees for p in t] + [0] * (T - 26))
    depth = []
    for t in trees:
        a = len(depth)
        for p in t:
            depth.append(0 if p < 0 else depth[a + p] + 1)
    offsets = i32(depth + [0] * (T - 26))
    tcu = i32([0] + torch.tensor([len(t) for t in trees]).cumsum(0).tolist())
    m = tcu[1:] - tcu[:-1]
    kc, vc = (torch.randn((n_pages, G, page, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    inv = (10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)).float()
    e = lambda *shape, **kw: torch.empty(shape, **{**bf, **kw})
    f32, ii = dict(dtype=torch.float32), dict(dtype=torch.int32)
    outs = dict(q=e(T, H * D), k=e(T, G * D), out=e(T, H * D), dec=e(T, H * D), tree=e(T, H * D), tq=e(T, H * D), dx=torch.empty_like(x),
                lse=e(H, T, **f32), dlse=e(H, T, **f32), tlse=e(H, T, **f32), kc=kc, vc=vc, refs=refs, forked=e(8, per, **ii),
                flens=e(8, **ii), grown=e(8, **ii), copies=e(8, 3, **ii), done=e(8, **ii))
    first = {k: outs[k].clone() for k in ("kc", "vc", "refs")}
    ws = {op: torch.empty(max(ub.ub_attn_required_bytes(op, cfg, T, 8), 16), dtype=torch.uint8, device="cuda")
          for op in (ub.UB_ATTN_PROMPT_WINDOW_BWD, ub.UB_ATTN_DECODE_WINDOW, ub.UB_ATTN_TREE)}
    rws = torch.empty(ub.ub_kv_resize_bytes(8), dtype=torch.uint8, device="cuda")
    cols = (0, H * D, (H + G) * D)
    hx, dh = [ub.heads(x, c) for c in cols], [ub.heads(outs["dx"], c) for c in cols]
    hd = {k: ub.heads(outs[k]) for k in ("q", "k", "out", "dec", "tree", "tq")}
    cache, dd = ub.make_kv_cache(kc, vc), ub.heads(d)
    rows = i32([0, 1, 2, 3, 0, 0, 3, 2])
    kept, kept_lens = i32([[0, 2, 3], [0, -1, -1], [0, 1, 2], [1, 2, 3]] * 2), i32([3, 0, 2, 3, 1, 1, 3, 3])
    want = e(8, **ii)

    def run(stream):
        h = s["h"]
        ub.ub_kv_append(h, *hx, hd["q"], hd["k"], inv, cu, None, n, None, None, cfg, stream)
        ub.ub_attn_prompt_window(h, hd["q"], hd["k"], hx[2], hd["out"], outs["lse"], cu, n, win, cfg, None, stream)
        ub.ub_attn_prompt_window_bwd(h, dd, hd["q"], hd["k"], hx[2], hd["out"], outs["lse"], *dh, cu, n, win, cfg,
                                     ws[ub.UB_ATTN_PROMPT_WINDOW_BWD], stream)
        ub.ub_attn_decode_window(h, hd["q"], cache, table, held, n, win, hd["dec"], outs["dlse"], cfg,
                                 ws[ub.UB_ATTN_DECODE_WINDOW], stream)
        ub.ub_kv_fork(h, outs["refs"], table, held, n, rows, outs["forked"], outs["flens"], 8, page, stream)
        with torch.cuda.stream(stream):
            torch.add(outs["flens"], m, out=want)
        ub.ub_kv_resize(h, outs["refs"], outs["forked"], outs["flens"], want, 8, outs["grown"], outs["copies"], page, None, rws, stream)
        ub.ub_kv_copy_pages(h, cache, outs["copies"], 8, cfg, stream)
        ub.ub_kv_append_at(h, *hx, hd["tq"], None, inv, offsets, tcu, outs["flens"], 8, cache, outs["forked"], cfg, stream)
        ub.ub_attn_tree(h, hd["tq"], cache, outs["forked"], outs["grown"], parents, tcu, 8, hd["tree"], outs["tlse"], cfg,
                        ws[ub.UB_ATTN_TREE], stream)
        ub.ub_kv_compact(h, cache, outs["forked"], outs["flens"], kept, kept_lens, 8, outs["done"], cfg, stream)

    def reset():
        for k, t in outs.items():
            t.copy_(first[k]) if k in first else t.zero_()

    s.update(run=run, outs=outs, reset=reset, keep=(buf, cu, held, table, parents, offsets, tcu, inv, ws, rws, rows, kept,
                                                    kept_lens, want))
    return s


def bits(outs):
    return {k: t.view(torch.uint8).clone() for k, t in outs.items()}


def same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_another_stream():
    s = calls(1)
    s["run"](torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = bits(s["outs"])
    assert s["outs"]["done"].tolist() == [304, 0, 3, 393, 302, 302, 393, 4]
    assert bool(torch.isfinite(s["outs"]["tree"]).all())
    s["reset"]()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s["run"](side)
    torch.cuda.current_stream().wait_stream(side)
    got = bits(s["outs"])
    torch.cuda.synchronize()
    same(want, got)
    s["ub"].ub_destroy(s["h"])


def test_graph():
    """Captured once, replayed with new inputs in the same buffers and eager work in between."""
    s = calls(2)
    s["run"](torch.cuda.current_stream())
    torch.cuda.synchronize()
    s["reset"]()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s["run"](torch.cuda.current_stream())
    for i in range(4):
        g = torch.Generator(device="cuda").manual_seed(50 + i)
        s["x"].copy_(torch.randn(s["x"].shape, generator=g, device="cuda"))
        s["d"].copy_(torch.randn(s["d"].shape, generator=g, device="cuda"))
        s["reset"]()
        s["run"](torch.cuda.current_stream())
        torch.cuda.synchronize()
        want = bits(s["outs"])
        s["reset"]()
        graph.replay()
        torch.cuda.synchronize()
        same(want, bits(s["outs"]))
        assert bool(torch.isfinite(s["outs"]["dx"]).all()) and math.isfinite(float(s["outs"]["tree"].float().sum()))
    s["ub"].ub_destroy(s["h"])


@pytest.mark.parametrize("W,S", [(50, 3), (3, 2), (16, 0), (1, 64)])
def test_windowed_training_step(W, S):
    """The gradient of all three projections under a window, dq and dk back through the rotation."""
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    H, G, D, hidden = 4, 2, 64, 128
    wqkv, wo = normal(1, hidden, (H + 2 * G) * D) / 11, normal(2, H * D, hidden) / 16
    b = AttentionBlock(wqkv, wo, H, G, D, capacity=800, max_seqs=4, max_len=16, tp=4, window=W, sinks=S)
    lens = [70, 0, 81, 600]
    rows = sum(lens)
    x, d = normal(3, rows, hidden), normal(4, rows, H * D)
    y, dqkv = b.train(x, lens, d)
    q, k = b.q[:rows].view(rows, H, D).double().cpu(), b.k[:rows].view(rows, G, D).double().cpu()
    v = b.qkv[:rows, (H + G) * D:].reshape(rows, G, D).double().cpu()
    cu = [0, 70, 70, 151, 751]
    o, _, t, _ = wref.prompt(q, k, v, cu, D ** -0.5, W, S)
    ref.check(b.attn[:rows].view(rows, H, D), o, t, "out")
    (dq, dk, dv), (tq, tk, tv) = wref.prompt_bwd(d.double().cpu().view(rows, H, D), q, k, v, cu, D ** -0.5, W, S)
    pos = torch.cat([torch.arange(n) for n in lens])
    got = dqkv.double().cpu()
    for name, w, t, c, n in (("dq", dq, tq, 0, H), ("dk", dk, tk, H * D, G)):
        z, e = ref.rotate(w, pos, -b.inv_freq.cpu(), False, D)
        # the bound of a pair's two entries, turned, and one more rounding
        both = t[..., : D // 2] + t[..., D // 2:]
        tol = (torch.cat([both, both], -1) + e) * (1 + ref.U16) + ref.U16 * z.abs()
        ref.check(got[:, c: c + n * D].reshape(rows, n, D), z, tol, name)
    ref.check(got[:, (H + G) * D:].reshape(rows, G, D), dv, tv, "dv")
    torch.cuda.synchronize()
    b.close()
