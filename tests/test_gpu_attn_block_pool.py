"""GPU tests of the attention block where its pool runs out of pages, and of captured decode steps as
sequences fork: what the cache holds, byte by byte, and each row against its definition."""

import random

import pytest
import torch

from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
H, G, D, HIDDEN, PAGE = 4, 2, 64, 256, 16


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_block(n_pages, max_seqs=3, max_len=100, **kw):
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    wqkv, wo = normal(1, HIDDEN, (H + 2 * G) * D) / 16, normal(2, H * D, HIDDEN) / 16
    return AttentionBlock(wqkv, wo, H, G, D, capacity=256, max_seqs=max_seqs, max_len=max_len, page=PAGE, n_pages=n_pages, **kw)


def held_bytes(b):
    return [c.view(torch.uint8).cpu().clone() for c in (b.k_cache, b.v_cache)]


def check_row(b, r, i, places, what):
    """Row r of the last attention call, of sequence i, sees these places of the cache."""
    places = torch.tensor(places)
    pg, off = b.pages[i].long().cpu()[places // PAGE], places % PAGE
    assert bool((pg >= 0).all()), what
    kc, vc = b.k_cache.double().cpu(), b.v_cache.double().cpu()
    for h in range(H):
        q = b.q[r: r + 1, h * D: (h + 1) * D].double().cpu()
        o, _, t, _ = ref.one(q, kc[pg, h // 2, off], vc[pg, h // 2, off], D ** -0.5, torch.ones((1, len(places)), dtype=torch.bool))
        ref.check(b.attn[r: r + 1, h * D: (h + 1) * D], o, t, what)


@pytest.mark.parametrize("free", [0, 1, 3])
def test_no_page_for_a_shared_last_page(free):
    """Three sequences share 4 tokens on a page of 16; `free` of them can have a page of their own."""
    b = make_block(2 + free)
    b.prefill(normal(3, 20, HIDDEN), [20])
    b.fork(i32([0, 0, 0]))
    before = held_bytes(b)
    y = b.decode(normal(4, 3, HIDDEN)).clone()
    for c, old in zip(held_bytes(b), before):
        assert torch.equal(c[:2], old[:2])  # the prompt's pages
        assert torch.equal(c[2 + free:], old[2 + free:])
    for i in range(3):
        if i < free:
            check_row(b, i, i, list(range(21)), f"row {i}")
            assert bool(torch.isfinite(y[i]).all())
        else:
            assert bool(torch.isnan(b.attn[i]).all()) and bool(torch.isnan(y[i]).all())
    torch.cuda.synchronize()
    b.close()


@pytest.mark.parametrize("free", [0, 1, 2])
def test_no_page_for_drafts(free):
    b = make_block(2 + free, max_seqs=2)
    b.prefill(normal(3, 20, HIDDEN), [20])
    b.fork(i32([0, 0]))
    before = held_bytes(b)
    trees = [[-1, 0, 0, 2], [-1, -1, 1, 2]]
    y = b.draft(normal(4, 8, HIDDEN), trees).clone()
    paths = [[0], [0, 1], [0, 2], [0, 2, 3], [0], [1], [1, 2], [1, 2, 3]]
    for r, path in enumerate(paths):
        if r // 4 < free:
            check_row(b, r, r // 4, list(range(20)) + [20 + p for p in path], f"node {r}")
            assert bool(torch.isfinite(y[r]).all())
        else:
            assert bool(torch.isnan(b.attn[r]).all()) and bool(torch.isnan(y[r]).all())
    b.accept(i32([[0, 2, 3], [1, 2, 3]]), i32([3 * (free > 0), 3 * (free > 1)]))
    for c, old in zip(held_bytes(b), before):
        assert torch.equal(c[:2], old[:2])
    assert b.lens.tolist() == [20 + 3 * (i < free) for i in range(2)]
    torch.cuda.synchronize()
    b.close()


def test_a_lost_token_stays_lost():
    """Pages that come free do not bring a lost token back; the other rows are what they would be."""
    b = make_block(5)
    b.prefill(normal(3, 64, HIDDEN), [32, 16, 16])
    b.decode(normal(4, 3, HIDDEN))
    check_row(b, 0, 0, list(range(33)), "served")
    assert bool(torch.isnan(b.attn[1:3]).all())
    b.fork(i32([-1, 1, 2]))
    for s in range(3):
        before, held = held_bytes(b), b.held.tolist()
        y = b.decode(normal(5 + s, 3, HIDDEN))
        check_row(b, 0, 0, list(range(s + 1)), f"new {s}")
        assert bool(torch.isnan(b.attn[1:3]).all()) and bool(torch.isnan(y[1:3]).all()) and bool(torch.isfinite(y[0]).all())
        assert b.held.tolist() == [s + 1] + held[1:]
        at = int(b.pages[0, 0])
        for c, old in zip(held_bytes(b), before):
            c[at], old[at] = 0, 0
            assert torch.equal(c, old)
    b.draft(normal(9, 3, HIDDEN), [[-1], [-1], [-1]])
    assert torch.isnan(b.attn[:3]).all(1).tolist() == [False, True, True]
    b.accept(i32([[0]] * 3), i32([1, 1, 0]))
    assert b.lens[0] == 4 and bool((b.lens[1:] >= 1 << 30).all())
    torch.cuda.synchronize()
    b.close()


@pytest.mark.parametrize("window", [None, 10])
def test_prompts_without_pages(window):
    """The rows of prompts that found no pages are NaN, those of the others their definition's, as
    are the tokens decoded after them."""
    kw = {} if window is None else dict(window=window, sinks=2)
    b, sound = make_block(5, max_seqs=4, **kw), make_block(50, max_seqs=4, **kw)
    lens = [40, 0, 33, 17]
    x = normal(3, sum(lens), HIDDEN)
    y, want = b.prefill(x, lens).clone(), sound.prefill(x, lens).clone()
    lost = torch.tensor([False] * 40 + [True] * 50, device="cuda")
    assert torch.isnan(y).all(1).tolist() == torch.isnan(y).any(1).tolist() == lost.tolist()
    assert torch.equal(y[:40], want[:40])
    b.decode(normal(4, 4, HIDDEN))
    seen = [u for u in range(41) if window is None or u < 2 or 40 - u < window]
    check_row(b, 0, 0, seen, "decode 0")
    check_row(b, 1, 1, [0], "decode 1")
    assert bool(torch.isnan(b.attn[2:4]).all())
    torch.cuda.synchronize()
    b.close()
    sound.close()


def test_a_pool_that_runs_out_under_a_graph():
    """A captured decode step, replayed until the pool has no pages: the eager steps' bits."""
    tokens = [normal(10 + s, 3, HIDDEN) for s in range(8)]

    def steps(b, step):
        b.prefill(normal(3, 44, HIDDEN), [14, 13, 17])
        out = []
        for t in tokens:
            out.append([x.clone().view(torch.uint8) for x in (step(t), b.lens, b.held, b.pages, b.refs, b.k_cache, b.v_cache)])
            normal(50, 64, 64) @ normal(51, 64, 64)  # eager work between the steps
            torch.cuda.synchronize()
        return out

    b = make_block(5)
    want = steps(b, b.decode)
    b.close()
    b = make_block(5)
    b.prefill(normal(3, 44, HIDDEN), [14, 13, 17])
    token = torch.zeros_like(tokens[0])
    b.decode(token)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.decode(token)
    keep = b.step

    def replay(t):
        token.copy_(t)
        graph.replay()
        return y

    got = steps(b, replay)
    for s, (w, g) in enumerate(zip(want, got)):
        # the rows of the cache that nothing has written since differ: the first block's are zeros
        for n, (a, c) in enumerate(zip(w[:5], g[:5])):
            assert torch.equal(a, c), (s, n)
    assert b.lens.tolist()[0] == 22 and b.lens[1] >= 1 << 30 and b.lens[2] == 25
    del keep
    b.close()


def test_fork_after_drafts():
    """Copies of a sequence whose drafts were not accepted write places of their own."""
    b = make_block(12, max_seqs=4)
    b.prefill(normal(3, 36, HIDDEN), [20, 16])
    b.draft(normal(4, 18, HIDDEN), [[-1] + list(range(13)), [-1, 0, 1, 2]])
    b.fork(i32([0, 0, 1, 1]))
    assert b.held.tolist() == b.lens.tolist() == [20, 20, 16, 16] and int((b.refs > 0).sum()) == 3
    b.decode(normal(5, 4, HIDDEN))
    n = H * D
    for i in range(4):
        at = int(b.lens[i]) - 1
        assert torch.equal(b.k_cache[b.pages[i, at // PAGE].long(), :, at % PAGE].reshape(-1), b.k[i])
        assert torch.equal(b.v_cache[b.pages[i, at // PAGE].long(), :, at % PAGE].reshape(-1), b.qkv[i, n + G * D:])
        check_row(b, i, i, list(range(at + 1)), f"decode {i}")
    torch.cuda.synchronize()
    b.close()


def test_a_captured_step_across_forks():
    """A decode step captured for two sequences, replayed after forks and new prompts, with eager work and
    new tensors between: the bits of eager steps, every time."""
    def steps(b, step):
        out = []
        b.prefill(normal(3, 50, HIDDEN), [20, 30])
        for s in range(6):
            if s in (2, 4):
                b.fork(i32([0, 1, 0]))
                b.decode(normal(30 + s, 3, HIDDEN))
                b.fork(i32([2, 1]) if s == 2 else i32([1, 0]))
            if s == 5:
                b.prefill(normal(4, 40, HIDDEN), [33, 7])
            junk = [torch.full((k,), 77, dtype=torch.int32, device="cuda") for k in range(1, 9)]
            y = step(normal(10 + s, 2, HIDDEN))
            out.append([x.clone().view(torch.uint8) for x in (y, b.attn[:2], b.lens, b.held, b.pages, b.refs)])
            normal(50, 64, 64) @ normal(51, 64, 64)
            torch.cuda.synchronize()
            assert len(junk) == 8
        return out

    b = make_block(20)
    want = steps(b, b.decode)
    b.close()
    b = make_block(20)
    b.prefill(normal(3, 50, HIDDEN), [20, 30])
    token = torch.zeros((2, HIDDEN), dtype=BF16, device="cuda")
    b.decode(token)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.decode(token)

    def replay(t):
        # the active shape that eager calls between the replays have set is not what a replay reads
        token.copy_(t)
        graph.replay()
        return y

    got = steps(b, replay)
    for s, (w, g) in enumerate(zip(want, got)):
        for n, (a, c) in enumerate(zip(w, g)):
            assert torch.equal(a, c), (s, n)
        assert not bool(torch.isnan(g[0].view(BF16)).any())
    b.close()


@pytest.mark.parametrize("seed", range(6))
def test_random_steps_as_modelled(monkeypatch, seed):
    """Prompts, decode steps, drafts, accepted paths and forks in any order: lengths, tables, counts, the rows
    that are NaN and the values in every slot are those of the model of test_attention_block_pool_host.py."""
    from tests import block_model as bm

    r = random.Random(seed)
    kw = dict(max_seqs=6, max_len=40, page=r.choice([1, 4, 16]))
    if seed % 3 == 0:
        kw.update(window=r.randint(1, 20), sinks=r.randint(0, 5))
    n_pages, count, ops, alive = r.randint(4, 14), 0, [], 0
    for _ in range(60):
        op = "prefill" if not alive else r.choice(["decode"] * 4 + ["draft"] * 3 * ("window" not in kw) + ["fork"] * 2 + ["prefill"])
        if op == "prefill":
            lens = [r.randint(0, 41) for _ in range(r.randint(1, 6))]
            if not sum(lens):
                continue
            args, n, alive = (lens,), sum(lens), len(lens)
        elif op == "decode":
            args, n = (), r.randint(1, alive)
        elif op == "draft":
            trees = [[r.randint(-1, j - 1) for j in range(r.randint(0, 7))] for _ in range(r.randint(1, alive))]
            if not sum(map(len, trees)):
                continue
            args, n = (trees,), sum(map(len, trees))
        else:
            args, n = ([r.randint(-1, alive) for _ in range(r.randint(1, 6))],), 0
            alive = len(args[0])
        ops.append((op, args, count, n))
        count += n
        if op == "draft" and r.random() < 0.8:
            kept = torch.full((r.randint(1, len(trees)), 8), -1, dtype=torch.int32)
            lens = []
            for i in range(kept.shape[0]):
                path, j = [], r.randint(-1, len(trees[i]) - 1)
                while j >= 0:
                    path.insert(0, j)
                    j = trees[i][j]
                kept[i, : len(path)] = torch.tensor(path, dtype=torch.int32)
                lens.append(len(path))
            ops.append(("accept", (kept, torch.tensor(lens, dtype=torch.int32)), count, 0))

    def run(b, rows, dev, after):
        for op, args, first, n in ops:
            if op == "fork":
                args = (torch.tensor(args[0], dtype=torch.int32),)
            args = [a.to(dev) if isinstance(a, torch.Tensor) else a for a in args]
            getattr(b, op)(*([rows(first, n)] if n else []), *args)
            after([t.cpu().clone() for t in (b.lens, b.held, b.pages, b.refs)],
                  torch.isnan(b.attn[:n].float()).all(1).tolist(), torch.isnan(b.attn[:n].float()).any(1).tolist())

    want = []
    with bm.modelled(monkeypatch) as (m, calls):
        b = bm.block(m, n_pages, **kw)
        run(b, bm.tokens, "cpu", lambda state, nan, some: want.append((state, nan, dict(calls.slots))))
        b.close()
    H, G, D, hidden = 2, 1, 64, 128
    wqkv, wo = normal(1, hidden, (H + 2 * G) * D) / 11, normal(2, H * D, hidden) / 11
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    b = AttentionBlock(wqkv, wo, H, G, D, capacity=256, n_pages=n_pages, **kw)
    x = normal(3, count, hidden)
    values = x.double().cpu() @ wqkv[:, (H + G) * D:].double().cpu()
    norms = 4e-3 * x.double().cpu().norm(dim=1)[:, None] * wqkv[:, (H + G) * D:].double().cpu().norm(dim=0)
    at, lost = 0, 0

    def after(state, nan, some):
        nonlocal at, lost
        (lens, held, pages, refs), rows, slots = want[at]
        what = (at, ops[at][0])
        assert nan == some == rows, what
        for g, w, name in zip(state, (lens, held, pages, refs), ("lens", "held", "pages", "refs")):
            assert torch.equal(g, w), (what, name)
        v, keys = b.v_cache.double().cpu(), [k for k, t in slots.items() if t is not None]
        if keys:  # (a matrix product's bound, as for the library's GEMMs)
            pg, off = torch.tensor(keys).unbind(1)
            t = torch.tensor([slots[k] for k in keys])
            assert bool(((v[pg, 0, off] - values[t]).abs() <= norms[t]).all()), what
        lost += sum(nan)
        at += 1

    run(b, lambda first, n: x[first: first + n], "cuda", after)
    assert at == len(want) and lost > 0
    b.close()
