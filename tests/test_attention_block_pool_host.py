"""Host-side tests of the attention block over a pool of pages (no GPU): what its calls store and read,
slot by slot, where the pages suffice and where they do not."""

import random

import pytest
import torch

pytest.importorskip("chunked_tp_overlap_amd.ub", reason="libub.so not built")
from tests.block_model import block, i32, modelled, tokens  # noqa: E402


@pytest.mark.parametrize("free", [0, 1, 2, 3])
def test_no_page_for_a_shared_last_page(monkeypatch, free):
    """Three sequences share a partly filled last page, and the pool has pages for `free` of them: the
    others' next tokens are stored nowhere, least of all on that page, and their rows are NaN."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 2 + free)
        b.prefill(tokens(0, 20), [20])
        b.fork(i32([0, 0, 0]))
        before = dict(calls.slots)
        b.decode(tokens(100, 3))
        assert calls.given == [i < free for i in range(3)] and calls.shared == []
        assert calls.rows == [list(range(20)) + [100 + i] if i < free else None for i in range(3)]
        assert {s: t for s, t in calls.slots.items() if s in before} == before
        b.close()


@pytest.mark.parametrize("free", [0, 1, 2])
def test_no_page_for_drafts(monkeypatch, free):
    """The same with trees of drafted tokens, of which a path is accepted: no node of a tree without pages
    is stored or moved, and a sequence of which none is accepted goes on."""
    trees, n = [[-1, 0, 0, 2], [-1, -1, 1, 2]], 4
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 2 + free, max_seqs=2)
        b.prefill(tokens(0, 20), [20])
        b.fork(i32([0, 0]))
        before = dict(calls.slots)
        b.draft(tokens(100, 2 * n), trees)
        assert calls.given == [i < free for i in range(2)] and calls.shared == []
        past = list(range(20))
        want = [past + [100], past + [100, 101], past + [100, 102], past + [100, 102, 103],
                past + [104], past + [105], past + [105, 106], past + [105, 106, 107]]
        assert calls.rows == [w if i // n < free else None for i, w in enumerate(want)]
        b.accept(i32([[0, 2, 3], [1, 2, 3]]), i32([3 * (free > 0), 3 * (free > 1)]))
        assert calls.shared == [] and {s: t for s, t in calls.slots.items() if s in before} == before
        assert b.lens.tolist() == [20 + 3 * (i < free) for i in range(2)]
        if free == 1:  # the first gave back what the other nodes had; the second's page is its own now
            b.decode(tokens(200, 2))
            assert calls.rows == [past + [100, 102, 103, 200], past + [201]] and calls.shared == []
        b.close()


def test_accept_goes_with_the_draft_before_it(monkeypatch):
    """Which sequences had pages for their drafts is known to the draft alone."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 8, max_seqs=3)
        kept, some = i32([[0], [0]]), i32([1, 1])
        b.prefill(tokens(0, 30), [20, 10])
        for between in (None, lambda: b.decode(tokens(70, 2)), lambda: b.fork(i32([1, 0])),
                        lambda: b.prefill(tokens(0, 30), [20, 10])):
            if between is not None:
                b.draft(tokens(50, 2), [[-1], [-1]])
                between()
            with pytest.raises(ValueError, match="accept"):
                b.accept(kept, some)
        b.draft(tokens(50, 2), [[-1], [-1]])
        with pytest.raises(ValueError, match="accept"):
            b.accept(i32([[0]] * 3), i32([1] * 3))
        before = b.lens.tolist()
        b.accept(kept, some)
        assert b.lens.tolist() == [before[0] + 1, before[1] + 1, 0]
        assert torch.equal(b.held, b.lens)
        b.close()


def test_a_lost_token_stays_lost(monkeypatch):
    """A sequence whose token was not stored is NaN from then on, with pages to spare too: the places that
    it never wrote hold other sequences' tokens.  It takes no more pages; what it has it keeps until it ends."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 5)
        b.prefill(tokens(0, 64), [32, 16, 16])
        b.decode(tokens(100, 3))  # all three need a page, the first gets it
        assert [r is None for r in calls.rows] == [False, True, True]
        b.fork(i32([-1, 1, 2]))  # the first ends: three pages are free
        for s in range(2):
            before, held = dict(calls.slots), b.held.tolist()
            b.decode(tokens(110 + 10 * s, 3))
            assert [r is None for r in calls.rows] == [False, True, True]  # the first is a new sequence
            assert b.held.tolist() == [held[0] + 1] + held[1:]
            assert sum(calls.slots.get(k) != v for k, v in before.items()) + len(calls.slots) - len(before) <= 1
        b.draft(tokens(150, 3), [[-1], [-1], [-1]])
        assert [r is None for r in calls.rows] == [False, True, True]
        b.accept(i32([[0]] * 3), i32([1, 1, 0]))
        b.fork(i32([0, 1, 1, 2]))  # copies of it are lost too
        b.decode(tokens(160, 4))
        assert [r is None for r in calls.rows] == [False, True, True, True]
        b.fork(i32([-1, -1, -1, -1]))
        assert int((b.refs == 0).sum()) == 5 and b.lens.tolist() == b.held.tolist() == [0] * 4
        b.prefill(tokens(0, 64), [32, 16, 16])
        assert b.lens.tolist() == [32, 16, 16, 0] and not bool(torch.isnan(b.attn[:64]).any())
        b.close()


def test_prompts_without_pages(monkeypatch):
    """A prompt that the pool has no pages for, or that is longer than a sequence can be: NaN, in its own rows
    and in all later ones."""
    with modelled(monkeypatch) as (m, calls):
        for lens, n_pages, lost in (([40, 0, 33, 17], 5, [0, 0, 1, 1]), ([65, 64], 9, [1, 0]), ([20], 1, [1]), ([16, 17], 2, [0, 1])):
            b = block(m, n_pages)
            b.prefill(tokens(0, sum(lens)), lens)
            nan = torch.isnan(b.attn[: sum(lens)].float())
            assert nan.all(1).tolist() == nan.any(1).tolist() == [bool(x) for n, x in zip(lens, lost) for _ in range(n)]
            b.fork(i32([i if x else -1 for i, x in enumerate(lost)]))  # the others end, pages are free
            first = len(calls.slots)
            b.decode(tokens(150, len(lens)))
            assert [r is None for r in calls.rows] == [bool(x) for x in lost]
            assert len(calls.slots) - first <= lost.count(0)
            b.close()
            calls.slots.clear()


def test_a_path_of_a_tree_without_pages(monkeypatch):
    """Its tokens were not stored: the sequence has lost them."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 2, max_seqs=3)
        b.prefill(tokens(0, 32), [16, 16])
        b.draft(tokens(50, 4), [[-1, 0], [-1, 0]])
        assert calls.rows == [None] * 4
        b.accept(i32([[0, 1], [0, 1]]), i32([0, 2]))
        assert b.lens[0] == 16 and b.lens[1] >= m.NOWHERE
        b.fork(i32([-1, 1, -1]))
        b.decode(tokens(60, 3))
        assert [r is None for r in calls.rows] == [False, True, True]  # one page: the first's
        b.close()


@pytest.mark.parametrize("accepted", [None, 1])
def test_fork_after_drafts(monkeypatch, accepted):
    """Drafts that were not accepted are no tokens of a sequence: its copies do not share their places,
    which all of them write next."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 12)
        b.prefill(tokens(0, 36), [20, 16])
        b.draft(tokens(50, 18), [[-1] + list(range(13)), [-1, 0, 1, 2]])
        if accepted is not None:  # of the first alone
            b.accept(i32([[0]]), i32([accepted]))
        first = list(range(20)) + ([50] if accepted else [])
        b.fork(i32([0, 0, 1, 1]))
        assert b.held.tolist() == b.lens.tolist() == [len(first)] * 2 + [16] * 2
        assert int((b.refs > 0).sum()) == 3
        b.decode(tokens(100, 4))
        assert calls.shared == []
        assert calls.rows == [first + [100], first + [101], list(range(20, 36)) + [102], list(range(20, 36)) + [103]]
        b.draft(tokens(110, 4), [[-1]] * 4)
        assert calls.shared == [] and calls.rows[1] == first + [101, 111]
        b.close()


@pytest.mark.parametrize("seed", range(12))
def test_random_steps(monkeypatch, seed):
    """Prompts, decode steps, drafts, accepted paths and forks in any order, in pools that run out: a row sees
    its sequence's own tokens, in order, or is NaN, and that from the first token that it lost."""
    r = random.Random(seed)
    window, sinks = (None, 0) if seed % 3 else (r.randint(1, 20), r.randint(0, 5))
    with modelled(monkeypatch) as (m, calls):
        b = block(m, r.randint(3, 14), max_seqs=6, max_len=40, page=r.choice([1, 4, 16]), window=window, sinks=sinks)
        count, past, alive = 0, [[] for _ in range(6)], 0  # past: a sequence's tokens, or None: it has lost one

        def new(n):
            nonlocal count
            count += n
            return list(range(count - n, count))

        def sees(tokens):
            n = len(tokens)
            return [t for u, t in enumerate(tokens) if window is None or n - 1 - u < window or u < sinks]

        def write(x, f):
            before = len(calls.shared)
            rows = torch.zeros((len(x), 128), dtype=torch.bfloat16)
            rows[:, 0], rows[:, 1] = torch.tensor(x) // 200, torch.tensor(x) % 200
            f(rows)
            assert len(calls.shared) == before

        for step in range(40):
            op = "prefill" if not alive else r.choice(["decode"] * 4 + ["draft"] * 3 * (window is None) + ["fork"] * 2 + ["prefill"])
            if op == "prefill":
                lens = [r.randint(0, 41) for _ in range(r.randint(1, 6))]
                if sum(lens) == 0:
                    continue
                x = new(sum(lens))
                write(x, lambda rows: b.prefill(rows, lens))
                nan, at, alive, past = torch.isnan(b.attn[: len(x), 0].float()).tolist(), 0, len(lens), [[] for _ in range(6)]
                for i, n in enumerate(lens):
                    past[i] = x[at: at + n] if calls.given[i] else None
                    assert nan[at: at + n] == [past[i] is None] * n
                    at += n
            elif op == "decode":
                n = r.randint(1, alive)
                x = new(n)
                write(x, b.decode)
                for i in range(n):
                    past[i] = past[i] + [x[i]] if past[i] is not None and calls.given[i] else None
                assert calls.rows == [None if past[i] is None else sees(past[i]) for i in range(n)]
            elif op == "draft":
                n = r.randint(1, alive)
                trees = [[r.randint(-1, j - 1) for j in range(r.randint(0, 7))] for _ in range(n)]
                if sum(map(len, trees)) == 0:
                    continue
                x = new(sum(map(len, trees)))
                write(x, lambda rows: b.draft(rows, trees))
                given, at, rows, paths, places = calls.given, 0, [], [], []
                for i, t in enumerate(trees):
                    of = []
                    for j, p in enumerate(t):
                        of.append((of[p] if p >= 0 else []) + [j])
                        rows.append(past[i] + [x[at + q] for q in of[j]] if past[i] is not None and given[i] else None)
                    places.append(of)
                    at += len(t)
                assert calls.rows == rows
                if r.random() < 0.8:
                    k, before, at = r.randint(1, n), len(calls.shared), 0
                    paths = [r.choice(of + [[]]) for of in places[:k]]
                    kept = torch.full((k, 8), -1, dtype=torch.int32)
                    for i, q in enumerate(paths):
                        kept[i, : len(q)] = torch.tensor(q, dtype=torch.int32)
                    b.accept(kept, i32([len(q) for q in paths]))
                    assert len(calls.shared) == before
                    for i, q in enumerate(paths):
                        if past[i] is not None and q:
                            past[i] = past[i] + [x[at + j] for j in q] if given[i] else None
                        at += len(trees[i])
            else:
                parents = [r.randint(-1, alive) for _ in range(r.randint(1, 6))]
                b.fork(i32(parents))
                past = [past[p] if 0 <= p < 6 else [] for p in parents] + [[] for _ in range(6 - len(parents))]
                alive = len(parents)
            for n, t in zip(b.lens.tolist(), past):
                assert n >= m.NOWHERE if t is None else n == len(t)
            want = torch.zeros_like(b.refs)
            for row, n in zip(b.pages.tolist(), b.held.tolist()):
                for p in row[: -(-n // b.page)]:
                    if p >= 0:
                        want[p] += 1
            assert torch.equal(b.refs, want)
        b.close()


@pytest.mark.parametrize("n_pages", [None, 20])
def test_addresses_a_captured_step_keeps(monkeypatch, n_pages):
    """A captured decode step holds the address of the rows' boundaries: it is the same, and says the same,
    after prompts and forks."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, n_pages)
        b.prefill(tokens(0, 30), [10, 20])
        b.decode(tokens(50, 2))
        step, boundaries = calls.appended[-1]
        others = []  # what the allocator gives a freed tensor's memory to
        if n_pages:
            b.fork(i32([0, 1, 0, 1]))
            others += [torch.full((k,), 77, dtype=torch.int32) for k in range(2, 6)]
            b.decode(tokens(60, 4))
            assert calls.appended[-1] == (step, [0, 1, 2, 3, 4])
            b.fork(i32([1, 0]))
        b.prefill(tokens(0, 30), [30])
        others += [torch.full((k,), 77, dtype=torch.int32) for k in range(2, 6)]
        b.prefill(tokens(0, 30), [20, 10])
        b.decode(tokens(50, 2))
        assert calls.appended[-1] == (step, boundaries)
        with pytest.raises(ValueError):  # no third sequence
            b.decode(tokens(50, 3))
        b.close()


def test_rows_of_no_sequence(monkeypatch):
    """More rows than sequences, or rows before there are any: refused before a page is given."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 20)
        for f in (lambda: None, lambda: b.prefill(tokens(0, 30), [10, 20]), lambda: b.fork(i32([1]))):
            f()
            n = len(calls.calls)
            with pytest.raises(ValueError, match="decode"):
                b.decode(tokens(50, 3))
            assert "ub_kv_resize" not in calls.calls[n:] and torch.equal(b.held, b.lens)
        b.close()


def test_refused_before_anything_changes(monkeypatch):
    """Prompts and drafts that are refused leave every sequence its pages and tokens."""
    with modelled(monkeypatch) as (m, calls):
        b = block(m, 20, max_seqs=3)
        x = tokens(0, 30)
        b.prefill(x, [10, 20])
        state = lambda: [t.clone() for t in (b.lens, b.held, b.pages, b.refs)] + [dict(calls.slots)]
        before = state()
        many = tokens(0, 4)
        for f in (lambda: b.prefill(x.float(), [10, 20]), lambda: b.prefill(x[:, :100], [10, 20]), lambda: b.prefill(x[0], [30]),
                  lambda: b.prefill(many, [1, 1, 1, 1]), lambda: b.prefill(x, [10, 21]), lambda: b.prefill(x, [-1, 20]),
                  lambda: b.prefill(torch.cat([tokens(0, 200)] * 2), [400]),
                  lambda: b.draft(many, [[-1]] * 4), lambda: b.draft(many.float(), [[-1, 0, 1, 2]]),
                  lambda: b.draft(tokens(0, 300), [[-1] * 150] * 2)):
            with pytest.raises((ValueError, m.ub.UBError)):
                f()
            after = state()
            assert all(torch.equal(p, q) for p, q in zip(before, after[:-1])) and before[-1] == after[-1]
        b.decode(tokens(100, 2))
        assert calls.rows == [list(range(10)) + [100], list(range(10, 30)) + [101]]
        b.close()
