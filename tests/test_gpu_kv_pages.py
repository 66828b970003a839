"""GPU tests of a cache's pages against a plain model on the CPU: forks, growth with copies of
shared last pages, pages taken back, windows, a pool that runs out, and bad tables."""

import random

import pytest
import torch

from tests.test_gpu_attn import BF16, F8, Rank, i32, make_cache, raw, ub  # noqa: F401

pytestmark = pytest.mark.gpu


def pages_of(n, page):
    return -(-n // page)


class Pool:
    """The pages' model: rows of ids, lengths, counts."""

    def __init__(self, n_pages, page, per):
        self.refs, self.page, self.per = [0] * n_pages, page, per
        self.rows, self.lens = [], []

    def add_empty(self, n):
        self.rows += [[-1] * self.per for _ in range(n)]
        self.lens += [0] * n

    def held(self, i):
        return [x for x in self.rows[i][: pages_of(self.lens[i], self.page)] if 0 <= x < len(self.refs)]

    def fork(self, parents):
        old = self.rows, self.lens
        for i in range(len(old[0])):
            uses = sum(p == i for p in parents) - 1
            for x in self.held(i):
                self.refs[x] += uses
        self.rows, self.lens = [], []
        for p in parents:
            some = 0 <= p < len(old[0])
            k = pages_of(old[1][p], self.page) if some else 0
            self.rows.append((old[0][p][:k] if some else []) + [-1] * (self.per - k))
            self.lens.append(old[1][p] if some else 0)

    def resize(self, new, window=None):
        page, copies, plan, end, open_ = self.page, [], [], 0, True
        free = [x for x, r in enumerate(self.refs) if r == 0]
        before = list(self.refs)
        for i, want in enumerate(new):
            had, has = pages_of(self.lens[i], page), pages_of(max(want, 0), page)
            fits = want <= self.per * page
            part, begin = 0, had
            if fits and want > self.lens[i] and self.lens[i] % page:
                last = self.rows[i][had - 1]
                if 0 <= last < len(before) and before[last] > 1:
                    part, begin = self.lens[i] % page, had - 1
            need = has - begin if fits and want > self.lens[i] else 0
            end += need
            plan.append((need == 0 or end <= len(free), fits, part, begin, need, end))
        for i, want in enumerate(new):
            served, fits, part, begin, need, end = plan[i]
            if not fits:
                copies.append([-1, -1, 0])
                new_len = self.lens[i]
            elif want > self.lens[i]:
                row = self.rows[i]
                if not served:
                    copies.append([-1, -1, 0])
                    new_len = self.lens[i]
                else:
                    src = row[begin] if part else -1
                    for j in range(need):
                        row[begin + j] = free[end - need + j]
                        self.refs[free[end - need + j]] += 1
                    if part:
                        self.refs[src] -= 1
                    copies.append([src, row[begin], part] if part else [-1, -1, 0])
                    new_len = want
            else:
                new_len = max(want, 0)
                for e in range(pages_of(new_len, page), pages_of(self.lens[i], page)):
                    self.drop(i, e)
                copies.append([-1, -1, 0])
            self.lens[i] = new_len
            if window and new_len > window[0]:
                for e in range(pages_of(window[1], page), (new_len - window[0]) // page):
                    self.drop(i, e)
                    if copies[i][2] and e == begin:
                        copies[i] = [-1, -1, 0]
        return copies

    def drop(self, i, e):
        x = self.rows[i][e]
        if 0 <= x < len(self.refs):
            self.refs[x] -= 1
        self.rows[i][e] = -1


class Device:
    """The same on the GPU."""

    def __init__(self, ub, h, pool):  # noqa: F811
        self.ub, self.h, self.per, self.page = ub, h, pool.per, pool.page
        self.refs = i32(pool.refs)
        self.set(pool)

    def set(self, pool):
        n = len(pool.rows)
        self.n, self.table = n, torch.tensor(pool.rows, dtype=torch.int32).view(n, self.per).cuda()
        self.lens = torch.tensor(pool.lens, dtype=torch.int32).cuda()

    def fork(self, parents):
        n = len(parents)
        table = torch.full((n, self.per), 99, dtype=torch.int32, device="cuda")
        lens = torch.full((n,), 99, dtype=torch.int32, device="cuda")
        self.ub.ub_kv_fork(self.h, self.refs, self.table, self.lens, self.n, torch.tensor(parents, dtype=torch.int32).cuda(),
                           table, lens, n, self.page)
        self.n, self.table, self.lens = n, table, lens

    def resize(self, new, window=None):
        copies = torch.full((self.n, 3), 77, dtype=torch.int32, device="cuda")
        ws = torch.full((max(self.ub.ub_kv_resize_bytes(self.n), 16),), 0xFF, dtype=torch.uint8, device="cuda")
        self.ub.ub_kv_resize(self.h, self.refs, self.table, self.lens, torch.tensor(new, dtype=torch.int32).cuda(), self.n,
                             self.lens, copies, self.page, self.ub.make_attn_window(*window) if window else None, ws)
        return copies

    def same(self, pool, what):
        assert self.lens.tolist() == pool.lens, what
        assert self.table.tolist() == pool.rows, what
        assert self.refs.tolist() == pool.refs, what


@pytest.mark.parametrize("page,n_pages,per,rows", [(16, 400, 40, 12), (1, 900, 70, 9), (64, 60, 8, 20), (5, 20000, 300, 100)])
@pytest.mark.parametrize("window", [None, (20, 3)])
def test_random_steps(ub, page, n_pages, per, rows, window):  # noqa: F811
    """Steps of forks, growth, shrinking, reordering and ends, with pools that run out."""
    r = random.Random(page * 1000 + rows)
    pool = Pool(n_pages, page, per)
    pool.add_empty(rows)
    with Rank(ub, 8) as h:
        dev = Device(ub, h, pool)
        for step in range(40):
            n = len(pool.rows)
            if step % 3 == 2:
                parents = [r.randrange(-1, n + 1) if r.random() < 0.3 else r.randrange(n) for _ in range(r.randint(1, rows))]
                pool.fork(parents)
                dev.fork(parents)
            else:
                cap = per * page
                new = [r.choice([x, x + r.randint(0, cap // 4), r.randint(0, cap), max(0, x - r.randint(0, cap)), cap, cap + 1, -5])
                       for x in pool.lens]
                want = pool.resize(new, window)
                got = dev.resize(new, window)
                assert got.tolist() == want, step
            dev.same(pool, step)
        # every row ends: nothing is held
        pool.fork([-1])
        dev.fork([-1])
        dev.same(pool, "end")
        assert not any(pool.refs)


def test_large_pool(ub):  # noqa: F811
    """Free pages far apart in a pool of many turns of the walk, with counts past its end."""
    n_pages, page, per = 50003, 16, 600
    pool = Pool(n_pages, page, per)
    r = random.Random(3)
    pool.refs = [0 if r.random() < 0.01 else 1 for _ in range(n_pages)]
    pool.refs[-1] = 0
    free = pool.refs.count(0)
    pool.add_empty(1500)
    new = [r.randint(0, 3) * page for _ in range(1500)]
    assert sum(x // page for x in new) > free  # it runs out
    with Rank(ub, 8) as h:
        dev = Device(ub, h, pool)
        assert dev.resize(new).tolist() == pool.resize(new)
        dev.same(pool, "out")
        few = [x // 2 for x in pool.lens]
        assert dev.resize(few).tolist() == pool.resize(few)
        dev.same(pool, "back")


@pytest.mark.parametrize("f8,token_major,page,G,D", [(False, False, 16, 1, 128), (True, True, 24, 3, 80), (False, True, 64, 4, 40)])
def test_copies(ub, f8, token_major, page, G, D):  # noqa: F811
    """Forked rows that grow each hold their parent's tokens on a page of their own."""
    pool = Pool(64, page, 6)
    pool.add_empty(3)
    kc, vc = make_cache(G, D, page, 64, f8, token_major, 5)
    cfg, cache = ub.make_attn_cfg(G, G, D, rotary_dim=0), ub.make_kv_cache(kc, vc)
    with Rank(ub, 8) as h:
        dev = Device(ub, h, pool)
        first = [page + 3, 2 * page, 1]
        dev.resize(first), pool.resize(first)
        parents = [0, 0, 0, 1, 1, 2, 2]
        dev.fork(parents), pool.fork(parents)
        old = [raw(c).view(64, G, page, -1) for c in (kc, vc)]
        grow = [page + 4, page + 3, 3 * page, 2 * page + 1, 2 * page, page + 1, 5]
        copies = dev.resize(grow)
        records = pool.resize(grow)
        assert copies.tolist() == records
        assert [x[2] for x in records] == [3, 0, 3, 0, 0, 1, 1]
        ub.ub_kv_copy_pages(h, cache, copies, len(grow), cfg)
        torch.cuda.synchronize()
    for c, was in zip((kc, vc), old):
        want = was.clone()
        for src, dst, n in records:
            if n:
                want[dst, :, :n] = was[src, :, :n]
        assert torch.equal(raw(c).view(64, G, page, -1), want)


def test_copy_records(ub):  # noqa: F811
    """Records of bad pages, equal pages, no or too many tokens."""
    G, D, page, n = 2, 64, 4, 8
    kc, vc = make_cache(G, D, page, n, False, False, 5)
    was = raw(kc).view(n, G, page, -1)
    records = [[0, 1, 99], [2, 8, 4], [-1, 3, 4], [4, 4, 4], [5, 6, 0], [1 << 30, 7, 2], [2, 7, -3], [0, 5, 2]]
    with Rank(ub, 8) as h:
        ub.ub_kv_copy_pages(h, ub.make_kv_cache(kc, vc), i32(records), len(records), ub.make_attn_cfg(G, G, D, rotary_dim=0))
        torch.cuda.synchronize()
    want = was.clone()
    want[1] = was[0]
    want[5, :, :2] = was[0, :, :2]
    assert torch.equal(raw(kc).view(n, G, page, -1), want)


def test_bad_tables(ub):  # noqa: F811
    """Ids outside the pool are skipped, lengths past a row's entries are cut to them."""
    pool = Pool(10, 4, 3)
    pool.rows, pool.lens, pool.refs = [[0, -7, 1 << 30], [3, 10, 2]], [12, 9], [1, 0, 1, 1] + [0] * 6
    with Rank(ub, 8) as h:
        dev = Device(ub, h, pool)
        dev.lens = i32([50, 9])  # the first row's is cut to 12
        dev.fork([0, 0, 1, 5])
        pool.fork([0, 0, 1, 5])
        dev.same(pool, "fork")
        new = [2, 0, 12, 13]
        assert dev.resize(new).tolist() == pool.resize(new)
        dev.same(pool, "resize")


@pytest.mark.parametrize("window", [None, (40, 3)])
def test_thousands_of_rows(ub, window):  # noqa: F811
    """More rows than the giving workgroup keeps at hand, with shared last pages, in a pool that runs out."""
    rows, page, per = 5001, 16, 8
    r = random.Random(7)
    pool = Pool(9000, page, per)
    pool.add_empty(rows)
    with Rank(ub, 8) as h:
        dev = Device(ub, h, pool)
        for step in range(3):
            new = [min(per * page, x + r.choice([0, 1, 5, 16, 30])) for x in pool.lens]
            assert dev.resize(new, window).tolist() == pool.resize(new, window), step
            dev.same(pool, step)
            short = sum(a != b for a, b in zip(new, pool.lens))
            parents = [r.randrange(rows) if r.random() < 0.1 else i for i in range(rows)]
            pool.fork(parents)
            dev.fork(parents)
            dev.same(pool, f"fork {step}")
        assert short > 1000  # the last step's pages ran out
