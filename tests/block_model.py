"""The attention block on the host, over a model of the calls that it makes: which token each slot of
the cache holds, which slots an attention row reads, and the plain table of test_gpu_kv_pages.py for
the pages.  A token is its row of x, numbered in x's first two columns."""

import contextlib

import torch

import chunked_tp_overlap_amd.ub as ub
from tests.test_attention_block_host import Stream, on_host
from tests.test_gpu_kv_pages import Pool

HIDDEN = 128
BASE = 200  # bf16 holds whole numbers up to 256


def tokens(first, n):
    """n rows of x, tokens first, first + 1, ..."""
    x = torch.zeros((n, HIDDEN), dtype=torch.bfloat16)
    at = torch.arange(first, first + n)
    x[:, 0], x[:, 1] = at // BASE, at % BASE
    return x


class Model:
    """What the calls do, on host tensors.  slots: token of (page, place in it); rows: of the last
    attention call, the tokens that each row sees, or None where its output is NaN; given: of
    the last ub_kv_resize, whether a row has the tokens it was to have."""

    def __init__(self):
        self.slots, self.x, self.rows, self.given = {}, None, None, None
        self.calls, self.shared = [], []  # shared: writes to a page that several rows hold
        self.refs = None
        self.appended = []

    def ub_copy_in(self, h, src, rows, *a):
        self.x = [int(r[0]) * BASE + int(r[1]) for r in src.float()]

    def at(self, pages, i, place, page):
        if not 0 <= place < pages.shape[1] * page:
            return None
        p = int(pages[i, place // page])
        return (p, place % page) if p >= 0 else None

    def write(self, slot, token):
        if self.refs is not None and int(self.refs[slot[0]]) > 1:
            self.shared.append(slot)
        self.slots[slot] = token

    def append(self, cu, past, n, cache, pages, page):
        self.appended.append((cu.data_ptr(), cu[: n + 1].tolist()))
        if cache is None:
            return
        for i in range(n):
            for j in range(int(cu[i + 1]) - int(cu[i])):
                slot = self.at(pages, i, (0 if past is None else int(past[i])) + j, page)
                if slot is not None:
                    self.write(slot, self.x[int(cu[i]) + j])

    def ub_kv_append(self, h, q, k, v, qo, ko, inv, cu, past, n, cache, pages, cfg, stream):
        self.append(cu, past, n, cache, pages, None if cache is None else cache.page_size)

    def ub_kv_append_at(self, h, q, k, v, qo, ko, inv, offsets, cu, past, n, cache, pages, cfg, stream):
        self.append(cu, past, n, cache, pages, cache.page_size)

    def read(self, pages, i, places, length, page):
        slots = [self.at(pages, i, p, page) for p in places]
        if length > pages.shape[1] * page or None in slots:
            return None
        return [self.slots.get(s) for s in slots]

    def done(self, out, rows):
        self.rows = rows
        for r, x in enumerate(rows):
            out.tensor[r] = float("nan") if x is None else 1.0

    def ub_attn_prompt(self, h, q, k, v, out, lse, cu, n, cfg, ws, stream):
        ends = cu.tolist()
        self.done(out, [self.x[a: r + 1] for a, b in zip(ends, ends[1:]) for r in range(a, b)])

    def ub_attn_prompt_window(self, h, q, k, v, out, lse, cu, n, window, cfg, ws, stream):
        ends = cu.tolist()
        self.done(out, [[self.x[u] for u in range(a, r + 1) if r - u < window.window or u - a < window.sinks]
                        for a, b in zip(ends, ends[1:]) for r in range(a, b)])

    def ub_attn_decode(self, h, q, cache, pages, lens, n, out, lse, cfg, ws, stream):
        lens = lens.tolist()
        over = pages.shape[1] * cache.page_size
        self.done(out, [self.read(pages, i, range(min(lens[i], over)), lens[i], cache.page_size) for i in range(n)])

    def ub_attn_decode_window(self, h, q, cache, pages, lens, n, window, out, lse, cfg, ws, stream):
        lens = lens.tolist()
        over = pages.shape[1] * cache.page_size
        self.done(out, [self.read(pages, i, [u for u in range(min(m, over)) if m - 1 - u < window.window or u < window.sinks],
                                  m, cache.page_size) for i, m in enumerate(lens[:n])])

    def ub_attn_tree(self, h, q, cache, pages, lens, parents, cu, n, out, lse, cfg, ws, stream):
        rows, page = [], cache.page_size
        for i in range(n):
            a, m, length = int(cu[i]), int(cu[i + 1]) - int(cu[i]), int(lens[i])
            whole = self.read(pages, i, range(min(length, pages.shape[1] * page)), length, page) if length >= m else None
            for j in range(m):
                path = []
                while j >= 0:
                    path.append(j)
                    j = int(parents[a + j])
                rows.append(None if whole is None else whole[: length - m] + [whole[length - m + p] for p in sorted(path)])
        self.done(out, rows)

    def ub_kv_resize(self, h, refs, pages, lens, new_lens, n, lens_out, copies, page, window, ws, stream):
        pool = Pool(refs.shape[0], page, pages.shape[1])
        pool.refs, pool.rows, pool.lens = refs.tolist(), pages[:n].tolist(), lens[:n].tolist()
        new = new_lens[:n].tolist()
        records = pool.resize(new, (window.window, window.sinks) if window else None)
        refs.copy_(torch.tensor(pool.refs, dtype=torch.int32))
        if n:
            pages[:n] = torch.tensor(pool.rows, dtype=torch.int32)
            lens_out[:n] = torch.tensor(pool.lens, dtype=torch.int32)
            copies[:n] = torch.tensor(records, dtype=torch.int32)
        self.refs, self.given = refs, [a == b for a, b in zip(pool.lens, new)]

    def ub_kv_copy_pages(self, h, cache, copies, n, cfg, stream):
        for src, dst, m in copies[:n].tolist():
            for o in range(m if src >= 0 and dst >= 0 else 0):
                self.slots[dst, o] = self.slots.get((src, o))

    def ub_kv_fork(self, h, refs, pages, lens, n, parents, pages_out, lens_out, n_out, page, stream):
        pool = Pool(refs.shape[0], page, pages.shape[1])
        pool.refs, pool.rows, pool.lens = refs.tolist(), pages[:n].tolist(), lens[:n].tolist()
        pool.fork(parents.tolist())
        refs.copy_(torch.tensor(pool.refs, dtype=torch.int32))
        pages_out[:n_out] = torch.tensor(pool.rows, dtype=torch.int32).view(n_out, -1)
        lens_out[:n_out] = torch.tensor(pool.lens, dtype=torch.int32)

    def ub_kv_compact(self, h, cache, pages, lens, kept, kept_lens, n, lens_out, cfg, stream):
        page = cache.page_size
        cap = pages.shape[1] * page
        for i in range(n):
            base, last, moved = min(max(int(lens[i]), 0), cap), -1, []
            for x in kept[i, : max(int(kept_lens[i]), 0)].tolist():
                if x <= last or base + x >= cap:
                    break
                last = x
                moved.append(x)
            have = [self.at(pages, i, base + x, page) for x in moved]
            have = [s and self.slots.get(s) for s in have]
            for d, (x, token) in enumerate(zip(moved, have)):
                to = self.at(pages, i, base + d, page)
                if x != d and to is not None and self.at(pages, i, base + x, page) is not None:
                    self.write(to, token)
            lens_out[i] = base + len(moved)


@contextlib.contextmanager
def modelled(monkeypatch):
    """The block's module, and the model that stands in for the calls that issue work."""
    from chunked_tp_overlap_amd import attention_block as m

    model = Model()
    with monkeypatch.context() as p:
        for name in ("zeros", "empty", "arange", "full"):
            p.setattr(torch, name, on_host(getattr(torch, name)))
        p.setattr(torch.Tensor, "cuda", lambda self, *a, **kw: self)
        p.setattr(torch.cuda, "current_stream", lambda *a: Stream)
        for name in ("ub_gemm_ag_chunked", "ub_gemm_rs_chunked"):
            p.setattr(ub, name, lambda *a: None)
        for name in ub.EXPORTS:
            if hasattr(Model, name):
                def call(*a, f=getattr(model, name), name=name):
                    model.calls.append(name)
                    return f(*a)
                p.setattr(ub, name, call)
        yield m, model


def block(m, n_pages, max_seqs=4, max_len=64, page=16, capacity=256, **kw):
    H, G, D = 2, 1, 64
    w = torch.zeros(HIDDEN, (H + 2 * G) * D, dtype=torch.bfloat16), torch.zeros(H * D, HIDDEN, dtype=torch.bfloat16)
    return m.AttentionBlock(*w, H, G, D, capacity=capacity, max_seqs=max_seqs, max_len=max_len, page=page, n_pages=n_pages, **kw)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)
