"""One rank's attention block over the library's calls: prompts, training steps and decode.

    python -m chunked_tp_overlap_amd.attention_block

``AttentionBlock`` holds what a serving or training program keeps between calls (the
registered UserBuffer, a paged key-value cache, the weights, workspaces) and runs, for each
microbatch of packed tokens:

    x -> ub_copy_in -> ub_gemm_ag_chunked (QKV) -> ub_kv_append (rotation, cache)
      -> ub_attn_prompt or ub_attn_decode -> ub_gemm_rs_chunked (output projection) -> y

With a window the attention calls are the windowed ones.  ``draft`` runs trees of drafted tokens
after the cached ones (ub_kv_append_at, ub_attn_tree) and ``accept`` keeps a path of each
(ub_kv_compact).  A block with a pool of pages deals them to its sequences as they grow and takes
them back (ub_kv_resize, ub_kv_copy_pages), and ``fork`` lets sequences share them (ub_kv_fork).

Rows of a microbatch beyond its tokens (T is a multiple of tp_size) are padding.  Only device
memory comes from torch.  A call's work runs on torch's current stream, in order with the torch
operations around it; a decode step can be captured into a graph.
"""

import torch

import chunked_tp_overlap_amd.ub as ub

BF16 = torch.bfloat16
NOWHERE = 1 << 30  # a place past any table: nothing is stored there, and a sequence that long is NaN


class AttentionBlock:
    """Heads of one rank: wqkv [hidden, (heads + 2 kv_heads) dim] and wo [heads dim, hidden], both
    contiguous bf16 matrices, which are kept and not copied.  The cache has room for `max_len` tokens
    of each of `max_seqs` sequences, as bf16 or (with scales k_scale and v_scale) E4M3; with
    `n_pages`, a pool of so many pages, for as many tokens of sequences up to that long as they hold.
    Where the pool has no pages for a sequence's new tokens (or its row of the table no entries) they are not
    stored, and their rows are NaN; once it has lost a token so, all its later rows are, and its copies',
    and its entry of `lens`, the cached tokens of each, is NOWHERE or more.  What it held is free when it
    ends (`fork`, `prefill`).  Drafts are no tokens of their sequence before they are accepted.  window:
    how many tokens a token sees, itself among them, besides the first `sinks`; a pool gets the pages of
    tokens that no later one sees back with the next decoded token, and has to hold whole prompts till then."""

    def __init__(self, wqkv, wo, heads, kv_heads, dim, capacity, max_seqs, max_len, page=64, tp=1, cache=BF16,
                 k_scale=1.0, v_scale=1.0, rope_base=10000.0, window=None, sinks=0, n_pages=None):
        for name, w, shape in (("wqkv", wqkv, (wqkv.shape[0], (heads + 2 * kv_heads) * dim)),
                               ("wo", wo, (heads * dim, wqkv.shape[0]))):
            if tuple(w.shape) != shape or w.dtype is not BF16 or not w.is_contiguous():
                raise ValueError(f"{name}: a contiguous bf16 {list(shape)} matrix")
        self.wqkv, self.wo, self.tp, self.hidden = wqkv, wo, tp, wqkv.shape[0]
        self.heads, self.kv_heads, self.dim, self.max_seqs = heads, kv_heads, dim, max_seqs
        bf16 = dict(dtype=BF16, device="cuda")
        ub_bytes, ws_bytes = ub.ub_required_bytes(capacity, self.hidden, tp)
        self.buf = torch.zeros(ub_bytes // 2, **bf16)
        self.rs_ws = torch.zeros(ws_bytes // 2, **bf16)
        self.h = ub.ub_init(capacity, self.hidden, tp, ub.UB_DTYPE_BF16, self.buf, ub_bytes, self.rs_ws, ws_bytes)
        self.gemm = ub.make_cfg("ring_exchange", tp, atomic_gemm=True)
        self.cfg = ub.make_attn_cfg(heads, kv_heads, dim)
        n = heads + 2 * kv_heads
        self.qkv, self.dqkv = (torch.zeros((capacity, n * dim), **bf16) for _ in range(2))
        self.q, self.attn = (torch.zeros((capacity, heads * dim), **bf16) for _ in range(2))
        self.k = torch.zeros((capacity, kv_heads * dim), **bf16)
        self.y = torch.zeros((capacity, self.hidden), **bf16)
        r = self.cfg.rotary_dim
        self.inv_freq = (rope_base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
        per_seq = -(-max_len // page)
        self.pool = n_pages is not None
        if self.pool and per_seq * page > NOWHERE:
            raise ValueError(f"max_len: {NOWHERE} tokens at most with a pool, not {max_len}")
        shape = (n_pages if self.pool else max_seqs * per_seq, kv_heads, page, dim)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=cache, device="cuda") for _ in range(2))
        self.cache = ub.make_kv_cache(self.k_cache, self.v_cache, k_scale, v_scale)
        self.pages = torch.arange(max_seqs * per_seq, dtype=torch.int32, device="cuda").view(max_seqs, per_seq)
        self.lens, self.next_lens, self.past = (torch.zeros(max_seqs, dtype=torch.int32, device="cuda") for _ in range(3))
        # a decode step's boundaries, one row to a sequence, where a captured step finds them
        self.step = torch.arange(max_seqs + 1, dtype=torch.int32, device="cuda")
        self.page, self.seqs, self.drafted = page, 0, 0  # sequences there are; drafted for, not yet accepted
        if self.pool:  # no sequence holds any of them
            self.pages.fill_(-1)
            self.other_pages = torch.zeros_like(self.pages)
            self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
            self.held = torch.zeros(max_seqs, dtype=torch.int32, device="cuda")  # tokens a row has pages for
            self.copies = torch.zeros((max_seqs, 3), dtype=torch.int32, device="cuda")
            self.resize_ws = torch.zeros(ub.ub_kv_resize_bytes(max_seqs), dtype=torch.uint8, device="cuda")
        self.window = None if window is None else ub.make_attn_window(window, sinks)
        need = [ub.ub_attn_required_bytes(op, self.cfg, capacity, max_seqs)
                for op in (ub.UB_ATTN_PROMPT, ub.UB_ATTN_PROMPT_BWD, ub.UB_ATTN_DECODE, ub.UB_ATTN_TREE)]
        if window is not None:
            need.append(ub.ub_attn_required_bytes(ub.UB_ATTN_PROMPT_WINDOW_BWD, self.cfg, capacity, max_seqs))
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
        cols = (0, heads * dim, (heads + kv_heads) * dim)
        self.hqkv = [ub.heads(self.qkv, c) for c in cols]
        self.hdqkv = [ub.heads(self.dqkv, c) for c in cols]
        self.hq, self.hk, self.hattn = ub.heads(self.q), ub.heads(self.k), ub.heads(self.attn)

    def _check(self, x):
        if x.dim() != 2 or x.shape[1] != self.hidden or x.dtype is not BF16:
            raise ValueError(f"x: a bf16 matrix of hidden size {self.hidden}, not {x.dtype} {tuple(x.shape)}")

    def _project_in(self, x):
        """QKV of x's rows; the active shape becomes their number, rounded up to tp."""
        self._check(x)
        rows = x.shape[0]
        T = -(-rows // self.tp) * self.tp
        stream = torch.cuda.current_stream()
        ub.ub_set_active_shape(self.h, (T, self.hidden))
        ub.ub_copy_in(self.h, x.contiguous(), rows, 0, stream)
        n = self.qkv.shape[1]
        ub.ub_gemm_ag_chunked(self.h, self.wqkv, n, n, self.qkv, n, self.gemm, stream)
        return T

    def _append(self, cu, past, n, cache):
        ub.ub_kv_append(self.h, *self.hqkv, self.hq, self.hk, self.inv_freq, cu, past, n, cache,
                        None if cache is None else self.pages, self.cfg, torch.cuda.current_stream())

    def _hold(self, lens, n, window=None):
        """Pages for so many tokens of the first n sequences, those that drop out given back; a last
        page that others hold too is replaced by a copy."""
        if not self.pool:
            return
        stream = torch.cuda.current_stream()
        ub.ub_kv_resize(self.h, self.refs, self.pages, self.held, lens, n, self.held, self.copies, self.page, window,
                        self.resize_ws, stream)
        ub.ub_kv_copy_pages(self.h, self.cache, self.copies, n, self.cfg, stream)

    def _lose(self, lens, wanted):
        """After `_hold` of so many tokens: where the pool had no pages for them, a sequence's next place is
        nowhere (a last page that others hold too is then still in its table), and its length stays past
        what the pool gives pages for."""
        lens.masked_fill_(self.held[: lens.shape[0]] < wanted, NOWHERE)

    def _project_out(self, rows):
        k = self.heads * self.dim
        ub.ub_gemm_rs_chunked(self.h, self.attn, k, k, self.wo, self.hidden, self.y, self.hidden, self.gemm,
                              torch.cuda.current_stream())
        return self.y[:rows]

    def prefill(self, x, lens):
        """Prompts x [sum(lens), hidden], one after another, of new sequences 0, 1, ...: fills the
        cache and returns the block's output rows (valid until the next call)."""
        self._check(x)
        lens = [int(m) for m in lens]
        n = len(lens)
        if n > self.max_seqs:
            raise ValueError(f"prefill: {n} prompts, {self.max_seqs} at most")
        if min(lens, default=0) < 0 or sum(lens) > x.shape[0]:
            raise ValueError(f"prefill: prompts of {lens} tokens, x is {tuple(x.shape)}")
        self._project_in(x)  # whose checks come before the sequences end, too
        cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        self.drafted = 0
        if self.pool:  # the sequences before them end
            self.lens.zero_()
            self._hold(self.lens, self.max_seqs)
        self.lens[:n] = cu[1:] - cu[:-1]
        self._hold(self.lens, n)
        if self.pool:
            self._lose(self.lens[:n], self.lens[:n])
        self._append(cu, None, n, self.cache)
        stream = torch.cuda.current_stream()
        if self.window is None:
            ub.ub_attn_prompt(self.h, self.hq, self.hk, self.hqkv[2], self.hattn, None, cu, n, self.cfg, self.ws, stream)
        else:
            ub.ub_attn_prompt_window(self.h, self.hq, self.hk, self.hqkv[2], self.hattn, None, cu, n, self.window, self.cfg,
                                     self.ws, stream)
        if self.pool:  # a prompt without pages is seen here, not only in the tokens after it
            rows = torch.arange(x.shape[0], dtype=torch.int32, device="cuda")
            lost = torch.cat((self.lens[:n] >= NOWHERE, torch.zeros(1, dtype=torch.bool, device="cuda")))
            self.attn[: x.shape[0]].masked_fill_(lost[torch.bucketize(rows, cu[1:], right=True)][:, None], float("nan"))
        self.seqs = n
        return self._project_out(x.shape[0])

    def decode(self, x):
        """The next token's rows x [sequences, hidden] of the sequences that prefill or fork set up."""
        self._check(x)
        n = x.shape[0]
        if n > self.seqs:
            raise ValueError(f"decode: rows for {n} sequences, there are {self.seqs}")
        self._project_in(x)
        self.drafted = 0
        if self.pool:
            torch.add(self.lens, 1, out=self.next_lens)
            self._hold(self.next_lens, n, self.window)
            self._lose(self.lens[:n], self.next_lens[:n])
        self._append(self.step, self.lens, n, self.cache)
        self.lens[:n] += 1
        stream = torch.cuda.current_stream()
        if self.window is None:
            ub.ub_attn_decode(self.h, self.hq, self.cache, self.pages, self.lens, n, self.hattn, None, self.cfg, self.ws,
                              stream)
        else:
            ub.ub_attn_decode_window(self.h, self.hq, self.cache, self.pages, self.lens, n, self.window, self.hattn, None,
                                     self.cfg, self.ws, stream)
        return self._project_out(n)

    def draft(self, x, trees):
        """Rows x [nodes, hidden] of a tree of drafted tokens for each sequence, one tree after another:
        trees[i] lists for each node the one before it on its path, by its number in the tree, or -1
        after the sequence's last token.  Returns the nodes' output rows; `accept` says which stay."""
        if self.window is not None:
            raise ValueError("draft: no trees under a window")
        if len(trees) > self.max_seqs:
            raise ValueError(f"draft: {len(trees)} trees, {self.max_seqs} at most")
        depths = []
        for i, tree in enumerate(trees):
            first = len(depths)
            for j, p in enumerate(tree):
                if not -1 <= p < j:
                    raise ValueError(f"draft: tree {i}: the node before {j} is one of 0 to {j - 1}, or -1, not {p}")
                depths.append(0 if p < 0 else depths[first + p] + 1)
            if len(tree) > ub.UB_ATTN_MAX_TREE:
                raise ValueError(f"draft: tree {i} has {len(tree)} nodes, {ub.UB_ATTN_MAX_TREE} at most")
        if x.dim() != 2 or x.shape[0] != len(depths):
            raise ValueError(f"draft: {len(depths)} nodes, x is {tuple(x.shape)}")
        n, stream = len(trees), torch.cuda.current_stream()
        T = self._project_in(x)
        pad = [0] * (T - len(depths))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
        cu, depths = i32([0] + [len(t) for t in trees]).cumsum(0, dtype=torch.int32), i32(depths + pad)
        parents = i32([p for t in trees for p in t] + pad)
        nodes = cu[1:] - cu[:-1]
        torch.add(self.lens[:n], nodes, out=self.next_lens[:n])
        self._hold(self.next_lens, n)
        past = self.past[:n]
        past.copy_(self.lens[:n])
        if self.pool:
            self._lose(past, self.next_lens[:n])
            torch.add(past, nodes, out=self.next_lens[:n])
        self.drafted = n
        ub.ub_kv_append_at(self.h, *self.hqkv, self.hq, self.hk, self.inv_freq, depths, cu, past, n, self.cache,
                           self.pages, self.cfg, stream)
        ub.ub_attn_tree(self.h, self.hq, self.cache, self.pages, self.next_lens, parents, cu, n, self.hattn, None, self.cfg,
                        self.ws, stream)
        return self._project_out(x.shape[0])

    def accept(self, kept, kept_lens):
        """Of the trees of the `draft` just before, sequence i's first kept_lens[i] nodes in row i of kept, a
        path from its last token, become its next tokens (int32 tensors on the device)."""
        n = kept.shape[0]
        if n > self.drafted:
            raise ValueError(f"accept: rows for {n} sequences, the call before it drafted for {self.drafted}")
        ub.ub_kv_compact(self.h, self.cache, self.pages, self.past, kept, kept_lens, n, self.next_lens, self.cfg,
                         torch.cuda.current_stream())
        self.drafted = 0
        if self.pool:  # of a tree without pages no node was stored
            some = (kept_lens[:n] > 0) & (kept[:, :1] >= 0).any(1)
            self.lens[:n] = torch.where(self.past[:n] < NOWHERE, self.next_lens[:n], self.lens[:n].masked_fill(some, NOWHERE))
        else:
            self.lens[:n] = self.next_lens[:n]
        self._hold(self.lens, n)  # what the other nodes had is given back

    def fork(self, parents):
        """Sequence i becomes a copy of sequence parents[i] (an int32 tensor on the device; -1: none),
        sharing its pages; sequences that are nobody's parent end, and so do drafts that were not accepted."""
        if not self.pool:
            raise ValueError("fork: a block without a pool has no pages to share")
        n = parents.shape[0]
        if n > self.max_seqs:
            raise ValueError(f"fork: {n} sequences, {self.max_seqs} at most")
        self.drafted = 0
        # A row that holds pages past its tokens would have them to write in, and share them
        self._hold(self.lens, self.max_seqs)
        ub.ub_kv_fork(self.h, self.refs, self.pages, self.held, self.max_seqs, parents, self.other_pages, self.next_lens, n,
                      self.page, torch.cuda.current_stream())
        self.other_pages[n:] = -1
        self.next_lens[n:] = 0
        self.pages.copy_(self.other_pages)  # in place, as all that a captured decode step reads
        self.held.copy_(self.next_lens)
        some = (parents >= 0) & (parents < self.max_seqs)
        lens = torch.where(some, self.lens[parents.clamp(0, self.max_seqs - 1).long()], 0)
        self.lens.zero_()
        self.lens[:n] = lens
        self.seqs = n

    def train(self, x, lens, dattn):
        """A training step's attention: the block's output for documents x, and the gradient of
        the projected q, k and v for the gradient dattn [rows, heads dim] of the attention's output.
        (The gradients of the projections, before and after it, are the caller's.)"""
        cu = torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        n, rows, stream = len(lens), x.shape[0], torch.cuda.current_stream()
        T = self._project_in(x)
        self._append(cu, None, n, None)
        lse = torch.empty((self.heads, T), dtype=torch.float32, device="cuda")
        d = torch.zeros((T, self.heads * self.dim), dtype=BF16, device="cuda")
        d[:rows] = dattn
        qkv = self.hq, self.hk, self.hqkv[2]
        grads = ub.heads(d), *qkv, self.hattn, lse, *self.hdqkv
        if self.window is None:
            ub.ub_attn_prompt(self.h, *qkv, self.hattn, lse, cu, n, self.cfg, self.ws, stream)
            y = self._project_out(rows)
            ub.ub_attn_prompt_bwd(self.h, *grads, cu, n, self.cfg, self.ws, stream)
        else:
            ub.ub_attn_prompt_window(self.h, *qkv, self.hattn, lse, cu, n, self.window, self.cfg, self.ws, stream)
            y = self._project_out(rows)
            ub.ub_attn_prompt_window_bwd(self.h, *grads, cu, n, self.window, self.cfg, self.ws, stream)
        # back through the rotation: the negated frequencies, in place
        dq, dk, _ = self.hdqkv
        ub.ub_kv_append(self.h, dq, dk, None, dq, dk, -self.inv_freq, cu, None, n, None, None, self.cfg, stream)
        return y, self.dqkv[:rows]

    def close(self):
        ub.ub_destroy(self.h)


def main():
    torch.manual_seed(0)
    hidden, heads, kv_heads, dim = 1024, 8, 1, 128
    normal = lambda *s: torch.randn(s, device="cuda").to(BF16)
    wqkv, wo = normal(hidden, (heads + 2 * kv_heads) * dim) / 32, normal(heads * dim, hidden) / 32
    block = AttentionBlock(wqkv, wo, heads, kv_heads, dim, capacity=4096, max_seqs=4, max_len=4096, tp=4)
    lens = [700, 33, 1500]
    y = block.prefill(normal(sum(lens), hidden), lens)
    print("prefill", tuple(y.shape), "mean square", float(y.float().square().mean()))
    for _ in range(4):
        y = block.decode(normal(len(lens), hidden))
    print("decode ", tuple(y.shape), "cached", block.lens[: len(lens)].tolist())
    y, dqkv = block.train(normal(sum(lens), hidden), lens, normal(sum(lens), heads * dim))
    print("train  ", tuple(y.shape), tuple(dqkv.shape), "gradient's mean square", float(dqkv.float().square().mean()))
    block.close()

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    block = AttentionBlock(wqkv, wo, heads, kv_heads, dim, capacity=4096, max_seqs=6, max_len=4096, tp=4, n_pages=100)
    block.prefill(normal(sum(lens), hidden), lens)
    block.fork(i32([0, 0, 1, 2, 2, 2]))
    trees = [[-1, 0, 0, 1]] * 6
    y = block.draft(normal(24, hidden), trees)
    block.accept(i32([[0, 1, 3]] * 6), i32([3, 0, 1, 2, 3, 3]))
    print("draft  ", tuple(y.shape), "cached", block.lens.tolist(), "free pages", int((block.refs == 0).sum()))
    block.close()

    block = AttentionBlock(wqkv, wo, heads, kv_heads, dim, capacity=4096, max_seqs=4, max_len=4096, tp=4, window=512,
                           sinks=4, n_pages=100)
    block.prefill(normal(sum(lens), hidden), lens)
    y = block.decode(normal(len(lens), hidden))
    print("window ", tuple(y.shape), "free pages", int((block.refs == 0).sum()))
    block.close()


if __name__ == "__main__":
    main()
