"""One rank's attention block over the library's calls: prompts, training steps and decode.

    python -m chunked_tp_overlap_amd.attention_block

``AttentionBlock`` holds what a serving or training program keeps between calls (the
registered UserBuffer, a paged key-value cache, the weights, workspaces) and runs, for each
microbatch of packed tokens:

    x -> ub_copy_in -> ub_gemm_ag_chunked (QKV) -> ub_kv_append (rotation, cache)
      -> ub_attn_prompt or ub_attn_decode -> ub_gemm_rs_chunked (output projection) -> y

Rows of a microbatch beyond its tokens (T is a multiple of tp_size) are padding.  Only device
memory comes from torch.  A call's work runs on torch's current stream, in order with the torch
operations around it; a decode step can be captured into a graph.
"""

import torch

import chunked_tp_overlap_amd.ub as ub

BF16 = torch.bfloat16


class AttentionBlock:
    """Heads of one rank: wqkv [hidden, (heads + 2 kv_heads) dim] and wo [heads dim, hidden], both
    contiguous bf16 matrices, which are kept and not copied.  The cache has room for `max_len` tokens
    of each of `max_seqs` sequences, as bf16 or (with scales k_scale and v_scale) E4M3."""

    def __init__(self, wqkv, wo, heads, kv_heads, dim, capacity, max_seqs, max_len, page=64, tp=1, cache=BF16,
                 k_scale=1.0, v_scale=1.0, rope_base=10000.0):
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
        shape = (max_seqs * per_seq, kv_heads, page, dim)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=cache, device="cuda") for _ in range(2))
        self.cache = ub.make_kv_cache(self.k_cache, self.v_cache, k_scale, v_scale)
        self.pages = torch.arange(max_seqs * per_seq, dtype=torch.int32, device="cuda").view(max_seqs, per_seq)
        self.lens = torch.zeros(max_seqs, dtype=torch.int32, device="cuda")
        need = [ub.ub_attn_required_bytes(op, self.cfg, capacity, max_seqs)
                for op in (ub.UB_ATTN_PROMPT, ub.UB_ATTN_PROMPT_BWD, ub.UB_ATTN_DECODE)]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
        cols = (0, heads * dim, (heads + kv_heads) * dim)
        self.hqkv = [ub.heads(self.qkv, c) for c in cols]
        self.hdqkv = [ub.heads(self.dqkv, c) for c in cols]
        self.hq, self.hk, self.hattn = ub.heads(self.q), ub.heads(self.k), ub.heads(self.attn)

    def _project_in(self, x):
        """QKV of x's rows; the active shape becomes their number, rounded up to tp."""
        if x.dim() != 2 or x.shape[1] != self.hidden or x.dtype is not BF16:
            raise ValueError(f"x: a bf16 matrix of hidden size {self.hidden}, not {x.dtype} {tuple(x.shape)}")
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

    def _project_out(self, rows):
        k = self.heads * self.dim
        ub.ub_gemm_rs_chunked(self.h, self.attn, k, k, self.wo, self.hidden, self.y, self.hidden, self.gemm,
                              torch.cuda.current_stream())
        return self.y[:rows]

    def prefill(self, x, lens):
        """Prompts x [sum(lens), hidden], one after another, of new sequences 0, 1, ...: fills the
        cache and returns the block's output rows (valid until the next call)."""
        cu = torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        n = len(lens)
        self._project_in(x)
        self._append(cu, None, n, self.cache)
        ub.ub_attn_prompt(self.h, self.hq, self.hk, self.hqkv[2], self.hattn, None, cu, n, self.cfg, self.ws,
                          torch.cuda.current_stream())
        self.lens[:n] = cu[1:] - cu[:-1]
        self.step = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        return self._project_out(x.shape[0])

    def decode(self, x):
        """The next token's rows x [sequences, hidden] of the sequences that prefill set up."""
        n = x.shape[0]
        self._project_in(x)
        self._append(self.step, self.lens, n, self.cache)
        self.lens[:n] += 1
        ub.ub_attn_decode(self.h, self.hq, self.cache, self.pages, self.lens, n, self.hattn, None, self.cfg, self.ws,
                          torch.cuda.current_stream())
        return self._project_out(n)

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
        ub.ub_attn_prompt(self.h, self.hq, self.hk, self.hqkv[2], self.hattn, lse, cu, n, self.cfg, self.ws, stream)
        y = self._project_out(rows)
        ub.ub_attn_prompt_bwd(self.h, ub.heads(d), self.hq, self.hk, self.hqkv[2], self.hattn, lse, *self.hdqkv, cu, n,
                              self.cfg, self.ws, stream)
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


if __name__ == "__main__":
    main()
