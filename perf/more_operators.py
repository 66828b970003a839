"""Attention with a sliding window, drafted trees, and the pages of a cache, case by case.

Calls of one tensor-parallel rank next to its causal attention: attention over packed tokens
with a sliding window and a few first tokens that stay visible (prompts, a training step, one
new token over a paged cache); attention of drafted trees over a paged cache, the append of
their tokens and the move of the accepted ones; and forks of cached sequences that share
their pages.  ``run`` with ``own`` false computes them with elementary torch operations in 32
bits; with ``own`` true it makes the library's calls.
"""

import math
import random

import torch

own = False

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def listed():
    return [
        # Short prompts of a small windowed model: 2 heads of 64.  Latency.
        dict(name="window_prompt_tiny", kind="prompt", tokens=500, seqs=3, heads=2, kv_heads=2, dim=64, window=128, sinks=4,
             pad=1, pack=1),
        # One long document on the GQA shard, where the window leaves a sixth of the keys.
        dict(name="window_prompt_gqa_long", kind="prompt", tokens=24392, seqs=1, heads=8, kv_heads=1, dim=128, window=2048,
             sinks=4, pad=0, pack=2),
        # A training step's attention of one pack of the QKV shard, without sinks.
        dict(name="window_train_qkv", kind="train", tokens=8184, seqs=5, heads=4, kv_heads=4, dim=128, window=512, sinks=0,
             pad=3, pack=3),
        # The same of one pack of longer documents on the GQA shard, with sinks.
        dict(name="window_train_gqa", kind="train", tokens=16264, seqs=2, heads=8, kv_heads=1, dim=128, window=2048, sinks=4,
             pad=0, pack=4),
        # One user's next token over a long cache of which the window is left.  Latency.
        dict(name="window_decode_one_gqa", kind="decode", seqs=1, shortest=32520, longest=32520, heads=8, kv_heads=1, dim=128,
             page=64, cache="bf16", token_major=False, window=4096, sinks=4, pad=0, pack=5),
        # A ragged batch, as many key-value heads as query heads.
        dict(name="window_decode_batch_qkv", kind="decode", seqs=64, shortest=1, longest=16264, heads=4, kv_heads=4, dim=128,
             page=16, cache="bf16", token_major=True, window=4096, sinks=16, pad=0, pack=6),
        # One user's draft of 24 tokens over a long cache.  Latency.
        dict(name="tree_one_gqa", kind="tree", seqs=1, shortest=32520, longest=32520, nodes=24, heads=8, kv_heads=1, dim=128,
             page=64, cache="bf16", token_major=False, pad=0, pack=7),
        # A ragged batch's drafts of up to 60 tokens over an E4M3 cache.
        dict(name="tree_batch_gqa_e4m3", kind="tree", seqs=64, shortest=100, longest=16264, nodes=60, heads=8, kv_heads=1,
             dim=128, page=64, cache="e4m3", token_major=False, pad=0, pack=8),
        # A small batch's drafts enter the cache, and the accepted ones move to their places.  Latency.
        dict(name="commit_step_gqa", kind="commit", seqs=16, shortest=100, longest=2000, nodes=24, heads=8, kv_heads=1,
             dim=128, page=16, cache="bf16", token_major=False, pad=0, pack=9),
        # The same of a large batch, as many key-value heads as query heads.
        dict(name="commit_batch_qkv", kind="commit", seqs=256, shortest=1, longest=2000, nodes=60, heads=4, kv_heads=4,
             dim=128, page=16, cache="bf16", token_major=True, pad=0, pack=10),
        # A few prompts, each forked into 4 samples that take some tokens and end.  Latency.
        dict(name="fork_samples_gqa", kind="fork", seqs=8, shortest=100, longest=2000, samples=4, grow=40, heads=8, kv_heads=1,
             dim=128, page=16, spare=0.5, cache="bf16", token_major=False, pack=11),
        # Many prompts, each forked into 8.
        dict(name="fork_batch_qkv", kind="fork", seqs=64, shortest=1, longest=8192, samples=8, grow=200, heads=4, kv_heads=4,
             dim=128, page=64, spare=1.0, cache="bf16", token_major=True, pack=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["prompt", "train", "decode", "tree", "commit", "fork"])
    heads, kv_heads, dim = rng.choice([(2, 2, 64), (4, 4, 128), (8, 1, 128), (8, 2, 128), (6, 3, 80), (5, 1, 64), (16, 1, 128)])
    c = dict(kind=kind, heads=heads, kv_heads=kv_heads, dim=dim, pack=rng.randrange(1 << 30))
    if kind != "fork":
        c["pad"] = rng.choice([0, 0, 1, 7])
    if kind in ("prompt", "train", "decode"):
        c.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 0, 1, 4, 16, 64]))
    if kind in ("prompt", "train"):
        c.update(seqs=rng.randint(1, 12), tokens=_log(rng, 16, 8192 if kind == "prompt" else 6000))
        return c
    c.update(page=rng.choice([1, 16, 24, 64, 128]), cache=rng.choice(["bf16", "e4m3"]), token_major=rng.random() < 0.5)
    c["longest"] = _log(rng, 1, {"decode": 16384, "tree": 8192, "commit": 2000, "fork": 2000}[kind])
    c["shortest"] = rng.choice([0 if kind in ("decode", "tree") else 1, c["longest"], (c["longest"] + 2) // 3])
    c["seqs"] = _log(rng, 1, {"decode": 160, "tree": 40, "commit": 64, "fork": 32}[kind])
    if kind in ("tree", "commit"):
        c["nodes"] = _log(rng, 1, 64)
    if kind == "fork":
        c.update(samples=rng.randint(1, 8), grow=_log(rng, 1, 200), spare=rng.choice([0.1, 1.0]))
    return c


# ---- what a case's lengths, trees and tables are -------------------------------------------
def lengths(c):
    """Tokens of each sequence: of a pack (their sum is `tokens`), or cached before the call."""
    r, n = random.Random(c["pack"]), c["seqs"]
    if "longest" in c:
        return [r.randint(c["shortest"], c["longest"]) for _ in range(n)]
    w = [r.uniform(0.2, 1.0) for _ in range(n)]
    lens = [int(c["tokens"] * x / sum(w)) for x in w]
    if n >= 4:  # packs also hold single tokens and, after filtering, empty sequences
        lens[1], lens[2] = 0, 1
    lens[0] += c["tokens"] - sum(lens)
    return lens


def trees(c):
    """Each sequence's drafted nodes as (parents, depths, an accepted path): a node's parent comes
    before it, -1 for a child of the last cached token."""
    r, out = random.Random(c["pack"] + 2), []
    for _ in range(c["seqs"]):
        m = c["nodes"] if c["seqs"] == 1 else r.randint((c["nodes"] + 1) // 2, c["nodes"])
        parents = [max(-1, j - 1 - int(r.expovariate(0.4))) for j in range(m)]
        depths = []
        for p in parents:
            depths.append(depths[p] + 1 if p >= 0 else 0)
        path, j = [], r.randrange(m)
        while j >= 0:
            path.insert(0, j)
            j = parents[j]
        out.append((parents, depths, path[: r.randint(0, len(path))]))
    return out


def grown(c):
    """New lengths of a fork's rows: the prompts' own, then the samples'."""
    r, lens = random.Random(c["pack"] + 3), lengths(c)
    return lens + [n + r.randint(1, c["grow"]) for n in lens for _ in range(c["samples"])]


def _cumulated(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _pages(n, page):
    return -(-n // page)


def _rotary(c):
    return c["dim"] // 16 * 16


def _item(c):
    return 1 if c.get("cache") == "e4m3" else 2


def seen(c, n):
    """Pairs of a row and a key that it sees, in a sequence of n tokens."""
    w, s = c["window"], c["sinks"]
    hidden = max(n - w - s, 0)  # rows that some key is hidden from: they hide 1, 2, ... keys
    return n * (n + 1) // 2 - hidden * (hidden + 1) // 2


def work(case):
    c, lens, kind = case, lengths(case), case["kind"]
    H, G, D = c["heads"], c["kv_heads"], c["dim"]
    if kind in ("prompt", "train"):
        rows, pairs = sum(lens) + c["pad"], sum(seen(c, n) for n in lens)
        if kind == "prompt":
            return {"bytes": rows * (2 * H + 2 * G) * D * 2 + rows * H * 4, "flops": 4 * D * H * pairs}
        return {"bytes": rows * (4 * H + 4 * G) * D * 2 + rows * H * 4, "flops": 14 * D * H * pairs}
    kv = 2 * G * D * _item(c)  # key and value of a token
    if kind == "decode":
        keys = sum(min(n, c["window"] + c["sinks"]) for n in lens)
        return {"bytes": keys * kv + 2 * (c["seqs"] + c["pad"]) * H * D * 2, "flops": 4 * D * H * keys}
    if kind == "fork":
        lens2, page = grown(c), c["page"]
        rows = len(lens2)
        copied = sum(lens[(i - c["seqs"]) // c["samples"]] % page for i in range(c["seqs"], rows))
        entries = sum(_pages(n, page) for n in lens) + rows * _pages(max(lens2), page) + 2 * sum(_pages(n, page) for n in lens2)
        return {"bytes": 2 * copied * kv + 4 * entries, "flops": 0}
    t = trees(c)
    nodes = sum(len(p) for p, _, _ in t)
    if kind == "tree":
        pairs = sum(len(p) * n + sum(d) + len(d) for n, (p, d, _) in zip(lens, t))
        return {"bytes": (sum(lens) + nodes) * kv + 2 * (nodes + c["pad"]) * H * D * 2, "flops": 4 * D * H * pairs}
    moved = sum(len([0 for i, j in enumerate(path) if i != j]) for _, _, path in t)
    return {"bytes": nodes * (H + 2 * G) * D * 2 + (nodes + c["pad"]) * H * D * 2 + (nodes + 2 * moved) * kv,
            "flops": 3 * nodes * (H + G) * _rotary(c)}


# ---- inputs ------------------------------------------------------------------------------
def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + c["pack"] % 1000003)
    H, G, D, n, kind = c["heads"], c["kv_heads"], c["dim"], c["seqs"], c["kind"]
    lens = lengths(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=c, n=n, lens_host=lens, scale=1.0 / math.sqrt(D))
    s["lens"] = torch.tensor(lens, **i32)
    if kind in ("tree", "commit"):
        t = trees(c)
        nodes = [len(p) for p, _, _ in t]
        s["nodes"], s["most_nodes"] = sum(nodes), max(nodes)
        s["cu"] = torch.tensor(_cumulated(nodes), **i32)
        s["parents"] = torch.tensor([p for x in t for p in x[0]], **i32)
        s["depths"] = torch.tensor([d for x in t for d in x[1]], **i32)
        s["full"] = torch.tensor([a + b for a, b in zip(lens, nodes)], **i32)  # the drafts appended
        s["kept"] = torch.zeros((n, max(nodes)), **i32)
        for i, x in enumerate(t):
            if x[2]:
                s["kept"][i, : len(x[2])] = torch.tensor(x[2], **i32)
        s["kept_lens"] = torch.tensor([len(x[2]) for x in t], **i32)
        s["lens_out"] = torch.zeros(n, **i32)
        held = [a + b for a, b in zip(lens, nodes)]
    else:
        s["cu"] = torch.tensor(_cumulated(lens), **i32)
        held = lens
    rows = {"prompt": sum(lens), "train": sum(lens), "decode": n}.get(kind, s.get("nodes", 0)) + c.get("pad", 0)
    s["rows"], s["longest"] = rows, max(max(held), 1)
    if kind in ("decode", "tree"):
        s["q"] = _normal(g, (rows, H * D), 1.5)
    elif kind != "fork":  # the QKV projection's rows: q, k and v side by side
        s["qkv"] = _normal(g, (rows, (H + 2 * G) * D))
        s["qkv"][:, : H * D] *= 1.5
    s["out"] = torch.empty((rows, H * D), dtype=BF16, device="cuda")
    s["lse"] = torch.empty((H, rows), dtype=torch.float32, device="cuda")
    if kind == "train":
        s["dout"] = _normal(g, (rows, H * D))
        s["dqkv"] = torch.empty_like(s["qkv"])
    if "cache" in c:
        _cache(s, c, g, held)
    r = _rotary(c)
    s["inv_freq"] = (500000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)).float()
    if own:
        _handles(s)
    return s


def _cache(s, c, g, held):
    """A pool of pages, dealt to the sequences in a random order."""
    G, D, n, page = c["kv_heads"], c["dim"], c["seqs"], c["page"]
    i32 = dict(dtype=torch.int32, device="cuda")
    s["e4m3"], s["k_scale"], s["v_scale"] = c["cache"] == "e4m3", 40.0, 60.0
    need = [_pages(m, page) for m in held]
    used, most = max(sum(need), 1), max(max(need), 1)
    n_pages = used
    if c["kind"] == "fork":
        s["new_lens"] = torch.tensor(grown(c), **i32)
        most = _pages(max(grown(c)), page)
        extra = sum(_pages(a, page) for a in grown(c)[n:])
        n_pages += extra + int(c["spare"] * used)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.full((n, most), -1, **i32), 0
    refs = torch.zeros(n_pages, **i32)
    for i, m in enumerate(need):
        table[i, :m] = order[at: at + m]
        at += m
    refs[order[:at].long()] = 1
    if c["kind"] == "decode":  # pages that the window left behind are given back: their entries hold nothing
        e = torch.arange(most, device="cuda")
        gone = (e * page >= c["sinks"]) & ((e + 1) * page <= s["lens"][:, None] - c["window"])
        table[gone] = -1
    s["pages"], s["refs"], s["n_pages"] = table, refs, n_pages
    shape = (n_pages, page, G, D) if c["token_major"] else (n_pages, G, page, D)
    for name, scale in (("k_cache", s["k_scale"]), ("v_cache", s["v_scale"])):
        x = _normal(g, shape)
        x = (x.float() * scale).clamp_(-448, 448).to(F8) if s["e4m3"] else x
        s[name] = x.transpose(1, 2) if c["token_major"] else x  # [pages, heads, tokens, dim]
    if c["kind"] == "fork":
        rows = n * (1 + c["samples"])
        own_rows, copies = list(range(n)), [i for i in range(n) for _ in range(c["samples"])]
        s["forked"], s["ended"] = torch.tensor(own_rows + copies, **i32), torch.tensor(own_rows, **i32)
        s["fork_rows"] = rows
        s["pages_fork"], s["lens_fork"] = torch.empty((rows, most), **i32), torch.empty(rows, **i32)
        s["lens_grown"], s["copies"] = torch.empty(rows, **i32), torch.empty((rows, 3), **i32)
        s["pages_end"], s["lens_end"] = torch.empty((n, most), **i32), torch.empty(n, **i32)


def _handles(s):
    """What a program keeps between calls: the registered buffer, descriptors, workspaces."""
    import chunked_tp_overlap_amd.ub as ub

    c = s["case"]
    H, G, D, rows, kind = c["heads"], c["kv_heads"], c["dim"], max(s["rows"], 1), c["kind"]
    s["ub"] = ub
    s["buf"] = torch.empty(rows * H * D, dtype=BF16, device="cuda")
    s["h"] = ub.ub_init(rows, H * D, 1, ub.UB_DTYPE_BF16, s["buf"], rows * H * D * 2)
    s["cfg"] = ub.make_attn_cfg(H, G, D, rotary_dim=_rotary(c))
    if kind in ("tree", "commit"):  # a value for each active row, those of no sequence too
        s["row_parents"], s["row_depths"] = (torch.nn.functional.pad(s[x], (0, rows - s["nodes"])) for x in ("parents", "depths"))
    if "window" in c:
        s["win"] = ub.make_attn_window(c["window"], c["sinks"])
    s["hout"] = ub.heads(s["out"])
    if "q" in s:
        s["hq"] = ub.heads(s["q"])
    if "qkv" in s:
        s["hq"], s["hk"], s["hv"] = (ub.heads(s["qkv"], col) for col in (0, H * D, (H + G) * D))
    if kind == "train":
        s["hdout"] = ub.heads(s["dout"])
        s["hdq"], s["hdk"], s["hdv"] = (ub.heads(s["dqkv"], col) for col in (0, H * D, (H + G) * D))
    if "cache" in c:
        s["cache"] = ub.make_kv_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    op = {"train": ub.UB_ATTN_PROMPT_WINDOW_BWD, "decode": ub.UB_ATTN_DECODE_WINDOW, "tree": ub.UB_ATTN_TREE}.get(kind)
    nbytes = 0
    if op is not None:
        nbytes = ub.ub_attn_required_bytes(op, s["cfg"], rows, s["n"])
    elif kind == "fork":
        nbytes = ub.ub_kv_resize_bytes(s["fork_rows"])
    s["ws"] = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device="cuda")


# ---- one pass ------------------------------------------------------------------------------
def run(state):
    s, kind = state, state["case"]["kind"]
    if own:
        return _own(s, kind)
    if kind == "prompt":
        out, lse, _ = _prompt(s)
        return {"out": out, "lse": lse}
    return {"train": _train, "decode": _decode, "tree": _tree, "commit": _commit, "fork": _fork}[kind](s)


def _own(s, kind):
    ub, h, cfg = s["ub"], s["h"], s["cfg"]
    stream = torch.cuda.current_stream()
    if kind == "prompt":
        ub.ub_attn_prompt_window(h, s["hq"], s["hk"], s["hv"], s["hout"], s["lse"], s["cu"], s["n"], s["win"], cfg, None, stream)
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "train":
        ub.ub_attn_prompt_window(h, s["hq"], s["hk"], s["hv"], s["hout"], s["lse"], s["cu"], s["n"], s["win"], cfg, None, stream)
        ub.ub_attn_prompt_window_bwd(h, s["hdout"], s["hq"], s["hk"], s["hv"], s["hout"], s["lse"], s["hdq"], s["hdk"],
                                     s["hdv"], s["cu"], s["n"], s["win"], cfg, s["ws"], stream)
        return {"out": s["out"], "lse": s["lse"], "dqkv": s["dqkv"]}
    if kind == "decode":
        ub.ub_attn_decode_window(h, s["hq"], s["cache"], s["pages"], s["lens"], s["n"], s["win"], s["hout"], s["lse"], cfg,
                                 s["ws"], stream)
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "tree":
        ub.ub_attn_tree(h, s["hq"], s["cache"], s["pages"], s["full"], s["row_parents"], s["cu"], s["n"], s["hout"], s["lse"],
                        cfg, s["ws"], stream)
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "commit":
        ub.ub_kv_append_at(h, s["hq"], s["hk"], s["hv"], s["hout"], None, s["inv_freq"], s["row_depths"], s["cu"], s["lens"],
                           s["n"], s["cache"], s["pages"], cfg, stream)
        ub.ub_kv_compact(h, s["cache"], s["pages"], s["lens"], s["kept"], s["kept_lens"], s["n"], s["lens_out"], cfg, stream)
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["lens_out"]}
    page, rows = s["case"]["page"], s["fork_rows"]
    ub.ub_kv_fork(h, s["refs"], s["pages"], s["lens"], s["n"], s["forked"], s["pages_fork"], s["lens_fork"], rows, page, stream)
    ub.ub_kv_resize(h, s["refs"], s["pages_fork"], s["lens_fork"], s["new_lens"], rows, s["lens_grown"], s["copies"], page,
                    None, s["ws"], stream)
    ub.ub_kv_copy_pages(h, s["cache"], s["copies"], rows, cfg, stream)
    ub.ub_kv_fork(h, s["refs"], s["pages_fork"], s["lens_grown"], rows, s["ended"], s["pages_end"], s["lens_end"], s["n"],
                  page, stream)
    return {"pages": s["pages_fork"], "lens": s["lens_grown"], "copies": s["copies"], "k_cache": s["k_cache"],
            "v_cache": s["v_cache"], "refs": s["refs"], "pages_end": s["pages_end"], "lens_end": s["lens_end"]}


def _padded(s, x, heads):
    """[rows, heads * dim] -> [seqs, heads, longest, dim] in 32 bits, zeros past a sequence."""
    n, L = s["n"], s["longest"]
    at = torch.arange(L, device="cuda", dtype=torch.int32)
    lens = s["cu"][1:] - s["cu"][:-1]
    valid = at < lens[:, None]
    row = torch.where(valid, s["cu"][:-1, None] + at, 0).long()
    x = x[row].float().view(n, L, heads, -1) * valid[:, :, None, None]
    return x.transpose(1, 2)


def _packed(s, x, total, fill=0.0):
    """[seqs, heads, longest, w] -> [rows, heads * w], `fill` in rows of no sequence."""
    token = torch.arange(total, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], token, right=True)
    out = torch.full((s["rows"], x.shape[1] * x.shape[3]), fill, dtype=x.dtype, device="cuda")
    out[:total] = x[seq, :, (token - s["cu"][seq]).long()].reshape(total, -1)
    return out


def _prompt(s):
    c, L, t = s["case"], s["longest"], sum(s["lens_host"])
    H, G, D, n = c["heads"], c["kv_heads"], c["dim"], s["n"]
    q = _padded(s, s["qkv"][:, : H * D], H).reshape(n, G, H // G, L, D)
    k = _padded(s, s["qkv"][:, H * D: (H + G) * D], G)[:, :, None]
    v = _padded(s, s["qkv"][:, (H + G) * D:], G)[:, :, None]
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    u = torch.arange(L, device="cuda")
    row = u[:, None]
    p.masked_fill_((u > row) | ((row - u >= c["window"]) & (u >= c["sinks"])), -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total)
    out = _packed(s, torch.matmul(p, v).reshape(n, H, L, D), t)
    lse = _packed(s, (m + total.log()).reshape(n, H, L, 1), t, -math.inf)
    return out.to(BF16), lse.t().contiguous(), (q, k, v, p, out)


def _train(s):
    c, L, t = s["case"], s["longest"], sum(s["lens_host"])
    H, G, D, n = c["heads"], c["kv_heads"], c["dim"], s["n"]
    out, lse, (q, k, v, p, o) = _prompt(s)
    do = _padded(s, s["dout"], H).reshape(n, G, H // G, L, D)
    o = _padded(s, o, H).reshape(n, G, H // G, L, D)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2).contiguous()).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k).reshape(n, H, L, D)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    dqkv = torch.cat([_packed(s, x, t) for x in (dq, dk, dv)], -1).to(BF16)
    return {"out": out, "lse": lse, "dqkv": dqkv}


def _rows_of(s, name, scale, page, off):
    """Keys or values [seqs, positions, heads, dim] at pages and places, in 32 bits."""
    if s["e4m3"]:
        return s[name].view(torch.uint8)[page, :, off].view(F8).float() / scale
    return s[name][page, :, off].float()


def _attend(q, k, v, allowed, scale):
    """q [n, G, rows, D], k and v [n, L, G, D], allowed broadcastable to [n, G, rows, L]; a row that
    sees nothing gets 0 and -inf."""
    p = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).mul_(scale)
    p = torch.where(allowed, p, -math.inf)
    m = p.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = (p - m0).exp()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v.transpose(1, 2).contiguous()) / torch.where(total == 0, 1.0, total), m0 + total.log()


def _decode(s):
    c, L = s["case"], s["longest"]
    H, G, D, n = c["heads"], c["kv_heads"], c["dim"], s["n"]
    u = torch.arange(L, device="cuda")
    left = s["lens"][:, None] - u  # 1 at the last token
    seen = (left > 0) & ((left <= c["window"]) | (u < c["sinks"]))
    page = torch.where(seen, s["pages"][:, u // c["page"]], 0).long()
    off = (u % c["page"]).expand(n, L)
    k, v = (_rows_of(s, name, s[name[0] + "_scale"], page, off) for name in ("k_cache", "v_cache"))
    v = v * seen[:, :, None, None]
    o, l = _attend(s["q"][:n].float().view(n, G, H // G, D), k, v, seen[:, None, None], s["scale"])
    out = torch.zeros((s["rows"], H * D), dtype=BF16, device="cuda")
    out[:n] = o.reshape(n, H * D).to(BF16)
    lse = torch.full((H, s["rows"]), -math.inf, dtype=torch.float32, device="cuda")
    lse[:, :n] = l.reshape(n, H).t()
    return {"out": out, "lse": lse}


def _closed(step, doublings):
    """Paths of any length up to 2 ** doublings, from those of length 0 and 1."""
    return step if doublings == 0 else _closed(torch.matmul(step, step).clamp_(max=1.0), doublings - 1)


def _tree(s):
    c, L, M = s["case"], s["longest"], s["most_nodes"]
    H, G, D, n = c["heads"], c["kv_heads"], c["dim"], s["n"]
    j = torch.arange(M, device="cuda", dtype=torch.int32)
    node = j < (s["cu"][1:] - s["cu"][:-1])[:, None]
    row = torch.where(node, s["cu"][:-1, None] + j, 0).long()
    parent = torch.where(node, s["parents"][row], -1)
    path = _closed(((parent[:, :, None] == j) | (j[:, None] == j)).float(), max(M - 1, 1).bit_length()) > 0
    u = torch.arange(L, device="cuda", dtype=torch.int32)
    drafted = u - s["lens"][:, None]
    at = drafted.clamp(0, M - 1).long()[:, None].expand(n, M, L)
    seen = (drafted < 0)[:, None] | ((u < s["full"][:, None])[:, None] & path.gather(2, at))
    held = u < s["full"][:, None]
    page = torch.where(held, s["pages"][:, (u // c["page"]).long()], 0).long()
    off = (u % c["page"]).long().expand(n, L)
    k, v = (_rows_of(s, name, s[name[0] + "_scale"], page, off) for name in ("k_cache", "v_cache"))
    q = s["q"][row].float().view(n, M, G, H // G, D).permute(0, 2, 3, 1, 4).reshape(n, G, H // G * M, D)
    o, l = _attend(q, k, v, seen[:, None, None].expand(n, G, H // G, M, L).reshape(n, G, -1, L), s["scale"])
    out = _packed(s, o.reshape(n, H, M, D), s["nodes"]).to(BF16)
    lse = _packed(s, l.reshape(n, H, M, 1), s["nodes"], -math.inf)
    return {"out": out, "lse": lse.t().contiguous()}


def _bytes(s, name):
    return s[name].view(torch.uint8) if s["e4m3"] else s[name]


def _commit(s):
    c = s["case"]
    H, G, D, t = c["heads"], c["kv_heads"], c["dim"], s["nodes"]
    r = _rotary(c)
    token = torch.arange(t, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], token, right=True)
    first = s["lens"][seq]
    angle = (first + s["depths"]).double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = s["qkv"][:t].float().view(t, H + 2 * G, D)
    a, b = x[:, : H + G, : r // 2], x[:, : H + G, r // 2: r]
    qk = torch.cat((a * cos - b * sin, b * cos + a * sin, x[:, : H + G, r:]), -1)
    pos = (first + token - s["cu"][seq]).long()
    page, off = s["pages"][seq, pos // c["page"]].long(), pos % c["page"]
    d = torch.arange(s["most_nodes"], device="cuda")
    moved = d < s["kept_lens"][:, None]
    to = torch.where(moved, s["lens"][:, None] + d, 0)
    of = torch.where(moved, s["lens"][:, None] + s["kept"], 0)  # the others: the first token stays where it is
    i = torch.arange(s["n"], device="cuda")[:, None]
    of_page, of_off = s["pages"][i, of // c["page"]].long(), (of % c["page"]).long()
    to_page, to_off = s["pages"][i, to // c["page"]].long(), (to % c["page"]).long()
    for name, y, scale in (("k_cache", qk[:, H:], s["k_scale"]), ("v_cache", x[:, H + G:], s["v_scale"])):
        cache = _bytes(s, name)
        cache[page, :, off] = (y * scale).clamp(-448, 448).to(F8).view(torch.uint8) if s["e4m3"] else y.to(BF16)
        cache[to_page, :, to_off] = cache[of_page, :, of_off]
    out = torch.zeros((s["rows"], H * D), dtype=BF16, device="cuda")
    out[:t] = qk[:, :H].reshape(t, H * D).to(BF16)
    return {"q": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["lens"] + s["kept_lens"]}


def _share(s, refs, pages, lens, parents, page):
    """Rows `parents` of a table in place of all its rows; refs count a page's holders."""
    e = torch.arange(pages.shape[1], device="cuda")
    held = e < (lens[:, None] + page - 1) // page
    uses = torch.zeros(len(lens), dtype=torch.int32, device="cuda").index_add_(0, parents, torch.ones_like(parents)) - 1
    refs = refs.index_add(0, torch.where(held, pages, 0).long().flatten(), torch.where(held, uses[:, None], 0).flatten())
    return refs, torch.where(held, pages, -1)[parents.long()], lens[parents.long()]


def _fork(s):
    c, rows = s["case"], s["fork_rows"]
    page = c["page"]
    refs, pages, lens = _share(s, s["refs"], s["pages"], s["lens"], s["forked"], page)
    new, e, i = s["new_lens"], torch.arange(pages.shape[1], device="cuda"), torch.arange(rows, device="cuda")
    had, has = (lens + page - 1) // page, (new + page - 1) // page
    last = pages[i, (had - 1).long()]
    part = torch.where((new > lens) & (refs[last.long()] > 1), lens % page, 0)  # tokens of a shared last page
    begin = had - (part > 0).int()
    need = has - begin
    end = need.cumsum(0)
    free = torch.argsort((refs > 0).int(), stable=True)
    served = (need == 0) | (end <= (refs == 0).sum())
    taken = served[:, None] & (e >= begin[:, None]) & (e < has[:, None])
    rank = torch.where(taken, (end - need - begin)[:, None] + e, 0)
    given = torch.where(taken, free[rank].int(), pages)
    part = torch.where(served, part, 0)
    refs = refs.index_add(0, torch.where(taken, given, 0).long().flatten(), taken.flatten().int())
    refs = refs.index_add(0, last.long(), -(part > 0).int())
    to = torch.where(part > 0, given[i, (had - 1).long()], last)
    token = torch.arange(page, device="cuda")[None, None, :, None] < part[:, None, None, None]
    for name in ("k_cache", "v_cache"):
        cache = _bytes(s, name)
        cache[to.long()] = torch.where(token, cache[last.long()], cache[to.long()])
    grown = torch.where(served, new, lens)
    copies = torch.stack((torch.where(part > 0, last, -1), torch.where(part > 0, to, -1), part), 1)
    refs, pages_end, lens_end = _share(s, refs, given, grown, s["ended"], page)
    return {"pages": given, "lens": grown, "copies": copies, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "refs": refs,
            "pages_end": pages_end, "lens_end": lens_end}


# ---- 64 bits, from the definitions ---------------------------------------------------------
def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "fork":
        return _exact_fork(c, s)
    if kind == "commit":
        return _exact_commit(c, s)
    H, G, D, lens = c["heads"], c["kv_heads"], c["dim"], lengths(c)
    f64 = dict(dtype=torch.float64, device="cuda")
    out = torch.zeros((s["rows"], H, D), **f64)
    lse = torch.full((H, s["rows"]), -math.inf, **f64)
    res = {"out": out.view(s["rows"], H * D), "lse": lse}
    if kind in ("decode", "tree"):
        first, drafts = 0, trees(c) if kind == "tree" else [([], [], [])] * len(lens)
        for i, n in enumerate(lens):
            parents = drafts[i][0]
            m = len(parents) if kind == "tree" else 1
            total = n + len(parents)
            if not total:  # one row for each sequence of a decode step, the empty ones too
                first += m
                continue
            see = torch.ones((m, total), dtype=torch.bool)
            if kind == "tree":
                see[:, n:] = False
                for j, p in enumerate(parents):
                    if p >= 0:
                        see[j] = see[p]
                    see[j, n + j] = True
            else:
                see[0, min(c["sinks"], total): max(total - c["window"], 0)] = False
            see, at = see.cuda(), torch.arange(total, device="cuda")
            page, off = s["pages"][i].long()[at // c["page"]].clamp(min=0), at % c["page"]
            for h in range(H):
                k, v = ((s[name].view(torch.uint8)[page, h // (H // G), off].view(F8) if s["e4m3"]
                         else s[name][page, h // (H // G), off]).double() / (s[sc] if s["e4m3"] else 1.0)
                        for name, sc in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
                q = s["q"][first: first + m, h * D: (h + 1) * D].double()
                x = (q @ k.t().contiguous() * D ** -0.5).masked_fill_(~see, -math.inf)
                lse[h, first: first + m] = x.logsumexp(1)
                out[first: first + m, h] = (x - lse[h, first: first + m, None]).exp() @ v
            first += m
        return res
    train = kind == "train"
    grad = torch.zeros((s["rows"], H + 2 * G, D), **f64)
    x = s["qkv"].view(s["rows"], H + 2 * G, D)
    for i, n in enumerate(lens):
        a = sum(lens[:i])
        for h in range(H if n else 0):
            g = h // (H // G)
            q, k, v = (x[a: a + n, w].double() for w in (h, H + g, H + G + g))
            for r0 in range(0, n, 8192):  # blocks of rows: a long document's square does not fit at once
                r1 = min(n, r0 + 8192)
                y = (q[r0:r1] @ k[:r1].t().contiguous()) * D ** -0.5
                back = torch.arange(r0, r1, device="cuda")[:, None] - torch.arange(r1, device="cuda")
                hidden = back >= c["window"]
                hidden[:, : c["sinks"]] = False
                y.masked_fill_(hidden | (back < 0), -math.inf)
                l = y.logsumexp(1)
                y = y.sub_(l[:, None]).exp_()
                lse[h, a + r0: a + r1] = l
                o = y @ v[:r1]
                out[a + r0: a + r1, h] = o
                if train:
                    do = s["dout"].view(s["rows"], H, D)[a + r0: a + r1, h].double()
                    grad[a: a + r1, H + G + g] += y.t().contiguous() @ do
                    z = y * (do @ v[:r1].t().contiguous() - (do * o).sum(1, keepdim=True)) * D ** -0.5
                    grad[a + r0: a + r1, h] += z @ k[:r1]
                    grad[a: a + r1, H + g] += z.t().contiguous() @ q[r0:r1]
    if train:
        res["dqkv"] = grad.flatten(1)
    return res


def _exact_commit(c, s):
    """Values before their rounding to the output's type; slots of the cache that are not written
    hold what they held."""
    H, G, D, r = c["heads"], c["kv_heads"], c["dim"], _rotary(c)
    out = torch.zeros((s["rows"], H, D), dtype=torch.float64, device="cuda")
    caches = {name: s[name].double() for name in ("k_cache", "v_cache")}
    one, first = torch.ones((), dtype=torch.float64, device="cuda"), 0
    for i, (n, (parents, depths, path)) in enumerate(zip(lengths(c), trees(c))):
        m = len(parents)
        x = s["qkv"][first: first + m].double().view(m, H + 2 * G, D)
        angle = (n + torch.tensor(depths, device="cuda")).double()[:, None] * s["inv_freq"].double()
        z = torch.complex(x[:, : H + G, : r // 2].contiguous(), x[:, : H + G, r // 2: r].contiguous()) * torch.polar(one, angle)[:, None]
        y = x.clone()
        y[:, : H + G, : r // 2], y[:, : H + G, r // 2: r] = z.real, z.imag
        out[first: first + m] = y[:, :H]
        order = path + list(range(len(path), m))  # what the slots after the cached tokens hold at the end
        pos = n + torch.arange(m, device="cuda")
        page, off = s["pages"][i].long()[pos // c["page"]], pos % c["page"]
        for name, at, sc in (("k_cache", H, "k_scale"), ("v_cache", H + G, "v_scale")):
            w = y[order, at: at + G]
            caches[name][page, :, off] = (w * s[sc]).clamp(-448, 448) if s["e4m3"] else w
        first += m
    return {"q": out.flatten(1), **caches, "lens": None}


def _exact_fork(c, s):
    """What the caches hold after the copies of shared last pages, row by row; the tables and counts
    are whole numbers."""
    page, n, lens, table = c["page"], c["seqs"], lengths(c), s["pages"].tolist()
    held = [table[i][: _pages(m, page)] for i, m in enumerate(lens)]
    used = {p for row in held for p in row}
    free = (p for p in range(s["n_pages"]) if p not in used)
    caches = {name: s[name].double() for name in ("k_cache", "v_cache")}
    res = {"pages": None, "lens": None, "copies": None, **caches, "refs": None, "pages_end": None, "lens_end": None}
    for row, new in enumerate(grown(c)[n:]):
        i = row // c["samples"]
        part = lens[i] % page if new > lens[i] else 0
        given = [next(free) for _ in range(_pages(new, page) - len(held[i]) + (part > 0))]
        if part:
            for x in caches.values():
                x[given[0], :, :part] = x[held[i][-1], :, :part]
    return res
