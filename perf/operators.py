"""The attention operators of one tensor-parallel rank, case by case.

Four calls over packed (THD) tokens: the rotation of q and k with the append to a paged
key-value cache, causal attention over whole prompts, its gradient (a training step runs
both), and the attention of one new token per sequence over the paged cache.  ``run`` with
``own`` false computes them with elementary torch operations in 32 bits; with ``own`` true
it makes the library's calls.
"""

import math
import random

import torch

own = False

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def listed():
    return [
        # One decode step of a small batch: 16 sequences append their new token (GQA shard:
        # 8 query heads on 1 key-value head).  Latency.
        dict(name="append_step_gqa", kind="append", tokens=16, seqs=16, step=True, past=4096, heads=8, kv_heads=1,
             dim=128, page=16, cache="bf16", token_major=False, pairs="half", pad=0, pack=1),
        # The prompts of one pack enter the cache (QKV shard with 4 heads of 128).
        dict(name="append_prompt_qkv", kind="append", tokens=8184, seqs=5, step=False, past=0, heads=4, kv_heads=4,
             dim=128, page=64, cache="bf16", token_major=True, pairs="half", pad=3, pack=2),
        # A long chunk of prompts joins sequences that are cached already, as E4M3.
        dict(name="append_prompt_gqa_e4m3", kind="append", tokens=32520, seqs=7, step=False, past=2000, heads=8,
             kv_heads=1, dim=128, page=64, cache="e4m3", token_major=False, pairs="half", pad=0, pack=3),
        # Short prompts of a small model: 2 heads of 64.  Latency.
        dict(name="prompt_tiny", kind="prompt", tokens=256, seqs=3, heads=2, kv_heads=2, dim=64, pad=1, pack=4),
        # One pack of prompts of the QKV shard.
        dict(name="prompt_qkv", kind="prompt", tokens=8184, seqs=5, heads=4, kv_heads=4, dim=128, pad=3, pack=5),
        # One long document on the GQA shard.
        dict(name="prompt_gqa_long", kind="prompt", tokens=24392, seqs=1, heads=8, kv_heads=1, dim=128, pad=0, pack=6),
        # A training step's attention, forward and backward, of a small model.
        dict(name="train_tiny", kind="train", tokens=1000, seqs=6, heads=2, kv_heads=2, dim=64, pad=5, pack=7),
        # The same of one pack of the QKV shard.
        dict(name="train_qkv", kind="train", tokens=8184, seqs=5, heads=4, kv_heads=4, dim=128, pad=3, pack=8),
        # The same of one pack of longer documents on the GQA shard.
        dict(name="train_gqa", kind="train", tokens=16264, seqs=2, heads=8, kv_heads=1, dim=128, pad=0, pack=9),
        # One user's next token over a long cache.
        dict(name="decode_one_gqa", kind="decode", seqs=1, shortest=32520, longest=32520, heads=8, kv_heads=1, dim=128,
             page=64, cache="bf16", token_major=False, pad=0, pack=10),
        # A batch of ragged lengths, as many key-value heads as query heads.
        dict(name="decode_batch_qkv", kind="decode", seqs=64, shortest=1, longest=8192, heads=4, kv_heads=4, dim=128,
             page=16, cache="bf16", token_major=True, pad=0, pack=11),
        # A large ragged batch over an E4M3 cache.
        dict(name="decode_batch_gqa_e4m3", kind="decode", seqs=128, shortest=100, longest=32520, heads=8, kv_heads=1,
             dim=128, page=64, cache="e4m3", token_major=False, pad=0, pack=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["append", "prompt", "train", "decode"])
    heads, kv_heads, dim = rng.choice([(2, 2, 64), (4, 4, 128), (8, 1, 128), (8, 2, 128), (6, 3, 80), (5, 1, 64), (16, 1, 128)])
    c = dict(kind=kind, heads=heads, kv_heads=kv_heads, dim=dim, pad=rng.choice([0, 0, 1, 7]), pack=rng.randrange(1 << 30))
    if kind in ("append", "decode"):
        c.update(page=rng.choice([1, 16, 24, 64, 128]), cache=rng.choice(["bf16", "e4m3"]),
                 token_major=rng.random() < 0.5)
    if kind == "append":
        step = rng.random() < 0.4
        c.update(step=step, past=rng.choice([0, _log(rng, 1, 8192)]), pairs=rng.choice(["half", "half", "next"]))
        c["seqs"] = _log(rng, 1, 64) if step else rng.randint(1, 12)
        c["tokens"] = c["seqs"] if step else _log(rng, 16, 16384)
    elif kind == "decode":
        c["seqs"] = _log(rng, 1, 160)
        c["longest"] = _log(rng, 1, 16384)
        c["shortest"] = rng.choice([0, c["longest"], c["longest"] // 3])
    else:
        c["seqs"] = rng.randint(1, 12)
        c["tokens"] = _log(rng, 16, 8192 if kind == "prompt" else 6000)
    return c


def lengths(c):
    """Tokens of each sequence: of a pack (their sum is `tokens`), or in the cache before a
    decode step's attention."""
    r, n = random.Random(c["pack"]), c["seqs"]
    if c["kind"] == "decode":
        return [r.randint(c["shortest"], c["longest"]) for _ in range(n)]
    if c.get("step"):
        return [1] * n
    w = [r.uniform(0.2, 1.0) for _ in range(n)]
    lens = [int(c["tokens"] * x / sum(w)) for x in w]
    if n >= 4:  # packs also hold single tokens and, after filtering, empty sequences
        lens[1], lens[2] = 0, 1
    lens[0] += c["tokens"] - sum(lens)
    return lens


def pasts(c):
    r = random.Random(c["pack"] + 1)
    return [r.randint(0, c["past"]) for _ in range(c["seqs"])]


def _rotary(c):
    return c["dim"] // 16 * 16


def _item(c):
    return 1 if c.get("cache") == "e4m3" else 2


def work(case):
    c, lens = case, lengths(case)
    H, G, D = c["heads"], c["kv_heads"], c["dim"]
    tokens, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
    rows = tokens + c["pad"]
    if c["kind"] == "append":
        read = tokens * (H + 2 * G) * D * 2
        return {"bytes": read + rows * H * D * 2 + tokens * 2 * G * D * _item(c), "flops": 3 * tokens * (H + G) * _rotary(c)}
    if c["kind"] == "prompt":
        return {"bytes": rows * (2 * H + 2 * G) * D * 2 + rows * H * 4, "flops": 4 * D * H * pairs}
    if c["kind"] == "train":
        return {"bytes": rows * (4 * H + 4 * G) * D * 2 + rows * H * 4, "flops": 14 * D * H * pairs}
    return {"bytes": tokens * 2 * G * D * _item(c) + 2 * (c["seqs"] + c["pad"]) * H * D * 2, "flops": 4 * D * H * tokens}


# ---- inputs ------------------------------------------------------------------------------
def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + c["pack"] % 1000003)
    H, G, D = c["heads"], c["kv_heads"], c["dim"]
    lens = lengths(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=c, n=c["seqs"], lens_host=lens, longest=max(max(lens), 1), scale=1.0 / math.sqrt(D))
    rows = c["seqs"] + c["pad"] if c["kind"] == "decode" else sum(lens) + c["pad"]
    s["rows"] = rows
    total = [0]
    for n in lens:
        total.append(total[-1] + n)
    s["cu"] = torch.tensor(total, **i32)
    if c["kind"] == "decode":
        s["q"] = _normal(g, (rows, H * D), 1.5)
    else:  # the QKV projection's rows: q, k and v side by side
        s["qkv"] = _normal(g, (rows, (H + 2 * G) * D))
        s["qkv"][:, : H * D] *= 1.5
    s["out"] = torch.empty((rows, H * D), dtype=BF16, device="cuda")
    s["lse"] = torch.empty((H, rows), dtype=torch.float32, device="cuda")
    if c["kind"] == "train":
        s["dout"] = _normal(g, (rows, H * D))
        s["dqkv"] = torch.empty_like(s["qkv"])
    if "cache" in c:
        past = pasts(c) if c["kind"] == "append" else [0] * c["seqs"]
        s["past"] = torch.tensor(past, **i32)
        s["lens"] = torch.tensor(lens, **i32)
        s["e4m3"], s["k_scale"], s["v_scale"] = c["cache"] == "e4m3", 40.0, 60.0
        need = [-(-(p + n) // c["page"]) for p, n in zip(past, lens)]
        n_pages, most = max(sum(need), 1), max(max(need), 1)
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        pages, at = torch.full((c["seqs"], most), -1, **i32), 0
        for i, m in enumerate(need):
            pages[i, :m] = order[at: at + m]
            at += m
        s["pages"] = pages
        shape = (n_pages, c["page"], G, D) if c["token_major"] else (n_pages, G, c["page"], D)
        for name, scale in (("k_cache", s["k_scale"]), ("v_cache", s["v_scale"])):
            x = _normal(g, shape)
            x = (x.float() * scale).clamp_(-448, 448).to(F8) if s["e4m3"] else x
            s[name] = x.transpose(1, 2) if c["token_major"] else x  # [pages, heads, tokens, dim]
    r = _rotary(c)
    s["inv_freq"] = (500000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)).float()
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps between calls: the registered buffer, descriptors, workspaces."""
    import chunked_tp_overlap_amd.ub as ub

    c = s["case"]
    H, G, D, rows = c["heads"], c["kv_heads"], c["dim"], max(s["rows"], 1)
    s["ub"] = ub
    s["buf"] = torch.empty(rows * H * D, dtype=BF16, device="cuda")
    s["h"] = ub.ub_init(rows, H * D, 1, ub.UB_DTYPE_BF16, s["buf"], rows * H * D * 2)
    s["cfg"] = ub.make_attn_cfg(H, G, D, rotary_dim=_rotary(c), rope_interleaved=c.get("pairs") == "next")
    s["hout"] = ub.heads(s["out"])
    if c["kind"] == "decode":
        s["hq"] = ub.heads(s["q"])
    else:
        s["hq"], s["hk"], s["hv"] = (ub.heads(s["qkv"], col) for col in (0, H * D, (H + G) * D))
    if c["kind"] == "train":
        s["hdout"] = ub.heads(s["dout"])
        s["hdq"], s["hdk"], s["hdv"] = (ub.heads(s["dqkv"], col) for col in (0, H * D, (H + G) * D))
    if "cache" in c:
        s["cache"] = ub.make_kv_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    op = {"prompt": ub.UB_ATTN_PROMPT, "train": ub.UB_ATTN_PROMPT_BWD, "decode": ub.UB_ATTN_DECODE}.get(c["kind"])
    if op is not None:
        nbytes = ub.ub_attn_required_bytes(op, s["cfg"], rows, s["n"])
        s["ws"] = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    if c["kind"] == "train":
        nbytes = ub.ub_attn_required_bytes(ub.UB_ATTN_PROMPT, s["cfg"], rows, s["n"])
        s["ws_fwd"] = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device="cuda")


# ---- one pass ------------------------------------------------------------------------------
def run(state):
    s, kind = state, state["case"]["kind"]
    if own:
        return _own(s, kind)
    if kind == "append":
        return _append(s)
    if kind == "prompt":
        out, lse, _ = _prompt(s)
        return {"out": out, "lse": lse}
    if kind == "train":
        return _train(s)
    return _decode(s)


def _own(s, kind):
    ub, h, cfg = s["ub"], s["h"], s["cfg"]
    stream = torch.cuda.current_stream()
    if kind == "append":
        ub.ub_kv_append(h, s["hq"], s["hk"], s["hv"], s["hout"], None, s["inv_freq"], s["cu"], s["past"], s["n"],
                        s["cache"], s["pages"], cfg, stream)
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if kind == "prompt":
        ub.ub_attn_prompt(h, s["hq"], s["hk"], s["hv"], s["hout"], s["lse"], s["cu"], s["n"], cfg, s["ws"], stream)
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "train":
        ub.ub_attn_prompt(h, s["hq"], s["hk"], s["hv"], s["hout"], s["lse"], s["cu"], s["n"], cfg, s["ws_fwd"], stream)
        ub.ub_attn_prompt_bwd(h, s["hdout"], s["hq"], s["hk"], s["hv"], s["hout"], s["lse"], s["hdq"], s["hdk"],
                              s["hdv"], s["cu"], s["n"], cfg, s["ws"], stream)
        return {"out": s["out"], "lse": s["lse"], "dqkv": s["dqkv"]}
    ub.ub_attn_decode(h, s["hq"], s["cache"], s["pages"], s["lens"], s["n"], s["hout"], s["lse"], cfg, s["ws"], stream)
    return {"out": s["out"], "lse": s["lse"]}


def _store(s, x, scale):
    """Rows for the cache: bf16, or E4M3 codes of x * scale as bytes."""
    return (x * scale).clamp_(-448, 448).to(F8).view(torch.uint8) if s["e4m3"] else x.to(BF16)


def _load(s, x, scale):
    return x.float() / scale if s["e4m3"] else x.float()


def _rotate(s, x, angle, pairs):
    r = 2 * angle.shape[-1]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if pairs == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., r:]), -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., r:]), -1)


def _append(s):
    c = s["case"]
    H, G, D, t = c["heads"], c["kv_heads"], c["dim"], sum(s["lens_host"])
    token = torch.arange(t, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], token, right=True)
    pos = (s["past"][seq] + token - s["cu"][seq]).long()
    angle = pos.double()[:, None] * s["inv_freq"].double()
    x = s["qkv"][:t].float()
    q = _rotate(s, x[:, : H * D].view(t, H, D), angle, c["pairs"])
    k = _rotate(s, x[:, H * D: (H + G) * D].view(t, G, D), angle, c["pairs"])
    v = x[:, (H + G) * D:].view(t, G, D)
    page, off = s["pages"][seq, pos // c["page"]].long(), pos % c["page"]
    for name, rows, scale in (("k_cache", k, s["k_scale"]), ("v_cache", v, s["v_scale"])):
        cache = s[name].view(torch.uint8) if s["e4m3"] else s[name]
        cache[page, :, off] = _store(s, rows, scale)
    out = torch.zeros((s["rows"], H * D), dtype=BF16, device="cuda")
    out[:t] = q.reshape(t, H * D).to(BF16)
    return {"q": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _padded(s, x, heads):
    """[rows, heads * dim] -> [seqs, heads, longest, dim] in 32 bits, zeros past a sequence."""
    n, L = s["n"], s["longest"]
    at = torch.arange(L, device="cuda", dtype=torch.int32)
    lens = s["cu"][1:] - s["cu"][:-1]
    valid = at < lens[:, None]
    row = torch.where(valid, s["cu"][:-1, None] + at, 0).long()
    x = x[row].float().view(n, L, heads, -1) * valid[:, :, None, None]
    return x.transpose(1, 2)


def _packed(s, x, fill=0.0):
    """[seqs, heads, longest, w] -> [rows, heads * w], `fill` in rows of no sequence."""
    t = sum(s["lens_host"])
    token = torch.arange(t, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], token, right=True)
    out = torch.full((s["rows"], x.shape[1] * x.shape[3]), fill, dtype=x.dtype, device="cuda")
    out[:t] = x[seq, :, (token - s["cu"][seq]).long()].reshape(t, -1)
    return out


def _prompt(s):
    c, L = s["case"], s["longest"]
    H, G, D, n = c["heads"], c["kv_heads"], c["dim"], s["n"]
    q = _padded(s, s["qkv"][:, : H * D], H).reshape(n, G, H // G, L, D)
    k = _padded(s, s["qkv"][:, H * D: (H + G) * D], G)[:, :, None]
    v = _padded(s, s["qkv"][:, (H + G) * D:], G)[:, :, None]
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    at = torch.arange(L, device="cuda")
    p.masked_fill_(at > at[:, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total)
    out = _packed(s, torch.matmul(p, v).reshape(n, H, L, D))
    lse = _packed(s, (m + total.log()).reshape(n, H, L, 1), -math.inf)
    return out.to(BF16), lse.t().contiguous(), (q, k, v, p, out)


def _train(s):
    c, L = s["case"], s["longest"]
    H, G, D, n = c["heads"], c["kv_heads"], c["dim"], s["n"]
    out, lse, (q, k, v, p, o) = _prompt(s)
    do = _padded(s, s["dout"], H).reshape(n, G, H // G, L, D)
    o = _padded(s, o, H).reshape(n, G, H // G, L, D)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2).contiguous()).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k).reshape(n, H, L, D)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    dqkv = torch.cat([_packed(s, x) for x in (dq, dk, dv)], -1).to(BF16)
    return {"out": out, "lse": lse, "dqkv": dqkv}


def _decode(s):
    c, L = s["case"], s["longest"]
    H, G, D, n = c["heads"], c["kv_heads"], c["dim"], s["n"]
    pos = torch.arange(L, device="cuda")
    valid = pos < s["lens"][:, None]
    page = torch.where(valid, s["pages"][:, pos // c["page"]], 0).long()
    off = (pos % c["page"]).expand(n, L)
    k = _load(s, s["k_cache"].view(torch.uint8)[page, :, off].view(F8) if s["e4m3"] else s["k_cache"][page, :, off], s["k_scale"])
    v = _load(s, s["v_cache"].view(torch.uint8)[page, :, off].view(F8) if s["e4m3"] else s["v_cache"][page, :, off], s["v_scale"])
    q = s["q"][:n].float().view(n, G, H // G, D)
    p = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).mul_(s["scale"])
    p = torch.where(valid[:, None, None], p, -math.inf)
    m = p.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = (p - m0).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(1, 2).contiguous()) / torch.where(total == 0, 1.0, total)
    out = torch.zeros((s["rows"], H * D), dtype=BF16, device="cuda")
    out[:n] = o.reshape(n, H * D).to(BF16)
    lse = torch.full((H, s["rows"]), -math.inf, dtype=torch.float32, device="cuda")
    lse[:, :n] = (m0 + total.log()).reshape(n, H).t()
    return {"out": out, "lse": lse}


# ---- 64 bits, from the definitions ---------------------------------------------------------
def exact(case, seed):
    c, s = case, prepare(case, seed)
    H, G, D, lens = c["heads"], c["kv_heads"], c["dim"], lengths(case)
    f64 = dict(dtype=torch.float64, device="cuda")
    if c["kind"] == "append":
        return _exact_append(c, s, lens)
    out = torch.zeros((s["rows"], H, D), **f64)
    lse = torch.full((H, s["rows"]), -math.inf, **f64)
    if c["kind"] == "decode":
        for i, n in enumerate(lens):
            if not n:
                continue
            at = torch.arange(n, device="cuda")
            page, off = s["pages"][i].long()[at // c["page"]], at % c["page"]
            for h in range(H):
                k, v = ((s[name].view(torch.uint8)[page, h // (H // G), off].view(F8) if s["e4m3"]
                         else s[name][page, h // (H // G), off]).double() / (s[sc] if s["e4m3"] else 1.0)
                        for name, sc in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
                x = (k @ s["q"][i, h * D: (h + 1) * D].double()) * D ** -0.5
                lse[h, i] = x.logsumexp(0)
                out[i, h] = (x - lse[h, i]).exp() @ v
        return {"out": out.flatten(1), "lse": lse}
    train = c["kind"] == "train"
    grad = torch.zeros((s["rows"], H + 2 * G, D), **f64)
    x = s["qkv"].view(s["rows"], H + 2 * G, D)
    for i, n in enumerate(lens):
        a = sum(lens[:i])
        for h in range(H if n else 0):
            j = h // (H // G)
            q, k, v = (x[a: a + n, w].double() for w in (h, H + j, H + G + j))
            for r0 in range(0, n, 8192):  # blocks of rows: a long document's square does not fit at once
                r1 = min(n, r0 + 8192)
                y = (q[r0:r1] @ k[:r1].t().contiguous()) * D ** -0.5
                y.masked_fill_(torch.arange(r1, device="cuda") > torch.arange(r0, r1, device="cuda")[:, None], -math.inf)
                l = y.logsumexp(1)
                y = y.sub_(l[:, None]).exp_()
                lse[h, a + r0: a + r1] = l
                o = y @ v[:r1]
                out[a + r0: a + r1, h] = o
                if train:
                    do = s["dout"].view(s["rows"], H, D)[a + r0: a + r1, h].double()
                    grad[a: a + r1, H + G + j] += y.t().contiguous() @ do
                    z = y * (do @ v[:r1].t().contiguous() - (do * o).sum(1, keepdim=True)) * D ** -0.5
                    grad[a + r0: a + r1, h] += z @ k[:r1]
                    grad[a: a + r1, H + j] += z.t().contiguous() @ q[r0:r1]
    res = {"out": out.flatten(1), "lse": lse}
    if train:
        res["dqkv"] = grad.flatten(1)
    return res


def _exact_append(c, s, lens):
    """Values before their rounding to the output's type; slots of the cache that are not
    written hold what they held."""
    H, G, D, r = c["heads"], c["kv_heads"], c["dim"], _rotary(c)
    out = torch.zeros((s["rows"], H, D), dtype=torch.float64, device="cuda")
    caches = {name: s[name].double() for name in ("k_cache", "v_cache")}
    first = 0
    for i, n in enumerate(lens):
        x = s["qkv"][first: first + n].double().view(n, H + 2 * G, D)
        pos = pasts(c)[i] + torch.arange(n, device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * s["inv_freq"].double())[:, None]
        y = x.clone()
        one, two = (slice(0, r // 2), slice(r // 2, r)) if c["pairs"] == "half" else (slice(0, r, 2), slice(1, r, 2))
        z = torch.complex(x[:, : H + G, one].contiguous(), x[:, : H + G, two].contiguous()) * turn
        y[:, : H + G, one], y[:, : H + G, two] = z.real, z.imag
        out[first: first + n] = y[:, :H]
        page, off = s["pages"][i].long()[pos // c["page"]], pos % c["page"]
        for name, at, sc in (("k_cache", H, "k_scale"), ("v_cache", H + G, "v_scale")):
            caches[name][page, :, off] = (y[:, at: at + G] * s[sc]).clamp(-448, 448) if s["e4m3"] else y[:, at: at + G]
        first += n
    return {"q": out.flatten(1), **caches}
