"""GPU tests of the attention calls as a program uses them: the attention block of one rank
(chunked_tp_overlap_amd/attention_block.py), on another stream, and captured into a HIP graph."""

import math

import pytest
import torch

from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


@pytest.mark.parametrize("tp,cache", [(1, BF16), (4, F8)])
def test_block(tp, cache):
    """Prompts, then decode steps: each stage against its definition from the stage before it,
    and a decoded row against the same row of the longer prompt."""
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    H, G, D, hidden = 4, 2, 64, 256
    ks, vs = (30.0, 50.0) if cache is F8 else (1.0, 1.0)
    wqkv, wo = normal(1, hidden, (H + 2 * G) * D) / 16, normal(2, H * D, hidden) / 16
    b = AttentionBlock(wqkv, wo, H, G, D, capacity=512, max_seqs=3, max_len=300, page=16, tp=tp, cache=cache,
                       k_scale=ks, v_scale=vs)
    lens, steps = [200, 1, 33], 3
    x = normal(3, sum(lens), hidden)
    y = b.prefill(x, lens).clone()
    tokens = [normal(10 + s, len(lens), hidden) for s in range(steps)]

    def gate(got, a, w):  # a matrix product's bound, as for the library's GEMMs
        want = a.double() @ w.double()
        tol = 4e-3 * a.double().norm(dim=1)[:, None] * w.double().norm(dim=0)
        assert bool(((got.double() - want).abs() <= tol).all())

    rows = sum(lens)
    gate(b.qkv[:rows], x, wqkv)
    gate(y, b.attn[:rows], wo)
    split = lambda t: [t[:, : H * D].reshape(-1, H, D), t[:, H * D:(H + G) * D].reshape(-1, G, D), t[:, (H + G) * D:].reshape(-1, G, D)]
    q, k, v = (t.double().cpu() for t in split(b.qkv[:rows]))
    pos = torch.cat([torch.arange(n) for n in lens])
    for got, src in ((b.q[:rows].view(rows, H, D), q), (b.k[:rows].view(rows, G, D), k)):
        w, e = ref.rotate(src, pos, b.inv_freq.cpu(), False, D)
        ref.check(got, w, e * (1 + ref.U16) + ref.U16 * w.abs(), "rotated")
    cu = [0, 200, 201, 234]
    o, _, t, _ = ref.prompt(b.q[:rows].view(rows, H, D).double().cpu(), b.k[:rows].view(rows, G, D).double().cpu(), v, cu, D ** -0.5)
    ref.check(b.attn[:rows].view(rows, H, D), o, t, "prompt")
    for s, token in enumerate(tokens):
        y = b.decode(token)
        n = len(lens)
        gate(b.qkv[:n], token, wqkv)
        gate(y, b.attn[:n], wo)
        assert b.lens.tolist() == [m + s + 1 for m in lens]
        for i, m in enumerate(lens):
            at = torch.arange(m + s + 1)
            pg, off = b.pages[i].long().cpu()[at // 16], at % 16
            kc, vc = (c.view(torch.uint8).cpu().view(F8).double() if cache is F8 else c.double().cpu()
                      for c in (b.k_cache, b.v_cache))
            for g in range(G):
                xq = b.q[i].double().cpu().view(H, D)[g * 2: g * 2 + 2]
                o, _, t, _ = ref.one(xq, kc[pg, g, off] / ks, vc[pg, g, off] / vs, D ** -0.5,
                                     torch.ones(2, m + s + 1, dtype=torch.bool))
                ref.check(b.attn[i].view(H, D)[g * 2: g * 2 + 2], o, t, f"decode {s} {i} {g}")
    decoded = y.clone()
    full = torch.cat([torch.cat([x[a: a + m]] + [t[i: i + 1] for t in tokens]) for i, (a, m) in enumerate(zip(cu, lens))])
    again = b.prefill(full, [m + steps for m in lens])
    last = torch.tensor([m + steps for m in lens]).cumsum(0) - 1
    # both within the attention's and the product's roundings of the same rows; E4M3 keys and
    # values are half a step (2^-4) off besides
    near = (2.0 ** -4 if cache is F8 else 2.0 ** -6) * again[last.cuda()].double().norm(dim=1)
    assert bool(((decoded.double() - again[last.cuda()].double()).norm(dim=1) <= near).all())
    torch.cuda.synchronize()
    b.close()


def test_block_training_step():
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    H, G, D, hidden = 4, 1, 64, 128
    wqkv, wo = normal(1, hidden, (H + 2 * G) * D) / 11, normal(2, H * D, hidden) / 16
    b = AttentionBlock(wqkv, wo, H, G, D, capacity=256, max_seqs=2, max_len=16, tp=4)
    lens = [70, 0, 81]
    rows = sum(lens)
    x, d = normal(3, rows, hidden), normal(4, rows, H * D)
    _, dqkv = b.train(x, lens, d)
    q, k = b.q[:rows].view(rows, H, D).double().cpu(), b.k[:rows].view(rows, G, D).double().cpu()
    v = b.qkv[:rows, (H + G) * D:].reshape(rows, G, D).double().cpu()
    cu = [0, 70, 70, 151]
    (dq, dk, dv), (tq, tk, tv) = ref.prompt_bwd(d.double().cpu().view(rows, H, D), q, k, v, cu, D ** -0.5)
    pos = torch.cat([torch.arange(n) for n in lens])
    got = dqkv.double().cpu()
    for name, w, t, c, n in (("dq", dq, tq, 0, H), ("dk", dk, tk, H * D, G)):
        y, e = ref.rotate(w, pos, -b.inv_freq.cpu(), False, D)
        # the bound of a pair's two entries, turned, and one more rounding
        both = t[..., : D // 2] + t[..., D // 2:]
        tol = (torch.cat([both, both], -1) + e) * (1 + ref.U16) + ref.U16 * y.abs()
        ref.check(got[:, c: c + n * D].reshape(rows, n, D), y, tol, name)
    ref.check(got[:, (H + G) * D:].reshape(rows, G, D), dv, tv, "dv")
    torch.cuda.synchronize()
    b.close()


def calls(seed):
    """The four calls on fixed buffers: what they need, and a function that makes them."""
    import chunked_tp_overlap_amd.ub as ub

    H, G, D, T, page = 8, 2, 128, 600, 16
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, (H + 2 * G) * D), generator=g, device="cuda").to(BF16)
    d = torch.randn((T, H * D), generator=g, device="cuda").to(BF16)
    buf = torch.empty(T * 64, dtype=BF16, device="cuda")
    s = dict(x=x, d=d, buf=buf, ub=ub, T=T)
    s["h"] = ub.ub_init(T, 64, 1, ub.UB_DTYPE_BF16, buf, T * 64 * 2)
    cfg = ub.make_attn_cfg(H, G, D)
    lens = [301, 0, 1, 290]
    cu = torch.tensor([0, 301, 301, 302, 592], dtype=torch.int32, device="cuda")
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    per = -(-max(lens) // page)
    table = torch.arange(len(lens) * per, dtype=torch.int32, device="cuda").view(len(lens), per)
    kc, vc = (torch.zeros((len(lens) * per, G, page, D), dtype=BF16, device="cuda") for _ in range(2))
    inv = (10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)).float()
    outs = dict(q=torch.empty((T, H * D), dtype=BF16, device="cuda"), k=torch.empty((T, G * D), dtype=BF16, device="cuda"),
                out=torch.empty((T, H * D), dtype=BF16, device="cuda"), dec=torch.empty((T, H * D), dtype=BF16, device="cuda"),
                dx=torch.empty_like(x), lse=torch.empty((H, T), device="cuda"), dlse=torch.empty((H, T), device="cuda"),
                kc=kc, vc=vc)
    ws = {op: torch.empty(max(ub.ub_attn_required_bytes(op, cfg, T, len(lens)), 16), dtype=torch.uint8, device="cuda")
          for op in (ub.UB_ATTN_PROMPT_BWD, ub.UB_ATTN_DECODE)}
    cols = (0, H * D, (H + G) * D)
    hq, hk, hv = (ub.heads(x, c) for c in cols)
    dh = [ub.heads(outs["dx"], c) for c in cols]
    q, k, out, dec, dd = (ub.heads(outs["q"]), ub.heads(outs["k"]), ub.heads(outs["out"]), ub.heads(outs["dec"]), ub.heads(d))
    cache = ub.make_kv_cache(kc, vc)

    def run(stream):
        h, n = s["h"], len(lens)
        ub.ub_kv_append(h, hq, hk, hv, q, k, inv, cu, None, n, cache, table, cfg, stream)
        ub.ub_attn_prompt(h, q, k, hv, out, outs["lse"], cu, n, cfg, None, stream)
        ub.ub_attn_prompt_bwd(h, dd, q, k, hv, out, outs["lse"], *dh, cu, n, cfg, ws[ub.UB_ATTN_PROMPT_BWD], stream)
        ub.ub_attn_decode(h, q, cache, table, kv_lens, n, dec, outs["dlse"], cfg, ws[ub.UB_ATTN_DECODE], stream)

    s.update(run=run, outs=outs, keep=(cu, kv_lens, table, inv, ws))
    return s


def bits(outs):
    return {k: t.view(torch.uint8).clone() for k, t in outs.items()}


def same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_another_stream():
    """The same bits from another stream than the tensors' own, ordered by events only."""
    s = calls(1)
    s["run"](torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = bits(s["outs"])
    side = torch.cuda.Stream()
    for t in s["outs"].values():
        t.zero_()
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
    s["run"](torch.cuda.current_stream())  # a kernel's first launch sets its attributes
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s["run"](torch.cuda.current_stream())
    for i in range(4):
        g = torch.Generator(device="cuda").manual_seed(50 + i)
        s["x"].copy_(torch.randn(s["x"].shape, generator=g, device="cuda"))
        s["d"].copy_(torch.randn(s["d"].shape, generator=g, device="cuda"))
        for t in s["outs"].values():
            t.zero_()
        s["run"](torch.cuda.current_stream())
        torch.cuda.synchronize()
        want = bits(s["outs"])
        for t in s["outs"].values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(want, bits(s["outs"]))
        assert bool(torch.isfinite(s["outs"]["dx"]).all()) and math.isfinite(float(s["outs"]["dec"].float().sum()))
    s["ub"].ub_destroy(s["h"])
