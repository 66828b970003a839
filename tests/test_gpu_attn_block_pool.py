"""GPU tests of the attention block where its pool runs out of pages, and of captured decode steps as
sequences fork: what the cache holds, byte by byte, and each row against its definition."""

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
