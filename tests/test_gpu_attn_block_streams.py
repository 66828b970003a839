"""GPU tests of the attention block on a stream of the caller's: its own torch operations and the
library's calls in one order, and a decode step captured into a HIP graph."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
H, G, D, HIDDEN, LENS = 4, 2, 64, 256, [200, 1, 33]


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


def make_block():
    from chunked_tp_overlap_amd.attention_block import AttentionBlock

    wqkv, wo = normal(1, HIDDEN, (H + 2 * G) * D) / 16, normal(2, H * D, HIDDEN) / 16
    return AttentionBlock(wqkv, wo, H, G, D, capacity=512, max_seqs=3, max_len=300, page=16, tp=4)


def inputs():
    return dict(x=normal(3, sum(LENS), HIDDEN), tokens=[normal(10 + s, len(LENS), HIDDEN) for s in range(3)],
                dattn=normal(20, sum(LENS), H * D))


def steps(b, i):
    """Prompts, decode steps and a training step: all outputs, cloned in the order of the work."""
    out = [b.prefill(i["x"], LENS).clone()]
    for t in i["tokens"]:
        out.append(b.decode(t).clone())
    out += [b.lens.clone(), b.k_cache.clone(), b.v_cache.clone()]
    out += [t.clone() for t in b.train(i["x"], LENS, i["dattn"])]
    return out


def same(got, want):
    assert len(got) == len(want)
    for n, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), n


def test_block_on_another_stream():
    """The same bits, with the stream held up before every step, so that work on any other
    stream would come first."""
    b, i = make_block(), inputs()
    want = steps(b, i)
    torch.cuda.synchronize()
    b.close()

    b, side = make_block(), torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        def hold(f):
            def g(*a):
                for _ in range(4):
                    busy @ busy
                return f(*a)
            return g
        b.prefill, b.decode, b.train = hold(b.prefill), hold(b.decode), hold(b.train)
        got = steps(b, i)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    same(got, want)
    b.close()


def test_decode_step_in_a_graph():
    """A decode step captured once and replayed as the sequences grow, against eager steps."""
    b, i = make_block(), inputs()
    b.prefill(i["x"], LENS)
    token = torch.zeros_like(i["tokens"][0])
    start = [t.clone() for t in (b.lens, b.k_cache, b.v_cache)]

    def reset():
        for t, s in zip((b.lens, b.k_cache, b.v_cache), start):
            t.copy_(s)

    want = []
    for s in range(4):
        token.copy_(normal(30 + s, len(LENS), HIDDEN))
        want.append([b.decode(token).clone(), b.lens.clone(), b.k_cache.clone()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.decode(token)
    reset()
    for s in range(4):
        token.copy_(normal(30 + s, len(LENS), HIDDEN))
        graph.replay()
        torch.cuda.synchronize()
        same([y, b.lens, b.k_cache], want[s])
        normal(50, 64, 64) @ normal(51, 64, 64)  # eager work between the replays
        torch.cuda.synchronize()
    b.close()
