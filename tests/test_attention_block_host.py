"""Host-side test of the attention block's streams (no GPU): every call that issues work gets
torch's current stream, on which the block's own tensor operations run."""

import contextlib
import inspect

import pytest
import torch

ub = pytest.importorskip("chunked_tp_overlap_amd.ub", reason="libub.so not built")


class Stream:
    cuda_stream = 0x1234


def on_host(f):
    def g(*a, **kw):
        kw.pop("device", None)
        return f(*a, **kw)
    return g


@contextlib.contextmanager
def recorded(monkeypatch):
    """The block on host tensors, with the calls that issue work recorded in place of made:
    (name, stream), and what ub_copy_in was given."""
    from chunked_tp_overlap_amd import attention_block as m

    calls, copied = [], []
    with monkeypatch.context() as p:
        for name in ("zeros", "empty", "arange", "full"):
            p.setattr(torch, name, on_host(getattr(torch, name)))
        p.setattr(torch.Tensor, "cuda", lambda self, *a, **kw: self)
        p.setattr(torch.cuda, "current_stream", lambda *a: Stream)
        for name in ub.EXPORTS:
            f = getattr(ub, name, None)
            if f is None or "stream" not in inspect.signature(f).parameters:
                continue

            def call(*a, f=f, name=name, **kw):
                given = inspect.signature(f).bind(*a, **kw).arguments
                calls.append((name, given.get("stream")))
                if name == "ub_copy_in":
                    copied.append(given["src"])
            p.setattr(ub, name, call)
        yield m, calls, copied


def make_block(m, H=4, G=2, D=64, hidden=128):
    w = torch.zeros(hidden, (H + 2 * G) * D, dtype=torch.bfloat16), torch.zeros(H * D, hidden, dtype=torch.bfloat16)
    return m.AttentionBlock(*w, H, G, D, capacity=16, max_seqs=2, max_len=32, tp=2)


def test_every_call_runs_on_the_current_stream(monkeypatch):
    H, D, hidden, lens = 4, 64, 128, [5, 1]
    with recorded(monkeypatch) as (m, calls, _):
        b = make_block(m)
        x = torch.zeros(6, hidden, dtype=torch.bfloat16)
        made = {}
        for name, f in (("prefill", lambda: b.prefill(x, lens)), ("decode", lambda: b.decode(x[:2])),
                        ("train", lambda: b.train(x, lens, torch.zeros(6, H * D, dtype=torch.bfloat16)))):
            calls.clear()
            f()
            made[name] = list(calls)
        b.close()
    ends = ["ub_copy_in", "ub_gemm_ag_chunked", "ub_kv_append"], ["ub_gemm_rs_chunked"]
    for name, middle in (("prefill", ["ub_attn_prompt"]), ("decode", ["ub_attn_decode"])):
        assert [c for c, _ in made[name]] == ends[0] + middle + ends[1]
    assert [c for c, _ in made["train"]] == ends[0] + ["ub_attn_prompt"] + ends[1] + ["ub_attn_prompt_bwd", "ub_kv_append"]
    for name, cs in made.items():
        assert [c for c, s in cs if s is not Stream] == [], name


def test_rows_of_any_layout(monkeypatch):
    """ub_copy_in takes an address and a number of rows: strided rows are laid out first, and what
    is no bf16 matrix of the hidden size is refused."""
    with recorded(monkeypatch) as (m, _, copied):
        b = make_block(m)
        wide = torch.randn(6, 256).bfloat16()
        for x in (wide[:, :128], wide[:, 128:], wide[::2, :128], wide.repeat(22, 1)[:128, :6].t()):
            b.prefill(x, [x.shape[0] - 1, 1])
            assert copied[-1].is_contiguous() and torch.equal(copied[-1], x)
        for bad in (wide, wide[:, :127], wide[:, :128].float(), wide[0, :128], wide[:, :128].half()):
            n = len(copied)
            for f in (lambda: b.prefill(bad, [1]), lambda: b.decode(bad), lambda: b.train(bad, [1], bad)):
                with pytest.raises(ValueError, match="hidden"):
                    f()
            assert len(copied) == n
        b.close()


def test_weights(monkeypatch):
    """The weights are kept, not copied, and read row by row: others than contiguous bf16 matrices
    of the block's sizes are refused."""
    with recorded(monkeypatch) as (m, _, _):
        wqkv, wo = torch.randn(128, 512).bfloat16(), torch.randn(256, 128).bfloat16()
        make = lambda a, b: m.AttentionBlock(a, b, 4, 2, 64, capacity=16, max_seqs=2, max_len=32)
        b = make(wqkv, wo)
        assert b.wqkv is wqkv and b.wo is wo
        b.close()
        for bad in ((wqkv.t().contiguous(), wo), (wqkv.t().contiguous().t(), wo), (wqkv.float(), wo), (wqkv[:, :504], wo)):
            with pytest.raises(ValueError, match="wqkv"):
                make(*bad)
        for bad in (wo.t().contiguous(), wo.t().contiguous().t(), wo.half(), wo[:, :120].contiguous(), wo[:255]):
            with pytest.raises(ValueError, match="wo:"):
                make(wqkv, bad)
