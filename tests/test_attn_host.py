"""Host-side tests of the attention calls (no GPU): refusals, workspace sizes, the binding's
own checks, and the paging arithmetic under sanitizers.  Every argument check runs before the
first HIP call, so placeholder device addresses are never dereferenced."""

import ctypes
import math
import os

import pytest
import torch

from tests import test_host_cpp as hc

ub = pytest.importorskip("chunked_tp_overlap_amd.ub", reason="libub.so not built")
FAKE = 0x7F0000000000
T = 64


@pytest.fixture
def h():
    x = ub.ub_init(T, 64, 1, ub.UB_DTYPE_BF16, FAKE, T * 64 * 2)
    yield x
    ub.ub_destroy(x)


def heads(ptr=FAKE, rs=1024, hs=0, rows=T):
    d = ub.ub_heads_t()
    d.ptr, d.row_stride, d.head_stride, d.rows = ptr, rs, hs, rows
    return d


def kv(k=FAKE, v=FAKE, ps=4096, hs=64, ts=256, n_pages=8, page=16, dtype=0, ks=1.0, vs=1.0):
    c = ub.ub_kv_cache_t()
    c.k, c.v, c.page_stride, c.head_stride, c.token_stride = k, v, ps, hs, ts
    c.n_pages, c.page_size, c.dtype, c.k_scale, c.v_scale = n_pages, page, dtype, ks, vs
    return c


def cfg(H=4, G=2, D=64, **kw):
    return ub.make_attn_cfg(H, G, D, **kw)


def status(name, *args):
    conv = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args]
    return ub.STATUS[ub.raw_call(name, *conv)]


def prompt(h, q=None, k=None, v=None, out=None, cu=FAKE, n=2, c=None):
    f = lambda x: heads() if x is None else x
    return status("ub_attn_prompt", h, f(q), f(k), f(v), f(out), None, cu, n, c or cfg(), None, 0, None)


BAD_CFGS = [dict(H=0), dict(G=0), dict(H=3, G=2), dict(D=0), dict(D=12), dict(D=-8), dict(rotary_dim=24),
            dict(rotary_dim=80), dict(rotary_dim=-16), dict(softmax_scale=0.0), dict(softmax_scale=-1.0),
            dict(softmax_scale=math.nan), dict(softmax_scale=math.inf), dict(H=1 << 20, G=1)]


@pytest.mark.parametrize("kw", BAD_CFGS)
def test_bad_cfg(h, kw):
    assert prompt(h, c=cfg(**kw)) == "UB_ERR_INVALID_ARG" and ub.ub_last_error(h)
    with pytest.raises(ub.UBError) as e:
        ub.ub_attn_required_bytes(ub.UB_ATTN_DECODE, cfg(**kw), 8, 1)
    assert e.value.name == "UB_ERR_INVALID_ARG"


def test_bad_interleave_and_null_cfg(h):
    c = cfg()
    c.rope_interleaved = 2
    assert prompt(h, c=c) == "UB_ERR_INVALID_ARG"
    assert status("ub_attn_prompt", h, heads(), heads(), heads(), heads(), None, FAKE, 1, None, None, 0, None) \
        == "UB_ERR_INVALID_ARG"


def test_head_dim_above_the_limit(h):
    assert prompt(h, c=cfg(D=136)) == "UB_ERR_UNSUPPORTED"
    assert prompt(h, c=cfg(D=ub.UB_ATTN_MAX_HEAD_DIM + 8)) == "UB_ERR_UNSUPPORTED"


BAD_HEADS = [(heads(ptr=None), "UB_ERR_INVALID_ARG"), (heads(ptr=FAKE + 2), "UB_ERR_INVALID_ARG"),
             (heads(rs=1020), "UB_ERR_INVALID_ARG"), (heads(rs=56), "UB_ERR_INVALID_ARG"),
             (heads(rs=1 << 22), "UB_ERR_INVALID_ARG"), (heads(rs=-64), "UB_ERR_INVALID_ARG"),
             (heads(hs=60), "UB_ERR_INVALID_ARG"), (heads(hs=56), "UB_ERR_INVALID_ARG"),
             (heads(hs=-64), "UB_ERR_INVALID_ARG"), (heads(rows=T - 1), "UB_ERR_BUFFER_TOO_SMALL")]


@pytest.mark.parametrize("bad,want", BAD_HEADS)
def test_bad_matrices(h, bad, want):
    for arg in ("q", "k", "v", "out"):
        assert prompt(h, **{arg: bad}) == want
        assert ub.ub_last_error(h).startswith(arg)
    names = ["dout", "q", "k", "v", "out", "dq", "dk", "dv"]
    for i, name in enumerate(names):
        hs = [heads() for _ in names]
        hs[i] = bad
        assert status("ub_attn_prompt_bwd", h, *hs[:5], FAKE, *hs[5:], FAKE, 1, cfg(), FAKE, 1 << 30, None) == want
        assert ub.ub_last_error(h).startswith(name)


def test_prompt_sequences(h):
    assert prompt(h, n=-1) == "UB_ERR_INVALID_ARG"
    assert prompt(h, cu=None) == "UB_ERR_INVALID_ARG"
    assert prompt(None) == "UB_ERR_NOT_INITIALIZED"


def test_gradient_lse_and_workspace(h):
    c = cfg()
    need = ub.ub_attn_required_bytes(ub.UB_ATTN_PROMPT_BWD, c, T, 1)
    call = lambda lse, ws, n: status("ub_attn_prompt_bwd", h, *[heads()] * 5, lse, *[heads()] * 3, FAKE, 1, c, ws, n, None)
    assert call(None, FAKE, need) == "UB_ERR_INVALID_ARG"
    assert call(FAKE, None, need) == "UB_ERR_INVALID_ARG"
    assert call(FAKE, FAKE + 8, need) == "UB_ERR_INVALID_ARG"
    assert call(FAKE, FAKE, need // 2) == "UB_ERR_BUFFER_TOO_SMALL"


def append(h, q=heads(), k=heads(), v=heads(), qo=heads(), ko=None, inv=FAKE, cu=FAKE, n=2, cache=None,
           table=FAKE, ld=8, per=8, c=None):
    return status("ub_kv_append", h, q, k, v, qo, ko, inv, cu, None, n, cache, table, ld, per, c or cfg(), None)


def decode(h, q=heads(), cache=None, table=FAKE, ld=8, per=8, lens=FAKE, n=2, out=heads(), ws=FAKE, wsb=1 << 30,
           c=None):
    return status("ub_attn_decode", h, q, cache or kv(), table, ld, per, lens, n, out, None, c or cfg(), ws, wsb, None)


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(ps=4100), dict(hs=60),
              dict(ts=12), dict(ps=-8), dict(n_pages=0), dict(n_pages=1 << 31), dict(page=0), dict(page=-1),
              dict(dtype=ub.UB_DTYPE_FP8_E4M3, hs=72), dict(dtype=ub.UB_DTYPE_FP8_E4M3, ks=0.0),
              dict(dtype=ub.UB_DTYPE_FP8_E4M3, vs=-1.0), dict(dtype=ub.UB_DTYPE_FP8_E4M3, ks=math.nan),
              dict(dtype=ub.UB_DTYPE_FP8_E4M3, vs=math.inf)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(h, kw):
    assert append(h, cache=kv(**kw)) == "UB_ERR_INVALID_ARG"
    assert decode(h, cache=kv(**kw)) == "UB_ERR_INVALID_ARG"


@pytest.mark.parametrize("dtype", (ub.UB_DTYPE_FP16, ub.UB_DTYPE_FP8_E5M2, 77, -1))
def test_cache_dtypes(h, dtype):
    assert append(h, cache=kv(dtype=dtype)) == "UB_ERR_DTYPE"
    assert decode(h, cache=kv(dtype=dtype)) == "UB_ERR_DTYPE"


def test_e4m3_head_dim(h):
    c = cfg(D=40, rotary_dim=32)
    f8 = kv(dtype=ub.UB_DTYPE_FP8_E4M3)
    assert append(h, cache=f8, c=c) == "UB_ERR_INVALID_ARG"
    assert decode(h, cache=f8, c=c) == "UB_ERR_INVALID_ARG"


def test_append_arguments(h):
    bad = "UB_ERR_INVALID_ARG"
    assert append(h, q=None) == bad and append(h, qo=None) == bad
    assert append(h, k=None, cache=kv()) == bad and append(h, k=None, ko=heads()) == bad
    assert append(h, v=None, cache=kv()) == bad
    assert append(h, inv=None) == bad and append(h, cu=None) == bad and append(h, n=-1) == bad
    assert append(h, cache=kv(), table=None) == bad
    assert append(h, cache=kv(), per=0) == bad and append(h, cache=kv(), ld=7) == bad
    assert append(None) == "UB_ERR_NOT_INITIALIZED"


def test_decode_arguments(h):
    bad = "UB_ERR_INVALID_ARG"
    assert decode(h, n=T + 1) == bad and decode(h, n=-1) == bad and decode(h, lens=None) == bad
    assert decode(h, table=None) == bad and decode(h, per=0) == bad and decode(h, ld=3) == bad
    assert decode(h, ws=None) == bad and decode(h, ws=FAKE + 8) == bad
    need = ub.ub_attn_required_bytes(ub.UB_ATTN_DECODE, cfg(), T, 2)
    assert decode(h, wsb=need - 1) == "UB_ERR_BUFFER_TOO_SMALL"
    assert decode(None) == "UB_ERR_NOT_INITIALIZED"


def test_required_bytes():
    c = cfg(8, 1, 128)
    for bad in ((7, c, 8, 1), (0, c, -1, 1), (0, c, 8, -1)):
        with pytest.raises(ub.UBError) as e:
            ub.ub_attn_required_bytes(*bad)
        assert e.value.name == "UB_ERR_INVALID_ARG"
    for op in (ub.UB_ATTN_PROMPT, ub.UB_ATTN_PROMPT_BWD, ub.UB_ATTN_DECODE):
        for c in (cfg(8, 1, 128), cfg(4, 4, 128), cfg(6, 3, 80), cfg(16, 1, 64)):
            rows = [ub.ub_attn_required_bytes(op, c, r, 4) for r in (0, 1, 127, 128, 129, 1000, 8184, 16384, 32520, 200000)]
            assert rows == sorted(rows)
            seqs = [ub.ub_attn_required_bytes(op, c, 1000, n) for n in (0, 1, 5, 64, 1000)]
            assert seqs == sorted(seqs)


def test_binding_checks(h):
    x = torch.zeros((T, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ub.heads(x.float())
    with pytest.raises(ValueError):
        ub.heads(x[0])
    with pytest.raises(ValueError):
        ub.heads(x.t())
    c = cfg(4, 2, 64)
    good = ub.heads(x)
    with pytest.raises(ValueError):  # 4 heads of 64 from column 64 of 256
        ub.ub_attn_prompt(h, ub.heads(x, 64), good, good, good, None, torch.zeros(2, dtype=torch.int32), 1, c)
    with pytest.raises(ValueError):  # lse of another shape
        ub.ub_attn_prompt(h, good, good, good, good, torch.zeros(4, T - 1), torch.zeros(2, dtype=torch.int32), 1, c)
    with pytest.raises(ValueError):  # cu_seqlens of another type
        ub.ub_attn_prompt(h, good, good, good, good, None, torch.zeros(2, dtype=torch.int64), 1, c)
    cache = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ub.make_kv_cache(cache, cache[:2])
    with pytest.raises(ValueError):  # one head too few
        ub.ub_kv_append(h, None, good, good, None, None, None, torch.zeros(2, dtype=torch.int32), None, 1,
                        ub.make_kv_cache(cache[:, :1], cache[:, :1]), torch.zeros((1, 4), dtype=torch.int32),
                        cfg(4, 2, 64, rotary_dim=0))
    with pytest.raises(ValueError):  # a table of too few rows
        ub.ub_kv_append(h, None, good, good, None, None, None, torch.zeros(3, dtype=torch.int32), None, 2,
                        ub.make_kv_cache(cache, cache), torch.zeros((1, 4), dtype=torch.int32),
                        cfg(4, 2, 64, rotary_dim=0))


@pytest.mark.skipif(hc._cxx() is None, reason="clang++ not available")
def test_paging_arithmetic(tmp_path):
    """Bad lengths, positions and page ids stay inside the table and the cache."""
    out = hc._build_and_run(tmp_path, "kv_pages_check", [os.path.join(hc.CPP, "kv_pages_check.cpp")])
    assert int(out.split()[1]) > 100000
