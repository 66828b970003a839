"""Host-side tests of the windowed calls, drafted trees and page operations (no GPU): refusals of the
C ABI, workspace sizes, and what the binding refuses before any address reaches a kernel."""

import ctypes
import math
import os

import pytest
import torch

from tests import test_host_cpp as hc
from tests.test_attn_binding import bf16, device, i32
from tests.test_attn_host import BAD_CACHES, BAD_CFGS, BAD_HEADS, FAKE, T, cfg, heads, kv, status

ub = pytest.importorskip("chunked_tp_overlap_amd.ub", reason="libub.so not built")
BAD = "UB_ERR_INVALID_ARG"


@pytest.fixture
def h():
    x = ub.ub_init(T, 64, 1, ub.UB_DTYPE_BF16, FAKE, T * 64 * 2)
    yield x
    ub.ub_destroy(x)


def win(w=8, s=2):
    return ub.make_attn_window(w, s)


def prompt(h, q=heads(), k=heads(), v=heads(), out=heads(), cu=FAKE, n=2, w=win(), c=None):
    return status("ub_attn_prompt_window", h, q, k, v, out, None, cu, n, w, c or cfg(), None, 0, None)


def bwd(h, hs=None, lse=FAKE, cu=FAKE, n=1, w=win(), c=None, ws=FAKE, wsb=1 << 40):
    hs = hs or [heads()] * 8
    return status("ub_attn_prompt_window_bwd", h, *hs[:5], lse, *hs[5:], cu, n, w, c or cfg(), ws, wsb, None)


def decode(h, q=heads(), cache=None, table=FAKE, ld=8, per=8, lens=FAKE, n=2, w=win(), out=heads(), ws=FAKE, wsb=1 << 30, c=None):
    return status("ub_attn_decode_window", h, q, cache or kv(), table, ld, per, lens, n, w, out, None, c or cfg(), ws, wsb, None)


def tree(h, q=heads(), cache=None, table=FAKE, ld=8, per=8, lens=FAKE, parents=FAKE, cu=FAKE, n=2, out=heads(), ws=FAKE,
         wsb=1 << 40, c=None):
    return status("ub_attn_tree", h, q, cache or kv(), table, ld, per, lens, parents, cu, n, out, None, c or cfg(), ws, wsb, None)


def append_at(h, q=heads(), k=heads(), v=heads(), qo=heads(), ko=None, inv=FAKE, off=FAKE, cu=FAKE, n=2, cache=None, table=FAKE,
              ld=8, per=8, c=None):
    return status("ub_kv_append_at", h, q, k, v, qo, ko, inv, off, cu, None, n, cache, table, ld, per, c or cfg(), None)


def compact(h, cache=None, table=FAKE, ld=8, per=8, lens=FAKE, kept=FAKE, kld=4, most=4, klens=FAKE, n=2, out=FAKE + 64, c=None):
    return status("ub_kv_compact", h, cache or kv(), table, ld, per, lens, kept, kld, most, klens, n, out, c or cfg(), None)


def fork(h, refs=FAKE, pages=8, table=FAKE, ld=8, per=8, lens=FAKE, n=2, parents=FAKE, tout=FAKE + 4096, old=8, oper=8,
         lout=FAKE + 64, nout=3, page=16):
    return status("ub_kv_fork", h, refs, pages, table, ld, per, lens, n, parents, tout, old, oper, lout, nout, page, None)


def resize(h, refs=FAKE, pages=8, table=FAKE, ld=8, per=8, lens=FAKE, new=FAKE + 64, n=2, out=FAKE, copies=FAKE, page=16, w=None,
           ws=FAKE, wsb=1 << 20):
    return status("ub_kv_resize", h, refs, pages, table, ld, per, lens, new, n, out, copies, page, w, ws, wsb, None)


def copy(h, cache=None, copies=FAKE, n=2, c=None):
    return status("ub_kv_copy_pages", h, cache or kv(), copies, n, c or cfg(), None)


@pytest.mark.parametrize("kw", BAD_CFGS)
def test_bad_cfg(h, kw):
    for call in (prompt, bwd, decode, tree, append_at, compact, copy):
        assert call(h, c=cfg(**kw)) == BAD and ub.ub_last_error(h)


@pytest.mark.parametrize("w", [None, win(0), win(-1), win(5, -1), win(5, ub.UB_ATTN_MAX_SINKS + 1)])
def test_bad_windows(h, w):
    assert prompt(h, w=w) == BAD and bwd(h, w=w) == BAD and decode(h, w=w) == BAD
    if w is not None:
        assert resize(h, w=w) == BAD


@pytest.mark.parametrize("bad,want", BAD_HEADS)
def test_bad_matrices(h, bad, want):
    for arg in ("q", "k", "v", "out"):
        assert prompt(h, **{arg: bad}) == want and ub.ub_last_error(h).startswith(arg)
    for i, name in enumerate(("dout", "q", "k", "v", "out", "dq", "dk", "dv")):
        hs = [heads()] * 8
        hs[i] = bad
        assert bwd(h, hs) == want and ub.ub_last_error(h).startswith(name)
    for arg in ("q", "out"):
        assert decode(h, **{arg: bad}) == want and tree(h, **{arg: bad}) == want


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(h, kw):
    for call in (decode, tree, append_at, compact, copy):
        assert call(h, cache=kv(**kw)) == BAD


@pytest.mark.parametrize("dtype", (ub.UB_DTYPE_FP16, ub.UB_DTYPE_FP8_E5M2, 77))
def test_cache_dtypes(h, dtype):
    for call in (decode, tree, append_at, compact, copy):
        assert call(h, cache=kv(dtype=dtype)) == "UB_ERR_DTYPE"


def test_window_and_tree_arguments(h):
    assert prompt(h, cu=None) == BAD and prompt(h, n=-1) == BAD and prompt(None) == "UB_ERR_NOT_INITIALIZED"
    assert bwd(h, lse=None) == BAD and bwd(h, ws=None) == BAD and bwd(h, ws=FAKE + 8) == BAD
    c = cfg()
    plain, more = (ub.ub_attn_required_bytes(op, c, T, 1) for op in (ub.UB_ATTN_PROMPT_BWD, ub.UB_ATTN_PROMPT_WINDOW_BWD))
    assert more >= plain and bwd(h, wsb=plain // 2, w=win(8, 0)) == "UB_ERR_BUFFER_TOO_SMALL"
    assert bwd(None) == decode(None) == tree(None) == append_at(None) == "UB_ERR_NOT_INITIALIZED"
    assert decode(h, n=T + 1) == BAD and decode(h, lens=None) == BAD and decode(h, table=None) == BAD and decode(h, ws=None) == BAD
    for kw in (dict(lens=None), dict(parents=None), dict(cu=None), dict(n=-1), dict(table=None), dict(per=0), dict(ld=7),
               dict(ws=None), dict(ws=FAKE + 8)):
        assert tree(h, **kw) == BAD, kw
    need = ub.ub_attn_required_bytes(ub.UB_ATTN_TREE, cfg(), T, 2)
    assert tree(h, wsb=need - 1) == "UB_ERR_BUFFER_TOO_SMALL"
    for kw in (dict(off=None), dict(q=None), dict(qo=None), dict(cu=None), dict(n=-1), dict(inv=None), dict(cache=kv(), table=None)):
        assert append_at(h, **kw) == BAD, kw


def test_page_arguments(h):
    assert compact(None) == fork(None) == resize(None) == copy(None) == "UB_ERR_NOT_INITIALIZED"
    for kw in (dict(lens=None), dict(kept=None), dict(klens=None), dict(out=None), dict(out=FAKE), dict(n=-1), dict(most=-1),
               dict(kld=3), dict(table=None), dict(per=0)):
        assert compact(h, **kw) == BAD, kw
    pool = (dict(refs=None), dict(refs=FAKE + 4), dict(pages=0), dict(pages=1 << 31), dict(page=0), dict(n=-1), dict(per=0),
            dict(ld=7), dict(lens=None), dict(table=None))
    for kw in (*pool, dict(parents=None), dict(lout=None), dict(tout=None), dict(tout=FAKE), dict(lout=FAKE), dict(oper=7), dict(nout=-1),
               dict(old=7)):
        assert fork(h, **kw) == BAD, kw
    for kw in (*pool, dict(new=None), dict(out=None), dict(out=FAKE + 64), dict(copies=None), dict(ws=None), dict(ws=FAKE + 4)):
        assert resize(h, **kw) == BAD, kw
    assert resize(h, wsb=ub.ub_kv_resize_bytes(2) - 1) == "UB_ERR_BUFFER_TOO_SMALL"
    assert copy(h, copies=None) == BAD and copy(h, n=-1) == BAD
    with pytest.raises(ub.UBError):
        ub.ub_kv_resize_bytes(-1)
    assert ub.raw_call("ub_kv_resize_bytes", 3, None) != 0
    sizes = [ub.ub_kv_resize_bytes(n) for n in (0, 1, 2, 100, 100000)]
    assert sizes == sorted(sizes)


def test_required_bytes():
    for op in (ub.UB_ATTN_PROMPT_WINDOW, ub.UB_ATTN_PROMPT_WINDOW_BWD, ub.UB_ATTN_DECODE_WINDOW, ub.UB_ATTN_TREE):
        for c in (cfg(8, 1, 128), cfg(4, 4, 128), cfg(6, 3, 80), cfg(16, 1, 64), cfg(600, 600, 16)):
            rows = [ub.ub_attn_required_bytes(op, c, r, 4) for r in (0, 1, 127, 128, 129, 1000, 8184, 16384, 32520, 200000)]
            assert rows == sorted(rows)
            seqs = [ub.ub_attn_required_bytes(op, c, 1000, n) for n in (0, 1, 5, 64, 1000)]
            assert seqs == sorted(seqs)


def test_windows_past_32_bits():
    assert ub.make_attn_window(1 << 40).window == (1 << 31) - 1 and ub.make_attn_window(7).sinks == 0


def test_host_tensors_and_sizes(h):
    """What the binding refuses, each by the argument's name."""
    c, w = ub.make_attn_cfg(4, 2, 64), win()
    q, k = ub.heads(bf16(T, 256)), ub.heads(bf16(T, 128))
    cache = ub.make_kv_cache(bf16(4, 2, 16, 64), bf16(4, 2, 16, 64))
    ws = device(torch.zeros(1 << 20, dtype=torch.uint8))
    hi = lambda *s: torch.zeros(s, dtype=torch.int32)
    tr = lambda lens=i32(1), par=i32(T), cu=i32(2), pages=i32(1, 4): ub.ub_attn_tree(h, q, cache, pages, lens, par, cu, 1, q, None, c, ws)
    co = lambda lens=i32(2), kept=i32(2, 3), kl=i32(2), out=i32(2), pages=i32(2, 4): ub.ub_kv_compact(
        h, cache, pages, lens, kept, kl, 2, out, c)
    fo = lambda refs=i32(8), pages=i32(2, 4), lens=i32(2), par=i32(3), out=i32(3, 4), lo=i32(3): ub.ub_kv_fork(
        h, refs, pages, lens, 2, par, out, lo, 3, 16)
    re = lambda refs=i32(8), pages=i32(2, 4), lens=i32(2), new=i32(2), lo=i32(2), cp=i32(2, 3): ub.ub_kv_resize(
        h, refs, pages, lens, new, 2, lo, cp, 16, None, ws)
    for match, call in (
            ("^kv_lens: .*device", lambda: tr(lens=hi(1))), ("^parents: .*device", lambda: tr(par=hi(T))),
            ("^parents: at least", lambda: tr(par=i32(T - 1))), ("^cu_seqlens: at least", lambda: tr(cu=i32(1))),
            ("^pages: .*device", lambda: tr(pages=hi(1, 4))),
            ("^offsets: at least", lambda: ub.ub_kv_append_at(h, q, k, k, q, None, device(torch.zeros(32)), i32(T - 1), i32(2), None, 1,
                                                              cache, i32(1, 4), c)),
            ("^lens: at least", lambda: co(lens=i32(1))), ("^kept: an int32", lambda: co(kept=i32(1, 3))),
            ("^kept: .*device", lambda: co(kept=hi(2, 3))), ("^kept_lens: .*device", lambda: co(kl=hi(2))),
            ("^lens_out: at least", lambda: co(out=i32(2).long())),
            ("^refs: .*device", lambda: fo(refs=hi(8))), ("^pages_out: an int32", lambda: fo(out=i32(2, 4))),
            ("^parents: at least", lambda: fo(par=i32(2))), ("^lens_out: at least", lambda: fo(lo=i32(2))),
            ("^new_lens: at least", lambda: re(new=i32(1))), ("^copies: at least", lambda: re(cp=i32(1, 3))),
            ("^copies: at least", lambda: ub.ub_kv_copy_pages(h, cache, i32(1, 3), 2, c)),
            ("^q: columns", lambda: ub.ub_attn_prompt_window(h, ub.heads(bf16(T, 256), 64), k, k, q, None, i32(2), 1, w, c)),
            ("^kv_lens: .*device", lambda: ub.ub_attn_decode_window(h, q, cache, i32(1, 4), hi(1), 1, w, q, None, c, ws))):
        with pytest.raises(ValueError, match=match):
            call()
    assert math.isfinite(c.softmax_scale) and ctypes.sizeof(ub.ub_attn_window_t) == 8


@pytest.mark.skipif(hc._cxx() is None, reason="clang++ not available")
def test_window_arithmetic(tmp_path):
    """The tiles and slots of windowed calls, and the page of a token by a product."""
    out = hc._build_and_run(tmp_path, "attn_window_check", [os.path.join(hc.CPP, "attn_window_check.cpp")])
    assert int(out.split()[1]) > 500000


def accepted(call, **kw):
    """The call passes the checks.  Its addresses are no memory: it is made only where there is no GPU to
    launch on."""
    return torch.cuda.is_available() or call(**kw) != BAD


def test_compact_outputs_clear_of_inputs(h):
    """A sequence's workgroups read its lists while one of them writes lens_out: it lies on none of what
    they read, in whole or in part.  (The next int32 after each, and the gap between rows, are free.)"""
    at = lambda **kw: compact(h, **{**dict(lens=FAKE, klens=FAKE + 1024, kept=FAKE + 2048, table=FAKE + 4096, n=2), **kw})
    for base, words in ((0, 2), (1024, 2), (2048, 8), (4096, 16)):
        for w in (-1, 0, words // 2, words - 1):
            assert at(out=FAKE + base + 4 * w) == BAD and "lens_out" in ub.ub_last_error(h), (base, w)
        for w in (-2, words):
            assert accepted(at, out=FAKE + base + 4 * w), (base, w, ub.ub_last_error(h))
    # rows of 3 entries, 8 apart: 5 are free between them, and all after the second
    for w in (2, 7, 8, 10):
        assert at(kld=8, most=3, out=FAKE + 2048 + 4 * w) == BAD, w
    for w in (3, 6, 11):
        assert accepted(at, kld=8, most=3, out=FAKE + 2048 + 4 * w), w
    assert at(kld=8, most=3, out=FAKE + 2048 + 2) == BAD and accepted(at, kld=1 << 61, most=3, out=FAKE + 64)
    assert accepted(at, most=0, kept=None, out=FAKE + 64)


def test_page_outputs_clear_of_inputs(h):
    """What ub_kv_fork and ub_kv_resize write lies on nothing that other workgroups or waves of the call still
    read; lens_out of a resize may be lens itself.  Two tables may be the columns of one array."""
    f = lambda **kw: fork(h, **{**dict(refs=FAKE + 65536, table=FAKE, lens=FAKE + 1024, parents=FAKE + 2048, tout=FAKE + 4096,
                                       lout=FAKE + 8192), **kw})
    r = lambda **kw: resize(h, **{**dict(refs=FAKE + 65536, table=FAKE, lens=FAKE + 1024, new=FAKE + 2048, out=FAKE + 4096,
                                         copies=FAKE + 8192), **kw})
    assert accepted(f) and accepted(r) and accepted(r, out=FAKE + 1024)
    # n 2, 3 rows of the new table, 8 entries a row
    for base, words in ((0, 16), (1024, 2), (2048, 3), (4096, 24)):
        for w in (-2, 0, words - 1):
            assert f(lout=FAKE + base + 4 * w) == BAD and "lens_out" in ub.ub_last_error(h), (base, w)
        for w in (-3, words):
            assert accepted(f, lout=FAKE + base + 4 * w), (base, w)
    for base, words in ((0, 16), (1024, 2), (2048, 3)):
        for w in (-23, 0, words - 1):
            assert f(tout=FAKE + base + 4 * w) == BAD and "table_out" in ub.ub_last_error(h), (base, w)
        for w in (-24, words):
            assert accepted(f, tout=FAKE + base + 4 * w), (base, w)
    assert accepted(f, ld=16, tout=FAKE + 32, old=16) and f(ld=16, tout=FAKE + 28, old=16) == BAD
    assert accepted(f, ld=16, tout=FAKE - 32, old=16) and f(ld=16, tout=FAKE - 28, old=16) == BAD
    assert accepted(f, ld=64, tout=FAKE + 32, old=16, nout=3) and f(ld=24, tout=FAKE + 32, old=16, nout=3) == BAD
    for base, words in ((0, 16), (2048, 2)):
        for w in (-1, 0, words - 1):
            assert r(out=FAKE + base + 4 * w) == BAD and "lens_out" in ub.ub_last_error(h), (base, w)
    assert r(out=FAKE + 1020) == BAD and r(out=FAKE + 1028) == BAD and accepted(r, out=FAKE + 1032)
    for base, words in ((0, 16), (1024, 2), (2048, 2), (4096, 2)):
        for w in (-5, 0, words - 1):
            assert r(copies=FAKE + base + 4 * w) == BAD and "copies" in ub.ub_last_error(h), (base, w)
        for w in (-6, words):
            assert accepted(r, copies=FAKE + base + 4 * w), (base, w)


@pytest.mark.skipif(hc._cxx() is None, reason="clang++ not available")
def test_path_bits(tmp_path):
    """Which of a group's keys a drafted token sees: a key of another group's is none that it has no score of."""
    out = hc._build_and_run(tmp_path, "attn_path_check", [os.path.join(hc.CPP, "attn_path_check.cpp")])
    assert int(out.split()[1]) > 5000000


@pytest.mark.parametrize("w,s", [(5 - (1 << 32), 0), (-(1 << 40) + 1, 0), (8, (1 << 32) + 3), (8, (1 << 31) + 1), (8, 4 - (1 << 32)), (0, 1 << 32)])
def test_windows_that_are_none(h, w, s):
    """What does not fit an int32 is not taken for its low bits, but refused like any window that is none."""
    x = win(w, s)
    assert prompt(h, w=x) == BAD and bwd(h, w=x) == BAD and decode(h, w=x) == BAD and resize(h, w=x) == BAD
