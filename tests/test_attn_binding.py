"""Host-side tests of what the attention calls' binding refuses before any address reaches a
kernel (no GPU): tensors that do not hold what a call would read or write."""

import pytest
import torch

ub = pytest.importorskip("chunked_tp_overlap_amd.ub", reason="libub.so not built")
FAKE = 0x7F0000000000
T = 64


@pytest.fixture
def h():
    x = ub.ub_init(T, 64, 1, ub.UB_DTYPE_BF16, FAKE, T * 64 * 2)
    yield x
    ub.ub_destroy(x)


class OnDevice(torch.Tensor):
    """A host tensor that says it is on the device, for the checks that come after that one."""
    is_cuda = True


def device(x):
    return x.as_subclass(OnDevice)


def i32(*shape):
    return device(torch.zeros(shape, dtype=torch.int32))


def bf16(*shape):
    return device(torch.zeros(shape, dtype=torch.bfloat16))


def test_page_table_strides():
    """A table is described by its own row stride; rows that overlap, or one row expanded to
    several sequences, are no layout that the calls take (they would be read `pages` entries
    apart, past the tensor's end)."""
    t = i32(3, 8)
    assert ub._table(t, 3) == (t.data_ptr(), 8, 8)
    wide = t[:, :5]
    assert ub._table(wide, 3) == (t.data_ptr(), 8, 5)
    for bad in (i32(1, 5).expand(3, 5), i32(40).as_strided((3, 8), (4, 1)), i32(2, 8).t()):
        with pytest.raises(ValueError, match="pages"):
            ub._table(bad, 2)
    one = i32(40).as_strided((1, 8), (3, 1))  # the stride of a single row means nothing
    assert ub._table(one, 1) == (one.data_ptr(), 8, 8)
    assert ub._table(i32(1, 5).expand(1, 5), 1)[1:] == (5, 5)
    # rows beyond the sequences are not read
    many = i32(1, 5).expand(3, 5)
    assert ub._table(many, 1)[1:] == (5, 5)


def test_heads_expanded_over_heads():
    """One head expanded to several has head stride 0, which a descriptor reads as head_dim."""
    x = torch.zeros((T, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="head"):
        ub.heads(x.expand(T, 8, 64))
    d = ub.heads(x.expand(T, 1, 64))
    assert (d.ptr, d.row_stride, d.rows) == (x.data_ptr(), 64, T)
    y = torch.zeros((4, T, 64), dtype=torch.bfloat16).transpose(0, 1)
    assert ub.heads(y).head_stride == T * 64


@pytest.mark.parametrize("dtype", (torch.float16, torch.int16, torch.uint16, torch.float32, torch.float8_e4m3fn))
def test_heads_dtype(dtype):
    """Matrices are bf16: other 2-byte values would have their bits read as bf16."""
    with pytest.raises(ValueError, match="bf16"):
        ub.heads(torch.zeros((T, 256), dtype=dtype))
    with pytest.raises(ValueError, match="bf16"):
        ub.heads(torch.zeros((T, 4, 64), dtype=dtype))


def test_heads_column():
    """A column before the matrix is an address before the tensor."""
    x = torch.zeros((T, 256), dtype=torch.bfloat16)
    for col in (-1, -8, -64):
        with pytest.raises(ValueError, match="col"):
            ub.heads(x, col)
    assert ub.heads(x, 64).ptr == x.data_ptr() + 128


def test_workspace_is_contiguous():
    """A workspace has the bytes that its tensor counts only if they lie side by side."""
    for bad in (device(torch.zeros(1, dtype=torch.uint8)).expand(1 << 20),
                device(torch.zeros((64, 64), dtype=torch.uint8))[:, :8]):
        with pytest.raises(ValueError, match="workspace"):
            ub._ws_arg(bad)
    assert ub._ws_arg(None) == (None, 0)
    assert ub._ws_arg(device(torch.zeros(48, dtype=torch.float32)))[1] == 192


def prompt_args(**kw):
    """ub_attn_prompt's arguments after the handle, all on the device."""
    a = dict(q=bf16(T, 256), k=bf16(T, 128), v=bf16(T, 128), out=bf16(T, 256), lse=device(torch.zeros(4, T)), cu=i32(2),
             ws=None)
    a.update(kw)
    return (*[ub.heads(a[x]) for x in ("q", "k", "v", "out")], a["lse"], a["cu"], 1, ub.make_attn_cfg(4, 2, 64), a["ws"])


@pytest.mark.parametrize("name", ("q", "k", "v", "out", "lse", "cu_seqlens", "workspace"))
def test_host_tensors_in_prompt(h, name):
    """Pageable host memory, which a kernel cannot address, is refused by the argument's name."""
    key = {"cu_seqlens": "cu", "workspace": "ws"}.get(name, name)
    host = {"q": torch.zeros(T, 256).bfloat16(), "k": torch.zeros(T, 128).bfloat16(), "v": torch.zeros(T, 128).bfloat16(),
            "out": torch.zeros(T, 256).bfloat16(), "lse": torch.zeros(4, T), "cu": torch.zeros(2, dtype=torch.int32),
            "ws": torch.zeros(64, dtype=torch.uint8)}[key]
    with pytest.raises(ValueError, match=f"^{name}: .*device"):
        ub.ub_attn_prompt(h, *prompt_args(**{key: host}))


def test_host_tensors_in_gradient(h):
    names = ["dout", "q", "k", "v", "out", "dq", "dk", "dv"]
    for bad in names:
        x = [ub.heads(torch.zeros(T, 256).bfloat16() if n == bad else bf16(T, 256)) for n in names]
        with pytest.raises(ValueError, match=f"^{bad}: .*device"):
            ub.ub_attn_prompt_bwd(h, *x[:5], device(torch.zeros(4, T)), *x[5:], i32(2), 1, ub.make_attn_cfg(4, 2, 64),
                                  device(torch.zeros(1 << 20, dtype=torch.uint8)))


def test_host_tensors_in_append_and_decode(h):
    cfg = ub.make_attn_cfg(4, 2, 64)
    host = dict(inv_freq=torch.zeros(32), cu_seqlens=torch.zeros(2, dtype=torch.int32),
                past_lens=torch.zeros(1, dtype=torch.int32), cache=torch.zeros(4, 2, 16, 64).bfloat16(),
                pages=torch.zeros((1, 4), dtype=torch.int32), kv_lens=torch.zeros(1, dtype=torch.int32))
    for bad, x in host.items():
        a = {n: device(t.clone()) for n, t in host.items()}
        a[bad] = x
        q, k = ub.heads(bf16(T, 256)), ub.heads(bf16(T, 128))
        cache = ub.make_kv_cache(a["cache"], a["cache"])
        if bad != "kv_lens":
            with pytest.raises(ValueError, match=f"^{bad}: .*device"):
                ub.ub_kv_append(h, q, k, k, q, None, a["inv_freq"], a["cu_seqlens"], a["past_lens"], 1, cache, a["pages"], cfg)
        if bad in ("cache", "pages", "kv_lens"):
            with pytest.raises(ValueError, match=f"^{bad}: .*device"):
                ub.ub_attn_decode(h, q, cache, a["pages"], a["kv_lens"], 1, q, None, cfg,
                                  device(torch.zeros(1 << 20, dtype=torch.uint8)))


def test_shapes_and_types_of_device_tensors(h):
    """What else the binding refuses, each by its own message."""
    cfg = ub.make_attn_cfg(4, 2, 64)
    x = ub.heads(bf16(T, 256))
    append = lambda cu=i32(3), cache=bf16(4, 2, 16, 64), pages=i32(2, 4), inv=device(torch.zeros(32)): ub.ub_kv_append(
        h, x, x, x, x, None, inv, cu, None, 2, ub.make_kv_cache(cache, cache), pages, cfg)
    for match, call in (
            ("^q: columns", lambda: ub.ub_attn_prompt(h, ub.heads(bf16(T, 256), 64), x, x, x, None, i32(2), 1, cfg)),
            ("^q: .* does not hold", lambda: ub.ub_attn_prompt(h, ub.heads(bf16(T, 3, 64)), x, x, x, None, i32(2), 1, cfg)),
            ("^lse: ", lambda: ub.ub_attn_prompt(h, x, x, x, x, device(torch.zeros(4, T - 1)), i32(2), 1, cfg)),
            ("^cu_seqlens: at least", lambda: ub.ub_attn_prompt(h, x, x, x, x, None, i32(2).long(), 1, cfg)),
            ("^cu_seqlens: at least", lambda: append(cu=i32(2))),
            ("^inv_freq: at least", lambda: append(inv=device(torch.zeros(31)))),
            ("^cache: ", lambda: append(cache=bf16(4, 1, 16, 64))),
            ("^pages: an int32", lambda: append(pages=i32(1, 4))),
            ("^workspace: a contiguous", lambda: ub.ub_attn_decode(
                h, x, ub.make_kv_cache(bf16(4, 2, 16, 64), bf16(4, 2, 16, 64)), i32(1, 4), i32(1), 1, x, None, cfg,
                device(torch.zeros(1, dtype=torch.uint8)).expand(1 << 20)))):
        with pytest.raises(ValueError, match=match):
            call()
