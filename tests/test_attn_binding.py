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


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


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
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros((64, 64), dtype=torch.uint8)[:, :8]):
        with pytest.raises(ValueError, match="workspace"):
            ub._ws_arg(bad)
    assert ub._ws_arg(None) == (None, 0)
    assert ub._ws_arg(torch.zeros(48, dtype=torch.float32))[1] == 192
