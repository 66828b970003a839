"""GPU tests of the workgroup -> (sequence, tile) map where the grid does not run at once: 17 to 65
sequences, and calls of more than 64 levels of tiles, with the kernels of one group of waves and
of four."""

import math

import pytest
import torch

from tests import attn_ref as ref
from tests import test_gpu_attn as base
from tests.test_gpu_attn import BF16, Rank, cu_of, i32, make, split, ub, workspace  # noqa: F401  (ub: a fixture)

pytestmark = pytest.mark.gpu


def ragged(n, longest, seed):
    """n lengths, empty ones and single tokens among them, the longest in the middle."""
    x = torch.randint(2, longest // 3, (n,), generator=torch.Generator().manual_seed(seed)).tolist()
    x[0], x[n // 3], x[n // 2], x[-1] = 0, 1, longest, 1
    return x


def workgroups(shape, lens, pad, rows):
    """Of the forward pass with tiles of `rows` rows; the gradient has more."""
    T = sum(lens) + pad
    return (T // rows + min(len(lens), T)) * shape[0]


def one_group(shape, lens, pad, below):
    """Whether a call of so many rows takes the kernels of one group of waves."""
    return (sum(lens) + pad) * shape[0] >= below * 1024 or len(lens) * shape[0] >= 96


@pytest.mark.parametrize("n,H,G,D,longest,grouped", [
    (17, 8, 2, 64, 900, False),
    (40, 8, 8, 40, 400, False),
    (63, 6, 3, 80, 150, False),
    (64, 8, 1, 64, 300, False),
    (65, 8, 1, 64, 300, False),
    (17, 4, 4, 64, 1001, True),
    (23, 4, 1, 128, 800, True),
    (31, 3, 1, 64, 900, True),
])
def test_many_sequences(ub, n, H, G, D, longest, grouped):
    shape, lens, pad = (H, G, D), ragged(n, longest, n), 3
    assert one_group(shape, lens, pad, 36) != grouped and one_group(shape, lens, pad, 44) != grouped
    assert workgroups(shape, lens, pad, 64 if grouped else 128) > 256
    base.test_prompt_and_gradient(ub, shape, lens, pad)


def on_device(f, *args):
    """f of device tensors in 64 bits, its results on the host."""
    with torch.device("cuda"):
        r = f(*[a.cuda() if isinstance(a, torch.Tensor) else a for a in args])
    host = lambda t: tuple(host(u) for u in t) if isinstance(t, tuple) else t.cpu()
    return host(r)


@pytest.mark.parametrize("H,G,D,lens,grouped", [
    (8, 8, 64, [60, 8321, 0, 1, 500], False),     # 70 levels of 128 rows
    (6, 1, 40, [1, 9000, 300], False),
    (8, 2, 64, [4200, 0, 97, 200], True),         # 71 levels of 64 rows
    (5, 1, 128, [63, 6500, 1, 400], True),
])
def test_long_sequences(ub, H, G, D, lens, grouped):
    shape, pad = (H, G, D), 2
    rows = 64 if grouped else 128
    assert one_group(shape, lens, pad, 36) != grouped and one_group(shape, lens, pad, 44) != grouped
    assert workgroups(shape, lens, pad, rows) > 256 and (sum(lens) + pad + rows - 1) // rows > 64
    x, T = make(shape, lens, pad, seed=D)
    cu, used, scale = cu_of(lens), sum(lens), D ** -0.5
    cfg = ub.make_attn_cfg(H, G, D)
    xd = x.cuda()
    do = torch.full((T, H * D), math.nan, dtype=BF16)
    do[:used] = base.normal(7, (used, H * D))
    dod, dx = do.cuda(), torch.full_like(xd, math.nan)
    out, lse = torch.full((T, H * D), math.nan, dtype=BF16, device="cuda"), torch.full((H, T), math.nan, device="cuda")
    cols = (0, H * D, (H + G) * D)
    hs, dh = [ub.heads(xd, c) for c in cols], [ub.heads(dx, c) for c in cols]
    ws = workspace(ub, ub.UB_ATTN_PROMPT_BWD, cfg, T, len(lens))
    with Rank(ub, T) as h:
        ub.ub_attn_prompt(h, *hs, ub.heads(out), lse, i32(cu), len(lens), cfg)
        ub.ub_attn_prompt_bwd(h, ub.heads(dod), *hs, ub.heads(out), lse, *dh, i32(cu), len(lens), cfg, ws)
        torch.cuda.synchronize()
    args = [t[:used].double() for t in split(x, shape)]
    o, l, to, tl = on_device(ref.prompt, *args, cu, scale)
    ref.check(out[:used].reshape(used, H, D), o, to, "out")
    ref.check(lse[:, :used], l, tl, "lse")
    want, tol = on_device(ref.prompt_bwd, do[:used].double().reshape(used, H, D), *args, cu, scale)
    for name, g, w, t in zip(("dq", "dk", "dv"), split(dx, shape), want, tol):
        ref.check(g[:used], w, t, name)
        assert bool((g[used:] == 0).all()), name
    assert bool((out[used:] == 0).all()) and bool((lse[:, used:] == -math.inf).all())
