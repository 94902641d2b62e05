"""The fp64 references of the block operators against hand-made values and
their gradients against differences."""
import math

import pytest
import torch

import block_ref as R


def test_log_rows_of_a_small_side():
    # side 8, far 64: rows 0..3 exact, then borders 4 * 16^(t/4) = 8, 16, 32
    got = [R.log_row(d, 8, 64) for d in (0, 3, 4, 7, 8, 15, 16, 31, 32, 63, 64, 1000)]
    assert got == [0, 3, 4, 4, 5, 5, 6, 6, 7, 7, 7, 7]


def test_relpos_rows_clip_and_groups():
    pos = torch.tensor([0, 5, 6], dtype=torch.int32)
    group = torch.tensor([0, 0, 1], dtype=torch.int32)
    rows = R.relpos_rows(pos, pos, 6, "clip", 0, group, group)  # radius 2, row 5 across groups
    assert rows.tolist() == [[[2, 4, 5], [0, 2, 5], [5, 5, 2]]]


def _directional(fn, args, dirs, eps=1e-6):
    plus = fn(*[a + eps * d for a, d in zip(args, dirs)])
    minus = fn(*[a - eps * d for a, d in zip(args, dirs)])
    return (plus - minus) / (2 * eps)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_block_gradient_against_differences(kind):
    g = torch.Generator().manual_seed(3)
    shapes = [(5, 12)] * 3 + [(12,)] * 5
    args = [torch.randn(s, generator=g, dtype=torch.float64, requires_grad=True) for s in shapes]
    wh, wy = torch.randn(5, 12, generator=g).double(), torch.randn(5, 12, generator=g).double()

    def loss(x, f, gate, scale, pw, pb, nw, nb):
        h, y = R.block(x, f, gate, scale, (pw, pb), (nw, nb), kind, 1e-5)
        return (h * wh).sum() + (y * wy).sum()

    grads = torch.autograd.grad(loss(*args), args)
    dirs = [torch.randn(s, generator=g, dtype=torch.float64) for s in shapes]
    with torch.no_grad():
        diff = _directional(loss, args, dirs)
    got = sum((gr * d).sum() for gr, d in zip(grads, dirs))
    assert abs(got - diff) <= 1e-7 * abs(diff) + 1e-7


def test_cross_gradient_against_differences_and_empty_rows():
    g = torch.Generator().manual_seed(4)
    q = torch.randn(2, 4, 3, 8, generator=g, dtype=torch.float64, requires_grad=True)
    k, v = (torch.randn(2, 2, 5, 8, generator=g, dtype=torch.float64, requires_grad=True) for _ in range(2))
    keep = torch.tensor([[1, 0, 1, 1, 0], [0, 0, 0, 0, 0]]).bool()
    w = torch.randn(2, 4, 3, 8, generator=g).double()

    def loss(q, k, v):
        return (R.cross(q, k, v, keep)[0] * w).sum()

    grads = torch.autograd.grad(loss(q, k, v), (q, k, v))
    dirs = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (q, k, v)]
    with torch.no_grad():
        diff = _directional(loss, (q, k, v), dirs)
        out, lse = R.cross(q, k, v, keep)
    assert abs(sum((a * b).sum() for a, b in zip(grads, dirs)) - diff) <= 1e-7 * abs(diff) + 1e-7
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all() and torch.isfinite(lse[0]).all()
    assert all((t[1] == 0).all() for t in grads)
