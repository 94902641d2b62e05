"""The choice among cross attention's forward kernels: shapes on either side of
every border give the reference's values, whichever kernel runs, and the same
bits every time.

`_kernel` repeats the library's rule with the clusters that a B200 of 148 SMs
holds; it only says which kernels the shapes are meant for.  Bounds as derived in
test_cross_attn.py, whose check is used."""
import pytest
import torch

import test_cross_attn as T
import pair_biased_attention_b200 as pba

TILES = {1: 148, 2: 74, 4: 33, 8: 15}
FEW = {1: 592, 2: 296, 3: 187, 4: 142, 5: 112, 6: 93, 7: 78, 8: 71}
FEW128 = {1: 296, 2: 148, 3: 93, 4: 71, 5: 56, 6: 45, 7: 37, 8: 33}
COST = {32: (5.5, 3.0, 0.34, 7.0, 5.8, 1.44, 1.5, 4.0), 64: (6.0, 3.0, 0.42, 9.25, 5.8, 1.44, 1.5, 11.0),
        128: (7.0, 6.0, 0.60, 8.75, 7.5, 2.06, 2.65, 20.0)}


def _up(a, b):
    return -(-a // b)


def _kernel(B, H, Hkv, Nq, Nk, D):
    """("rows", blocks to 16 rows) or ("tiles", CTAs to a unit)."""
    room = FEW128 if D == 128 else FEW
    start, more, step, rate, t_start, tile, shared, join = COST[D]
    units, n = B * Hkv * _up(H // Hkv * Nq, 16), 1
    while n < min(8, _up(Nk, 64)) and units <= room[n + 1]:
        n += 1
    steps, rounds = _up(_up(_up(Nk, 16), n), 4), _up(units * n, room[1])
    rows = start + more * (rounds - 1) + max(rounds * steps * step, units * n * steps * 64 * D * 4e-6 / rate)
    units, s = B * H * _up(Nq, 256), 1
    while s < 8 and units <= TILES[2 * s] and _up(Nk, 128) >= 4 * s:
        s *= 2
    per = _up(_up(Nk, 128), s)
    tiles = 8.0 + join / s + per * shared if s > 1 else t_start + _up(units, 148) * per * tile
    return ("rows", n) if rows <= tiles else ("tiles", s)


# B, H, Hkv, Nq, Nk, and the kernel of D = 64: around 15 and 16 units of clusters of eight, 33 and 34 of four, 74 and 75 of
# two; few rows around the units that 8, 6 and 3 blocks to 16 rows are held for, and one head of few queries
SHAPES = [
    ((1, 15, 15, 256, 2048), ("tiles", 8)), ((1, 16, 16, 256, 2048), ("tiles", 4)), ((1, 33, 33, 140, 1100), ("tiles", 4)),
    ((1, 34, 34, 250, 1100), ("tiles", 2)), ((2, 37, 37, 200, 600), ("tiles", 2)), ((1, 75, 75, 200, 600), ("tiles", 1)),
    ((1, 71, 71, 9, 1000), ("rows", 8)), ((1, 72, 72, 9, 1000), ("rows", 7)), ((3, 31, 31, 2, 640), ("rows", 6)),
    ((2, 47, 47, 3, 640), ("rows", 5)), ((11, 17, 17, 1, 300), ("rows", 3)), ((4, 47, 47, 1, 300), ("rows", 2)),
    ((1, 1, 1, 5, 9000), ("rows", 8)),
]


def test_shapes_are_meant_for_each_choice():
    assert all(_kernel(*s, 64) == k for s, k in SHAPES)
    # the shapes of test_cross_attn.py still reach every kernel that they are there for

    def name(B, H, Hkv, Nq, Nk, D):
        kernel, n = _kernel(B, H, Hkv, Nq, Nk, D)
        return kernel if kernel == "rows" else "clusters" if n > 1 else "tiles" if B * H * _up(Nq, 256) <= 148 else "persistent"

    for D in (32, 64, 128):
        for shapes in (T.SHAPES, T.MASKED, T.NANS, [T.MANY]):
            assert {name(*s, D) for s in shapes} >= {T._forward_kernel(*s, D) for s in shapes}


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("shape", [s for s, _ in SHAPES])
def test_values_around_every_border(cuda_device, shape, D):
    B, H, Hkv, Nq, Nk = shape
    q, k, v, dout, g = T._inputs(*shape, D, seed=H)
    k_len = torch.randint(1, Nk + 1, (B,), generator=g, dtype=torch.int32)
    out, lse = T._check(q, k, v, dout, k_len, backward=False)[:2]
    again = pba.pba_cross_attn_forward(q.cuda(), k.cuda(), v.cuda(), k_len.cuda())
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
