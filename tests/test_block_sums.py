"""The per-channel sums of the norms' gradients: every row once, and as exact as
the header says (fp32 over at most 512 rows of a thread, 64 bits beyond, a
block's share kept as fp32).

Whole numbers whose sums stay below 2^24 come out exactly, in any order of
addition: a row left out or taken twice shows.  Row counts lie on both sides of
what the launch takes at once: `_shape` repeats the launch's rule, for these
counts and for the bounds."""
import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _shape(C):
    """Rows of a block and blocks of one round of the launch for C channels."""
    lanes = -(-C // 8)
    if lanes > 32:
        threads = -(-lanes // 32) * 32
        return 1, 148 * max(1, 512 // threads)
    lanes = 1 << (lanes - 1).bit_length()
    return 256 // lanes, 296


def _counts(C):
    y, blocks = _shape(C)
    turn = y * blocks
    return sorted({1, y, y + 1, turn - 1, turn, turn + 1, 2 * turn + y + 1, 4 * turn + 3})


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [8, 20, 64, 128, 300, 512, 1021, 4104])
def test_whole_numbers_are_exact(cuda_device, C, dtype):
    g = torch.Generator("cuda").manual_seed(C)
    for rows in _counts(C):
        def ints(n=8):
            return torch.randint(-n, n + 1, (rows, C), generator=g, device="cuda").to(dtype)

        dy, dh, f, h = ints(), ints(), ints(), ints()
        w = torch.ones((C,), dtype=dtype, device="cuda")
        zero = torch.zeros_like(w)
        # dpre_b; dscale without a norm or a gate, with t = dh (a norm of weight 0 passes nothing on)
        got = pba.pba_block_norm_backward(h, dh, dy, f, None, w, None, (zero, zero), "layer")
        assert torch.equal(got[7].double(), dy.double().sum(0)), (rows, C)
        assert torch.equal(got[3].double(), (dh.double() * f.double()).sum(0)), (rows, C)
        # dpost_b
        got = pba.pba_block_norm_backward(None, dh, None, f, None, None, (w, zero), None, "layer")
        assert torch.equal(got[5].double(), dh.double().sum(0)), (rows, C)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,C", [(20001, 64), (5000, 512), (9473, 100)])
def test_weights_gradients_within_the_real_chain(cuda_device, rows, C, dtype):
    """dpre_w and dpost_w.  A thread adds ceil(rows / (rows of a round)) <= 512 terms in fp32; the block's join and all
    beyond are in 64 bits, a block's share and the result rounded once each.  A term is off by at most 128 u of
    |dy| (|v_hat| + max|v| rs) (the statistics: 18 and 24 u, the products 3 u)."""
    g = torch.Generator().manual_seed(rows)
    h, f, dy, dh = (torch.randn((rows, C), generator=g).to(dtype) for _ in range(4))
    w = torch.rand((C,), generator=g).to(dtype) + 0.5
    zero = torch.zeros((C,), dtype=dtype)
    y, blocks = _shape(C)
    chain = -(-rows // (y * blocks))
    for kind in ("layer", "rms"):
        got = pba.pba_block_norm_backward(h.cuda(), dh.cuda(), dy.cuda(), f.cuda(), None, None, (w.cuda(), None),
                                          (zero.cuda(), None), kind, 1e-5)
        for value, x, d in ((got[6], h, dy), (got[4], f, dh)):
            x, d = R.d64(x), R.d64(d)
            v = R.norm(x, (torch.ones(C).double(), None), kind, 1e-5)
            c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
            big = x.abs().amax(-1, keepdim=True) / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5)
            mag = (d.abs() * (v.abs() + big)).sum(0)
            assert ((R.d64(value) - (d * v).sum(0)).abs() <= (chain + 2 + 128) * U * mag).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [1, 64, 128, 256])
def test_a_blocks_rows_are_joined_in_64_bits(cuda_device, C, dtype):
    """One row of 2^24 among ones, a row to a thread: the block's share is rounded once, half a step of 2."""
    y, _ = _shape(C)
    dy = torch.ones((y, C), dtype=dtype, device="cuda")
    dy[0] = 2.0 ** 24
    w = torch.ones((C,), dtype=dtype, device="cuda")
    got = pba.pba_block_norm_backward(torch.zeros_like(dy), None, dy, None, None, None, None, (w, w), "layer")
    assert ((got[7].double() - (2.0 ** 24 + y - 1)).abs() <= 1).all()


@pytest.mark.parametrize("C", [8, 512])
def test_a_thread_takes_at_most_512_rows(cuda_device, C):
    """2^24 in the first row and ones in 1100 rounds of rows: what a thread's fp32 sum loses are the at most 511 ones
    that follow the first row in its share; the block's share is rounded by 1 at most (steps of 2 from 2^24 on), the
    result by half its own step."""
    y, blocks = _shape(C)
    rows = 1100 * y * blocks
    dy = torch.ones((rows, C), dtype=torch.bfloat16, device="cuda")
    dy[0] = 2.0 ** 24
    w = torch.ones((C,), dtype=torch.bfloat16, device="cuda")
    h = torch.zeros((1, C), dtype=torch.bfloat16, device="cuda").expand(rows, C)
    got = pba.pba_block_norm_backward(h, None, dy, None, None, None, None, (w, w), "layer")[7].double()
    want = 2.0 ** 24 + rows - 1
    step = 2.0 ** (int(want).bit_length() - 24)
    assert ((got - want).abs() <= 511 + 1 + step / 2).all()
