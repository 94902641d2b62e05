"""Outputs whose rows lie on one another (a stride of 0 on an axis longer than 1,
as torch's expand makes them) are refused: several rows would be written to one
place at once."""
import ctypes

import pytest
import torch

import pair_biased_attention_b200 as pba

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: each call below fails its checks first
BAD = pba.PBA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return pba.load_library()


def _relpos(**kw):
    d = pba.PbaRelposDesc()
    d.B, d.H, d.Nq, d.Nk, d.dtype, d.rows = 2, 4, 16, 16, pba.PBA_BF16, 9
    d.out_stride[:] = (4 * 256, 256, 16)
    return d


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_bias(lib, axis):
    d = _relpos()
    d.out_stride[axis] = 0
    assert lib.pba_relpos_bias_forward(ctypes.byref(d), FAKE, FAKE, None, None, FAKE, None, FAKE, None) == BAD


def test_norms(lib):
    names = ["x", "f", "gate", "h", "y", "dh", "dy", "dx", "df", "dgate"]
    for zero in ("h", "y", "dx", "df", "dgate"):
        d = pba.PbaNormDesc()
        d.rows, d.C, d.eps = 4, 64, 1e-5
        for n in names:
            setattr(d, n + "_stride", 0 if n == zero else 64)
        if zero in ("h", "y"):
            assert lib.pba_block_norm_forward(ctypes.byref(d), *([FAKE] * 10), None) == BAD
        else:
            assert lib.pba_block_norm_backward(ctypes.byref(d), *([FAKE] * 19), 1 << 40, None) == BAD


@pytest.mark.parametrize("which", ["out_stride", "lse_stride"])
@pytest.mark.parametrize("axis", [0, 1, 2])
def test_cross_attention(lib, which, axis):
    d = pba.PbaCrossDesc(2, 4, 2, 16, 16, 64, pba.PBA_BF16)
    for s, n in ((d.q_stride, 4), (d.out_stride, 4), (d.k_stride, 2), (d.v_stride, 2)):
        s[:] = (n * 16 * 64, 16 * 64, 64)
    d.lse_stride[:] = (64, 16, 1)
    getattr(d, which)[axis] = 0
    args = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE]
    assert lib.pba_cross_attn_forward(ctypes.byref(d), *args, None) == BAD


@pytest.mark.gpu
def test_public_calls(cuda_device):
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    table = torch.ones((5, 2), device="cuda")
    with pytest.raises(pba.PbaError):
        pba.pba_relpos_bias_forward(table, pos, pos, out=torch.zeros((1, 2, 1, 8), device="cuda").expand(1, 2, 8, 8))
    x = torch.ones((4, 64), device="cuda")
    one = torch.ones((1, 64), device="cuda")
    for kw in (dict(h=one.expand(4, 64)), dict(y=one.expand(4, 64))):
        with pytest.raises(pba.PbaError):
            pba.pba_block_norm_forward(x, x, pre=(one[0], None), **kw)
    # a single row, and inputs that are shared, are as before
    h, y = pba.pba_block_norm_forward(one.expand(4, 64), x, pre=(one[0], None))
    assert (h == 2).all()
    q = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pba.PbaError):
        pba.pba_cross_attn_forward(q, q, q, out=q[:, :1].expand(2, 2, 3, 64))
    with pytest.raises(pba.PbaError):
        pba.pba_cross_attn_forward(q, q, q, lse=torch.zeros((1,), device="cuda").expand(2, 2, 3))
    # a shared gradient of the bias is read, not written
    dbias = torch.ones((1, 1, 1, 8), device="cuda").expand(2, 2, 8, 8)
    want = pba.pba_relpos_bias_backward(dbias.contiguous(), pos, pos, 5)
    assert torch.equal(pba.pba_relpos_bias_backward(dbias, pos, pos, 5), want)
