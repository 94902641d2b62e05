"""The relative position bias goes into pba_forward and pba_partial as it comes,
whatever the number of keys: bf16 rows lie a multiple of eight elements apart
(fp32 rows are taken wherever they lie).

No tolerances: the bias is the table's own value, and the attention of a bias
is, bit for bit, that of a copy of it, in bf16 with rows padded by the caller."""
import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba

pytestmark = pytest.mark.gpu


def _padded(t):
    """A copy, in bf16 with rows a multiple of eight elements apart."""
    *lead, n = t.shape
    if t.dtype == torch.float32:
        return t.clone()
    out = t.new_zeros((*lead, n + 8 - n % 8))[..., :n]
    return out.copy_(t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,Nq,Nk", [(1, 16, 1, 2047), (2, 3, 9, 1), (1, 4, 203, 203), (2, 5, 70, 130), (1, 2, 64, 264),
                                       (3, 1, 5, 7)])
def test_attention_takes_the_bias(cuda_device, B, H, Nq, Nk, dtype):
    g = torch.Generator().manual_seed(Nk)
    q, k, v = (torch.randn((B, H, n, 64), generator=g).to(dtype).cuda() for n in (Nq, Nk, Nk))
    table = torch.randn((33, H), generator=g).to(dtype).cuda()
    q_pos = torch.randint(0, 300, (B, Nq), generator=g, dtype=torch.int32).cuda()
    k_pos = torch.randint(0, 300, (B, Nk), generator=g, dtype=torch.int32).cuda()
    mask = (torch.rand((B, Nk), generator=g) < 0.9).to(torch.uint8).cuda()
    ref = R.relpos_bias(table, R.relpos_rows(q_pos, k_pos, 33, "clip", 0))
    for base in (None, torch.zeros((B, H, Nq, Nk), dtype=dtype, device="cuda")):
        bias = pba.pba_relpos_bias_forward(table, q_pos, k_pos, base=base)
        assert tuple(bias.shape) == (B, H, Nq, Nk) and torch.equal(R.d64(bias), ref)
        out, lse = pba.pba_forward(q, k, v, bias, mask)
        want, want_lse = pba.pba_forward(q, k, v, _padded(bias), mask)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        parts = pba.pba_partial(q, k, v, bias, mask)
        assert all(torch.equal(a, b) for a, b in zip(parts, pba.pba_partial(q, k, v, _padded(bias), mask)))
    assert pba.pba_last_device_error() == pba.PBA_OK


def test_layer_of_an_odd_number_of_tokens(cuda_device):
    """Norm, bias and attention of 203 tokens as a layer runs them, against fp64.  Bound: y, q, k and v carry one bf16
    rounding (2^-8), P and the result one more each; at most eight such roundings in a row, sqrt(8) 2^-8 = 1.1e-2 of the
    tensor's norm (see test_block_chain.py), and 2e-2 is asserted as there."""
    B, H, N, D, rows = 2, 4, 203, 32, 34
    g = torch.Generator().manual_seed(3)

    def t(*shape, std=1.0, at=0.0):
        return (torch.randn(shape, generator=g) * std + at).to(torch.bfloat16)

    x, table, pair, w, b = t(B, N, H * D), t(rows, H, std=0.5), t(B, H, N, N, std=0.5), t(H * D, std=0.1, at=1.0), t(H * D)
    pos = torch.arange(N).int()
    chain = (pos >= 120).int()
    mask = (torch.rand((B, N), generator=g) < 0.9).to(torch.uint8)

    def heads(y):
        return y.reshape(B, N, H, D).transpose(1, 2)

    index = R.relpos_rows(pos, pos, rows, "clip", 0, chain, chain)
    y64 = heads(R.norm(R.d64(x), (R.d64(w), R.d64(b)), "layer", 1e-5))
    s = y64 @ y64.transpose(-1, -2) / D ** 0.5 + R.relpos_bias(table, index, pair)
    ref = torch.softmax(s.masked_fill(mask[:, None, None, :] == 0, -float("inf")), -1) @ y64
    c = [v.cuda() for v in (x, table, pair, w, b, pos, chain, mask)]
    _, y = pba.pba_block_norm_forward(c[0], pre=(c[3], c[4]))
    bias = pba.pba_relpos_bias_forward(c[1], c[5], c[5], q_group=c[6], k_group=c[6], base=c[2])
    qkv = heads(y).contiguous()
    out, _ = pba.pba_forward(qkv, qkv, qkv, bias, c[7])
    assert float((R.d64(out) - ref).norm() / ref.norm()) <= 2e-2
