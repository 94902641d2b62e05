"""The operators around the attention block run together, as a layer of a pair or
token model uses them, and their gradients through the whole chain.

One self-attention layer with a learned relative position bias, and one cross
attention layer to an encoder's states, each between a norm before and a gated,
scaled residual after:

    bias   = relpos(table, positions, chains) + pair bias
    x, y0  = block_norm(x0, pre)                       y0 feeds the projections
    a      = pba(q(y0), k(y0), v(y0), bias, key mask)
    h1, y1 = block_norm(x, a, gate, scale, post, pre)
    c      = cross(q(y1), k(enc), v(enc), k_len)
    h2, _  = block_norm(h1, c, scale, post)

Projections are fixed reshapes with sign flips (so that they round nothing).
The chain runs on the GPU kernels in bf16 and, from the same bf16 inputs, in
fp64 by the definitions; gradients by the kernels' backward calls in reverse
against autograd in fp64.

Bounds.  Every stored tensor along the chain is rounded to bf16, 2^-8 of itself,
and each operator adds its own rounding of P, dS and its result (2^-8 each).  A
quantity passes through at most 16 such roundings forward and 16 backward;
relative to the tensor's root mean square they are independent of each other's
sign, so 2^-8 sqrt(32) = 2.2e-2 is one standard deviation at the most
unfavourable alignment of all of them (each half step at its extreme), which
the relative L2 error over a whole tensor stays below; 4e-2 is asserted for
gradients and half of it for the forward."""
import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba

pytestmark = pytest.mark.gpu
B, H, N, D, NE, ROWS = 2, 4, 200, 32, 264, 34
C = H * D


def heads(y, sign):
    """[B,N,C] -> [B,H,N,D], every other feature's sign flipped for sign < 0."""
    f = torch.ones(C, dtype=y.dtype, device=y.device)
    if sign < 0:
        f[::2] = -1
    return (y * f).reshape(B, -1, H, D).transpose(1, 2)


def merge(o):
    return o.transpose(1, 2).reshape(B, -1, C)


def attention64(q, k, v, bias, keep):
    s = q @ k.transpose(-1, -2) / D ** 0.5 + bias
    s = s.masked_fill(~keep[:, None, None, :], -float("inf"))
    return torch.softmax(s, -1) @ v


def rel(a, b):
    a, b = R.d64(a), R.d64(b)
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("captured", [False, True])
def test_layer_forward_and_backward(cuda_device, captured):
    g = torch.Generator().manual_seed(21)

    def t(*shape, std=1.0, at=0.0):
        return (torch.randn(shape, generator=g) * std + at).to(torch.bfloat16)

    leaves = dict(x0=t(B, N, C), enc=t(B, NE, C), table=t(ROWS, H, std=0.5), pair=t(B, H, N, N, std=0.5),
                  gate=t(B, N, C), scale1=t(C, std=0.2, at=0.7), scale2=t(C, std=0.2, at=0.7),
                  w0=t(C, std=0.1, at=1.0), b0=t(C, std=0.1), w1=t(C, std=0.1, at=1.0), b1=t(C, std=0.1),
                  w2=t(C, std=0.1, at=1.0), b2=t(C, std=0.1), w3=t(C, std=0.1, at=1.0), b3=t(C, std=0.1))
    pos = torch.stack([torch.arange(N), torch.cat([torch.arange(120), torch.arange(N - 120)])]).int()
    chain = torch.stack([torch.zeros(N), (torch.arange(N) >= 120).float()]).int()
    mask = (torch.rand((B, N), generator=g) < 0.9).to(torch.uint8)
    k_len = torch.tensor([NE, 150], dtype=torch.int32)
    dh2 = t(B, N, C)

    # fp64
    L = {n: R.d64(v).requires_grad_() for n, v in leaves.items()}
    index = R.relpos_rows(pos, pos, ROWS, "clip", 0, chain, chain)
    bias = L["table"][index].permute(0, 3, 1, 2) + L["pair"]
    _, y0 = R.block(L["x0"], None, None, None, None, (L["w0"], L["b0"]), "layer", 1e-5)
    a = merge(attention64(heads(y0, 1), heads(y0, -1), heads(y0, 1), bias, mask != 0))
    h1, y1 = R.block(L["x0"], a, L["gate"], L["scale1"], (L["w1"], L["b1"]), (L["w2"], L["b2"]), "layer", 1e-5)
    keep = torch.arange(NE)[None, :] < k_len[:, None]
    c = merge(R.cross(heads(y1, 1), heads(L["enc"], -1), heads(L["enc"], 1), keep)[0])
    h2, _ = R.block(h1, c, None, L["scale2"], (L["w3"], L["b3"]), None, "layer", 1e-5)
    h2.backward(R.d64(dh2))

    # the kernels
    G = {n: v.cuda() for n, v in leaves.items()}
    posc, chainc, maskc, lenc, dh2c = (v.cuda() for v in (pos, chain, mask, k_len, dh2))
    enc = G["enc"]

    def run():
        bias = pba.pba_relpos_bias_forward(G["table"], posc, posc, "clip", q_group=chainc, k_group=chainc,
                                           base=G["pair"])
        _, y0 = pba.pba_block_norm_forward(G["x0"], pre=(G["w0"], G["b0"]))
        q, k, v = (heads(y0, s).contiguous() for s in (1, -1, 1))
        a, lse = pba.pba_forward(q, k, v, bias, maskc)
        am = merge(a).contiguous()
        args1 = (am, G["gate"], G["scale1"], (G["w1"], G["b1"]), (G["w2"], G["b2"]))
        h1, y1 = pba.pba_block_norm_forward(G["x0"], *args1)
        cq, ck, cv = (heads(y1, 1), heads(enc, -1), heads(enc, 1))
        c, clse = pba.pba_cross_attn_forward(cq, ck, cv, lenc)
        cm = merge(c).contiguous()
        args2 = (cm, None, G["scale2"], (G["w3"], G["b3"]), None)
        h2, _ = pba.pba_block_norm_forward(h1, *args2)
        # backward
        dh1, dcm, _, ds2, dw3, db3, _, _ = pba.pba_block_norm_backward(h2, dh2c, None, *args2)
        dcq, dck, dcv = pba.pba_cross_attn_backward(cq, ck, cv, c, clse, heads(dcm, 1), lenc)
        f = torch.ones(C, dtype=torch.bfloat16, device="cuda")
        f[::2] = -1
        dy1 = merge(dcq).contiguous()
        denc = merge(dck) * f + merge(dcv)
        dx, dam, dgate, ds1, dw1, db1, dw2, db2 = pba.pba_block_norm_backward(h1, dh1, dy1, *args1)
        dq, dk, dv, dbias, _ = pba.pba_backward(q, k, v, bias, maskc, a, lse, heads(dam, 1).contiguous())
        dtable = pba.pba_relpos_bias_backward(dbias, posc, posc, ROWS, "clip", q_group=chainc, k_group=chainc)
        dy0 = (merge(dq + dv) + merge(dk) * f.float()).to(torch.bfloat16)
        dx0, _, _, _, _, _, dw0, db0 = pba.pba_block_norm_backward(G["x0"], dx, dy0, pre=(G["w0"], G["b0"]))
        return h2, dict(x0=dx0, enc=denc, table=dtable, pair=dbias, gate=dgate, scale1=ds1, scale2=ds2, w0=dw0, b0=db0,
                        w1=dw1, b1=db1, w2=dw2, b2=db2, w3=dw3, b3=db3)

    got, grads = run()
    if captured:
        want, wgrads = got, grads
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got, grads = run()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(torch.equal(grads[n], wgrads[n]) for n in grads)
    torch.cuda.synchronize()
    assert pba.pba_last_device_error() == pba.PBA_OK
    assert rel(got, h2) <= 2e-2
    for n, v in grads.items():
        assert rel(v, L[n].grad) <= 4e-2, (n, rel(v, L[n].grad))
