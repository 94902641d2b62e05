"""The gate's gradient over the whole range of the sigmoid: dgate = t u s (1 - s)
keeps its relative accuracy on both sides, where s is next to 0 and next to 1.

The weights of the norms are 0, so that t is dh and u the norm's bias (or f)
exactly.  Bound, u = 2^-24: s and 1 - s are each a quotient of an exponential
whose exponent is off by |gate| u, units good to 4 u, and an addition, so
(|gate| + 12) u relative; four products more: (2 |gate| + 32) u covers it, and
half a step of the type for the result.  Below 1e-37 fp32 ends."""
import math

import pytest
import torch

import pair_biased_attention_b200 as pba

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("parts", ["gate", "gate-pre", "gate-post-pre", "gate-post"])
@pytest.mark.parametrize("C", [64, 100, 768, 8192])
def test_gradient_of_large_gates(cuda_device, C, parts, dtype):
    rows = 7
    g = torch.Generator().manual_seed(C)

    def t(*s):
        return torch.randn(s, generator=g).to(dtype)

    f, dh, dy, h = (t(rows, C) for _ in range(4))
    gate = ((torch.rand((rows, C), generator=g) - 0.5) * 160).to(dtype)
    gate[0, :6] = torch.tensor([0.0, 17.0, -17.0, 40.0, math.inf, -math.inf], dtype=dtype)
    zero, b = torch.zeros((C,), dtype=dtype), t(C)
    pre = (zero, None) if "pre" in parts else None
    post = (zero, b) if "post" in parts else None
    cuda = [None if p is None else tuple(None if e is None else e.cuda() for e in p) for p in (post, pre)]
    got = pba.pba_block_norm_backward(h.cuda(), dh.cuda(), dy.cuda() if pre else None, f.cuda(), gate.cuda(), None, *cuda)
    assert torch.equal(got[0].cpu(), dh)
    x = gate.double()
    s, c = torch.sigmoid(x), torch.sigmoid(-x)
    u = (b if post else f).double()
    ref = dh.double() * u * s * c
    rel = (2 * x.abs().clamp(max=100) + 32) * U
    half = torch.finfo(dtype).eps / 2
    err = (got[2].double().cpu() - ref).abs()
    assert (err <= (rel * (1 + half) + half) * ref.abs() + 1e-37).all()
    assert (got[2][0, 4:6] == 0).all()
    if not post:  # df = dh s
        df = dh.double() * s
        err = (got[1].double().cpu() - df).abs()
        assert (err <= (rel * (1 + half) + half) * df.abs() + 1e-37).all()
