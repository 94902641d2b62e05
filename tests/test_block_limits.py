"""The operators around the attention block at their limits: infinities and NaN
in places that count, offsets past 32 bits, and calls on two streams at once.

Values and tolerances are the other files'; here a result is compared with the
same call's on tensors without the peculiarity, bit for bit, wherever that one
is known to be right."""
import math

import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 + 64  # elements: an offset that 32 bits cannot hold, on 16 bytes for every type


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 3])  # rows on 16 bytes, and not
def test_table_gradient_keeps_infinities_in_their_rows(cuda_device, dtype, pad):
    """Three groups that share eights of keys, distances far on either side and near: an infinity or a NaN reaches
    the row of its own pair only, and leaves every other as it was."""
    B, H, Nq, Nk, rows = 1, 2, 96, 96, 18
    q = torch.arange(Nq, dtype=torch.int32)
    group = (torch.arange(Nk) // 20).clamp(max=2).int()
    index = R.relpos_rows(q, q, rows, "clip", 0, group, group)
    g = torch.Generator().manual_seed(2)
    clean = torch.randn((B, H, Nq, Nk), generator=g).to(dtype)
    call = [t.cuda() for t in (q, q)] + [rows, "clip", 0] + [group.cuda()] * 2
    for bad in (math.inf, math.nan):
        for i, j in ((0, 1), (30, 18), (30, 21), (70, 95), (95, 41), (95, 38), (5, 90)):
            d = torch.zeros((B, H, Nq, Nk + 16), dtype=dtype)[..., pad:pad + Nk]
            d.copy_(clean)
            d[0, 1, i, j] = bad
            hit = torch.zeros((rows, H), dtype=torch.bool)
            hit[index[0, i, j], 1] = True
            wide = d.new_zeros((B, H, Nq, Nk + 16)).cuda()
            view = wide[..., pad:pad + Nk]
            view.copy_(d)
            got = pba.pba_relpos_bias_backward(view, *call).cpu()
            view.copy_(clean)
            want = pba.pba_relpos_bias_backward(view, *call).cpu()
            assert torch.equal(~torch.isfinite(got), hit)
            assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("shape", [(2, 4, 2, 1, 300), (2, 8, 4, 513, 1000), (2, 16, 8, 600, 1000)])
def test_not_a_number_in_a_key_shows(cuda_device, shape, D):
    """A NaN in a key that counts makes every output and lse of the heads that read it NaN, and no other."""
    B, H, Hkv, Nq, Nk = shape
    g = torch.Generator().manual_seed(D)
    q, k, v = (torch.randn((B, h, n, D), generator=g).to(torch.bfloat16).cuda()
               for h, n in ((H, Nq), (Hkv, Nk), (Hkv, Nk)))
    want, want_lse = pba.pba_cross_attn_forward(q, k, v)
    for key in (0, 150, Nk - 1):
        bad = k.clone()
        bad[1, 1, key, 3] = math.nan
        out, lse = pba.pba_cross_attn_forward(q, bad, v)
        G = H // Hkv
        hit = torch.zeros((B, H), dtype=torch.bool)
        hit[1, G:2 * G] = True
        hit = hit.cuda()
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
        assert pba.pba_last_device_error() == pba.PBA_OK


def test_offsets_past_32_bits(cuda_device):
    """Heads, batches and rows that lie over 2^31 elements apart."""
    g = torch.Generator().manual_seed(4)
    field = torch.empty(BIG + 2 ** 22, dtype=torch.bfloat16, device="cuda")

    def far(t, axis, at=0):
        """t with the two entries of `axis` BIG elements apart in the field."""
        assert t.shape[axis] == 2
        strides = list(t.contiguous().stride())
        strides[axis] = BIG
        view = field.as_strided(t.shape, strides, at)
        view.copy_(t)
        return view

    for Nq in (2, 300):
        for axis in (0, 1):
            q, k, v, dout = (torch.randn((2, 2, n, 64), generator=g).to(torch.bfloat16).cuda()
                             for n in (Nq, 520, 520, Nq))
            out, lse = pba.pba_cross_attn_forward(q, k, v)
            grads = pba.pba_cross_attn_backward(q, k, v, out, lse, dout)
            fq, fk, fv, fo = (far(t, axis, i * 2 ** 19) for i, t in enumerate((q, k, v, dout)))
            fout = far(torch.zeros_like(out), axis, 4 * 2 ** 19)
            out2, lse2 = pba.pba_cross_attn_forward(fq, fk, fv, out=fout)
            assert torch.equal(out2, out) and torch.equal(lse2, lse)
            grads2 = pba.pba_cross_attn_backward(fq, fk, fv, fout, lse2, fo)
            assert all(torch.equal(a, b) for a, b in zip(grads, grads2))

    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    table = torch.randn((9, 2), generator=g).to(torch.bfloat16).cuda()
    base = torch.randn((2, 2, 40, 40), generator=g).to(torch.bfloat16).cuda()
    want = pba.pba_relpos_bias_forward(table, pos, pos, base=base)
    dtable = pba.pba_relpos_bias_backward(base, pos, pos, 9)
    for axis in (0, 1):
        for at in (0, 3):
            b = far(base, axis, at)
            out = far(torch.zeros_like(base), axis, 2 ** 20 + at)
            assert torch.equal(pba.pba_relpos_bias_forward(table, pos, pos, base=b, out=out), want)
            assert torch.equal(pba.pba_relpos_bias_backward(b, pos, pos, 9), dtable)

    x, f, dy = (torch.randn((2, 96), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    w = torch.rand((96,), generator=g).to(torch.bfloat16).cuda()
    want = pba.pba_block_norm_forward(x, f, pre=(w, None))
    grads = pba.pba_block_norm_backward(want[0], dy, dy, f, pre=(w, None))
    for at in (0, 3):
        fx, ff, fdy, fh, fy = (far(t, 0, at + 2 ** 10 * i)
                               for i, t in enumerate((x, f, dy, torch.zeros_like(x), torch.zeros_like(x))))
        got = pba.pba_block_norm_forward(fx, ff, pre=(w, None), h=fh, y=fy)
        bwd = pba.pba_block_norm_backward(got[0], fdy, fdy, ff, pre=(w, None))
        if at == 0:  # off 16 bytes the sums over a row go in another order
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(bwd, grads))
        else:
            # h is rounded from the same two terms; y is one rounding from an fp32 value good to 2^-18 of the
            # row's largest, which moves a bf16 result by one step of 2^-7 of itself at most
            assert torch.equal(got[0], want[0])
            close = (got[1].double() - want[1].double()).abs()
            assert (close <= 2.0 ** -7 * want[1].double().abs() + 2.0 ** -16).all()


def test_two_streams_at_once(cuda_device):
    """Calls that run next to each other on two streams give what each gives alone: no state is shared."""
    g = torch.Generator().manual_seed(6)

    def bf(*s):
        return torch.randn(s, generator=g).to(torch.bfloat16).cuda()

    pos = torch.arange(700, dtype=torch.int32, device="cuda")
    sets = []
    for Nq in (2, 600):
        sets.append(dict(q=bf(2, 16, Nq, 64), k=bf(2, 8, 1100, 64), v=bf(2, 8, 1100, 64), dout=bf(2, 16, Nq, 64),
                         table=bf(33, 4), base=bf(1, 4, 700, 700), x=bf(3000, 128), f=bf(3000, 128), w=bf(128)))

    def run(s):
        out, lse = pba.pba_cross_attn_forward(s["q"], s["k"], s["v"])
        grads = pba.pba_cross_attn_backward(s["q"], s["k"], s["v"], out, lse, s["dout"])
        bias = pba.pba_relpos_bias_forward(s["table"], pos, pos, base=s["base"])
        dtable = pba.pba_relpos_bias_backward(bias, pos, pos, 33)
        h, y = pba.pba_block_norm_forward(s["x"], s["f"], pre=(s["w"], None))
        back = pba.pba_block_norm_backward(h, y, y, s["f"], pre=(s["w"], None))
        return [out, lse, *grads, bias, dtable, h, y, *(t for t in back if t is not None)]

    alone = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    results = [[] for _ in sets]
    for _ in range(6):
        for i, (s, stream) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(stream):
                results[i].append(run(s))
    torch.cuda.synchronize()
    for want, many in zip(alone, results):
        for got in many:
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert pba.pba_last_device_error() == pba.PBA_OK
