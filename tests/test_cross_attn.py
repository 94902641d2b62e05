"""pba_cross_attn_forward and pba_cross_attn_backward: refusals (CPU), and on
the GPU outputs and gradients against the fp64 definition, element by element.

Bounds, u = 2^-24, half = 2^-8 (half a step of bf16).  A score is a chain of D
fp32 sums scaled once: off by at most E = (D + 8) u tau sum|q||k| + 2^-21, the
last term for the exponential unit and the subtraction of the maximum; a
probability then by 2 E of itself, plus half when it is rounded for the product
with V.  The sum of the probabilities is taken over them unrounded.  So
    |out - ref| <= (half + 3 E) sum_j P_j |v_j| + half |ref|
    |lse - ref| <= 2 E + (64 + Nk / 64) u + 4 u |ref|
and, dS rounded once, Delta from the rounded out,
    dS:  half |dS| + P (4 E (|dP| + |Delta|) + (D + 8) u sum|dout||v| + sum|dout| err(out))
    dq, dk: those sums times |k|, |q| and tau;  dv: (half + 4 E) sum P |dout|;
each plus half of itself for its own rounding."""
import ctypes
import math

import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: each call below fails its checks first
U, HALF = 2.0 ** -24, 2.0 ** -8


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    return pba.load_library()


def _desc(**kw):
    d = pba.PbaCrossDesc(1, 4, 2, 16, 16, 64, pba.PBA_BF16)
    for s, n in ((d.q_stride, 4), (d.out_stride, 4), (d.dout_stride, 4), (d.k_stride, 2), (d.v_stride, 2)):
        s[:] = (n * 16 * 64, 16 * 64, 64)
    d.lse_stride[:] = (64, 16, 1)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


BAD, UNSUP = pba.PBA_ERR_INVALID_ARG, pba.PBA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,expect", [
    ({"B": 0}, BAD), ({"H": 0}, BAD), ({"Hkv": 0}, BAD), ({"Hkv": 3}, BAD), ({"Nq": -1}, BAD), ({"Nk": 1 << 31}, BAD),
    ({"D": 48}, UNSUP), ({"dtype": pba.PBA_F32}, UNSUP),
    ({"softmax_scale": -1.0}, BAD), ({"softmax_scale": float("nan")}, BAD), ({"softmax_scale": float("inf")}, BAD),
    ({"q_stride": (4096, 1024, 60)}, BAD), ({"k_stride": (2048, 0, 64)}, BAD), ({"v_stride": (2048, 1024, -64)}, BAD),
    ({"out_stride": (4096, 1024, 68)}, BAD),
])
def test_rejects_bad_descriptors(lib, kw, expect):
    d = ctypes.byref(_desc(**kw))
    assert lib.pba_cross_attn_forward(d, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, None) == expect
    assert lib.pba_cross_attn_backward(d, *([FAKE] * 3), None, None, *([FAKE] * 7), None) == expect


def test_rejects_nulls_and_alignment(lib):
    d = ctypes.byref(_desc())
    assert lib.pba_cross_attn_forward(None, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, None) == BAD
    odd = ctypes.c_void_p(0x10002)
    for i in (0, 1, 2, 5):  # q, k, v, out
        for bad in (None, odd):
            args = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE]
            args[i] = bad
            assert lib.pba_cross_attn_forward(d, *args, None) == BAD
    for i in (3, 6):  # k_len, lse: only misaligned
        args = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE]
        args[i] = odd
        assert lib.pba_cross_attn_forward(d, *args, None) == BAD
    for i in (0, 1, 2, 5, 6, 7, 8, 9, 10, 11):
        for bad in (None, odd):
            args = [FAKE, FAKE, FAKE, None, None] + [FAKE] * 7
            args[i] = bad
            assert lib.pba_cross_attn_backward(d, *args, None) == BAD
    # a dout that tile loads cannot address
    d = ctypes.byref(_desc(dout_stride=(0, 0, 0)))
    assert lib.pba_cross_attn_backward(d, *([FAKE] * 3), None, None, *([FAKE] * 7), None) == BAD


def test_no_queries_forward(lib):
    assert lib.pba_cross_attn_forward(ctypes.byref(_desc(Nq=0)), *([None] * 7), None) == pba.PBA_OK


# ------------------------------------------------------------------ GPU
def _inputs(B, H, Hkv, Nq, Nk, D, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)

    def t(h, n):
        return (torch.randn((B, h, n, D), generator=g) * std).to(torch.bfloat16)

    return t(H, Nq), t(Hkv, Nk), t(Hkv, Nk), t(H, Nq), g


def _keep(B, Nk, k_len, mask):
    keep = torch.ones((B, Nk), dtype=torch.bool)
    if k_len is not None:
        keep &= torch.arange(Nk)[None, :] < k_len.cpu()[:, None]
    if mask is not None:
        keep &= mask.cpu() != 0
    return keep


def _check(q, k, v, dout, k_len=None, mask=None, scale=None, backward=True):
    """Both passes against the reference; returns what the kernels gave."""
    c = [None if t is None else t.cuda() for t in (k_len, mask)]
    qc, kc, vc = q.cuda(), k.cuda(), v.cuda()
    out, lse = pba.pba_cross_attn_forward(qc, kc, vc, *c, softmax_scale=scale)
    grads = pba.pba_cross_attn_backward(qc, kc, vc, out, lse, dout.cuda(), *c, softmax_scale=scale) if backward else ()
    torch.cuda.synchronize()
    assert pba.pba_last_device_error() == pba.PBA_OK
    _check_values(q, k, v, dout, _keep(q.shape[0], k.shape[2], k_len, mask), scale, out, lse, grads)
    return (out, lse, *grads)


def _check_values(q, k, v, dout, keep, scale, out, lse, grads):
    B, H, Nq, D = q.shape
    Hkv, Nk = k.shape[1:3]
    G = H // Hkv
    tau = scale or 1 / math.sqrt(D)
    zero = torch.zeros((), dtype=torch.float64)
    q64 = R.d64(q).requires_grad_()
    k64, v64 = (torch.where(keep[:, None, :, None], R.d64(t), zero).requires_grad_() for t in (k, v))
    ref, ref_lse = R.cross(q64, k64, v64, keep, scale)
    got, got_lse = R.d64(out), R.d64(lse)
    with torch.no_grad():
        kx, vx = k64.repeat_interleave(G, 1), v64.repeat_interleave(G, 1)
        some = torch.isfinite(ref_lse)
        s = (q64 @ kx.transpose(-1, -2)) * tau
        P = torch.where(keep[:, None, None, :] & some[..., None],
                        torch.exp(s - torch.where(some, ref_lse, zero)[..., None]), zero)
        A = (q64.abs() @ kx.abs().transpose(-1, -2)).amax(-1) * tau if Nk else torch.zeros_like(ref_lse)
        E = (D + 8) * U * A + 2.0 ** -21
        assert torch.equal(got_lse == -math.inf, ~some)
        lerr = 2 * E + (64 + Nk / 64) * U + 4 * U * torch.where(some, ref_lse.abs(), zero)
        assert ((got_lse - ref_lse)[some].abs() <= lerr[some]).all(), ((got_lse - ref_lse)[some].abs() - lerr[some]).max()
        oerr = (HALF + 3 * E[..., None]) * (P @ vx.abs()) + HALF * ref.abs()
        assert ((got - ref).abs() <= oerr).all(), ((got - ref).abs() - oerr).max()
        assert (got[~some] == 0).all()
    if not grads:
        return
    do = R.d64(dout)
    rq, rk, rv = torch.autograd.grad(ref, (q64, k64, v64), do)
    dq, dk, dv = (R.d64(t) for t in grads)
    with torch.no_grad():
        dP = do @ vx.transpose(-1, -2)
        delta = (do * ref).sum(-1, keepdim=True)
        dS = P * (dP - delta)
        E4 = 4 * E[..., None] + 2 * lerr[..., None]
        serr = HALF * dS.abs() + P * (E4 * (dP.abs() + delta.abs()) + (D + 8) * U * (do.abs() @ vx.abs().transpose(-1, -2))
                                      + (do.abs() * oerr).sum(-1, keepdim=True)) * (1 + HALF)

        def check(name, x, ref_x, err):
            err = err + HALF * ref_x.abs() + 1e-30
            assert ((x - ref_x).abs() <= err).all(), f"{name}: {((x - ref_x).abs() - err).max().item():.3e}"

        def grouped(t):
            return t.reshape(B, Hkv, G, Nk, D).sum(2)

        check("dq", dq, rq, tau * (serr @ kx.abs()))
        check("dk", dk, rk, grouped(tau * (serr.transpose(-1, -2) @ q64.abs())))
        check("dv", dv, rv, grouped(((HALF + E4) * P).transpose(-1, -2) @ do.abs()))
        assert (dk[(~keep)[:, None].expand(B, Hkv, Nk)] == 0).all()
        assert (dv[(~keep)[:, None].expand(B, Hkv, Nk)] == 0).all()


SHAPES = [
    # B, H, Hkv, Nq, Nk
    (1, 1, 1, 1, 1),
    (2, 4, 2, 1, 77),        # new tokens: keys split over blocks
    (2, 8, 2, 3, 1000),
    (1, 6, 6, 17, 129),
    (1, 4, 1, 16, 640),
    (2, 2, 1, 33, 5),
    (1, 3, 3, 65, 128),
    (2, 2, 2, 200, 300),
    (1, 4, 2, 257, 513),
    (1, 2, 1, 520, 64),
    (2, 8, 4, 1000, 2049),   # tiles, units shared by clusters
    (2, 8, 4, 513, 1000),
    (2, 16, 8, 600, 1000),   # tiles, a CTA to a unit
    (3, 32, 16, 520, 300),   # and several units to a CTA
]


def _forward_kernel(B, H, Hkv, Nq, Nk, D):
    """Which forward kernel the library's rule takes, so that the shapes here are known to reach each of them."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    units, tiles, s = B * H * up(Nq, 256), up(Nk, 128), 1
    while s < 8 and units * s * 2 <= 132 and tiles >= s * 4:
        s *= 2
    read = B * Hkv * up(H // Hkv * Nq, 16) * Nk * D * 4.0
    if read / 9e6 <= up(tiles, s) * up(units * s, 148) * (2.2 if D == 128 else 1.45) + 4:
        return "rows"
    return "clusters" if s > 1 else "tiles" if units <= 148 else "persistent"


def test_shapes_reach_every_forward_kernel():
    for D in (32, 64, 128):
        want = {"rows", "clusters", "tiles", "persistent"}
        assert {_forward_kernel(*s, D) for s in SHAPES} == want
        assert {_forward_kernel(*s, D) for s in MASKED} == {"rows", "clusters", "persistent"}
        assert {_forward_kernel(*s, D) for s in NANS} == {"rows", "clusters", "tiles"}
        assert _forward_kernel(*MANY, D) == "persistent"


MASKED = [(8, 4, 2, 2, 300), (8, 4, 2, 150, 300), (8, 2, 1, 1000, 1100), (8, 8, 2, 800, 300)]
NANS = [(2, 4, 4, 1, 333), (2, 4, 4, 300, 333), (2, 8, 4, 1000, 1303), (2, 16, 8, 600, 1000)]
MANY = (7, 16, 4, 600, 700)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_all_keys(cuda_device, shape, D):
    B, H, Hkv, Nq, Nk = shape
    q, k, v, dout, _ = _inputs(*shape, D, seed=Nq)
    _check(q, k, v, dout)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("shape", MASKED)
def test_lengths_and_masks(cuda_device, shape, D):
    """Lengths of 0, 1, inside and at the end of a tile, beyond Nk and below 0; masks that leave a sequence empty."""
    B, H, Hkv, Nq, Nk = shape
    q, k, v, dout, g = _inputs(B, H, Hkv, Nq, Nk, D, seed=D + Nq)
    k_len = torch.tensor([0, 1, 127, 128, 129, Nk, 5000, -3], dtype=torch.int32)
    mask = (torch.rand((B, Nk), generator=g) < 0.8).to(torch.uint8) * 3
    mask[4] = 0
    mask[5, :256] = 0  # whole tiles without a key, then some
    for args in ((k_len, None), (None, mask), (k_len, mask)):
        _check(q, k, v, dout, *args)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("shape", NANS)
def test_what_does_not_count_is_not_used(cuda_device, shape, D):
    """NaN and infinities behind the lengths and under the mask change no bit."""
    B, H, Hkv, Nq, Nk = shape
    q, k, v, dout, g = _inputs(B, H, Hkv, Nq, Nk, D, seed=7)
    k_len = torch.tensor([200, Nk], dtype=torch.int32)
    mask = (torch.rand((B, Nk), generator=g) < 0.7).to(torch.uint8)
    for args in ((k_len, None), (None, mask), (k_len, mask)):
        keep = _keep(B, Nk, *args)[:, None, :, None]
        want = _check(q, k, v, dout, *args)
        for bad in (math.nan, math.inf, torch.finfo(torch.bfloat16).min):
            fill = torch.tensor(bad, dtype=torch.bfloat16)
            got = _check(q, torch.where(keep, k, fill), torch.where(keep, v, fill), dout, *args)
            assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 4, 2, 3, 150), (2, 8, 4, 520, 1000), (2, 16, 8, 600, 700)])
def test_strides(cuda_device, shape):
    """Heads inside the token axis, padded rows, outputs given by the caller; what lies around an output stays."""
    (B, H, Hkv, Nq, Nk), D = shape, 64
    q, k, v, dout, _ = _inputs(B, H, Hkv, Nq, Nk, D, seed=3)
    want = _check(q, k, v, dout)

    def inside(t, pad):  # [B,h,n,D] as a view of [B, n, h + 1, D + pad]
        big = torch.zeros((t.shape[0], t.shape[2], t.shape[1] + 1, D + pad), dtype=t.dtype, device="cuda")
        view = big[:, :, :t.shape[1], :D].transpose(1, 2)
        view.copy_(t)
        return view

    qs, ks, vs, ds = inside(q, 8), inside(k, 16), inside(v, 0), inside(dout, 8)
    big = torch.full((B, Nq, H, D + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    out = big[..., :D].transpose(1, 2)
    lbig = torch.full((B, Nq, H + 1), 9.0, device="cuda")
    lse = lbig[..., :H].transpose(1, 2)
    o, l = pba.pba_cross_attn_forward(qs, ks, vs, out=out, lse=lse)
    assert o is out and l is lse and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (big[..., D:] == 9).all() and (lbig[..., H:] == 9).all()
    got = pba.pba_cross_attn_backward(qs, ks, vs, out, lse, ds)
    assert all(torch.equal(a, b) for a, b in zip(got, want[2:]))


@pytest.mark.gpu
@pytest.mark.parametrize("Nq,H", [(2, 2), (1500, 8), (2000, 40)])
def test_scales_and_large_scores(cuda_device, Nq, H):
    """A given scale, and scores far enough apart that rows keep one key (the running maximum is raised often)."""
    q, k, v, dout, _ = _inputs(1, H, H, Nq, 400, 64, seed=5, std=4.0)
    _check(q, k, v, dout)
    _check(q, k, v, dout, scale=1.0)
    _check(q, k, v, dout, scale=1e-3)
    # scores that rise tile by tile
    k = (torch.arange(400)[None, None, :, None] / 100.0 * torch.ones(1, H, 400, 64)).to(torch.bfloat16)
    q = torch.full((1, H, Nq, 64), 1.0, dtype=torch.bfloat16)
    _check(q, k, v, dout, scale=1.0)
    _check(-q, k, v, dout, scale=1.0)


@pytest.mark.gpu
def test_no_keys_and_no_queries(cuda_device):
    for Nq in (2, 200):
        q, k, v, dout, _ = _inputs(2, 4, 2, Nq, 0, 64)
        out, lse, dq, dk, dv = _check(q, k, v, dout, backward=False) + (None,) * 3
        dq, dk, dv = pba.pba_cross_attn_backward(q.cuda(), k.cuda(), v.cuda(), out, lse, dout.cuda())
        assert (dq == 0).all() and dk.numel() == 0 and dv.numel() == 0
    q, k, v, dout, _ = _inputs(2, 4, 2, 0, 50, 64)
    out, lse = pba.pba_cross_attn_forward(q.cuda(), k.cuda(), v.cuda())
    dq, dk, dv = pba.pba_cross_attn_backward(q.cuda(), k.cuda(), v.cuda(), out, lse, dout.cuda())
    assert (dk == 0).all() and (dv == 0).all() and dq.numel() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 16, 4, 1, 4096), (1, 8, 8, 700, 1500)])
def test_repeatable_other_stream_and_captured(cuda_device, shape):
    q, k, v, dout, g = _inputs(*shape, 64, seed=11)
    B, Nk = shape[0], shape[4]
    k_len = torch.tensor([Nk - 5 * b for b in range(B)], dtype=torch.int32).cuda()
    q, k, v, dout = (t.cuda() for t in (q, k, v, dout))

    def both(stream=None):
        o, l = pba.pba_cross_attn_forward(q, k, v, k_len, stream=stream)
        return (o, l, *pba.pba_cross_attn_backward(q, k, v, o, l, dout, k_len, stream=stream))

    want = both()
    assert all(torch.equal(a, b) for a, b in zip(want, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert pba.pba_last_device_error() == pba.PBA_OK


@pytest.mark.gpu
def test_many_units_walk_the_card(cuda_device):
    """More units than SMs, of different lengths, some empty: every ring and barrier phase runs on across units."""
    (B, H, Hkv, Nq, Nk), D = MANY, 64
    q, k, v, dout, g = _inputs(B, H, Hkv, Nq, Nk, D, seed=13)
    k_len = torch.tensor([700, 0, 130, 1, 0, 512, 333], dtype=torch.int32)
    _check(q, k, v, dout, k_len)


@pytest.mark.gpu
def test_gradient_against_differences(cuda_device):
    """dq, dk, dv along one direction against differences of the fp64 definition.  Each gradient element is within the
    bound of test_all_keys; 2^-6 of the sum of magnitudes covers those (half for P, dS, out and the result)."""
    q, k, v, dout, g = _inputs(2, 4, 2, 140, 200, 64, seed=17)
    keep = torch.ones((2, 200), dtype=torch.bool)
    flat = [R.d64(t) for t in (q, k, v)]
    dirs = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in flat]

    def loss(*a):
        return (R.cross(*a, keep)[0] * R.d64(dout)).sum()

    eps = 1e-5
    diff = (loss(*[t + eps * d for t, d in zip(flat, dirs)]) - loss(*[t - eps * d for t, d in zip(flat, dirs)])) / (2 * eps)
    c = [t.cuda() for t in (q, k, v)]
    out, lse = pba.pba_cross_attn_forward(*c)
    parts = [R.d64(t) * d for t, d in zip(pba.pba_cross_attn_backward(*c, out, lse, dout.cuda()), dirs)]
    assert abs(sum(p.sum() for p in parts) - diff) <= 2.0 ** -6 * sum(p.abs().sum() for p in parts)


@pytest.mark.gpu
def test_binding_refuses(cuda_device):
    q, k, v, dout, _ = (t.cuda() if torch.is_tensor(t) and t.dim() == 4 else t for t in _inputs(2, 4, 2, 8, 16, 64))
    with pytest.raises(ValueError):
        pba.pba_cross_attn_forward(q.cpu(), k, v)
    with pytest.raises(ValueError):
        pba.pba_cross_attn_forward(q, k[:, :, :8], v)
    with pytest.raises(ValueError):
        pba.pba_cross_attn_forward(q, k.float(), v)
    with pytest.raises(ValueError):
        pba.pba_cross_attn_forward(q, k, v, torch.tensor([3], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        pba.pba_cross_attn_forward(q, k, v, None, torch.ones((2, 16), device="cuda"))
    with pytest.raises(pba.PbaError):
        pba.pba_cross_attn_forward(q.float(), k.float(), v.float())
    with pytest.raises(pba.PbaError):
        pba.pba_cross_attn_forward(q[:, :3], k, v)
