"""pba_block_norm_forward and pba_block_norm_backward: refusals (CPU), and on the GPU
every combination of gate, scale and norms against the fp64 definition (its
gradients by autograd).

Bounds, with u = 2^-24, half = half a step of the type, C channels.  A row sum
in fp32 is eight terms per thread, at most five shuffles and five more over the
warps: 8 + 10 additions, so the mean is off by at most 18 u max|v|, the mean
square by 2 * 19 u of itself, its root by half that (plus 2 u for rsqrtf).  A
normalised value is then off by at most 18 u max|v| rs + 24 u |v_hat|; times
the weight, plus three more roundings: 64 u (max|v| rs + |v_hat|) |w| covers
it, and the gate's exponential and quotient (8 u on the sigmoid, more where
|gate| is large: |gate| u in the exponent) add (16 + 2 |gate|) u.  The written value adds
half a step of its type.

A gradient through a norm is three such terms, each bounded by rs times the
largest |w dy| of the row times (1 + |v_hat|): 128 u rs (1 + max|v_hat|)^2
max|w dy| covers them with the statistics' own errors (max|v| rs enters as the
size of an uncentred value).  Sums over rows: each thread adds at most rows /
(rows in flight) + the block's rows terms in fp32, so (rows + 64) u times the
sum of magnitudes covers them for the small row counts here, the terms' own
errors (128 u relative to their magnitudes) included."""
import ctypes
import itertools

import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: each call below fails its checks first
U = 2.0 ** -24


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    return pba.load_library()


def _desc(**kw):
    d = pba.PbaNormDesc()
    d.rows, d.C, d.eps = 4, 64, 1e-5
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,expect", [
    ({"rows": -1}, pba.PBA_ERR_INVALID_ARG),
    ({"C": 0}, pba.PBA_ERR_INVALID_ARG),
    ({"C": 8193}, pba.PBA_ERR_UNSUPPORTED),
    ({"dtype": 9}, pba.PBA_ERR_UNSUPPORTED),
    ({"param_dtype": 9}, pba.PBA_ERR_UNSUPPORTED),
    ({"kind": 2}, pba.PBA_ERR_INVALID_ARG),
    ({"eps": 0.0}, pba.PBA_ERR_INVALID_ARG),
    ({"eps": float("nan")}, pba.PBA_ERR_INVALID_ARG),
    ({"eps": float("inf")}, pba.PBA_ERR_INVALID_ARG),
])
def test_rejects_bad_descriptors(lib, kw, expect):
    d = _desc(**kw)
    assert lib.pba_block_norm_forward(ctypes.byref(d), *([FAKE] * 10), None) == expect
    assert lib.pba_block_norm_backward(ctypes.byref(d), *([FAKE] * 19), 1 << 40, None) == expect


def test_rejects_combinations_nulls_and_alignment(lib):
    d = ctypes.byref(_desc())
    bad = pba.PBA_ERR_INVALID_ARG
    names = ["x", "f", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b", "h", "y"]

    def fwd(**kw):
        return lib.pba_block_norm_forward(d, *[kw.get(n, FAKE) for n in names], None)

    assert lib.pba_block_norm_forward(None, *([FAKE] * 10), None) == bad
    assert fwd(x=None) == bad and fwd(h=None) == bad and fwd(y=None) == bad
    assert fwd(f=None) == bad                                       # a gate without a block
    assert fwd(f=None, gate=None, scale=None) == bad                # a norm after no block
    assert fwd(post_w=None) == bad and fwd(pre_w=None) == bad       # a bias without its weight
    none = dict(f=None, gate=None, scale=None, post_w=None, post_b=None, pre_w=None, pre_b=None)
    assert fwd(**none) == bad                                       # nothing to do
    for n in names:
        assert fwd(**{n: ctypes.c_void_p(0x10001)}) == bad
    need = ctypes.c_int64()
    assert lib.pba_block_norm_backward_workspace(d, ctypes.byref(need)) == pba.PBA_OK and need.value > 0
    assert lib.pba_block_norm_backward_workspace(d, None) == bad
    bn = ["h", "f", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b", "dh", "dy", "dx", "df", "dgate", "dscale",
          "dpost_w", "dpost_b", "dpre_w", "dpre_b", "work"]

    def bwd(size=need.value, **kw):
        return lib.pba_block_norm_backward(d, *[kw.get(n, FAKE) for n in bn], size, None)

    assert bwd(size=need.value - 1) == bad
    for n in ("h", "dy", "dx", "df", "dgate", "work"):
        assert bwd(**{n: None}) == bad
    for n in bn:
        assert bwd(**{n: ctypes.c_void_p(0x10001)}) == bad
    assert bwd(pre_w=None, pre_b=None, dh=None) == bad


def test_no_rows_forward(lib):
    d = _desc(rows=0)
    args = [None] * 10
    args[6] = FAKE
    assert lib.pba_block_norm_forward(ctypes.byref(d), *args, None) == pba.PBA_OK


# ------------------------------------------------------------------ GPU
def _inputs(rows, C, dtype, parts, kind, seed=0, param_dtype=None, mean=0.3):
    """x, f, gate, scale, post, pre (CPU), dh, dy; parts: which of post, gate, scale, pre, f there are."""
    g = torch.Generator().manual_seed(seed)
    pd = param_dtype or dtype

    def t(std=1.0, at=0.0):
        return (torch.randn((rows, C), generator=g) * std + at).to(dtype)

    def c(std, at):
        return (torch.randn((C,), generator=g) * std + at).to(pd)

    bias = kind == "layer"
    d = dict(x=t(2.0, mean), f=t() if "f" in parts else None, gate=t(1.5) if "gate" in parts else None,
             scale=c(0.3, 0.5) if "scale" in parts else None,
             post=(c(0.2, 1.0), c(0.1, 0.0) if bias else None) if "post" in parts else None,
             pre=(c(0.2, 1.0), c(0.1, 0.0) if bias else None) if "pre" in parts else None)
    return d, t(), t()


def _cuda(d):
    return {k: (tuple(None if e is None else e.cuda() for e in v) if isinstance(v, tuple)
                else None if v is None else v.cuda()) for k, v in d.items()}


def _d64(d):
    return {k: (tuple(R.d64(e) for e in v) if isinstance(v, tuple) else R.d64(v)) for k, v in d.items()}


def _norm_err(v, params, kind, eps):
    """64 u (max|v| rs + |v_hat|) |w| of one norm, and rs, v_hat."""
    c = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    rs = (c.square().mean(-1, keepdim=True) + eps).rsqrt()
    big = v.abs().amax(-1, keepdim=True) * rs
    err = 64 * U * (big + (c * rs).abs()) * params[0].abs()
    return (err if params[1] is None else err + 2 * U * params[1].abs()), rs, c * rs, big


def _check_forward(d, kind, eps, h, y):
    r = _d64(d)
    ref_h, ref_y = R.block(r["x"], r["f"], r["gate"], r["scale"], r["post"], r["pre"], kind, eps)
    dtype = d["x"].dtype
    half = torch.finfo(dtype).eps / 2
    err = torch.zeros_like(ref_h)
    if r["f"] is not None:
        u = r["f"] if r["post"] is None else R.norm(r["f"], r["post"], kind, eps)
        err = torch.zeros_like(u) if r["post"] is None else _norm_err(r["f"], r["post"], kind, eps)[0]
        if r["gate"] is not None:
            s = torch.sigmoid(r["gate"])
            err = err * s + (u * s).abs() * (16 + 2 * r["gate"].abs()) * U
            u = u * s
        if r["scale"] is not None:
            err = err * r["scale"].abs()
            u = u * r["scale"]
        err = err + 4 * U * (u.abs() + r["x"].abs())
        assert ((R.d64(h) - ref_h).abs() <= err * (1 + half) + half * ref_h.abs() + 1e-37).all()
    if ref_y is not None:
        e, rs, _, _ = _norm_err(ref_h, r["pre"], kind, eps)
        # an error in h enters its own value, the mean and the mean square
        e = e + 3 * err.amax(-1, keepdim=True) * rs * r["pre"][0].abs() * (1 + (ref_y.abs()).amax(-1, keepdim=True))
        assert ((R.d64(y) - ref_y).abs() <= e * (1 + half) + half * ref_y.abs() + 1e-37).all()


PARTS = [p for p in (("f",) + tuple(n for n, on in zip(("post", "gate", "scale", "pre"), bits) if on)
                     for bits in itertools.product((0, 1), repeat=4))] + [("pre",)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("parts", PARTS, ids=lambda p: "-".join(p))
def test_every_combination(cuda_device, parts, kind, dtype):
    for rows, C in ((5, 64), (3, 300)):
        d, dh, dy = _inputs(rows, C, dtype, parts, kind)
        c = _cuda(d)
        h, y = pba.pba_block_norm_forward(**c, kind=kind)
        assert (y is None) == ("pre" not in parts) and (h is c["x"]) == ("f" not in parts)
        _check_forward(d, kind, 1e-5, h, y)
        _check_backward(d, dh, dy, kind, 1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("parts", [p for p in PARTS if "pre" in p and "scale" not in p], ids=lambda p: "-".join(p))
def test_sets_of_parts_over_many_rows(cuda_device, parts, kind, dtype):
    """The sets of parts whose gradients have kernels of their own and the others, with several rows to a thread and a
    ragged end: rows that share a block, and rows of a block."""
    for rows, C in ((20001, 64), (1500, 512)):
        d, dh, dy = _inputs(rows, C, dtype, parts, kind, seed=rows)
        _check_backward(d, dh, dy, kind, 1e-5)


SHAPES = [(1, 1), (1, 8), (7, 100), (300, 128), (33, 256), (5, 257), (9, 384), (2, 768), (3, 1021), (2, 4096),
          (3, 4100), (2, 8192), (1000, 24)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_shapes(cuda_device, rows, C, dtype):
    parts = ("f", "post", "gate", "scale", "pre")
    for kind in ("layer", "rms"):
        d, dh, dy = _inputs(rows, C, dtype, parts, kind, seed=C)
        c = _cuda(d)
        h, y = pba.pba_block_norm_forward(**c, kind=kind, eps=1e-3)
        _check_forward(d, kind, 1e-3, h, y)
        _check_backward(d, dh, dy, kind, 1e-3)


def _check_backward(d, dh, dy, kind, eps, h=None):
    """Against autograd in fp64 from the stored h."""
    dtype = d["x"].dtype
    half = torch.finfo(dtype).eps / 2
    h = d["x"] if h is None else h
    c = _cuda(d)
    pre, post = d["pre"] is not None, d["post"] is not None
    got = pba.pba_block_norm_backward(h.cuda(), dh.cuda(), dy.cuda() if pre else None, c["f"], c["gate"], c["scale"],
                                  c["post"], c["pre"], kind, eps)
    r = _d64(d)
    h64, t = R.d64(h), R.d64(dh)
    terr = 2 * U * t.abs()
    rows = h64.shape[0]
    if pre:
        w, b = r["pre"]
        hv = h64.clone().requires_grad_()
        wv = w.clone().requires_grad_()
        out = R.norm(hv, (wv, b), kind, eps)
        gx, gw = torch.autograd.grad(out, (hv, wv), R.d64(dy))
        t = t + gx
        _, rs, v, big = _norm_err(h64, r["pre"], kind, eps)
        m = (w * R.d64(dy)).abs().amax(-1, keepdim=True)
        terr = terr + 128 * U * rs * (1 + v.abs().amax(-1, keepdim=True) + big) ** 2 * m + 4 * U * t.abs()
        mag = (R.d64(dy).abs() * (v.abs() + big)).sum(0)
        assert ((R.d64(got[6]) - gw).abs() <= (rows + 192) * U * mag).all()
        if b is not None:
            assert ((R.d64(got[7]) - R.d64(dy).sum(0)).abs() <= (rows + 64) * U * R.d64(dy).abs().sum(0)).all()
        else:
            assert got[7] is None
    else:
        assert got[6] is None and got[7] is None
    assert ((R.d64(got[0]) - t).abs() <= terr * (1 + half) + half * t.abs()).all()
    if d["f"] is None:
        assert got[1] is None and got[2] is None and got[3] is None
        return
    f = r["f"]
    leaves = [f, r["gate"], r["scale"], *(r["post"] or (None, None))]
    leaves = [None if x is None else x.clone().requires_grad_() for x in leaves]
    out = R.block(torch.zeros_like(f), leaves[0], leaves[1], leaves[2], (leaves[3], leaves[4]) if post else None,
                  None, kind, eps)[0]
    grads = torch.autograd.grad(out, [x for x in leaves if x is not None], t)
    grads = iter(grads)
    df, dg, ds, dpw, dpb = (None if x is None else next(grads) for x in leaves)
    s = torch.sigmoid(r["gate"]) if r["gate"] is not None else torch.ones_like(f)
    sc = r["scale"].abs() if r["scale"] is not None else torch.ones(f.shape[-1]).double()
    u, uerr = f, 2 * U * f.abs()
    if post:
        u = R.norm(f, r["post"], kind, eps)
        uerr, rs, v, big = _norm_err(f, r["post"], kind, eps)
    gate_rel = (16 + 2 * r["gate"].abs()) * U if r["gate"] is not None else torch.zeros_like(f)
    # relative errors of t s sc, and the errors of t and u themselves
    da = (t * s).abs() * sc
    daerr = da * (gate_rel + 8 * U) + terr * s * sc
    if dg is not None:
        e = (t.abs() * sc * s * (1 - s)) * (uerr + u.abs() * (2 * gate_rel + 16 * U)) + terr * sc * s * u.abs()
        # 1 - s carries an absolute error of s gate_rel + u
        e = e + t.abs() * sc * s * u.abs() * (s * gate_rel + 2 * U)
        assert ((R.d64(got[2]) - dg).abs() <= e * (1 + half) + half * dg.abs() + 1e-37).all()
    if ds is not None:
        e = ((t * s).abs() * uerr + (t * s * u).abs() * (gate_rel + 8 * U) + terr * s * u.abs()).sum(0)
        assert ((R.d64(got[3]) - ds).abs() <= e + (rows + 64) * U * (t * s * u).abs().sum(0)).all()
    else:
        assert got[3] is None
    if post:
        e = (da * 64 * U * (big + v.abs()) + daerr * v.abs()).sum(0) + (rows + 64) * U * (da * v.abs()).sum(0)
        assert ((R.d64(got[4]) - dpw).abs() <= e).all()
        if dpb is not None:
            assert ((R.d64(got[5]) - dpb).abs() <= daerr.sum(0) + (rows + 64) * U * da.sum(0)).all()
        else:
            assert got[5] is None
        w = r["post"][0].abs()
        m = (da * w).amax(-1, keepdim=True)
        span = (1 + v.abs().amax(-1, keepdim=True) + big) ** 2
        e = rs * span * (128 * U * m + 3 * (daerr * w).amax(-1, keepdim=True))
        assert ((R.d64(got[1]) - df).abs() <= e * (1 + half) + half * df.abs() + 1e-37).all()
    else:
        assert got[4] is None and got[5] is None
        assert ((R.d64(got[1]) - df).abs() <= daerr * (1 + half) + half * df.abs() + 1e-37).all()


@pytest.mark.gpu
def test_large_mean_keeps_its_variance(cuda_device):
    """Values near 1000 with a spread of 1: the squares are taken around the mean."""
    d, dh, dy = _inputs(6, 128, torch.float32, ("f", "post", "pre"), "layer", seed=9, mean=1000.0)
    d["f"] = d["f"] + 500.0
    h, y = pba.pba_block_norm_forward(**_cuda(d), kind="layer")
    _check_forward(d, "layer", 1e-5, h, y)


@pytest.mark.gpu
def test_fp32_parameters_with_bf16_rows(cuda_device):
    for C in (128, 520):
        d, dh, dy = _inputs(6, C, torch.bfloat16, ("f", "post", "gate", "scale", "pre"), "layer", seed=2,
                            param_dtype=torch.float32)
        h, y = pba.pba_block_norm_forward(**_cuda(d), kind="layer")
        _check_forward(d, "layer", 1e-5, h, y)
        _check_backward(d, dh, dy, "layer", 1e-5, h=h.cpu())


@pytest.mark.gpu
def test_zero_and_huge_rows(cuda_device):
    x = torch.zeros((4, 96))
    x[1] = 1e18
    x[2, 3] = 1e15
    for kind in ("layer", "rms"):
        w = torch.ones(96)
        h, y = pba.pba_block_norm_forward(x.cuda(), pre=(w.cuda(), None), kind=kind)
        ref = R.norm(x.double(), (w.double(), None), kind, 1e-5)
        assert torch.isfinite(y).all() and (y[0] == 0).all()
        # row 1 is constant: its exact layer norm is 0, and 18 u 1e18 off the mean is all that rounding can leave
        rows = [0, 2, 3] if kind == "layer" else [0, 1, 2, 3]
        assert ((y.double().cpu() - ref)[rows].abs() <= 64 * U * (1 + ref[rows].abs()) * 10).all()


@pytest.mark.gpu
def test_row_strides_views_and_in_place(cuda_device):
    d, dh, dy = _inputs(12, 72, torch.bfloat16, ("f", "post", "gate", "pre"), "rms", seed=4)
    c = _cuda(d)
    h, y = pba.pba_block_norm_forward(**c, kind="rms")
    wide = torch.full((4, 3, 100), 5.0, dtype=torch.bfloat16, device="cuda")
    for at in (8, 5):  # rows on 16 bytes, and not
        view = wide[..., at:at + 72]
        view.copy_(c["x"].view(4, 3, 72))
        h2, y2 = pba.pba_block_norm_forward(view, c["f"].view(4, 3, 72), c["gate"].view(4, 3, 72), None, c["post"],
                                        c["pre"], "rms", h=view)
        assert h2 is view and torch.equal(view.reshape(12, 72), h) and torch.equal(y2.reshape(12, 72), y)
        assert (wide[..., :at] == 5).all() and (wide[..., at + 72:] == 5).all()
        wide.fill_(5.0)
    with pytest.raises(ValueError):
        pba.pba_block_norm_forward(c["x"].view(4, 3, 72).transpose(0, 1), pre=c["pre"])
    g1 = pba.pba_block_norm_backward(h, dh.cuda(), dy.cuda(), c["f"], c["gate"], None, c["post"], c["pre"], "rms")
    pad = torch.zeros((12, 80), dtype=torch.bfloat16, device="cuda")
    pad[:, :72] = dy.cuda()
    g2 = pba.pba_block_norm_backward(h, dh.cuda(), pad[:, :72], c["f"], c["gate"], None, c["post"], c["pre"], "rms")
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(g1, g2))


@pytest.mark.gpu
def test_no_residual_gradient_no_rows_and_only_pre(cuda_device):
    d, dh, dy = _inputs(5, 64, torch.float32, ("f", "pre"), "layer", seed=6)
    c = _cuda(d)
    a = pba.pba_block_norm_backward(c["x"], None, dy.cuda(), c["f"], None, None, None, c["pre"])
    b = pba.pba_block_norm_backward(c["x"], torch.zeros_like(dh).cuda(), dy.cuda(), c["f"], None, None, None, c["pre"])
    assert all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))
    none = torch.zeros((0, 64), device="cuda")
    h, y = pba.pba_block_norm_forward(none, none, pre=c["pre"])
    assert h.shape == (0, 64) and y.shape == (0, 64)
    g = pba.pba_block_norm_backward(none, none, none, none, None, None, None, c["pre"])
    assert (g[6] == 0).all() and (g[7] == 0).all()


@pytest.mark.gpu
def test_repeatable_other_stream_and_captured(cuda_device):
    d, dh, dy = _inputs(3000, 128, torch.bfloat16, ("f", "post", "gate", "scale", "pre"), "layer", seed=8)
    c = _cuda(d)
    dh, dy = dh.cuda(), dy.cuda()

    def both(stream=None):
        h, y = pba.pba_block_norm_forward(**c, stream=stream)
        return (h, y, *pba.pba_block_norm_backward(h, dh, dy, c["f"], c["gate"], c["scale"], c["post"], c["pre"],
                                               stream=stream))

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


@pytest.mark.gpu
def test_gradient_against_differences(cuda_device):
    """The kernel's gradients against differences of the fp64 definition along one direction.  The fp32 sums behind the
    directional derivative are each within 1e-5 of exact (see the bounds above); the difference itself is good to
    about eps^2."""
    d, dh, dy = _inputs(40, 96, torch.float32, ("f", "post", "gate", "scale", "pre"), "layer", seed=12)
    c = _cuda(d)
    r = _d64(d)
    g = torch.Generator().manual_seed(1)
    flat = [r["x"], r["f"], r["gate"], r["scale"], *r["post"], *r["pre"]]
    dirs = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in flat]

    def loss(x, f, gate, scale, pw, pb, nw, nb):
        h, y = R.block(x, f, gate, scale, (pw, pb), (nw, nb), "layer", 1e-5)
        return (h * R.d64(dh)).sum() + (y * R.d64(dy)).sum()

    eps = 1e-5
    diff = (loss(*[t + eps * v for t, v in zip(flat, dirs)]) - loss(*[t - eps * v for t, v in zip(flat, dirs)])) / (2 * eps)
    h, _ = pba.pba_block_norm_forward(**c)
    grads = pba.pba_block_norm_backward(h, dh.cuda(), dy.cuda(), c["f"], c["gate"], c["scale"], c["post"], c["pre"])
    parts = [(R.d64(a) * v) for a, v in zip(grads, dirs)]
    got, mag = sum(p.sum() for p in parts), sum(p.abs().sum() for p in parts)
    assert abs(got - diff) <= 1e-5 * mag
