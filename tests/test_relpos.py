"""pba_relpos_bias_forward and pba_relpos_bias_backward: refusals (CPU), and on the GPU
the gathered values, the sum with a base and the table's gradient against the
fp64 reference.

Bounds.  Without a base the output is the table's own value, bit for bit.  With
one it is one fp32 sum (2^-24 relative) rounded to the output's type (half a
step).  The table's gradient is added in fp32 by threads that take eight keys of
at most 512 queries each, so a word of a thread's receives at most 8 min(512,
Nq) values one by one (and once each of the sums kept in registers, three
additions deep); then come four such words and five shuffles per block, 64-bit
sums beyond, and the result's own rounding.  With u = 2^-24 the error is below
(8 min(512, Nq) + 16) u times the sum of the magnitudes."""
import ctypes

import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: each call below fails its checks first


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    return pba.load_library()


def _desc(**kw):
    d = pba.PbaRelposDesc()
    d.B, d.H, d.Nq, d.Nk, d.dtype, d.rows = 1, 4, 16, 16, pba.PBA_BF16, 9
    for k, v in kw.items():
        setattr(d, k, v)
    return d


LOG, CAUSAL = pba.PBA_RELPOS_LOG, pba.PBA_RELPOS_LOG_CAUSAL


@pytest.mark.parametrize("kw,expect", [
    ({"B": 0}, pba.PBA_ERR_INVALID_ARG),
    ({"H": 70000}, pba.PBA_ERR_INVALID_ARG),
    ({"Nq": -1}, pba.PBA_ERR_INVALID_ARG),
    ({"Nk": 1 << 31}, pba.PBA_ERR_INVALID_ARG),
    ({"B": 3, "Nq": 1 << 30}, pba.PBA_ERR_INVALID_ARG),
    ({"dtype": 5}, pba.PBA_ERR_UNSUPPORTED),
    ({"rule": 3}, pba.PBA_ERR_INVALID_ARG),
    ({"rows": 8}, pba.PBA_ERR_INVALID_ARG),                                     # clip: an even number of buckets
    ({"rows": 2000}, pba.PBA_ERR_UNSUPPORTED),
    ({"rule": LOG, "rows": 9, "max_distance": 128}, pba.PBA_ERR_INVALID_ARG),   # both sides: an odd number
    ({"rule": LOG, "rows": 2, "max_distance": 128}, pba.PBA_ERR_INVALID_ARG),
    ({"rule": LOG, "rows": 32, "max_distance": 8}, pba.PBA_ERR_INVALID_ARG),    # not past the exact distances
    ({"rule": CAUSAL, "rows": 32, "max_distance": (1 << 30) + 1}, pba.PBA_ERR_INVALID_ARG),
    ({"rule": CAUSAL, "rows": 1, "max_distance": 128}, pba.PBA_ERR_INVALID_ARG),
])
def test_rejects_bad_descriptors(lib, kw, expect):
    d = _desc(**kw)
    assert lib.pba_relpos_bias_forward(ctypes.byref(d), FAKE, FAKE, None, None, FAKE, None, FAKE, None) == expect
    assert lib.pba_relpos_bias_backward(ctypes.byref(d), FAKE, FAKE, None, None, FAKE, FAKE, FAKE, 1 << 40,
                                    None) == expect


def test_rejects_nulls_alignment_and_small_workspaces(lib):
    d = _desc()
    p = ctypes.byref(d)
    bad = pba.PBA_ERR_INVALID_ARG
    odd = ctypes.c_void_p(0x10001)
    assert lib.pba_relpos_bias_forward(None, FAKE, FAKE, None, None, FAKE, None, FAKE, None) == bad
    for i in (0, 1, 4, 6):  # q_pos, k_pos, table, out
        for value in (None, odd):
            args = [FAKE, FAKE, None, None, FAKE, None, FAKE]
            args[i] = value
            assert lib.pba_relpos_bias_forward(p, *args, None) == bad
    d.rows = 10  # one group array alone
    assert lib.pba_relpos_bias_forward(p, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, None) == bad
    d.rows = 9
    need = ctypes.c_int64()
    assert lib.pba_relpos_bias_backward_workspace(p, ctypes.byref(need)) == pba.PBA_OK and need.value > 0
    assert lib.pba_relpos_bias_backward_workspace(p, None) == bad
    assert lib.pba_relpos_bias_backward(p, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, need.value - 1, None) == bad
    for i in (0, 1, 4, 5, 6):
        args = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE]
        args[i] = None
        assert lib.pba_relpos_bias_backward(p, *args, need.value, None) == bad


def test_empty_forward_writes_nothing(lib):
    assert lib.pba_relpos_bias_forward(ctypes.byref(_desc(Nq=0)), None, None, None, None, None, None, None,
                                   None) == pba.PBA_OK


# ------------------------------------------------------------------ GPU
def _positions(g, B, n, spread):
    """Sorted with gaps, or anywhere in +-spread."""
    if spread:
        return torch.randint(-spread, spread + 1, (B, n), generator=g, dtype=torch.int32)
    return (1 + (torch.rand((B, n), generator=g) < 0.1).int() * 6).cumsum(1).int()


CASES = [
    # B, H, Nq, Nk, rule, buckets, far, groups, spread
    (1, 1, 1, 1, "clip", 1, 0, False, 0),
    (1, 3, 1, 77, "log_causal", 32, 128, False, 0),
    (2, 4, 33, 65, "clip", 65, 0, True, 0),
    (3, 5, 19, 40, "log", 32, 128, True, 200),
    (1, 2, 130, 520, "log", 8, 64, False, 0),
    (2, 16, 64, 8, "clip", 9, 0, True, 4),
    (1, 7, 50, 1031, "log", 64, 1024, False, 2000),
    (1, 2, 9, 31, "log_causal", 2, 5, False, 7),
    (1, 2, 40, 24, "clip", 1023, 0, True, 600),   # the widest table
    (2, 1, 25, 16, "log", 4, 3, False, 9),
]


def _grad_bound(mag, Nq):
    return (8 * min(512, Nq) + 16) * 2 ** -24 * mag


def _make(case, dtype, device, seed=0):
    B, H, Nq, Nk, rule, buckets, far, groups, spread = case
    g = torch.Generator().manual_seed(seed)
    q_pos, k_pos = _positions(g, B, Nq, spread), _positions(g, B, Nk, spread)
    q_group = torch.randint(0, 3, (B, Nq), generator=g, dtype=torch.int32) if groups else None
    k_group = (torch.arange(Nk) * 3 // Nk).int().expand(B, Nk).contiguous() if groups else None
    rows = buckets + groups
    table = torch.randn((rows, H), generator=g).to(dtype)
    cpu = (q_pos, k_pos, q_group, k_group)
    index = R.relpos_rows(q_pos, k_pos, rows, rule, far, q_group, k_group)
    return table.to(device), [None if t is None else t.to(device) for t in cpu], index, rows, g


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_forward(cuda_device, case, dtype):
    B, H, Nq, Nk, rule, _, far, _, _ = case
    table, (q, k, qg, kg), index, rows, g = _make(case, dtype, cuda_device)
    out = pba.pba_relpos_bias_forward(table, q, k, rule, far, qg, kg)
    assert torch.equal(out.double().cpu(), R.relpos_bias(table, index).expand(B, H, Nq, Nk))
    base = torch.randn((B, H, Nq, Nk), generator=g).to(dtype).to(cuda_device)
    ref = R.relpos_bias(table, index, base)
    got = pba.pba_relpos_bias_forward(table, q, k, rule, far, qg, kg, base=base)
    half = torch.finfo(dtype).eps / 2
    bound = (half + 2 ** -24) * ref.abs() + (2 ** -24 * (ref - d_base(base)).abs())
    assert ((got.double().cpu() - ref).abs() <= bound).all()
    # the base itself as output
    again = pba.pba_relpos_bias_forward(table, q, k, rule, far, qg, kg, base=base, out=base)
    assert again is base and torch.equal(base, got)


def d_base(base):
    return base.double().cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_table_gradient(cuda_device, case, dtype):
    B, H, Nq, Nk, rule, _, far, _, _ = case
    table, (q, k, qg, kg), index, rows, g = _make(case, dtype, cuda_device, seed=1)
    dbias = torch.randn((B, H, Nq, Nk), generator=g).to(dtype).to(cuda_device)
    got = pba.pba_relpos_bias_backward(dbias, q, k, rows, rule, far, qg, kg)
    ref, mag = R.relpos_table_grad(dbias, index, rows)
    assert got.dtype == torch.float32 and tuple(got.shape) == (rows, H)
    assert ((got.double().cpu() - ref).abs() <= _grad_bound(mag, Nq)).all()
    assert torch.equal(got, pba.pba_relpos_bias_backward(dbias, q, k, rows, rule, far, qg, kg))


@pytest.mark.gpu
def test_long_columns_and_shared_positions(cuda_device):
    """A batch that shares one position row, many queries (several splits), strided matrices."""
    B, H, Nq, Nk, rows = 2, 3, 1500, 264, 33
    g = torch.Generator().manual_seed(5)
    pos = _positions(g, 1, Nq, 0)[0]
    q, k = pos.cuda(), pos[:Nk].cuda()
    index = R.relpos_rows(pos, pos[:Nk], rows, "clip", 0)
    wide = torch.randn((H, B, Nq, Nk + 24), generator=g).to(torch.bfloat16).cuda()
    dbias = wide[..., 8:8 + Nk].transpose(0, 1)
    got = pba.pba_relpos_bias_backward(dbias, q, k, rows)
    ref, mag = R.relpos_table_grad(dbias, index, rows)
    assert ((got.double().cpu() - ref).abs() <= _grad_bound(mag, Nq)).all()
    odd = wide[..., 3:3 + Nk].transpose(0, 1)  # not on 16 bytes: element by element
    ref, mag = R.relpos_table_grad(odd, index, rows)
    assert ((pba.pba_relpos_bias_backward(odd, q, k, rows).double().cpu() - ref).abs() <= _grad_bound(mag, Nq)).all()
    # forward into a window of a larger matrix: what lies around it stays
    table = torch.randn((rows, H), generator=g).to(torch.bfloat16).cuda()
    for at in (8, 3):
        field = torch.full((1, H, Nq, Nk + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        pba.pba_relpos_bias_forward(table, q, k, out=field[..., at:at + Nk])
        assert torch.equal(field[..., at:at + Nk].double().cpu(), R.relpos_bias(table, index))
        assert (field[..., :at] == 7).all() and (field[..., at + Nk:] == 7).all()


@pytest.mark.gpu
def test_positions_at_the_ends_of_int32(cuda_device):
    lo, hi = -2 ** 31, 2 ** 31 - 1
    pos = torch.tensor([lo, lo + 1, -1, 0, 1, hi - 1, hi], dtype=torch.int32)
    for rule, rows, far in (("clip", 5, 0), ("log", 32, 128), ("log_causal", 16, 1 << 30)):
        table = torch.randn((rows, 2), generator=torch.Generator().manual_seed(1)).cuda()
        index = R.relpos_rows(pos, pos, rows, rule, far)
        out = pba.pba_relpos_bias_forward(table, pos.cuda(), pos.cuda(), rule, far)
        assert torch.equal(out.double().cpu(), R.relpos_bias(table, index))
        dbias = torch.randn((1, 2, 7, 7), generator=torch.Generator().manual_seed(2)).cuda()
        ref, mag = R.relpos_table_grad(dbias, index, rows)
        got = pba.pba_relpos_bias_backward(dbias, pos.cuda(), pos.cuda(), rows, rule, far).double().cpu()
        assert ((got - ref).abs() <= _grad_bound(mag, 7)).all()


@pytest.mark.gpu
def test_every_border_of_the_logarithmic_rule(cuda_device):
    for rows, far in ((32, 128), (64, 1024), (16, 37), (128, 65536), (1024, 1 << 20), (34, 300)):
        side = rows // 2
        ds = sorted({d + o for b in (R_border(side, far, t) for t in range(1, side - side // 2)) for d in (b,)
                     for o in (-1, 0, 1) if d + o >= 0})
        k = torch.tensor(ds, dtype=torch.int32)
        table = torch.arange(rows, dtype=torch.float32)[:, None].contiguous().cuda()
        out = pba.pba_relpos_bias_forward(table, torch.zeros(1, dtype=torch.int32, device="cuda"), (-k).cuda(), "log",
                                      far)
        want = torch.tensor([R.log_row(d, side, far) for d in ds]).double()
        assert torch.equal(out.reshape(-1).double().cpu(), want)


def R_border(side, far, t):
    e = side // 2
    return int(round(e * (far / e) ** (t / (side - e))))


@pytest.mark.gpu
def test_empty_gradient_is_zero(cuda_device):
    none = torch.zeros((0,), dtype=torch.int32, device="cuda")
    some = torch.zeros((4,), dtype=torch.int32, device="cuda")
    for q, k in ((none, some), (some, none)):
        dbias = torch.zeros((1, 2, q.numel(), k.numel()), device="cuda")
        assert (pba.pba_relpos_bias_backward(dbias, q, k, 5) == 0).all()
        assert pba.pba_relpos_bias_forward(torch.zeros((5, 2), device="cuda"), q, k).numel() == 0


@pytest.mark.gpu
def test_other_stream_and_captured(cuda_device):
    case = CASES[2]
    B, H, Nq, Nk, rule, _, far, _, _ = case
    table, (q, k, qg, kg), index, rows, g = _make(case, torch.bfloat16, cuda_device, seed=3)
    dbias = torch.randn((B, H, Nq, Nk), generator=g).cuda()
    want = pba.pba_relpos_bias_forward(table, q, k, rule, far, qg, kg), pba.pba_relpos_bias_backward(dbias, q, k, rows, rule,
                                                                                             far, qg, kg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (pba.pba_relpos_bias_forward(table, q, k, rule, far, qg, kg, stream=side),
           pba.pba_relpos_bias_backward(dbias, q, k, rows, rule, far, qg, kg, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):  # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = (pba.pba_relpos_bias_forward(table, q, k, rule, far, qg, kg),
                 pba.pba_relpos_bias_backward(dbias, q, k, rows, rule, far, qg, kg))
        graphs.append((graph, r))
    for graph, r in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, r in graphs:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


@pytest.mark.gpu
def test_binding_refuses(cuda_device):
    table = torch.zeros((5, 2), device="cuda")
    pos = torch.zeros((4,), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_forward(table, pos.long(), pos)
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_forward(table, pos.cpu(), pos)
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_forward(table, pos, pos, "nearest")
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_forward(table, pos, pos, q_group=pos)
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_forward(table, pos, pos, base=torch.zeros((1, 2, 4, 5), device="cuda"))
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_forward(table.half(), pos, pos)
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_backward(torch.zeros((2, 2, 4, 4), device="cuda"), pos.expand(3, 4), pos, 5)
    with pytest.raises(pba.PbaError):
        pba.pba_relpos_bias_forward(table[:4].contiguous(), pos, pos)
