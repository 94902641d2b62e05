"""The table's gradient takes every pair once, and its workspace is asked for
within the call's limits."""
import ctypes

import pytest
import torch

import block_ref as R
import pair_biased_attention_b200 as pba


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 3])  # rows on 16 bytes, and not
@pytest.mark.parametrize("B,H,Nq,Nk,rule,buckets,far,groups", [
    (1, 2, 1500, 264, "clip", 33, 0, True), (2, 1, 700, 1031, "log", 32, 128, False), (1, 3, 513, 40, "log_causal", 16, 64, True),
    (1, 1, 4100, 9, "clip", 1, 0, False), (3, 2, 65, 2000, "log", 64, 1024, True)])
def test_whole_numbers_are_exact(cuda_device, B, H, Nq, Nk, rule, buckets, far, groups, pad, dtype):
    """Sums below 2^24 come out exactly in any order: a pair left out or taken twice shows."""
    g = torch.Generator().manual_seed(Nq)
    q, k = (torch.randint(0, 1500, (B, n), generator=g, dtype=torch.int32).sort(-1)[0] for n in (Nq, Nk))
    qg, kg = ((torch.arange(n) * 3 // n).int().expand(B, n).contiguous() if groups else None for n in (Nq, Nk))
    rows = buckets + groups
    wide = torch.randint(-8, 9, (B, H, Nq, Nk + 13 - (Nk + 13) % 8 + 8), generator=g).to(dtype).cuda()
    dbias = wide[..., pad:pad + Nk]
    ref, _ = R.relpos_table_grad(dbias, R.relpos_rows(q, k, rows, rule, far, qg, kg), rows)
    got = pba.pba_relpos_bias_backward(dbias, *[None if t is None else t.cuda() for t in (q, k)], rows, rule, far,
                                       *[None if t is None else t.cuda() for t in (qg, kg)])
    assert torch.equal(got.double().cpu(), ref)


def test_workspace_of_a_problem_beyond_the_limits():
    """Where the number of partial tables passes 31 bits the backward refuses the call, and so does the question for its
    workspace, whose bytes would pass 64."""
    lib = pba.load_library()
    d = pba.PbaRelposDesc()
    d.B, d.H, d.Nq, d.Nk, d.dtype, d.rows = 65535, 65535, 32000, 2 ** 31 - 2 ** 21, pba.PBA_BF16, 1025
    need = ctypes.c_int64()
    assert lib.pba_relpos_bias_backward_workspace(ctypes.byref(d), ctypes.byref(need)) == pba.PBA_ERR_INVALID_ARG
    d.B = d.H = 1
    d.Nk = 4096
    assert lib.pba_relpos_bias_backward_workspace(ctypes.byref(d), ctypes.byref(need)) == pba.PBA_OK and need.value > 0
