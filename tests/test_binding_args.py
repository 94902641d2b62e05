"""Whole numbers and scales that a descriptor's narrower field would change are
refused by the binding, not cut."""
import pytest
import torch

import pair_biased_attention_b200 as pba


def _relpos(rows, max_distance, rule="log"):
    pos = torch.zeros((4,), dtype=torch.int32)
    return pba._relpos_desc(rows, 2, torch.bfloat16, pos, pos, rule, max_distance, None, None)


@pytest.mark.parametrize("max_distance", [2 ** 32 + 128, 2 ** 31, -2 ** 32 + 128, 128.5, float("nan"), float("inf")])
def test_max_distance_is_not_cut(max_distance):
    with pytest.raises(ValueError):
        _relpos(32, max_distance)


@pytest.mark.parametrize("rows", [2 ** 32 + 33, 2 ** 31, -2 ** 32 + 33, 33.5])
def test_rows_are_not_cut(rows):
    with pytest.raises(ValueError):
        _relpos(rows, 0, "clip")


def test_whole_numbers_of_any_kind_are_taken():
    for v in (128, 128.0, torch.tensor(128)):
        d = _relpos(32, v)
        assert d.max_distance == 128 and d.rows == 32


@pytest.mark.parametrize("scale", [1e-50, -1e-50, 1e39])
def test_scale_outside_fp32(scale):
    """1e-50 as a float is 0, which stands for 1/sqrt(D)."""
    q, k = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 5, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pba._cross_desc(q, k, k, None, None, scale)
    assert pba._cross_desc(q, k, k, None, None, 0.5).softmax_scale == 0.5
    assert pba._cross_desc(q, k, k, None, None, None).softmax_scale == 0.0


@pytest.mark.gpu
def test_public_calls_refuse(cuda_device):
    table = torch.zeros((32, 2), device="cuda")
    pos = torch.zeros((4,), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_forward(table, pos, pos, "log", 2 ** 32 + 128)
    dbias = torch.zeros((1, 2, 4, 4), device="cuda")
    with pytest.raises(ValueError):
        pba.pba_relpos_bias_backward(dbias, pos, pos, 2 ** 32 + 33)
