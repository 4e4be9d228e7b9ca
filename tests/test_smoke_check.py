"""The smoke run's check of the FP8 experts, on the CPU: what it lets through and what not."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import __graft_entry__ as entry  # noqa: E402
from expert_reference import cast_rows, wide_rows  # noqa: E402


@pytest.fixture
def experts():
    gen = torch.Generator().manual_seed(3)
    h = torch.randn(40, 256, generator=gen) * 10.0 ** torch.linspace(-9, 3, 40)[:, None]   # the smallest under the scale's floor
    w = torch.randn(96, 256, generator=gen) / 16.0
    return (wide_rows(*cast_rows(h)).float() @ w.T).bfloat16().float(), h, w


def test_the_cast_of_the_rows_is_let_through(experts):
    assert entry.experts_agree(*experts)


@pytest.mark.parametrize("row,col,value", [(5, 7, float("nan")), (5, slice(None), float("nan")), (5, slice(None), 0.0),
                                           (39, slice(None), 0.0), (slice(None), 7, 0.0), (30, 11, float("inf"))])
def test_one_wrong_value_row_or_channel_is_not(experts, row, col, value):
    y, h, w = experts
    y[row, col] = value
    assert not entry.experts_agree(y, h, w)
