"""The 2-norm bounds see a lost term where the bounds per value do not (CPU)."""
import pytest
import torch

from expert_reference import BF16, sum_bound
from norm_bounds import bf16_bound, relative


@pytest.mark.parametrize("k", [512, 7168])
def test_a_lost_term_is_seen(k):
    gen = torch.Generator().manual_seed(k)
    x, w = (torch.randn(n, k, generator=gen).bfloat16() for n in (48, 64))
    want = x.double() @ w.double().T
    assert relative((x.float() @ w.float().T).bfloat16(), want) <= bf16_bound(k)
    for lost in (0, k // 2, k - 1):
        keep = torch.arange(k) != lost
        bad = (x[:, keep].double() @ w[:, keep].double().T).bfloat16()
        assert relative(bad, want) > 2.0 * bf16_bound(k)
    if k == 7168:       # the bound per value sees the same mistake only where the term is a large one
        tol = BF16 * want.abs() + sum_bound(k, x.double().abs() @ w.double().abs().T)
        assert float(((bad.double() - want).abs() <= tol).double().mean()) > 0.9
