"""GPU checks of the expert operators at the edges of their groups, ranges and handles."""
import pytest
import torch

from test_gpu_experts import _setup, check_wgrad, group  # noqa: F401  (_setup: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,k", [(136, 264), (520, 200)])
def test_wgrad_clears_what_lies_behind_every_group(n, k, dtype):
    """Each remainder of a group's rows modulo 64, in short groups and behind full
    blocks of 64, with NaN in the rows that follow: the lines that both CTAs of a
    pair clear before the products read them, the same bits every time."""
    counts = list(range(0, 65)) + [64 * b + r for b in (1, 3, 9) for r in (1, 15, 16, 17, 31, 32, 47, 48, 63)]
    buf, h, grp = group(counts, padded=True)
    first = check_wgrad(buf, h, grp, n, k, dtype)
    for _ in range(3):
        assert torch.equal(check_wgrad(buf, h, grp, n, k, dtype), first)
