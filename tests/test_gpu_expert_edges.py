"""GPU checks of the expert operators at the edges of their groups, ranges and handles."""
import pytest
import torch

from expert_reference import receive
from test_gpu_experts import _setup, check_wgrad, done, group  # noqa: F401  (_setup: the module's fixture)

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


@pytest.mark.parametrize("rows", [384, 1024, 6000])
def test_wgrad_in_fp32_drifts_no_more_than_an_fp32_product(rows):
    """Sums of equal sign.  An addition in the tensor cores drops half an ulp of the
    running sum on average, 0.72 * 2^-24 of it over all mantissas; 16 of them in a
    piece of 256 rows, whose sum grows evenly, 17 / 2 * 0.72 * 2^-24 = 3.7e-7.  The
    pieces' sums in fp32 add 24 random roundings at most, 1.5e-7.  Together (2-norm)
    below 2^-21, where pieces of 384 rows (5.4e-7) are not."""
    buf, h, grp = group([rows])
    dy, x = receive(buf.rows, 136, grp, 5).abs(), receive(buf.rows, 264, grp, 6).abs()
    dw = buf.expert_wgrad(dy, x, h)
    done(buf)
    want = dy.double().T @ x.double()
    assert float((dw[0].double() - want).norm() / want.norm()) < 2.0 ** -21
