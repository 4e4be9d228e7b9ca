"""2-norm bounds for long sums, beside the bounds per value.

A bound per value has to allow for every rounding going one way, which at k = 7168
is more than most of the sum's terms.  In the 2-norm of a row or a column a rounding
to bf16 (8 significand bits) is at most 2^-8 of it, and the sum's own error is small: k / 16 additions
in the tensor cores that drop less than 2^-23 of a partial sum each, partial sums
that are no larger than the result in the mean and go up and down with it, so
k / 16 * 2^-23 (5e-5 at k = 7168).  A lost term is 1 / sqrt(k) of the result
(1.2e-2 there)."""
import torch


def relative(got: torch.Tensor, want: torch.Tensor) -> float:
    """The largest relative 2-norm error of a row or column."""
    d = got.double() - want
    return max(float((d.norm(dim=i) / want.norm(dim=i)).max()) for i in (0, 1))


def bf16_bound(k: int) -> float:
    return 2.0 ** -8 + 2.0 * k / 16 * 2.0 ** -23


def fp32_bound(k: int) -> float:
    return 2.0 * k / 16 * 2.0 ** -23
