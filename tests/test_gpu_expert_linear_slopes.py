"""GPU checks of the epilogue's backward pass where its bounds of 8 bits do not look."""
import pytest
import torch

from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from expert_reference import in_use, receive
from test_gpu_expert_linear import ACTS, group, slope64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    epbuild.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("act", ACTS[1:])
def test_a_nan_in_z_is_not_hidden(act):
    """It is NaN in the forward pass: dz there and the channel's bias gradient are too, and nothing else changes."""
    buf, h, grp = group([5, 40, 0, 300])
    n = 72
    dy, z = receive(buf.rows, n, grp, 1), receive(buf.rows, n, grp, 2)
    dz, db = buf.expert_linear_backward(dy, z, h, activation=act)
    spots = [(0, 0, 0), (7, 71, 1), (44, 9, 1), (45, 8, 3), (344, 33, 3)]     # row, channel, expert
    bad = z.clone()
    for r, c, _ in spots:
        bad[r, c] = float("nan")
    dz2, db2 = buf.expert_linear_backward(dy, bad, h, activation=act)
    used = in_use(buf.rows, grp)
    hit, hit_db = torch.zeros_like(dz, dtype=torch.bool), torch.zeros_like(db, dtype=torch.bool)
    for r, c, e in spots:
        hit[r, c], hit_db[e, c] = True, True
    assert bool(dz2[hit].isnan().all()) and bool(db2[hit_db].isnan().all())
    assert torch.equal(dz2[used][~hit[used]], dz[used][~hit[used]]) and torch.equal(db2[~hit_db], db[~hit_db])
    assert buf.device_status() == ep.EP_OK


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_of_bias_gradients_are_good_to_32_bits(act):
    """dy = 1 and one row: the bias gradient is the slope as it is added up, before dz's rounding.

    The slopes (1.13 at most) come out of at most eight roundings and approximations of numbers of that size or
    less, each off by 2^-24 at most where it is a rounding and 2^-23 or 2^-22 of itself where it is the fast reciprocal or
    exponential (whose factor is half or less): spread evenly, 2^-24 / sqrt(3) and as much for those, of which numbers
    below 1/2 make a half or less, so in the root of the mean square sqrt(8) * 2^-24 / sqrt(3) * 0.6 = 2^-24, and
    6 * 2^-24 at most for any."""
    buf, h, _ = group([1])
    g = torch.Generator("cuda").manual_seed(3)
    for scale in (1.0, 3.0):
        z = (torch.randn(1, 65536, generator=g, device="cuda") * scale).bfloat16()
        _, db = buf.expert_linear_backward(torch.ones_like(z), z, h, activation=act)
        error = db[0].double() - slope64(z[0].double(), act)
        assert float(error.square().mean().sqrt()) <= 2.0 ** -24 and float(error.abs().max()) <= 6 * 2.0 ** -24
    assert buf.device_status() == ep.EP_OK
