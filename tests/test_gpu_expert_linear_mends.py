"""GPU checks of the epilogue's backward pass where its bounds of 8 bits do not look."""
import pytest
import torch

from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from expert_reference import in_use, receive
from test_gpu_expert_linear import ACTS, group

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
