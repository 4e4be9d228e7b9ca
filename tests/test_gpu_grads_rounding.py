"""GPU checks of the gradients' norm and factor to the last rounding, and at both ends of fp32's range.

Whole numbers' squares add up exactly, in fp32 and fp64, so what is left is the kernel's own: the root and the
quotient are good to 2^-44 and each is rounded once, 2^-24 of it."""
import math
import random

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer
from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from test_gpu_grads import NORM, check, norm_of

pytestmark = pytest.mark.gpu

ONCE = 2.0 ** -24 * (1 + 2.0 ** -16)
F32, B16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def buf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    epbuild.build()
    torch.cuda.set_device(0)
    return Buffer(1, 1, 128, 1, 1)


@pytest.mark.parametrize("two", [False, True])      # in place, or into another tensor
def test_norm_and_factor_are_rounded_once(buf, two):
    """1, 2 and 4 times the factor are the factor's own bits: off by one rounding at most."""
    r = random.Random(5)
    for _ in range(300):
        n = [r.randint(1, 5000) for _ in range(3)]
        flat = torch.zeros(sum(n) + 2, device="cuda")
        g = flat[:sum(n)]
        g[:n[0]], g[n[0]:n[0] + n[1]], g[n[0] + n[1]:] = 1.0, 2.0, -4.0
        total = n[0] + 4 * n[1] + 16 * n[2]
        limit = float(torch.tensor(math.sqrt(total) * math.exp(r.uniform(-40.0, 0.0)), dtype=F32))
        if limit >= math.sqrt(total):
            continue
        out = torch.empty_like(g) if two else g
        norm = float(buf.clip_grads([g], limit, out=[out] if two else None))
        assert abs(norm - math.sqrt(total)) <= ONCE * math.sqrt(total), (n, norm)
        exact = limit / math.sqrt(total)
        for i, v in ((0, 1.0), (n[0], 2.0), (n[0] + n[1], -4.0)):
            assert abs(float(out[i]) - v * exact) <= ONCE * abs(v) * exact, (n, limit, float(out[i]), v * exact)


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("scale", [1e-42, 1e-40, 1e-36, 3e35, 5e36, 9e36])
def test_norms_at_both_ends_of_the_range(buf, dtype, scale):
    """Down to subnormal values, and norms of 1e37 to 3.2e38: finite, and clipped."""
    grads = [torch.full((1000,), scale, device="cuda", dtype=dtype), torch.full((9,), scale * 5, device="cuda", dtype=dtype)]
    want = norm_of(grads)
    assert want < 3.4e38      # 0 for 1e-42 in bf16, whose smallest number is 9.2e-41
    if scale > 1e-37:
        check(buf, [g.clone() for g in grads], want * 0.5)
        return
    # subnormal numbers are rounded to 2^-149 (bf16: 2^-133)
    kept = [g.clone() for g in grads]
    norm = buf.clip_grads(grads, want * 0.5)
    assert abs(float(norm) - want) <= NORM * want + 2.0 ** -149
    factor = float(torch.tensor(want * 0.5, dtype=F32)) / want if want else 1.0
    for g, k in zip(grads, kept):
        step = 2.0 ** -149 if dtype == F32 else 2.0 ** -133
        assert bool(((g.double() - k.double() * factor).abs() <= step).all())


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("scale", [1.2e37, 3e37, 3e38])
def test_finite_values_whose_norm_passes_the_range_are_not_scaled(buf, dtype, scale):
    grads = [torch.full((1000,), scale, device="cuda", dtype=dtype), torch.full((9,), scale, device="cuda", dtype=dtype)]
    assert norm_of(grads) > 3.5e38 and all(bool(g.isfinite().all()) for g in grads)
    kept, out = [g.clone() for g in grads], [torch.zeros_like(g) for g in grads]
    for to in (out, None):
        assert float(buf.clip_grads(grads, 1.0, out=to)) == math.inf
        for g, k, o in zip(grads, kept, out):
            assert torch.equal(g, k) and torch.equal(o, k)
    assert ep.ep_get_device_status(buf.ctx) == ep.EP_OK
