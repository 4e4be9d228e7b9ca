"""GPU checks of the gradients' norm and clipping against 64 bits.

Tolerances: a thread's 16 or 32 squares are summed in fp32 (32 roundings of 2^-24 of the sum, half of that in
the root: 2^-20), everything else in fp64; the factor is rounded once, the product once, bf16 results once more."""
import math

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer
from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from expert_reference import BF16, assert_close

pytestmark = pytest.mark.gpu

NORM = 2.0 ** -20 + 2.0 ** -23
F32, B16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def buf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    epbuild.build()
    torch.cuda.set_device(0)
    return Buffer(1, 1, 128, 1, 1)


def tensors(sizes, types, seed=0, scale=1.0, offset=0):
    """Views of larger buffers whose neighbours are sentinels; offset: elements past an aligned address."""
    g = torch.Generator("cuda").manual_seed(seed)
    whole, views = [], []
    for i, n in enumerate(sizes):
        dtype = types[i % len(types)]
        b = torch.full((n + offset + 24,), 333.0, device="cuda", dtype=dtype)
        v = b[offset:offset + n]
        v.copy_(torch.randn(n, generator=g, device="cuda") * scale * 10.0 ** -(i % 3))
        whole.append(b)
        views.append(v)
    return whole, views


def norm_of(ts):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))


def check(buf, grads, max_norm, out=None, whole=(), norm_want=None):
    kept = [g.clone() for g in grads]
    want = norm_of(kept) if norm_want is None else norm_want
    norm = buf.clip_grads(grads, max_norm, out=out)
    got = float(norm)
    assert abs(got - want) <= NORM * want, (got, want)
    coef = min(1.0, max_norm / want) if want else 1.0
    for i, (g, o) in enumerate(zip(kept, grads if out is None else out)):
        exact = g.double() * coef
        if coef == 1.0:
            assert torch.equal(o, g)
        else:
            rel = NORM + 2.0 ** -23 + (BF16 if g.dtype == B16 else 2.0 ** -24)
            assert_close(o, exact, rel * exact.abs() + 2.0 ** -133, f"tensor {i}")
    for b, g in zip(whole, grads if out is None else out):
        at = (g.data_ptr() - b.data_ptr()) // b.element_size()
        edge = torch.cat([b[:at], b[at + g.numel():]])
        assert bool((edge == 333.0).all()), "a neighbour was written"
    return got


SIZES = [[1], [0, 1, 0], [7, 8, 9], [4096, 4095, 4097], [8192, 1, 8193, 16383], [100003, 0, 65536, 31], [3_000_001]]


@pytest.mark.parametrize("types", [[F32], [B16], [B16, F32]])
@pytest.mark.parametrize("offset", [0, 1, 3, 5])
@pytest.mark.parametrize("sizes", SIZES)
def test_clip_in_place(buf, sizes, types, offset):
    whole, grads = tensors(sizes, types, offset=offset)
    check(buf, grads, 0.3 * norm_of(grads), whole=whole)


@pytest.mark.parametrize("types", [[F32], [B16], [F32, B16]])
@pytest.mark.parametrize("offsets", [(0, 0), (1, 1), (0, 1), (3, 2)])
@pytest.mark.parametrize("limit", [0.3, 2.0])
def test_clip_to_other_tensors(buf, types, offsets, limit):
    sizes = [33, 0, 10007, 8192, 70001]
    _, grads = tensors(sizes, types, offset=offsets[0])
    whole, out = tensors(sizes, types, seed=5, offset=offsets[1])
    kept = [g.clone() for g in grads]
    check(buf, grads, limit * norm_of(grads), out=out, whole=whole)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


@pytest.mark.parametrize("count", [32, 33, 128, 129, 384, 385, 1024, 1025, 2500])
def test_many_tensors(buf, count):
    """One table, a larger one, several."""
    flat = torch.full((count * 70,), 0.0, device="cuda", dtype=B16).normal_(generator=torch.Generator("cuda").manual_seed(count))
    grads = [flat[70 * i:70 * i + 1 + i % 70] for i in range(count)]
    check(buf, grads, 0.5 * norm_of(grads))


def test_large_and_uneven(buf):
    whole, grads = tensors([1 << 26, 5, (1 << 25) + 3, 1000], [F32, B16], offset=1)
    check(buf, grads, 0.01 * norm_of(grads), whole=whole)


def test_more_than_32_bits_of_elements(buf):
    """2^32 + 9 bf16 elements in one tensor: what lies past 32 bits counts."""
    n = (1 << 32) + 9
    g = torch.zeros(n, device="cuda", dtype=B16)
    g[0], g[-1], g[n - 9] = 3.0, 4.0, 12.0
    norm = buf.clip_grads([g], 6.5)
    assert float(norm) == 13.0
    assert float(g[0]) == 1.5 and float(g[-1]) == 2.0 and float(g[n - 9]) == 6.0
    del g
    torch.cuda.empty_cache()


@pytest.mark.parametrize("types", [[F32], [B16]])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-19, 1e19, 3e37])
def test_squares_neither_overflow_nor_vanish(buf, types, scale):
    """Values whose squares fp32 does not hold (2e38 at the most, so that the norm is finite)."""
    grads = [torch.full((1000,), scale, device="cuda", dtype=types[0]), torch.full((9,), scale * 5, device="cuda", dtype=types[0])]
    want = norm_of(grads)
    if want < 3e38:
        check(buf, grads, want * 0.5)


def test_mixed_magnitudes(buf):
    grads = [torch.tensor([1e-30] * 100 + [1.0], device="cuda"), torch.full((5000,), 1e-25, device="cuda")]
    assert float(buf.clip_grads(grads, 1e9)) == 1.0


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [F32, B16])
def test_a_norm_that_is_not_finite_scales_nothing(buf, value, dtype):
    grads = [torch.randn(5000, device="cuda").to(dtype), torch.randn(77, device="cuda").to(dtype)]
    grads[1][13] = value
    kept, out = [g.clone() for g in grads], [torch.zeros_like(g) for g in grads]
    assert not math.isfinite(float(buf.clip_grads(grads, 1e-3, out=out)))
    assert not math.isfinite(float(buf.clip_grads(grads, 1e-3)))
    for g, k, o in zip(grads, kept, out):
        assert torch.equal(g.nan_to_num(9.0), k.nan_to_num(9.0)) and torch.equal(o.nan_to_num(9.0), k.nan_to_num(9.0))


def test_limits_zero_and_infinity(buf):
    grads = [torch.randn(1000, device="cuda"), torch.randn(31, device="cuda").bfloat16()]
    kept = [g.clone() for g in grads]
    norm = buf.clip_grads(grads, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept)) and abs(float(norm) - norm_of(kept)) <= NORM * float(norm)
    buf.clip_grads(grads, 0.0)
    assert all(bool((g == 0).all()) for g in grads)
    assert float(buf.clip_grads(grads, 0.0)) == 0.0 and all(bool((g == 0).all()) for g in grads)
    assert float(buf.clip_grads([], 1.0)) == 0.0


def test_below_the_limit_nothing_is_written(buf):
    """In place and within the limit: bits stay, NaN payloads and all neighbours too."""
    whole, grads = tensors([5000, 77, 12345], [B16, F32], offset=1)
    kept = [b.clone() for b in whole]
    buf.clip_grads(grads, 2 * norm_of(grads))
    assert all(torch.equal(a, b) for a, b in zip(whole, kept))


def test_repeats_and_works_in_graphs_on_two_streams(buf):
    sets = [tensors([40000, 3, 999], [B16, F32], seed=s)[1] for s in (1, 2)]
    outs = [[torch.zeros_like(g) for g in s] for s in sets]
    limits = [0.5 * norm_of(s) for s in sets]
    first = [buf.clip_grads(s, m, out=o).clone() for s, m, o in zip(sets, limits, outs)]
    want = [[t.clone() for t in o] for o in outs]
    graphs, norms = [], []
    torch.cuda.synchronize()
    for s, m, o in zip(sets, limits, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(buf.clip_grads(s, m, out=o))
        graphs.append(g)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for n, f, o, w in zip(norms, first, outs, want):
            assert torch.equal(n, f) and all(torch.equal(a, b) for a, b in zip(o, w))


def test_the_norm_of_two_processes(buf):
    """Partial sums added up between the calls: both sides clip by the norm of all tensors."""
    parts = [tensors([1000, 77], [F32], seed=s)[1] for s in (1, 2)]
    want = norm_of(parts[0] + parts[1])
    sums = []
    for ts in parts:
        p = torch.full((ep.EP_GRAD_PARTIALS,), 1e30, dtype=torch.float64, device="cuda")
        ep.ep_grad_norm(buf.ctx, ep.grad_list(ts), p)
        sums.append(p)
    total = sums[0] + sums[1]
    for ts in parts:
        kept = [t.clone() for t in ts]
        norm = torch.zeros(1, device="cuda")
        ep.ep_grad_clip(buf.ctx, ep.grad_list(ts), total, 0.25 * want, norm)
        assert abs(float(norm) - want) <= NORM * want
        for t, k in zip(ts, kept):
            assert_close(t, k.double() * 0.25, (NORM + 2.0 ** -22) * k.double().abs(), "scaled")


def test_max_sms(buf):
    _, grads = tensors([100000, 5], [B16])
    want = norm_of(grads)
    for sms in (1, 5, 152):
        small = Buffer(1, 1, 128, 1, 1, max_sms=sms)
        assert abs(float(small.clip_grads(grads, math.inf)) - want) <= NORM * want


def test_many_short_ctas_and_few_long_ones_clip_alike(buf):
    # 150 MB into other tensors: more CTAs than fit at a time, and with 7 SMs a few that go through all
    gen = torch.Generator(device="cuda").manual_seed(9)
    grads = [torch.randn(n, device="cuda", generator=gen).to(t) for n, t in ((30_000_001, torch.float32), (77, B16), (15_000_003, B16))]
    want = norm_of(grads)
    partials = torch.empty(ep.EP_GRAD_PARTIALS, dtype=torch.float64, device="cuda")
    ep.ep_grad_norm(buf.ctx, ep.grad_list(grads), partials)
    outs = []
    for b in (buf, Buffer(1, 1, 128, 1, 1, max_sms=7)):
        out, norm = [torch.full_like(g, math.nan) for g in grads], torch.zeros(1, device="cuda")
        ep.ep_grad_clip(b.ctx, ep.grad_list(grads, out), partials, 0.25 * want, norm)
        assert abs(float(norm) - want) <= NORM * want
        outs.append(out)
    for g, a, b in zip(grads, *outs):
        assert torch.equal(a, b)
        # the factor's own errors as above, and the rounding of the result
        rel = NORM + 2.0 ** -22 + torch.finfo(g.dtype).eps / 2
        assert_close(a, g.double() * 0.25, rel * g.double().abs() * 0.25 * 1.01, "scaled")


def test_refusals(buf):
    a, b = torch.ones(100, device="cuda"), torch.ones(100, device="cuda", dtype=B16)
    for grads, out in (([a.cpu()], None), ([a.view(10, 10).T], None), ([a.half()], None), ([a, b], [a]), ([a], [b]), ([a], [a[:50]])):
        with pytest.raises(ValueError):
            buf.clip_grads(grads, 1.0, out=out)
    for grads, out in (([a, a], None), ([a, a[50:]], None), ([a[:60], a[50:]], None), ([a[:50]], [a[10:60]]),
                       ([a[:50], a[50:]], [a[50:], a[:50]])):
        with pytest.raises(ep.EPError) as e:
            buf.clip_grads(grads, 1.0, out=out)
        assert e.value.status == ep.EP_ERR_INVALID_ARG
    for limit in (-1.0, math.nan):
        with pytest.raises(ep.EPError) as e:
            buf.clip_grads([a], limit)
        assert e.value.status == ep.EP_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((a == 1).all()) and bool((b == 1).all())
