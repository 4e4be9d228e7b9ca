"""GPU checks of the expert operators at the edges of their groups, ranges and handles."""
import ctypes
import time

import pytest
import torch

from combine_get_dispatch_02_gb300 import ep
from expert_reference import (BF16, assert_close, cast_blocks, cast_rows, in_use, receive, silu, weights, wide_block,
                              wide_rows)
from norm_bounds import bf16_bound, fp32_bound, relative
from test_gpu_experts import _setup, check_wgrad, done, group, sentinel  # noqa: F401  (_setup: the module's fixture)

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


@pytest.mark.parametrize("counts", [[3, 0, 40], [300, 700]])
def test_gate_is_good_to_24_bits_however_far_out(counts):
    """One gate value per block of 128 channels, the others zero: the block's scale is
    |h| / 448 in fp32.  exp is good to 1 ulp, 1 + e, g e and u to half a one, the
    division to 2 and the scale to half: 5 ulp of 2^-23, below 2^-20.  The last gates
    are past the range where a fast division by 1 + exp(-g) gives 0."""
    gates = [-1.0, -6.5, -12.0, -20.0, -26.0, -44.0, -60.0, -72.0, -80.0, -88.0, 1.0, 20.0, 60.0, 88.0]
    buf, h, _ = group(counts)
    E, inner = len(counts), 128 * len(gates)
    g = torch.tensor(gates, dtype=torch.float64)
    up = 2.0 ** (1 - silu(g).abs().log2().ceil())     # so that h lies between 1 and 4
    want = (silu(g) * up).abs().cuda()
    xq = torch.zeros(buf.rows, 128, device="cuda")
    xq[:, 0] = 1.0
    wq, ws = torch.zeros(E, 2 * inner, 128, device="cuda"), torch.ones(E, 2 * len(gates), 1, device="cuda")
    wq[:, 0:inner:128, 0] = g.float().cuda()
    wq[:, inner::128, 0] = 1.0
    ws[:, len(gates):, 0] = up.float().cuda()
    fp8 = torch.float8_e4m3fn
    hq, hs = buf.expert_gate_fp8((xq.to(fp8), torch.ones(buf.rows, 1, device="cuda")), (wq.to(fp8), ws), h)
    done(buf)
    assert_close(hs * 448.0, want.expand_as(hs), 2.0 ** -20 * want, "scales")
    assert bool((hq[:, ::128].float() == 448.0 * torch.sign(g.float()).cuda()).all())


def test_swiglu_far_out_with_large_factors():
    """Gates where exp(-g) overflows in fp32 while h and its gradient do not.  exp(g)
    is subnormal there, good to half of 2^-149; everything else to a few ulp."""
    gates = [-30.0, -60.0, -87.0, -88.5, -89.0, -92.0, -95.0, -98.0, 30.0, 60.0, 89.0, 98.0]
    g = torch.tensor(gates, dtype=torch.float64).cuda()
    u = torch.where(g < 0, 2.0 ** 100, 1.5)
    dh = torch.where(g < 0, 2.0 ** 30, 0.75)         # u dh alone is past fp32's range
    pad = torch.zeros(4, dtype=torch.float64, device="cuda")
    row = torch.cat((g, pad, u, pad)).bfloat16().expand(5, -1).contiguous()
    buf, h, _ = group([2, 3])
    out = buf.expert_swiglu(row, h)
    dgu, again = buf.expert_swiglu_backward(row, torch.cat((dh, pad)).bfloat16().expand(5, -1).contiguous(), h)
    done(buf)
    assert torch.equal(out, again)
    s, low = torch.sigmoid(g), 2.0 ** -149 * (1.0 + g.abs()) * u
    want = silu(g) * u
    assert_close(out[:, :12], want.expand(5, -1), (BF16 + 2.0 ** -19) * want.abs() + low, "h")
    want = dh * silu(g)
    assert_close(dgu[:, 16:28], want.expand(5, -1), (BF16 + 2.0 ** -19) * want.abs() + low / u * dh, "du")
    want = dh * u * s * (1 + g * (1 - s))
    assert_close(dgu[:, :12], want.expand(5, -1), (BF16 + 2.0 ** -19) * want.abs() + low * dh, "dg")


def held_by_captured_calls(h, want, seconds=10.0):
    """The captured calls' tile counters once they are ``want``: a graph's objects go
    on a thread of the driver's."""
    end = time.monotonic() + seconds
    while (n := ep.ep_get_test_counters(h.raw)[1]) != want and time.monotonic() < end:
        time.sleep(0.01)
    return n


def test_captured_calls_give_their_counters_back():
    """A program that captures its step again and again: every call of a graph that
    exists holds a counter, none does when the graphs are gone, and a graph that is
    destroyed while it runs keeps its counters until it has run."""
    buf, h, grp = group([300, 0, 17, 640, 128, 1, 77, 256] * 4)
    used = in_use(buf.rows, grp)
    x, w = receive(buf.rows, 256, grp, 1), weights(32, 2048, 256, 2)
    want, out = buf.expert_gemm(x, w, h), sentinel((buf.rows, 2048))
    torch.cuda.synchronize()
    for _ in range(4):      # 6000 calls in all
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(1500):
                buf.expert_gemm(x, w, h, out=out)
        assert ep.ep_get_test_counters(h.raw)[1] == 1500
        out.fill_(0)
        g.replay()
        done(buf)
        assert torch.equal(out[used], want[used])
        del g
        assert held_by_captured_calls(h, 0) == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(1500):
            buf.expert_gemm(x, w, h, out=out)
    for _ in range(4):
        g.replay()
    ran = torch.cuda.Event()
    ran.record()
    del g
    early = ep.ep_get_test_counters(h.raw)[1], ran.query()
    done(buf)
    assert early[1] or early[0] == 1500
    assert held_by_captured_calls(h, 0) == 0


def test_more_streams_than_counters():
    """Past the counters for streams the tiles come in a fixed order, with the same bits."""
    buf, h, grp = group([300, 0, 17, 640, 128, 1, 77, 256])
    used = in_use(buf.rows, grp)
    x, w = receive(buf.rows, 256, grp, 1), weights(8, 2560, 256, 2)
    want, out = buf.expert_gemm(x, w, h), sentinel((buf.rows, 2560))
    rt = torch.cuda.cudart()
    for _ in range(520):
        raw = ctypes.c_void_p()
        assert int(rt.cudaStreamCreate(ctypes.addressof(raw))) == 0
        out.fill_(0)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.ExternalStream(raw.value)):
            buf.expert_gemm(x, w, h, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out[used], want[used])
        assert int(rt.cudaStreamDestroy(raw.value)) == 0
    assert ep.ep_get_test_counters(h.raw)[0] == 512
    done(buf)


@pytest.mark.parametrize("sms", [1, 2, 3])
def test_products_on_one_pair_of_sms(sms):
    """The products take SMs in pairs, one pair at least: the same bits as on all."""
    counts = [0, 1, 31, 300, 700, 64]
    outs = []
    for n in (0, sms):
        buf, h, grp = group(counts, max_sms=n)
        x, w = receive(buf.rows, 256, grp, 1), weights(6, 512, 256, 2)
        outs.append((buf.expert_gemm(x, w, h)[in_use(buf.rows, grp)], buf.expert_wgrad(x, x, h)))
        done(buf)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# rows per expert of a long sum: a few (the FP8 products' column form), many (their row form)
LONG = [[33, 0, 130], [300, 520]]


@pytest.mark.parametrize("counts", LONG)
@pytest.mark.parametrize("op", ["gemm", "dgrad", "fp8"])
def test_long_sums_lose_no_term(op, counts):
    """k = 7168 in the 2-norm of each row and column of the result, where one lost
    term is three times the bound (see norm_bounds)."""
    n, k = 264, 7168
    buf, h, grp = group(counts)
    x = receive(buf.rows, k, grp, 1)
    if op == "fp8":
        xq, wq = cast_rows(x.float()), cast_blocks(weights(len(counts), n, k, 2))
        y = buf.expert_gemm_fp8(xq, wq, h)
        operands = lambda e, r: (wide_rows(xq[0][r], xq[1][r]), wide_block(wq[0][e], wq[1][e]))  # noqa: E731
    else:
        w = weights(len(counts), *((k, n) if op == "dgrad" else (n, k)), 2)
        y = buf.expert_gemm(x, w, h, transpose_w=op == "dgrad")
        operands = lambda e, r: (x[r].double(), (w[e].T if op == "dgrad" else w[e]).double())  # noqa: E731
    done(buf)
    for e, (b, c) in enumerate(grp):
        if c:
            xe, we = operands(e, slice(b, b + c))
            assert relative(y[b:b + c], xe @ we.T) <= bf16_bound(k), e


@pytest.mark.parametrize("rows", [7168, 7201])
def test_long_sums_over_rows_lose_no_row(rows):
    buf, h, grp = group([rows])
    dy, x = receive(buf.rows, 136, grp, 1), receive(buf.rows, 264, grp, 2)
    want = dy.double().T @ x.double()
    dw = buf.expert_wgrad(dy, x, h)
    dw16 = buf.expert_wgrad(dy, x, h, out=torch.empty(1, 136, 264, dtype=torch.bfloat16, device="cuda"))
    done(buf)
    assert relative(dw[0], want) <= fp32_bound(rows)
    assert relative(dw16[0], want) <= bf16_bound(rows)


@pytest.mark.parametrize("counts", LONG)
def test_gate_over_long_sums_loses_no_term(counts):
    """The scales of h, which are in fp32: a gate and an up sum off by k / 16 * 2^-23
    each and a gate's slope of 1.1 at most give 2^-12; a lost term is 1.2e-2."""
    inner, k = 256, 7168
    buf, h, grp = group(counts)
    xq, wq = cast_rows(receive(buf.rows, k, grp, 1).float()), cast_blocks(weights(len(counts), 2 * inner, k, 2))
    _, hs = buf.expert_gate_fp8(xq, wq, h)
    done(buf)
    for e, (b, c) in enumerate(grp):
        if c:
            v = wide_rows(xq[0][b:b + c], xq[1][b:b + c]) @ wide_block(wq[0][e], wq[1][e]).T
            want = (silu(v[:, :inner]) * v[:, inner:]).view(c, -1, 128).abs().amax(2) / 448
            assert relative(hs[b:b + c], want) <= 2.0 ** -12, e
