"""GPU checks of the expert operators against plain 64-bit references."""
import ctypes

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer
from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from expert_reference import (BF16, assert_close, assert_untouched, cast_blocks, cast_rows, groups, in_use, receive,
                              silu, sum_bound, topk_for_counts, weights, wide_block, wide_rows)

pytestmark = pytest.mark.gpu

# rows per expert where a tile can go wrong: none, one, around 32 / 128 / 256 and past two tiles
EDGES = [0, 1, 31, 32, 33, 127, 128, 129, 0, 255, 256, 257, 520]
# n, k: below one tile, no tile divides them, exact tiles, long
SHAPES = [(8, 8), (24, 72), (136, 64), (264, 200), (256, 256), (1000, 328)]
# the same with many rows per expert on average, where the FP8 products put the rows on the other side
EDGES_MANY = [0, 1, 16, 17, 127, 128, 129, 0, 144, 255, 256, 257, 300, 520, 1000, 777]
SHAPES_FP8 = [(8, 128), (136, 256), (264, 384), (256, 128), (1000, 1152)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    epbuild.build()
    torch.cuda.set_device(0)


def group(counts, padded=False, ranks=1, max_sms=0, seed=0):
    idx = topk_for_counts(counts, ranks, seed).cuda()
    buf = Buffer(ranks, idx.shape[1], 128, len(counts), 1, low_latency_mode=padded, max_sms=max_sms)
    h = buf.get_dispatch_layout(idx)[3]
    grp = groups(buf, h)
    assert [c for _, c in grp] == list(counts)
    return buf, h, grp


def sentinel(shape, dtype=torch.bfloat16):
    if dtype == torch.float32:
        return torch.full(shape, 12345.678, device="cuda")
    if dtype == torch.bfloat16:
        return torch.full(shape, -777.0, device="cuda", dtype=dtype)
    return torch.full(shape, 0x55, device="cuda", dtype=torch.uint8).view(dtype)


def done(buf):
    assert buf.device_status() == ep.EP_OK


def check_gemm(buf, h, grp, n, k, transpose, seed=1, x=None, w=None):
    E = len(grp)
    x = receive(buf.rows, k, grp, seed) if x is None else x
    w = weights(E, k, n, seed + 1) if transpose and w is None else (weights(E, n, k, seed + 1) if w is None else w)
    out = sentinel((buf.rows, n))
    before = out.clone()
    buf.expert_gemm(x, w, h, transpose_w=transpose, out=out)
    done(buf)
    assert_untouched(out, before, in_use(buf.rows, grp), "gemm")
    for e, (b, c) in enumerate(grp):
        if c == 0:
            continue
        xe, we = x[b:b + c].double(), (w[e].T if transpose else w[e]).double()
        want = xe @ we.T
        assert_close(out[b:b + c], want, BF16 * want.abs() + sum_bound(k, xe.abs() @ we.abs().T), f"expert {e}")
    return out


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("n,k", SHAPES)
def test_gemm_edges(n, k, transpose):
    buf, h, grp = group(EDGES, padded=(n == 264), ranks=13 if n == 24 else 1)
    check_gemm(buf, h, grp, n, k, transpose)


@pytest.mark.parametrize("transpose", [False, True])
def test_gemm_few_tokens_and_long_sums(transpose):
    buf, h, grp = group([1, 0, 2, 1, 0, 0, 4, 1], padded=True, ranks=4)
    check_gemm(buf, h, grp, 776, 7168, transpose)


def test_gemm_many_experts_and_big_groups():
    buf, h, grp = group([3, 0, 1500] + [5] * 253, seed=3)
    check_gemm(buf, h, grp, 512, 128, False)


def check_fp8(buf, h, grp, n, k, seed=1):
    E = len(grp)
    rows = buf.rows
    x = receive(rows, k, grp, seed).float()
    x *= 10.0 ** (torch.rand(rows, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) * 4 - 2)
    xq, xs = cast_rows(x)   # NaN rows stay NaN: codes and scales
    wq, ws = cast_blocks(weights(E, n, k, seed + 1))
    out = sentinel((rows, n))
    before = out.clone()
    buf.expert_gemm_fp8((xq, xs), (wq, ws), h, out=out)
    done(buf)
    assert_untouched(out, before, in_use(rows, grp), "gemm_fp8")
    for e, (b, c) in enumerate(grp):
        if c == 0:
            continue
        xe, we = wide_rows(xq[b:b + c], xs[b:b + c]), wide_block(wq[e], ws[e])
        want = xe @ we.T
        assert_close(out[b:b + c], want, BF16 * want.abs() + sum_bound(k, xe.abs() @ we.abs().T), f"expert {e}")


@pytest.mark.parametrize("n,k", SHAPES_FP8)
def test_gemm_fp8_edges(n, k):
    buf, h, grp = group(EDGES, padded=(n == 264))
    check_fp8(buf, h, grp, n, k)


@pytest.mark.parametrize("n,k", SHAPES_FP8)
def test_gemm_fp8_edges_of_many_rows(n, k):
    buf, h, grp = group(EDGES_MANY, padded=(n == 264))
    check_fp8(buf, h, grp, n, k)


def test_gemm_fp8_few_tokens_and_long_sums():
    buf, h, grp = group([1, 0, 2, 1, 0, 0, 4, 1], padded=True, ranks=4)
    check_fp8(buf, h, grp, 776, 7168)


def check_gate(buf, h, grp, inner, k, seed=1):
    E, rows = len(grp), buf.rows
    xq, xs = cast_rows(receive(rows, k, grp, seed, scale=3.0).float())
    wq, ws = cast_blocks(weights(E, 2 * inner, k, seed + 1))
    hq, hs = sentinel((rows, inner), torch.float8_e4m3fn), sentinel((rows, inner // 128), torch.float32)
    before = hq.clone(), hs.clone()
    buf.expert_gate_fp8((xq, xs), (wq, ws), h, out=(hq, hs))
    done(buf)
    used = in_use(rows, grp)
    assert_untouched(hq, before[0], used, "gate codes")
    assert_untouched(hs, before[1], used, "gate scales")
    for e, (b, c) in enumerate(grp):
        if c == 0:
            continue
        xe, we = wide_rows(xq[b:b + c], xs[b:b + c]), wide_block(wq[e], ws[e])
        v = xe @ we.T
        g, u = v[:, :inner], v[:, inner:]
        off = sum_bound(k, xe.abs() @ we.abs().T)
        want = silu(g) * u
        # |silu'| <= 1.1; the fp32 activation itself is good to 2^-20
        tol = 1.1 * u.abs() * off[:, :inner] + silu(g).abs() * off[:, inner:] + off[:, :inner] * off[:, inner:] + \
            2.0 ** -20 * want.abs()
        s = hs[b:b + c].double()
        top = want.abs().view(c, -1, 128).amax(2).clamp_min(1e-4)
        assert_close(hs[b:b + c], top / 448, tol.view(c, -1, 128).amax(2) / 448 + 2.0 ** -21 * top / 448, f"scales of {e}")
        wide_s = s.repeat_interleave(128, 1)
        got = hq[b:b + c].float().double() * wide_s
        assert_close(got, want, 2.0 ** -4 * (want.abs() + tol) + 2.0 ** -10 * wide_s + tol, f"expert {e}")


@pytest.mark.parametrize("inner,k", [(128, 128), (256, 384), (384, 1152), (640, 256)])
def test_gate_fp8_edges(inner, k):
    buf, h, grp = group(EDGES, padded=(inner == 384))
    check_gate(buf, h, grp, inner, k)


@pytest.mark.parametrize("inner,k", [(128, 128), (256, 384), (384, 1152), (640, 256)])
def test_gate_fp8_edges_of_many_rows(inner, k):
    buf, h, grp = group(EDGES_MANY, padded=(inner == 384))
    check_gate(buf, h, grp, inner, k)


def test_gate_fp8_few_tokens_and_long_sums():
    buf, h, grp = group([1, 0, 2, 1, 0, 0, 4, 1], padded=True, ranks=4)
    check_gate(buf, h, grp, 256, 7168)


def test_gate_fp8_zero_rows_get_the_floor_scale():
    buf, h, grp = group([5, 40])
    xq = torch.zeros(buf.rows, 256, device="cuda").to(torch.float8_e4m3fn)
    xs = torch.ones(buf.rows, 2, device="cuda")
    w = buf.cast_weights(weights(2, 256, 256, 3))
    hq, hs = buf.expert_gate_fp8((xq, xs), w, h)
    done(buf)
    assert bool((hq.view(torch.uint8) & 0x7F == 0).all())
    assert bool((hs.cpu() == torch.tensor(1e-4) / torch.tensor(448.0)).all())


def check_wgrad(buf, h, grp, n, k, dtype, accumulate=False, seed=1):
    E = len(grp)
    dy, x = receive(buf.rows, n, grp, seed), receive(buf.rows, k, grp, seed + 1)
    dw = sentinel((E, n, k), dtype)
    before = dw.clone()
    buf.expert_wgrad(dy, x, h, out=dw, accumulate=accumulate)
    done(buf)
    for e, (b, c) in enumerate(grp):
        d, v = dy[b:b + c].double(), x[b:b + c].double()
        want = d.T @ v
        tol = sum_bound(c, d.abs().T @ v.abs())
        if accumulate:
            want = want + before[e].double()
            tol = tol + 2.0 ** -24 * want.abs()
        if dtype == torch.bfloat16:
            tol = tol + BF16 * want.abs()
        assert_close(dw[e], want, tol, f"expert {e}")
    return dw


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,k", SHAPES)
def test_wgrad_edges(n, k, dtype):
    buf, h, grp = group(EDGES, padded=(n == 264), ranks=13 if n == 24 else 1)
    check_wgrad(buf, h, grp, n, k, dtype)


def test_wgrad_accumulates():
    buf, h, grp = group([0, 1, 100, 300, 65])
    check_wgrad(buf, h, grp, 136, 264, torch.float32, accumulate=True)


def test_wgrad_long_sum_in_fp32_keeps_24_bits():
    """Sums of equal sign over many rows: a sum kept in fp32 that loses a bit
    per addition would drift; the result stays within 2^-20 of the sum."""
    buf, h, grp = group([6000, 17])
    dy = receive(buf.rows, 64, grp, 5).abs()
    x = receive(buf.rows, 72, grp, 6).abs()
    dw = buf.expert_wgrad(dy, x, h)
    done(buf)
    for e, (b, c) in enumerate(grp):
        want = dy[b:b + c].double().T @ x[b:b + c].double()
        assert_close(dw[e], want, 2.0 ** -20 * want, f"expert {e}")


@pytest.mark.parametrize("inner", [8, 72, 256, 1000])
@pytest.mark.parametrize("padded", [False, True])
def test_swiglu_and_its_gradient(inner, padded):
    buf, h, grp = group([0, 1, 33, 200, 0, 7], padded=padded, ranks=3)
    gu = receive(buf.rows, 2 * inner, grp, 1, scale=4.0)
    dh = receive(buf.rows, inner, grp, 2)
    used = in_use(buf.rows, grp)
    g, u, d = gu[used][:, :inner].double(), gu[used][:, inner:].double(), dh[used].double()
    s = torch.sigmoid(g)
    want_h, want_u = silu(g) * u, d * silu(g)
    slope = s * (1 + g * (1 - s))
    want_g = d * u * slope
    # fp32 steps: 2^-19 of the terms' magnitudes
    tol_g = BF16 * want_g.abs() + 2.0 ** -19 * (d * u * s).abs() * (1 + g.abs() * (1 - s))
    out = sentinel((buf.rows, inner))
    before = out.clone()
    buf.expert_swiglu(gu, h, out=out)
    done(buf)
    assert_untouched(out, before, used, "swiglu")
    assert_close(out[used], want_h, BF16 * want_h.abs() + 2.0 ** -19 * want_h.abs(), "h")
    dgu, h2 = sentinel((buf.rows, 2 * inner)), sentinel((buf.rows, inner))
    before = dgu.clone()
    buf.expert_swiglu_backward(gu, dh, h, out=(dgu, h2))
    done(buf)
    assert_untouched(dgu, before, used, "swiglu gradient")
    assert torch.equal(h2.view(torch.int16), out.view(torch.int16))
    assert_close(dgu[used][:, :inner], want_g, tol_g, "dg")
    assert_close(dgu[used][:, inner:], want_u, BF16 * want_u.abs() + 2.0 ** -19 * want_u.abs(), "du")
    # without h
    only = sentinel((buf.rows, 2 * inner))
    ep.ep_expert_swiglu_backward(buf.ctx, h.raw, gu, dh, inner, only)
    done(buf)
    assert torch.equal(only.view(torch.int16), dgu.view(torch.int16))


def test_swiglu_extremes():
    """Gates far out: silu goes to 0 and to g without overflow on the way."""
    buf, h, grp = group([4])
    g = torch.tensor([0.0, -0.0, 1e-30, 20.0, -20.0, 88.0, -88.0, -100.0, 100.0, 3e38, -3e38, 1.0, -1.0, 0.5, -0.5, 2.0])
    u = torch.full((16,), 2.0)
    u[9] = 0.5
    gu = torch.cat((g, u)).bfloat16().cuda().repeat(4, 1)
    out = buf.expert_swiglu(gu, h)
    done(buf)
    want = silu(gu[:, :16].double()) * gu[:, 16:].double()
    assert_close(out, want, BF16 * want.abs() + 1e-37, "extremes")


@pytest.mark.parametrize("n,k", [(8, 128), (128, 256), (264, 384)])
def test_cast_weights_bit_exact(n, k):
    buf, _, _ = group([1, 2, 3])
    w = weights(3, n, k, 9)
    w[1] *= 1e-6
    w[2, :, :128] *= 1000.0
    q, s = buf.cast_weights(w)
    done(buf)
    wq, ws = cast_blocks(w)
    same = torch.equal(q.view(torch.uint8), wq.view(torch.uint8)), torch.equal(s, ws)
    assert same == (True, True)


# ------------------------------------------------------------------ behaviour around the kernels

def test_no_rows_at_all():
    """T = 0 and layouts whose every entry is masked: outputs stay, dW is zero."""
    for tokens in (0, 6):
        buf = Buffer(2, 8, 128, 4, 2, low_latency_mode=False)
        idx = torch.full((2, tokens, 2), -1, dtype=torch.int64, device="cuda")
        h = buf.get_dispatch_layout(idx)[3]
        x = torch.full((buf.rows, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
        out = sentinel((buf.rows, 64))
        before = out.clone()
        buf.expert_gemm(x, weights(4, 64, 128, 1), h, out=out)
        buf.expert_gemm(x, weights(4, 128, 64, 1), h, transpose_w=True, out=out)
        xq, xs = cast_rows(x.float())
        buf.expert_gemm_fp8((xq, xs), cast_blocks(weights(4, 64, 128, 1)), h, out=out)
        assert torch.equal(out, before)
        for dtype in (torch.float32, torch.bfloat16):
            dw = sentinel((4, 64, 128), dtype)
            buf.expert_wgrad(out, x, h, out=dw)
            assert bool((dw == 0).all())
        dw = sentinel((4, 64, 128), torch.float32)
        buf.expert_wgrad(out, x, h, out=dw, accumulate=True)
        assert torch.equal(dw, sentinel((4, 64, 128), torch.float32))
        done(buf)


def test_infinities_stay_in_their_row_and_column():
    buf, h, grp = group([40, 300])
    x, w = receive(buf.rows, 200, grp, 1), weights(2, 264, 200, 2)
    x[grp[1][0] + 5, 3] = float("inf")
    w[0, 7, 100] = float("nan")
    out = buf.expert_gemm(x, w, h)
    done(buf)
    b0, b1 = grp[0][0], grp[1][0]
    bad = ~torch.isfinite(out.float())
    want = torch.zeros_like(bad)
    want[b0:b0 + 40, 7] = True
    want[b1 + 5] = True
    assert torch.equal(bad, want)


def test_same_bits_every_time_on_any_sm_count():
    outs = []
    for sms in (0, 0, 2, 37):
        buf, h, grp = group([0, 1, 31, 300, 700, 64], max_sms=sms)
        outs.append([check_gemm(buf, h, grp, 264, 200, False), check_gemm(buf, h, grp, 264, 200, True),
                     check_wgrad(buf, h, grp, 136, 200, torch.float32)])
        used = in_use(buf.rows, grp)
    for o in outs[1:]:
        assert torch.equal(o[0][used], outs[0][0][used]) and torch.equal(o[1][used], outs[0][1][used])
        assert torch.equal(o[2], outs[0][2])


@pytest.mark.parametrize("many", [False, True])
def test_fp8_same_bits_every_time_on_any_sm_count(many):
    counts = EDGES_MANY if many else EDGES
    outs = []
    for sms in (0, 0, 2, 37):
        buf, h, grp = group(counts, max_sms=sms)
        xq = cast_rows(receive(buf.rows, 512, grp, 1).float())
        w = buf.cast_weights(weights(len(counts), 768, 512, 2))
        y, (hq, hs) = buf.expert_gemm_fp8(xq, w, h), buf.expert_gate_fp8(xq, w, h)
        done(buf)
        used = in_use(buf.rows, grp)
        outs.append((y[used], hq.view(torch.uint8)[used], hs[used]))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_more_experts_than_the_kernels_keep_at_hand():
    """Past 256 experts counts and bases are read as they are needed, and the
    weights' gradient takes the experts in their own order."""
    counts = [(7 * e) % 5 for e in range(600)]
    counts[3], counts[599] = 260, 40
    buf, h, grp = group(counts)
    check_gemm(buf, h, grp, 72, 136, False)
    check_gemm(buf, h, grp, 72, 136, True)
    check_wgrad(buf, h, grp, 40, 72, torch.float32)
    check_fp8(buf, h, grp, 72, 128)
    check_gate(buf, h, grp, 128, 128)


def test_operators_of_one_handle_side_by_side():
    """A step's independent products on two streams: input and weight gradient
    of one handle, launched over and over without a wait between them."""
    buf, h, grp = group([300, 0, 17, 640, 128, 1, 77, 256] * 4)
    used = in_use(buf.rows, grp)
    dy, x, w = receive(buf.rows, 512, grp, 1), receive(buf.rows, 256, grp, 2), weights(32, 512, 256, 3)
    want_dx, want_dw = buf.expert_gemm(dy, w, h, transpose_w=True), buf.expert_wgrad(dy, x, h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dx, dw = sentinel((buf.rows, 256)), sentinel((32, 512, 256), torch.float32)
    torch.cuda.synchronize()
    for _ in range(20):
        buf.expert_gemm(dy, w, h, transpose_w=True, out=dx)
        with torch.cuda.stream(side):
            buf.expert_wgrad(dy, x, h, out=dw)
    torch.cuda.synchronize()
    done(buf)
    assert torch.equal(dx[used], want_dx[used]) and torch.equal(dw, want_dw)


def test_graphs_beside_eager_calls_and_each_other():
    """Products that draw their tiles from a counter: two graphs and an eager
    stream of one handle at once, each launched many times over."""
    buf, h, grp = group([300, 0, 17, 640, 128, 1, 77, 256] * 4)
    used = in_use(buf.rows, grp)
    x, w = receive(buf.rows, 256, grp, 1), weights(32, 2048, 256, 2)
    want = buf.expert_gemm(x, w, h)
    outs = [sentinel((buf.rows, 2048)) for _ in range(3)]
    torch.cuda.synchronize()
    graphs = []
    for out in outs[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(8):
                buf.expert_gemm(x, w, h, out=out)
    side = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        for _ in range(8):
            buf.expert_gemm(x, w, h, out=outs[2])
    torch.cuda.synchronize()
    done(buf)
    for out in outs:
        assert torch.equal(out[used], want[used])


def test_more_captured_calls_than_counters():
    """Past the tile counters of a handle the tiles come in a fixed order, with
    the same bits (and the weights' gradient adds each tile once)."""
    buf, h, grp = group([40, 0, 17, 64, 128, 1, 77, 56] * 4)
    used = in_use(buf.rows, grp)
    x, w = receive(buf.rows, 256, grp, 1), weights(32, 1024, 256, 2)
    dy = receive(buf.rows, 1024, grp, 3)
    want, want_dw = buf.expert_gemm(x, w, h), buf.expert_wgrad(dy, x, h)
    out, dw = sentinel((buf.rows, 1024)), torch.zeros((32, 1024, 256), dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4040):
            buf.expert_gemm(x, w, h, out=out)
        out.fill_(0)
        buf.expert_gemm(x, w, h, out=out)
        buf.expert_wgrad(dy, x, h, accumulate=True, out=dw)
    g.replay()
    torch.cuda.synchronize()
    done(buf)
    assert torch.equal(out[used], want[used]) and torch.equal(dw, want_dw)


def test_on_another_stream_and_in_a_graph():
    buf, h, grp = group([10, 0, 200, 33])
    x, w = receive(buf.rows, 256, grp, 1), weights(4, 512, 256, 2)
    want = check_gemm(buf, h, grp, 512, 256, False, x=x, w=w)
    wq = buf.cast_weights(w)
    xq = cast_rows(x.float())
    gate = buf.expert_gate_fp8(xq, wq, h)
    used = in_use(buf.rows, grp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = sentinel((buf.rows, 512))
    hq, hs = sentinel((buf.rows, 256), torch.float8_e4m3fn), sentinel((buf.rows, 2), torch.float32)
    with torch.cuda.stream(side):
        buf.expert_gemm(x, w, h, out=out)
    side.synchronize()
    assert torch.equal(out[used], want[used])
    g = torch.cuda.CUDAGraph()
    out.fill_(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        buf.expert_gemm(x, w, h, out=out)
        buf.expert_gate_fp8(xq, wq, h, out=(hq, hs))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[used], want[used])
    assert torch.equal(hq.view(torch.uint8)[used], gate[0].view(torch.uint8)[used]) and torch.equal(hs[used], gate[1][used])
    done(buf)


def test_offsets_past_32_bits():
    """A padded layout whose rows x channels pass 2^31: the last experts' rows."""
    E, cap, k, n = 64, 4160, 128, 8200   # 266240 rows x 8200 channels
    buf = Buffer(1, cap, 128, E, 1, low_latency_mode=True)
    idx = topk_for_counts([1, 0] * 31 + [3, 70]).cuda()
    h = buf.get_dispatch_layout(idx)[3]
    grp = groups(buf, h)
    x, w = torch.zeros(buf.rows, k, dtype=torch.bfloat16, device="cuda"), weights(E, n, k, 2)
    for b, c in grp:
        x[b:b + c] = receive(c, k, [(0, c)], b % 1000 + 1)
    out = torch.zeros(buf.rows, n, dtype=torch.bfloat16, device="cuda")
    buf.expert_gemm(x, w, h, out=out)
    done(buf)
    for e in (0, 2, 62, 63):
        b, c = grp[e]
        want = x[b:b + c].double() @ w[e].double().T
        assert_close(out[b:b + c], want,
                     BF16 * want.abs() + sum_bound(k, x[b:b + c].double().abs() @ w[e].double().abs().T), f"expert {e}")
    assert int((out != 0).any(1).sum()) == sum(c for _, c in grp)
    back = torch.zeros(buf.rows, k, dtype=torch.bfloat16, device="cuda")
    buf.expert_gemm(out, w, h, transpose_w=True, out=back)
    dw = buf.expert_wgrad(out, x, h)
    done(buf)
    for e in (0, 62, 63):
        b, c = grp[e]
        o, we, xe = out[b:b + c].double(), w[e].double(), x[b:b + c].double()
        want = o @ we
        assert_close(back[b:b + c], want, BF16 * want.abs() + sum_bound(n, o.abs() @ we.abs()), f"expert {e}")
        want = o.T @ xe
        assert_close(dw[e], want, sum_bound(c, o.abs().T @ xe.abs()), f"expert {e}")


def test_refusals():
    buf, h, grp = group([4, 4])
    other, h_other, _ = group([4, 4])
    L, P = ep.lib(), ctypes.c_void_p
    st = P(torch.cuda.current_stream().cuda_stream)
    x, w = receive(buf.rows, 128, grp, 1), weights(2, 256, 128, 2)
    y = torch.empty(buf.rows, 256, dtype=torch.bfloat16, device="cuda")
    xq, xs = cast_rows(x.float())
    wq, ws = cast_blocks(w)
    ptr = lambda t, off=0: P(t.data_ptr() + off)  # noqa: E731
    INV, UNS, NOL = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED, ep.EP_ERR_NO_LAYOUT
    gemm = lambda hh, a, b, n, k, t, c: L.ep_expert_gemm(buf.ctx, hh, a, b, n, k, t, c, st)  # noqa: E731
    assert gemm(h_other.raw, ptr(x), ptr(w), 256, 128, 0, ptr(y)) == INV
    assert gemm(buf.new_handle().raw, ptr(x), ptr(w), 256, 128, 0, ptr(y)) == NOL
    assert gemm(h.raw, None, ptr(w), 256, 128, 0, ptr(y)) == INV
    assert gemm(h.raw, ptr(x, 2), ptr(w), 256, 128, 0, ptr(y)) == INV
    assert gemm(h.raw, ptr(x), ptr(w), 250, 128, 0, ptr(y)) == INV
    assert gemm(h.raw, ptr(x), ptr(w), 256, 0, 0, ptr(y)) == INV
    assert gemm(h.raw, ptr(x), ptr(w), 256, 128, 2, ptr(y)) == INV
    assert gemm(h.raw, ptr(x), ptr(w), 65544, 128, 0, ptr(y)) == UNS
    fp8 = lambda k, s: L.ep_expert_gemm_fp8(buf.ctx, h.raw, ptr(xq), s, ptr(wq), ptr(ws), 256, k, ptr(y), st)  # noqa: E731
    assert fp8(64, ptr(xs)) == UNS and fp8(128, None) == INV and fp8(128, ptr(xs, 2)) == INV
    gate = lambda i: L.ep_expert_gate_fp8(buf.ctx, h.raw, ptr(xq), ptr(xs), ptr(wq), ptr(ws), i, 128, ptr(xq),  # noqa: E731
                                          ptr(xs), st)
    assert gate(64) == UNS and gate(4) == INV and gate(32896) == UNS
    wgrad = lambda f, a: L.ep_expert_wgrad(buf.ctx, h.raw, ptr(y), ptr(x), 256, 128, f, a, ptr(y), st)  # noqa: E731
    assert wgrad(0, 1) == INV and wgrad(2, 0) == INV
    # a rank-deduplicated layout has no experts' groups
    rl = Buffer(2, 4, 128, 4, 2)
    idx = torch.zeros(2, 4, 2, dtype=torch.int64, device="cuda")
    idx[..., 1] = 2
    hr = rl.get_rank_layout(idx)[3]
    assert L.ep_expert_swiglu(rl.ctx, hr.raw, ptr(x), 8, ptr(y), st) == NOL
    # the object API names the tensor
    with pytest.raises(ValueError, match="x must be"):
        buf.expert_gemm(x[:, :64].contiguous(), w, h)
    with pytest.raises(ValueError, match="w must be"):
        buf.expert_gemm(x, w[:1], h)
    with pytest.raises(ValueError, match="contiguous"):
        buf.expert_gemm(x, w.transpose(1, 2).contiguous().transpose(1, 2), h)
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        buf.expert_gemm(x.float(), w, h)
    with pytest.raises(ValueError, match="w scales"):
        buf.expert_gemm_fp8((xq, xs), (wq, ws[:, :1].contiguous()), h)
    with pytest.raises(ep.EPError):
        buf.expert_wgrad(y, x, h, out=torch.zeros(2, 256, 128, dtype=torch.bfloat16, device="cuda"), accumulate=True)
    with pytest.raises(ValueError, match="accumulate"):
        buf.expert_wgrad(y, x, h, accumulate=True)
    done(buf)


@pytest.mark.parametrize("op", ["gemm", "dgrad", "wgrad", "wgrad_fp32", "fp8", "gate"])
@pytest.mark.parametrize("counts", [[40, 0, 3, 130, 128, 9], [300, 700, 1, 256, 513, 40]])
def test_waits_run_out_then_the_context_works_again(op, counts):
    """An expert whose operands are never loaded: every wait in the kernel gives
    up after a millisecond, the call reports it, and the same calls afterwards
    give the same bits as before."""
    buf, h, grp = group(counts)
    E, used = len(counts), in_use(buf.rows, grp)
    x, dy, w = receive(buf.rows, 1024, grp, 1), receive(buf.rows, 1024, grp, 2), weights(E, 1024, 1024, 3)
    xq, wq = cast_rows(x.float()), buf.cast_weights(w)

    def call():
        if op == "gemm":
            return (buf.expert_gemm(x, w, h)[used],)
        if op == "dgrad":
            return (buf.expert_gemm(dy, w, h, transpose_w=True)[used],)
        if op == "fp8":
            return (buf.expert_gemm_fp8(xq, wq, h)[used],)
        if op == "gate":
            q, s = buf.expert_gate_fp8(xq, wq, h)
            return q.view(torch.uint8)[used], s[used]
        dtype = torch.float32 if op == "wgrad_fp32" else torch.bfloat16
        return (buf.expert_wgrad(dy, x, h, out=torch.empty(E, 1024, 1024, dtype=dtype, device="cuda")),)

    want = call()
    done(buf)
    ep.ep_set_test_hooks(buf.ctx, move_withhold_item=3, move_wait_ns=1_000_000)
    call()
    assert buf.device_status() == ep.EP_ERR_TIMEOUT
    ep.ep_set_test_hooks(buf.ctx)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    done(buf)


# ------------------------------------------------------------------ the operators as they are used together

def test_fp8_serving_path_from_dispatch_to_combine():
    """FP8 dispatch -> gate and up -> down -> combine, against 64 bits on the
    codes and scales that each step reads."""
    torch.manual_seed(4)
    R, T, H, E, K, inner = 4, 37, 256, 8, 3, 384
    buf = Buffer(R, T, H, E, K, low_latency_mode=True)
    x = torch.randn(R, T, H, device="cuda").bfloat16()
    idx = torch.rand(R * T, E, device="cuda").topk(K).indices.view(R, T, K)
    idx[0, :5, 1] = -1
    wts = torch.rand(R * T, K, device="cuda")
    wgu, wd = weights(E, 2 * inner, H, 1), weights(E, H, inner, 2)
    qgu, qd = buf.cast_weights(wgu), buf.cast_weights(wd)
    recv, _, h = buf.low_latency_dispatch(x, idx, T, E, use_fp8=True)
    hq = buf.expert_gate_fp8(recv, qgu, h)
    y = buf.expert_gemm_fp8(hq, qd, h)
    out = buf.low_latency_combine(y, idx, wts, h, E)
    done(buf)
    again = buf.expert_mlp_fp8(recv, qgu, qd, h)
    used = in_use(buf.rows, groups(buf, h))
    assert torch.equal(again[used], y[used])
    ye = y.double()
    for e, (b, c) in enumerate(groups(buf, h)):
        v = wide_rows(recv[0][b:b + c], recv[1][b:b + c]) @ wide_block(qgu[0][e], qgu[1][e]).T
        want = silu(v[:, :inner]) * v[:, inner:]
        got = wide_rows(hq[0][b:b + c], hq[1][b:b + c])
        top = hq[1][b:b + c].double().repeat_interleave(128, 1) * 448
        assert_close(got, want, 2.0 ** -4 * want.abs() + 2.0 ** -18 * top, f"h of expert {e}")
        want = got @ wide_block(qd[0][e], qd[1][e]).T
        assert_close(y[b:b + c], want, BF16 * want.abs() + 1e-4 * want.abs().amax(), f"y of expert {e}")
    slot = h.tensors()["slot"].long()
    want = torch.zeros(R * T, H, dtype=torch.float64, device="cuda")
    for j in range(K):
        m = slot[:, j] >= 0
        want[m] += wts[m, j:j + 1].double() * ye[slot[m, j]]
    assert_close(out, want, BF16 * want.abs() + 1e-5, "combine")


def test_training_step_gradients_against_formula_and_differences():
    """bf16 experts forward and backward between dispatch and combine: each
    gradient against autograd in 64 bits, and the whole against central
    differences of the 64-bit forward pass."""
    torch.manual_seed(5)
    R, T, H, E, K, inner = 2, 45, 136, 6, 2, 72
    buf = Buffer(R, T, H, E, K, low_latency_mode=False)
    x = torch.randn(R, T, H, device="cuda").bfloat16()
    idx = torch.rand(R * T, E - 1, device="cuda").topk(K).indices.view(R, T, K)   # the last expert gets none
    wgu, wd = weights(E, 2 * inner, H, 1), weights(E, H, inner, 2)
    recv, _, h = buf.low_latency_dispatch(x, idx, T, E, use_fp8=False)
    y, saved = buf.expert_mlp(recv, wgu, wd, h)
    dy = receive(buf.rows, H, groups(buf, h), 7)
    dx, dwgu, dwd = buf.expert_mlp_backward(dy, saved, wgu, wd, h)
    dtok = buf.low_latency_combine(dx, idx, None, h, E)
    done(buf)
    used = in_use(buf.rows, groups(buf, h))
    grp = groups(buf, h)

    def forward(rx, a, b):
        outs = []
        for e, (s, c) in enumerate(grp):
            v = rx[s:s + c] @ a[e].T
            outs.append(silu(v[:, :inner]) * v[:, inner:] @ b[e].T)
        return torch.cat(outs)

    args = [recv.double().requires_grad_(), wgu.double().requires_grad_(), wd.double().requires_grad_()]
    out = forward(*args)
    loss = (out * dy.double()).sum()
    grads = torch.autograd.grad(loss, args)
    # the step keeps gu, h, dh and dgu in bf16: relative errors of a few 2^-9 each, that sums of
    # independent roundings do not exceed by more than their number
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(y[used], out.detach()) < 4 * 2.0 ** -8
    for got, want, what in ((dx[used], grads[0][used], "dx"), (dwgu, grads[1], "dwgu"), (dwd, grads[2], "dwd")):
        assert rel(got, want) < 4 * 2.0 ** -8, what
    assert bool((dwgu[-1] == 0).all()) and bool((dwd[-1] == 0).all())
    dirs = [torch.randn_like(a) for a in args]
    eps = 1e-6
    with torch.no_grad():
        hi = (forward(*[a + eps * d for a, d in zip(args, dirs)]) * dy.double()).sum()
        lo = (forward(*[a - eps * d for a, d in zip(args, dirs)]) * dy.double()).sum()
    slope = (hi - lo) / (2 * eps)
    parts = [(g.double() * d)[torch.isfinite(g)].sum() for g, d in zip((dx, dwgu, dwd), dirs)]
    size = sum(float((g * d).square().sum().sqrt()) for g, d in zip(grads, dirs))
    assert abs(float(sum(parts) - slope)) < 8 * 2.0 ** -8 * size
    # the token's gradient is the sum over its experts' rows
    slot = h.tensors()["slot"].long()
    want = dx.double()[slot].sum(1)
    assert_close(dtok, want, BF16 * want.abs() + 1e-5, "token gradient")
