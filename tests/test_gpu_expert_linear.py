"""GPU checks of the product with bias, activation and residual, and of its backward pass, against their
definitions in 64 bits."""
import math

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer
from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from expert_reference import BF16, assert_close, assert_untouched, groups, in_use, receive, sum_bound, topk_for_counts, weights

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 31, 32, 33, 127, 128, 129, 0, 255, 256, 257, 520]
SHAPES = [(8, 8), (24, 72), (136, 64), (264, 200), (256, 256), (1000, 328)]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


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


def sentinel(shape):
    return torch.full(shape, -777.0, device="cuda", dtype=torch.bfloat16)


def bias_of(E, n, seed, dtype):
    return (torch.randn(E, n, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * 0.5).to(dtype)


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    p = torch.sigmoid(z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return p + z * p * (1 - p) * (1.0 if act == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z))


def check(buf, h, grp, n, k, act="none", bias=None, residual=False, save=False, seed=1, in_place=False, x=None, w=None):
    """The sum is off by sum_bound; the slopes are at most 1.13; the activation itself is good to 2^-14 of its
    value (the exponential's argument reaches 80 and carries a few roundings, 80 * 4 * 2^-24), and each
    addition to 2^-23."""
    E = len(grp)
    x = receive(buf.rows, k, grp, seed) if x is None else x
    w = weights(E, n, k, seed + 1) if w is None else w
    b = bias_of(E, n, seed + 2, bias) if bias is not None else None
    res = receive(buf.rows, n, grp, seed + 3) if residual else None
    kept = res.clone() if residual else None
    out = res if in_place else sentinel((buf.rows, n))
    before = out.clone()
    z = sentinel((buf.rows, n)) if save else None
    got = buf.expert_linear(x, w, h, bias=b, activation=act, residual=res, out=out, z=z)
    assert got is out and buf.device_status() == ep.EP_OK
    used = in_use(buf.rows, grp)
    assert_untouched(out, before, used, "linear")
    if save:
        assert_untouched(z, sentinel((buf.rows, n)), used, "z")
    for e, (at, c) in enumerate(grp):
        if c == 0:
            continue
        xe, we = x[at:at + c].double(), w[e].double()
        v, dv = xe @ we.T, sum_bound(k, xe.abs() @ we.abs().T)
        if b is not None:
            v = v + b[e].double()
            dv = dv + 2.0 ** -23 * v.abs()
        if save:
            assert_close(z[at:at + c], v, BF16 * v.abs() + dv * (1 + BF16), f"z of expert {e}")
        want = act64(v, act)
        tol = (dv if act == "none" else 1.13 * dv + 2.0 ** -14 * want.abs() + 1e-37)
        if residual:
            r = kept[at:at + c].double()
            tol = tol + 2.0 ** -23 * (want.abs() + r.abs())
            want = want + r
        assert_close(out[at:at + c], want, BF16 * want.abs() + tol * (1 + BF16), f"expert {e}")
    return out, z


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_edges_with_everything(n, k, act):
    buf, h, grp = group(EDGES, padded=(n == 264), ranks=13 if n == 24 else 1)
    check(buf, h, grp, n, k, act, bias=torch.float32 if n % 16 else torch.bfloat16, residual=True, save=True)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("bias", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("save", [False, True])
def test_each_part_on_its_own(act, bias, residual, save):
    buf, h, grp = group([3, 0, 70, 300])
    check(buf, h, grp, 136, 200, act, bias, residual, save)


def test_few_tokens_and_long_sums():
    buf, h, grp = group([1, 0, 2, 1, 0, 0, 4, 1], padded=True, ranks=4)
    check(buf, h, grp, 776, 7168, "silu", torch.bfloat16, True, True)


def test_many_experts_and_big_groups():
    buf, h, grp = group([3, 0, 1500] + [5] * 253, seed=3)
    check(buf, h, grp, 512, 128, "gelu_tanh", torch.float32, True)


def test_more_experts_than_are_kept_in_shared_memory():
    buf, h, grp = group([2] * 300 + [0] * 4, seed=3)
    check(buf, h, grp, 40, 24, "relu", torch.bfloat16, True, True)


def test_residual_may_be_the_output():
    buf, h, grp = group(EDGES)
    check(buf, h, grp, 264, 72, "silu", torch.bfloat16, residual=True, in_place=True)


@pytest.mark.parametrize("act", ACTS)
def test_activation_over_its_whole_range(act):
    """x one-hot, so z is the weight itself: every bf16 from the largest down to the subnormal ones."""
    buf, h, grp = group([8])
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[bits.isfinite()]
    bits = torch.cat([bits, bits[: -len(bits) % 64]]).view(1, -1, 8).contiguous().cuda()
    x = torch.eye(8, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(8, bits.shape[1], device="cuda", dtype=torch.bfloat16)
    buf.expert_linear(x, bits, h, activation=act, out=out)
    assert buf.device_status() == ep.EP_OK
    z = bits[0].T.double()
    want = act64(z, act)
    # below the smallest normal number the result may be zero
    assert_close(out, want, BF16 * want.abs() + 2.0 ** -14 * want.abs() + 2.0 ** -126, act)


@pytest.mark.parametrize("act", ACTS)
def test_slope_over_its_whole_range(act):
    """dy = 1: dz is the slope of every finite bf16 (2^-19 absolute: sums and products of terms up to 1.13)."""
    buf, h, grp = group([8])
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[bits.isfinite()]
    z = torch.cat([bits, bits[: -len(bits) % 64]]).view(8, -1).contiguous().cuda()
    dz, _ = buf.expert_linear_backward(torch.ones_like(z), z, h, activation=act, out=torch.empty_like(z))
    want = slope64(z.double().clamp(-1e30, 1e30), act)
    assert_close(dz, want, BF16 * want.abs() + 2.0 ** -19, act)


def test_nan_and_infinite_inputs_stay_in_their_rows():
    buf, h, grp = group([5, 40])
    x, w = receive(buf.rows, 72, grp, 1), weights(2, 136, 72, 2)
    clean, _ = check(buf, h, grp, 136, 72, "relu", x=x, w=w)
    x2 = x.clone()
    x2[3], x2[9, 7] = float("nan"), float("inf")
    got = buf.expert_linear(x2, w, h, activation="relu")
    assert bool(got[3].isnan().all())
    keep = torch.ones(45, dtype=torch.bool, device="cuda")
    keep[3] = keep[9] = False
    assert torch.equal(got[keep], clean[keep])


def test_no_epilogue_gives_the_plain_product():
    buf, h, grp = group(EDGES)
    x, w = receive(buf.rows, 200, grp, 1), weights(len(grp), 264, 200, 2)
    used = in_use(buf.rows, grp)
    assert torch.equal(buf.expert_linear(x, w, h)[used], buf.expert_gemm(x, w, h)[used])


# ------------------------------------------------------------------ backward

def check_backward(buf, h, grp, n, act, seed=1, accumulate=False, in_place=None, want_dz=True):
    """dz: the slope is good to 2^-19; db: that, and an fp32 sum of c terms (c + 16 roundings)."""
    E = len(grp)
    dy, z = receive(buf.rows, n, grp, seed), receive(buf.rows, n, grp, seed + 1, scale=2.0)
    d0, z0 = dy.clone(), z.clone()
    out = {"dy": dy, "z": z, None: sentinel((buf.rows, n))}[in_place]
    before = out.clone()
    db = torch.randn(E, n, device="cuda")
    db0 = db.clone()
    dz, got = buf.expert_linear_backward(dy, z, h, activation=act, out=out if want_dz else None, dbias=db, accumulate=accumulate)
    assert got is db and buf.device_status() == ep.EP_OK
    if want_dz:
        assert_untouched(out, before, in_use(buf.rows, grp), "dz")
    for e, (at, c) in enumerate(grp):
        a, v = d0[at:at + c].double(), z0[at:at + c].double()
        want = a * slope64(v, act)
        if want_dz:
            assert_close(dz[at:at + c], want, BF16 * want.abs() + 2.0 ** -18 * a.abs(), f"dz of expert {e}")
        total = want.sum(0) + (db0[e].double() if accumulate else 0.0)
        tol = 2.0 ** -18 * a.abs().sum(0) + (c + 16) * 2.0 ** -24 * want.abs().sum(0) + 2.0 ** -23 * db0[e].double().abs()
        assert_close(db[e], total, tol + 2.0 ** -23 * total.abs(), f"db of expert {e}")
    return dz, db


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n", [8, 136, 256, 264, 1000])
def test_backward_edges(n, act):
    buf, h, grp = group(EDGES, padded=(n == 264), ranks=13 if n == 136 else 1)
    check_backward(buf, h, grp, n, act, accumulate=n == 256)


@pytest.mark.parametrize("counts", [[0, 0, 0], [1], [4096], [5000, 3, 0, 900], [7] * 300, [2] * 1024])
def test_backward_of_every_kind_of_split(counts):
    buf, h, grp = group(counts)
    check_backward(buf, h, grp, 72, "silu")
    check_backward(buf, h, grp, 2048 if len(counts) < 8 else 264, "gelu", accumulate=True)


@pytest.mark.parametrize("where", ["dy", "z"])
def test_backward_in_place(where):
    buf, h, grp = group(EDGES)
    check_backward(buf, h, grp, 264, "gelu", in_place=where)


def test_backward_without_activation():
    buf, h, grp = group(EDGES)
    dy = receive(buf.rows, 136, grp, 1)
    dz, db = buf.expert_linear_backward(dy, None, h)
    assert dz is dy
    _, want = check_backward(buf, h, grp, 136, "none", want_dz=False)
    assert torch.equal(db, want)
    out = sentinel(dy.shape)
    buf.expert_linear_backward(dy, None, h, out=out)
    assert torch.equal(out[in_use(buf.rows, grp)], dy[in_use(buf.rows, grp)])


def test_backward_of_equal_signed_sums():
    """5000 rows of ones: the bias gradient is exact."""
    buf, h, grp = group([5000, 17])
    _, db = buf.expert_linear_backward(torch.ones(buf.rows, 264, device="cuda", dtype=torch.bfloat16), None, h)
    assert bool((db[0] == 5000).all()) and bool((db[1] == 17).all())


def test_backward_does_not_depend_on_max_sms_and_repeats():
    buf, h, grp = group([300, 1, 0, 77])
    first = check_backward(buf, h, grp, 264, "gelu_tanh")
    for sms in (1, 31, 152):
        buf, h, grp = group([300, 1, 0, 77], max_sms=sms)
        again = check_backward(buf, h, grp, 264, "gelu_tanh")
        assert torch.equal(first[1], again[1]) and torch.equal(first[0], again[0])


def test_gradients_against_differences():
    """d/ds of sum(dy * y) along random directions of x, w and the bias, y in 64 bits around the kernel's z."""
    counts, n, k, s = [5, 0, 33, 12], 40, 24, 1e-4
    buf, h, grp = group(counts)
    E = len(counts)
    x, w, b = receive(buf.rows, k, grp, 1), weights(E, n, k, 2), bias_of(E, n, 3, torch.float32)
    dy = receive(buf.rows, n, grp, 4)
    z = torch.zeros(buf.rows, n, device="cuda", dtype=torch.bfloat16)
    buf.expert_linear(x, w, h, bias=b, activation="gelu", z=z)
    dz, db = buf.expert_linear_backward(dy, z, h, activation="gelu")
    dx, dw = buf.expert_gemm(dz, w, h, transpose_w=True), buf.expert_wgrad(dz, x, h)
    g = torch.Generator("cuda").manual_seed(9)
    dirs = [torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in (x, w, b)]

    def loss(step):
        X, W, B = (t.double() + step * d for t, d in zip((x, w, b), dirs))
        return sum((dy[a:a + c].double() * act64(X[a:a + c] @ W[e].T + B[e], "gelu")).sum() for e, (a, c) in enumerate(grp))

    slope = float((loss(s) - loss(-s)) / (2 * s))
    got = sum(float((t[a:a + c].double() * d[a:a + c]).sum()) for t, d in ((dx, dirs[0]),) for a, c in grp)
    got += float((dw.double() * dirs[1]).sum() + (db.double() * dirs[2]).sum())
    # each factor of a gradient is rounded to bf16 at most three times (z, dz, dx), independently: 2-norms
    scale = math.sqrt(sum(float((t.double()[:] * d)[in_use(buf.rows, grp)].square().sum()) if t is dx else
                          float((t.double() * d).square().sum()) for t, d in ((dx, dirs[0]), (dw, dirs[1]), (db, dirs[2]))))
    assert abs(got - slope) <= 6 * 3 * BF16 * scale, (got, slope, scale)


def test_experts_with_biases_forward_and_backward():
    """expert_mlp and expert_mlp_backward with biases, as a training step calls them, in a graph too: against
    autograd in 64 bits on the same values (gu, h, dh, dgu each rounded to bf16 once)."""
    counts, H, I = [9, 0, 40, 17], 64, 48
    buf, h, grp = group(counts)
    E = len(counts)
    x, dy = receive(buf.rows, H, grp, 1), receive(buf.rows, H, grp, 2)
    w13, w2 = weights(E, 2 * I, H, 3), weights(E, H, I, 4)
    b = bias_of(E, 2 * I, 5, torch.bfloat16), bias_of(E, H, 6, torch.float32)
    grads = tuple(torch.zeros(t.shape, device="cuda") for t in (w13, w2))
    bias_grads = tuple(torch.zeros(t.shape, device="cuda") for t in b)

    def step():
        y, saved = buf.expert_mlp(x, w13, w2, h, biases=b)
        dx, *_ = buf.expert_mlp_backward(dy, saved, w13, w2, h, grads=grads, bias_grads=bias_grads)
        return y, dx

    y, dx = step()
    assert buf.device_status() == ep.EP_OK
    wide = [t.double().requires_grad_() for t in (x.nan_to_num(0.0), w13, w2, *b)]
    X, W13, W2, B13, B2 = wide
    rows = []
    for e, (a, c) in enumerate(grp):
        g, u = (X[a:a + c] @ W13[e].T + B13[e]).chunk(2, 1)
        rows.append((torch.nn.functional.silu(g) * u) @ W2[e].T + B2[e])
    want = torch.cat(rows)
    want.backward(dy[in_use(buf.rows, grp)].double())
    for got, ref in ((y[in_use(buf.rows, grp)], want), (dx[in_use(buf.rows, grp)], X.grad[in_use(buf.rows, grp)]), (grads[0], W13.grad),
                     (grads[1], W2.grad), (bias_grads[0], B13.grad), (bias_grads[1], B2.grad)):
        error = float((got.double() - ref.detach()).norm() / ref.detach().norm())
        assert error <= 5 * BF16, error
    kept = [t.clone() for t in grads + bias_grads]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y2, dx2 = step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2[in_use(buf.rows, grp)], y[in_use(buf.rows, grp)])
    assert torch.equal(dx2[in_use(buf.rows, grp)], dx[in_use(buf.rows, grp)])
    for got, once in zip(grads + bias_grads, kept):     # added up three times in all
        assert_close(got, 3 * once.double(), 2.0 ** -22 * 3 * once.double().abs(), "accumulated")


def test_refusals_touch_nothing():
    buf, h, grp = group([3, 5])
    x, w, z = receive(buf.rows, 24, grp, 1), weights(2, 40, 24, 2), receive(buf.rows, 40, grp, 3)
    out = sentinel((buf.rows, 40))
    with pytest.raises(ValueError):
        buf.expert_linear(x, w, h, activation="tanh", out=out)
    with pytest.raises(ValueError):
        buf.expert_linear(x, w, h, bias=torch.zeros(2, 40, device="cuda", dtype=torch.float16), out=out)
    with pytest.raises(ValueError):
        buf.expert_linear(x, w, h, residual=z.float(), out=out)
    with pytest.raises(ep.EPError) as e:
        buf.expert_linear(x, w, h, z=out, out=out)
    assert e.value.status == ep.EP_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        buf.expert_linear_backward(z, None, h, activation="relu")
    fresh = buf.new_handle()
    with pytest.raises(ep.EPError) as e:
        buf.expert_linear(x, w, fresh, out=out)
    assert e.value.status == ep.EP_ERR_NO_LAYOUT
    with pytest.raises(ep.EPError) as e:
        buf.expert_linear_backward(z, z, fresh, activation="relu")
    assert e.value.status == ep.EP_ERR_NO_LAYOUT
    lib, p = ep.lib(), lambda t: t.data_ptr()  # noqa: E731
    good = [buf.ctx, h.raw, p(x), p(w), 40, 24, None, 0, 0, None, None, p(out), None]
    for at, value in ((2, None), (3, None), (11, None), (2, p(x) + 2), (4, 12), (5, 0), (7, 2), (8, 5), (8, -1), (9, p(z) + 8), (10, p(z) + 2)):
        bad = list(good)
        bad[at] = value
        assert lib.ep_expert_linear(*bad) == ep.EP_ERR_INVALID_ARG, (at, value)
    bad = list(good)
    bad[4] = 65544
    assert lib.ep_expert_linear(*bad) == ep.EP_ERR_UNSUPPORTED
    db = torch.full((2, 40), 5.0, device="cuda")
    good = [buf.ctx, h.raw, p(z), p(z), 40, 1, 0, p(out), p(db), None]
    for at, value in ((2, None), (3, None), (2, p(z) + 2), (4, 12), (5, 9), (6, 2), (7, p(out) + 8), (8, p(db) + 2)):
        bad = list(good)
        bad[at] = value
        assert lib.ep_expert_linear_backward(*bad) == ep.EP_ERR_INVALID_ARG, (at, value)
    bad = list(good)
    bad[7] = bad[8] = None
    assert lib.ep_expert_linear_backward(*bad) == ep.EP_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((out == -777.0).all()) and bool((db == 5.0).all())


def test_empty_calls():
    """No tokens at all: outputs keep what they hold, the bias gradient is zero unless it is added to."""
    buf = Buffer(2, 4, 128, 4, 2, low_latency_mode=False)
    h = buf.get_dispatch_layout(torch.empty(2, 0, 2, dtype=torch.int64, device="cuda"))[3]
    z, out, db = sentinel((buf.rows, 40)), sentinel((buf.rows, 40)), torch.full((4, 40), 5.0, device="cuda")
    buf.expert_linear(sentinel((buf.rows, 24)), weights(4, 40, 24, 1), h, out=out)
    buf.expert_linear_backward(z, z, h, activation="relu", out=out, dbias=db, accumulate=True)
    assert bool((out == -777.0).all()) and bool((db == 5.0).all())
    buf.expert_linear_backward(z, z, h, activation="relu", out=out, dbias=db)
    assert bool((out == -777.0).all()) and bool((db == 0.0).all()) and buf.device_status() == ep.EP_OK


def test_the_input_is_no_output():
    buf, h, grp = group([3, 5])
    x, w, out = receive(buf.rows, 40, grp, 1), weights(2, 40, 40, 2), sentinel((buf.rows, 40))
    kept = x.clone()
    for kw in ({"out": x}, {"out": out, "z": x}):
        with pytest.raises(ep.EPError) as e:
            buf.expert_linear(x, w, h, activation="relu", **kw)
        assert e.value.status == ep.EP_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(x.view(torch.int16), kept.view(torch.int16)) and bool((out == -777.0).all())


@pytest.mark.parametrize("accumulate", [False, True])
def test_a_bias_in_one_of_the_two_products(accumulate):
    """The other one's is left out, forward and backward: the same bits as with zeros for it."""
    buf, h, grp = group([9, 0, 40, 17])
    H, I = 64, 48
    x, dy = receive(buf.rows, H, grp, 1), receive(buf.rows, H, grp, 2)
    w13, w2 = weights(4, 2 * I, H, 3), weights(4, H, I, 4)
    used = in_use(buf.rows, grp)
    for at, n in ((0, 2 * I), (1, H)):
        b, zeros = bias_of(4, n, 5, torch.bfloat16), torch.zeros(4, (H, 2 * I)[at], device="cuda")
        some, both = ((b, None), (b, zeros)) if at == 0 else ((None, b), (zeros, b))
        y, saved = buf.expert_mlp(x, w13, w2, h, biases=some)
        y0, saved0 = buf.expert_mlp(x, w13, w2, h, biases=both)
        assert torch.equal(y[used], y0[used])
        grads = tuple(torch.zeros(t.shape, device="cuda") for t in (w13, w2)) if accumulate else None
        db, db0 = torch.zeros(4, n, device="cuda"), [torch.zeros(4, c, device="cuda") for c in (2 * I, H)]
        dx, *_ = buf.expert_mlp_backward(dy, saved, w13, w2, h, grads=grads, bias_grads=(db, None) if at == 0 else (None, db))
        dx0, *_ = buf.expert_mlp_backward(dy, saved0, w13, w2, h, grads=grads, bias_grads=db0)
        assert torch.equal(dx[used], dx0[used]) and torch.equal(db, db0[at])
    assert buf.device_status() == ep.EP_OK
