"""GPU checks of the whole layer for a few tokens against its definition in 64 bits."""
import ctypes

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer
from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from expert_reference import BF16, assert_close, cast_blocks, silu, sum_bound, weights, wide_block
from norm_bounds import bf16_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    epbuild.build()
    torch.cuda.set_device(0)


def bf(shape, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


def route(N, E, K, seed, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    top = torch.randn(N, E, generator=g).topk(K, dim=1)
    idx = top.indices.clone()
    idx[torch.rand(N, K, generator=g) < drop] = -1
    return idx.cuda(), torch.softmax(top.values, -1).contiguous().cuda()


class Layer:
    """Weights, tokens and routing of one call, and its definition with error bounds.

    Bounds: a product of bf16 / e4m3 values is exact in fp32 and a sum of n of them off by
    sum_bound(n); silu's slope is at most 1.1; h is kept to 2^-17 and computed to 2^-20 of itself;
    the K shares add 2^-23 of their magnitudes each, the result's rounding BF16 of it."""

    def __init__(self, N, H, I, E, K, fp8=False, bias=False, residual=False, drop=0.0, seed=0, idx=None, max_sms=0):
        self.N, self.H, self.I, self.E, self.K, self.fp8 = N, H, I, E, K, fp8
        self.buf = Buffer(1, max(N, 1), H, E, K, max_sms=max_sms)
        self.x = bf((N, H), seed + 1)
        made, self.wts = route(N, max(E, K), K, seed, drop)     # with idx given, K may be more than E
        self.idx = made if idx is None else idx
        self.gu, self.down = weights(E, 2 * I, H, seed + 2), weights(E, H, I, seed + 3)
        if fp8:
            self.gu, self.down = cast_blocks(self.gu), cast_blocks(self.down)
        self.bias = (bf((E, 2 * I), seed + 4, 0.5), bf((E, H), seed + 5, 0.5)) if bias else None
        self.residual = bf((N, H), seed + 6) if residual else None

    def run(self, **kw):
        out = self.buf.expert_layer(self.x, self.idx, self.wts, self.gu, self.down, biases=self.bias, residual=self.residual, **kw)
        assert self.buf.device_status() == ep.EP_OK
        return out

    def want(self):
        wide = lambda w, e: wide_block(w[0][e], w[1][e]) if self.fp8 else w[e].double()  # noqa: E731
        out = torch.zeros(self.N, self.H, device="cuda", dtype=torch.float64)
        tol, mag = torch.zeros_like(out), torch.zeros_like(out)
        for e in range(self.E):
            t, k = (self.idx == e).nonzero(as_tuple=True)
            if t.numel() == 0:
                continue
            x, w = self.x[t].double(), wide(self.gu, e)
            v, dv = x @ w.T, sum_bound(self.H, x.abs() @ w.abs().T)
            if self.bias is not None:
                v = v + self.bias[0][e].double()
                dv = dv + 2.0 ** -23 * v.abs()
            (g, u), (dg, du) = v.chunk(2, 1), dv.chunk(2, 1)
            h = silu(g) * u
            dh = 1.1 * dg * (u.abs() + du) + silu(g).abs() * du + (2.0 ** -17 + 2.0 ** -20) * h.abs()
            w = wide(self.down, e)
            y, dy = h @ w.T, dh @ w.abs().T + sum_bound(2 * self.I, (h.abs() + dh) @ w.abs().T)
            if self.bias is not None:
                y = y + self.bias[1][e].double()
            p = self.wts[t, k].double().unsqueeze(1)
            out.index_add_(0, t, p * y)
            tol.index_add_(0, t, p.abs() * dy)
            mag.index_add_(0, t, (p * y).abs())
        if self.residual is not None:
            out += self.residual.double()
            mag += self.residual.double().abs()
        tol += (self.K + 2) * 2.0 ** -23 * mag
        return out, tol + BF16 * (out.abs() + tol)

    def check(self, **kw):
        got = self.run(**kw)
        want, tol = self.want()
        assert_close(got, want, tol, "layer")
        return got


# Two forms: the small one up to 96 MB of bf16 or 32 MB of e4m3 weights (of as many experts as there are entries)
# and 4 entries per expert, the large one past either.
# N, H, I, E, K: one token; tiles cut off on every side; more than 8 and 16 tokens of an expert; the most tokens
SIZES = [(1, 8, 8, 1, 1), (1, 1024, 512, 32, 4), (3, 264, 24, 5, 2), (7, 40, 200, 9, 3), (17, 520, 136, 2, 2), (32, 1000, 328, 64, 6),
         (128, 256, 64, 16, 8), (128, 72, 1016, 3, 1), (5, 2048, 16, 1024, 32)]
SIZES_FP8 = [(1, 128, 128, 1, 1), (1, 1024, 512, 32, 4), (3, 256, 128, 5, 2), (17, 640, 384, 2, 2), (31, 1152, 128, 40, 6), (128, 256, 640, 16, 8)]


# the large form: many tokens of few experts, odd channels; weights past the small form's
SIZES += [(5, 8, 8, 1, 1), (40, 264, 24, 5, 2), (33, 40, 200, 4, 3), (21, 1000, 328, 3, 1), (70, 2048, 16, 8, 8), (1, 4096, 2048, 16, 8),
          (3, 2824, 1416, 40, 6), (65, 200, 264, 2, 1), (128, 136, 72, 2, 2), (8, 72, 1016, 1, 1), (9, 72, 1016, 1, 1), (8, 1024, 512, 1024, 32)]
SIZES_FP8 += [(4, 128, 384, 1, 1), (5, 128, 128, 1, 1), (4, 1024, 512, 1024, 32), (33, 1152, 256, 4, 3), (1, 7168, 2048, 8, 8), (5, 2176, 1920, 20, 4), (100, 384, 640, 3, 2)]


# the most tokens, experts and entries of a token at a time
SIZES += [(128, 512, 264, 1024, 32)]
SIZES_FP8 += [(128, 512, 256, 1024, 32)]


@pytest.mark.parametrize("extras", [False, True])
@pytest.mark.parametrize("N,H,I,E,K", SIZES)
def test_layer_bf16(N, H, I, E, K, extras):
    Layer(N, H, I, E, K, bias=extras, residual=extras, drop=0.2 if extras and N > 1 else 0.0, seed=N).check()


@pytest.mark.parametrize("extras", [False, True])
@pytest.mark.parametrize("N,H,I,E,K", SIZES_FP8)
def test_layer_fp8(N, H, I, E, K, extras):
    Layer(N, H, I, E, K, fp8=True, bias=extras, residual=extras, drop=0.2 if extras and N > 1 else 0.0, seed=N).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_long_sums_in_the_norm(fp8):
    """Per row, where a lost channel of 7168 shows: the bf16 rounding and the sums' own error."""
    layer = Layer(6, 7168, 2048, 8, 2, fp8=fp8, seed=11)
    got, (want, _) = layer.check(), layer.want()
    error = (got.double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(error.max()) <= bf16_bound(7168) + 2.0 ** -17


@pytest.mark.parametrize("fp8", [False, True])
def test_one_expert_for_all_tokens_and_every_count(fp8):
    """1 to 40 tokens of one expert beside others, by number of masked entries."""
    for n in (1, 2, 7, 8, 9, 15, 16, 17, 24, 33, 40):
        idx = torch.full((40, 2), -1, dtype=torch.int64)
        idx[:n, 0] = 3
        idx[::3, 1] = 1
        Layer(40, 384, 128, 4, 2, fp8=fp8, idx=idx.cuda(), seed=n).check()
        Layer(40, 384, 128, 20, 2, fp8=fp8, idx=idx.cuda(), seed=n).check()     # the small form


@pytest.mark.parametrize("tokens", [3, 6])      # 3 and 6 entries per expert: the small and the large form
def test_same_expert_twice_in_a_token(tokens):
    idx = torch.tensor([[2, 2, 2], [2, 0, 2], [-1, 1, 1]]).repeat(tokens // 3, 1).cuda()
    Layer(tokens, 136, 72, 3, 3, idx=idx, bias=True).check()


@pytest.mark.parametrize("E", [4, 1])           # the small and the large form
def test_tokens_without_experts_get_their_residual_or_zeros(E):
    idx = torch.tensor([[-1, -1], [E - 1, -1], [-1, -1]]).cuda()
    buf = dict(N=3, H=264, I=40, E=E, K=2) if E > 1 else dict(N=3, H=264, I=40, E=1, K=1)
    idx = idx[:, :buf["K"]].contiguous()
    if E == 1:
        idx = idx.repeat(3, 1)
        buf["N"] = 9
    layer = Layer(**buf, idx=idx, residual=True)
    got = layer.check()
    assert torch.equal(got[0::3], layer.residual[0::3]) and torch.equal(got[2::3], layer.residual[2::3])
    layer = Layer(**buf, idx=torch.full_like(idx, -1), residual=True, bias=True)
    assert torch.equal(layer.run(), layer.residual)
    layer.residual = None
    out = torch.full((buf["N"], 264), 7.0, device="cuda", dtype=torch.bfloat16)
    assert torch.equal(layer.run(out=out), torch.zeros_like(out))


@pytest.mark.parametrize("tokens", [7, 19])     # the small and the large form
@pytest.mark.parametrize("fp8", [False, True])
def test_what_masked_entries_and_unnamed_experts_hold_does_not_matter(fp8, tokens):
    layer = Layer(tokens, 256, 128, 6, 3, fp8=fp8, bias=True, drop=0.3, seed=5)
    layer.idx[layer.idx == 4] = -1
    before = layer.check()
    layer.wts[layer.idx < 0] = float("nan")
    for w in (layer.gu, layer.down):
        if fp8:
            w[0].view(torch.uint8)[4] = 0x7F
            w[1][4] = float("inf")
        else:
            w[4] = float("nan")
    for b in layer.bias:
        b[4] = float("nan")
    assert torch.equal(layer.run(), before)


@pytest.mark.parametrize("copies", [1, 4])      # the small and the large form
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_nan_codes_of_fp8_weights_give_nan(byte, copies):
    """One code of a row: that channel of every token of the expert, and no other."""
    idx = torch.tensor([[0], [1], [1], [0]]).repeat(copies, 1).cuda()
    layer = Layer(4 * copies, 256, 128, 2, 1, fp8=True, idx=idx)
    second = idx[:, 0] == 1
    before = layer.check()
    layer.down[0].view(torch.uint8)[1, 77, 101] = byte
    got = layer.run()
    assert bool(got[second, 77].isnan().all())
    got[second, 77] = before[second, 77]
    assert torch.equal(got, before)
    layer.gu[0].view(torch.uint8)[0, 128 + 5, 255] = byte   # an up row: the whole token
    assert bool(layer.run()[~second].isnan().all())


@pytest.mark.parametrize("E", [1, 2])           # the large and the small form
def test_every_fp8_code(E):
    """Weights of all 254 finite codes against one-hot tokens: exact but for the roundings behind them."""
    layer = Layer(8, 256, 128, E, 1, fp8=True, seed=3, idx=torch.zeros(8, 1, dtype=torch.int64).cuda())
    codes = torch.arange(256, dtype=torch.int64)
    codes[(codes & 0x7F) == 0x7F] = 0
    layer.gu[0].view(torch.uint8)[0, :] = codes.to(torch.uint8).cuda()[(torch.arange(256)[:, None] + torch.arange(256)) % 256]
    layer.gu[1].fill_(0.02)
    layer.x.zero_()
    layer.x[torch.arange(8), torch.arange(8) * 37 % 256] = 1.0
    layer.check()


def test_infinities_and_large_values():
    """A token of infinities and a huge one, beside others that stay as they are, in both forms and types."""
    for copies in (1, 5):
        for fp8 in (False, True):
            layer = Layer(3 * copies, 128, 128, 3, 1, fp8=fp8, idx=torch.tensor([[0], [1], [1]]).repeat(copies, 1).cuda())
            before = layer.check()
            layer.x[0, 5] = float("inf")
            layer.x[1] *= 1e18
            out = layer.run()
            assert not bool(out[0].isfinite().all())
            want, _ = layer.want()
            assert bool((out[1].double() - want[1]).abs().max() <= want[1].abs().max() * 2.0 ** -7)
            assert torch.equal(out[2:], before[2:])


@pytest.mark.parametrize("fp8", [False, True])
def test_every_number_of_sms_and_repeated_calls(fp8):
    """The sums are cut into as many shares as there are SMs: within the bounds for each number, and the same bits
    every time for one."""
    for sms, N in [(s, n) for s in (0, 1, 7, 64, 151, 152) for n in (15, 21)]:    # the small and the large form
        layer = Layer(N=N, H=512, I=256, E=12, K=3, fp8=fp8, bias=True, residual=True, seed=2, max_sms=sms)
        first = layer.check()
        for _ in range(3):
            assert torch.equal(layer.run(), first)


@pytest.mark.parametrize("N", [13, 15])         # the small and the large form
def test_residual_may_be_the_output(N):
    layer = Layer(N, 328, 72, 7, 2, bias=True, residual=True)
    want = layer.check()
    layer.residual = layer.residual.clone()
    assert layer.run(out=layer.residual) is layer.residual
    assert torch.equal(layer.residual, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [13, 40])         # the small and the large form
def test_in_place_on_the_residual_stream(N, fp8):
    """x + layer(x) written to x."""
    layer = Layer(N, 512, 256, 8, 2, fp8=fp8, bias=True)
    layer.residual = layer.x
    want = layer.check()
    for _ in range(5):
        x = layer.x.clone()
        got = layer.buf.expert_layer(x, layer.idx, layer.wts, layer.gu, layer.down, biases=layer.bias, residual=x, out=x)
        assert got is x and layer.buf.device_status() == ep.EP_OK and torch.equal(x, want)


def test_long_sums_of_equal_sign():
    """x = 1 and positive weights, 7168 channels: the tensor cores drop what falls off when they add (16 at a time,
    2^-23 of the sum each at most), and nothing else is lost: both products, both forms (1 and 3 experts' weights)."""
    for E in (1, 12):
        layer = Layer(5, 7168, 64, E, 1, idx=torch.zeros(5, 1, dtype=torch.int64).cuda())
        layer.x.fill_(1.0)
        layer.gu.abs_()
        layer.down.abs_()
        got, (want, _) = layer.run(), layer.want()
        error = (got.double() - want).norm() / want.norm()
        assert float(error) <= 2.0 ** -8 + 2 * (7168 / 16 + 64 / 16) * 2.0 ** -23


def test_a_wide_range_of_values_in_a_token():
    """FP8 weights: channels over seven decades beside each other in blocks of 128 (two codes hold 2^-13 of a block's
    largest exactly, and 2^-21 of it below)."""
    for N in (4, 40):
        layer = Layer(N, 512, 256, 8, 2, fp8=True, seed=9)
        g = torch.Generator("cuda").manual_seed(1)
        layer.x *= 10.0 ** (torch.rand(layer.x.shape, generator=g, device="cuda") * 7.0 - 3.5)
        layer.check()


@pytest.mark.parametrize("N", [4, 11])          # the small and the large form
def test_bad_ids_are_reported_and_skipped(N):
    layer = Layer(N, 136, 64, 5, 2)
    clean = layer.idx.clone()
    clean[1, 0] = clean[3, 1] = -1
    layer.idx = clean
    want = layer.check()
    layer.idx = clean.clone()
    layer.idx[1, 0], layer.idx[3, 1] = 5, -(1 << 40)
    out = layer.buf.expert_layer(layer.x, layer.idx, layer.wts, layer.gu, layer.down)
    assert layer.buf.device_status() == ep.EP_ERR_BAD_EXPERT
    assert torch.equal(out, want)
    layer.idx = clean
    assert torch.equal(layer.run(), want)


@pytest.mark.parametrize("N", [5, 13])          # the small and the large form
def test_weights_none_are_ones(N):
    layer = Layer(N, 128, 64, 6, 2)
    layer.wts.fill_(1.0)
    want = layer.check()
    layer.wts = None
    assert torch.equal(layer.run(), want)


@pytest.mark.parametrize("N", [9, 21])          # the small and the large form
def test_side_by_side_on_streams_and_in_graphs(N):
    """Two calls of one context at once, and two captured ones replayed with other inputs."""
    a, b = (Layer(N, 1024, 256, 16, 4, fp8=f, seed=s, bias=True) for f, s in ((False, 1), (True, 2)))
    want = a.check(), b.check()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    b.buf = a.buf
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for layer, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(layer.buf.expert_layer(layer.x, layer.idx, layer.wts, layer.gu, layer.down, biases=layer.bias))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs, outs = [], []
    for layer in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.buf.expert_layer(layer.x, layer.idx, layer.wts, layer.gu, layer.down, biases=layer.bias))
        graphs.append(g)
    fresh = Layer(N, 1024, 256, 16, 4, seed=7, bias=True)
    for layer in (a, b):
        layer.x.copy_(fresh.x)
        layer.idx.copy_(fresh.idx)
        layer.wts.copy_(fresh.wts)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for layer, out in zip((a, b), outs):
            want, tol = layer.want()
            assert_close(out, want, tol, "replayed")


def test_agrees_with_dispatch_experts_combine():
    """The bf16 path through the receive layout rounds h and y to bf16; the layer does not."""
    layer = Layer(24, 512, 256, 8, 2, seed=4)
    recv, _, h = layer.buf.low_latency_dispatch(layer.x.view(1, 24, 512), layer.idx.view(1, 24, 2), 24, 8, use_fp8=False)
    y, _ = layer.buf.expert_mlp(recv, layer.gu, layer.down, h)
    out = layer.buf.low_latency_combine(y, layer.idx.view(1, 24, 2), layer.wts, h, 8)
    want, tol = layer.want()
    got = layer.check()
    # gu (twice), h and y rounded to bf16: 2-norm well within the sum of the four roundings
    assert float((out.double() - want).norm() / want.norm()) <= 5 * BF16
    assert float((got.double() - want).norm() / want.norm()) <= BF16


def test_refusals_touch_nothing():
    layer = Layer(4, 128, 64, 5, 2)
    buf, out = layer.buf, torch.full((4, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    call = lambda **kw: buf.expert_layer(**{**dict(x=layer.x, topk_idx=layer.idx, topk_weights=layer.wts, w_gate_up=layer.gu,  # noqa: E731
                                                   w_down=layer.down, out=out), **kw})
    with pytest.raises(ValueError):
        call(x=layer.x[:, :64].contiguous())
    with pytest.raises(ValueError):
        call(x=layer.x.float())
    with pytest.raises(ValueError):
        call(w_down=cast_blocks(bf((5, 128, 128), 0)))
    with pytest.raises(ValueError):
        call(topk_weights=layer.wts[:2])
    with pytest.raises(ValueError):
        call(biases=(bf((5, 64), 0), None))
    with pytest.raises(ValueError):
        call(residual=layer.x[:2].contiguous())
    with pytest.raises(ValueError):
        call(topk_idx=layer.idx.int())
    with pytest.raises(ep.EPError) as e:
        call(w_gate_up=bf((5, 24, 128), 0), w_down=bf((5, 128, 12), 0))
    assert e.value.status == ep.EP_ERR_INVALID_ARG
    big = Layer(ep.EP_LAYER_MAX_TOKENS + 1, 128, 64, 5, 2)
    with pytest.raises(ep.EPError) as e:
        big.run()
    assert e.value.status == ep.EP_ERR_UNSUPPORTED
    lib, p = ep.lib(), lambda t: t.data_ptr()  # noqa: E731
    ws = torch.empty(ep.ep_expert_layer_workspace(buf.ctx, 4, 64), dtype=torch.uint8, device="cuda")
    args = [buf.ctx, p(layer.x), p(layer.idx), p(layer.wts), 4, 64, p(layer.gu), None, None, p(layer.down), None, None, None, p(ws),
            p(out), None]
    for at, value in ((1, None), (2, None), (6, None), (9, None), (13, None), (14, None), (1, p(layer.x) + 2), (13, p(ws) + 8), (4, -1),
                      (5, 0), (7, p(layer.wts))):
        bad = list(args)
        bad[at] = value
        assert lib.ep_expert_layer(*bad) == ep.EP_ERR_INVALID_ARG, (at, value)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    zero = list(args)
    zero[4] = 0
    assert lib.ep_expert_layer(*zero) == ep.EP_OK
    assert buf.device_status() == ep.EP_OK and bool((out == 3.0).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_lists_cut_into_jobs_agree_between_the_sms(fp8):
    """128 tokens of one expert, few tiles, many SMs: the jobs of one list run on different SMs."""
    for seed in range(4):
        layer = Layer(128, 256, 128, 3, 2, fp8=fp8, seed=seed, bias=True)
        first = layer.check()
        for _ in range(5):
            assert torch.equal(layer.run(), first)


def test_the_same_expert_for_every_entry():
    """4096 entries of one expert, 32 of each token."""
    Layer(128, 64, 16, 32, 32, idx=torch.ones(128, 32, dtype=torch.int64).cuda()).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_wait_that_runs_out_is_reported_and_leaves_nothing_behind(fp8):
    """The large form, an expert whose weights never come, 1 ms waits: the status says so; the next call is right
    again."""
    layer = Layer(24, 1024, 512, 8, 2, fp8=fp8, seed=1)
    want = layer.check()
    for _ in range(2):
        ep.ep_set_test_hooks(layer.buf.ctx, move_withhold_item=int(layer.idx[3, 1]), move_wait_ns=1_000_000)
        layer.buf.expert_layer(layer.x, layer.idx, layer.wts, layer.gu, layer.down)
        assert layer.buf.device_status() == ep.EP_ERR_TIMEOUT
        ep.ep_set_test_hooks(layer.buf.ctx)
        for _ in range(3):
            assert torch.equal(layer.run(), want)


def test_more_streams_than_there_are_counters():
    """The large form: from the 513th stream on a barrier counter comes from the workspace."""
    layer = Layer(2, 64, 16, 2, 5, idx=torch.tensor([[0, 1, 0, 1, 1], [1, 1, 0, 0, 0]]).cuda())
    want = layer.check()
    raw = lambda s: ep.ep_expert_layer(layer.buf.ctx, layer.x, layer.idx, layer.wts, 2, 16, layer.gu, None, None, layer.down, None,  # noqa: E731
                                       None, None, ws, out, stream=s)
    rt = ctypes.CDLL("libcudart.so")
    made = []
    for i in range(530):
        h = ctypes.c_void_p()
        assert rt.cudaStreamCreate(ctypes.byref(h)) == 0
        made.append(h)
        ws = torch.empty(ep.ep_expert_layer_workspace(layer.buf.ctx, 2, 16), dtype=torch.uint8, device="cuda")
        out = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        raw(torch.cuda.ExternalStream(h.value))
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    for h in made:
        assert rt.cudaStreamDestroy(h) == 0
    assert layer.buf.device_status() == ep.EP_OK


# e4m3, many entries for the SMs: tokens are laid out as codes before the products
LAID = [(128, 1920, 1024, 8, 8, 0), (67, 1664, 1920, 5, 5, 0), (60, 1152, 640, 4, 3, 16), (128, 256, 640, 16, 8, 7), (9, 1152, 640, 2, 2, 1)]


@pytest.mark.parametrize("N,H,I,E,K,sms", LAID)
@pytest.mark.parametrize("extras", [False, True])
def test_tokens_laid_out_as_codes(N, H, I, E, K, sms, extras):
    layer = Layer(N, H, I, E, K, fp8=True, bias=extras, residual=extras, drop=0.2 if extras else 0.0, max_sms=sms, seed=3)
    first = layer.check()
    for _ in range(3):
        assert torch.equal(layer.run(), first)


def test_laid_out_tokens_do_not_touch_each_other():
    """Tokens of NaN, infinities, zeros and the largest and smallest numbers change their own rows only."""
    layer = Layer(60, 1152, 640, 4, 3, fp8=True, max_sms=16, seed=5)
    first = layer.check()
    layer.x = layer.x.clone()
    layer.x[3, 5], layer.x[17, 200], layer.x[41] = float("inf"), float("nan"), 0.0
    layer.x[50] *= 2.0 ** 100
    layer.x[51] *= 2.0 ** -100
    got = layer.run()
    others = torch.ones(60, dtype=torch.bool, device="cuda")
    others[[3, 17, 41, 50, 51]] = False
    assert torch.equal(got[others], first[others])
    assert not bool(got[3].isfinite().any()) and bool(got[17].isnan().all()) and bool((got[41] == 0).all())


def test_laid_out_tokens_on_streams_and_in_graphs():
    layer = Layer(60, 1152, 640, 4, 3, fp8=True, bias=True, max_sms=16, seed=6)
    want = layer.check()
    call = lambda: layer.buf.expert_layer(layer.x, layer.idx, layer.wts, layer.gu, layer.down, biases=layer.bias)  # noqa: E731
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, call()))
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        outs = []
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i < 2:
                    graphs[i][0].replay()
                    outs.append(graphs[i][1])
                else:
                    outs.append(call())
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        for _, o in graphs:
            o.zero_()
    assert layer.buf.device_status() == ep.EP_OK


def test_a_wait_that_runs_out_with_tokens_laid_out():
    layer = Layer(60, 1152, 640, 4, 3, fp8=True, max_sms=16, seed=7)
    want = layer.check()
    for _ in range(2):
        ep.ep_set_test_hooks(layer.buf.ctx, move_withhold_item=int(layer.idx[3, 1]), move_wait_ns=1_000_000)
        layer.buf.expert_layer(layer.x, layer.idx, layer.wts, layer.gu, layer.down)
        assert layer.buf.device_status() == ep.EP_ERR_TIMEOUT
        ep.ep_set_test_hooks(layer.buf.ctx)
        for _ in range(3):
            assert torch.equal(layer.run(), want)
