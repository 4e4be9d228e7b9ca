"""GPU checks of the whole layer: what a wait that runs out leaves behind, and which tensors may share memory."""
import ctypes

import pytest
import torch

from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from test_gpu_expert_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    epbuild.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_barrier_is_put_back_behind_all_arrivals(fp8):
    """With the context's 512 counters taken the barrier is the end of the workspace, where it can be looked at: zero
    behind every call, the waits run out or not (an expert whose weights never come, 1 ms waits)."""
    layer = Layer(24, 1024, 512, 8, 2, fp8=fp8, seed=1)
    want, ctx = layer.check(), layer.buf.ctx
    w, s = (layer.gu, layer.down), (None, None)
    if fp8:
        w, s = (layer.gu[0], layer.down[0]), (layer.gu[1], layer.down[1])
    ws = torch.empty(ep.ep_expert_layer_workspace(ctx, 24, 512), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)

    def call(stream):
        ep.ep_expert_layer(ctx, layer.x, layer.idx, layer.wts, 24, 512, w[0], s[0], None, w[1], s[1], None, None, ws, out, stream=stream)

    rt = ctypes.CDLL("libcudart.so")
    made = []
    for i in range(513):
        h = ctypes.c_void_p()
        assert rt.cudaStreamCreate(ctypes.byref(h)) == 0
        made.append(torch.cuda.ExternalStream(h.value))
        call(made[-1])
        torch.cuda.synchronize()
    try:
        for i in range(60):
            ws.fill_(0xA5)
            torch.cuda.synchronize()
            held = i % 3 < 2
            if held:
                ep.ep_set_test_hooks(ctx, move_withhold_item=int(layer.idx[i % 24, i % 2]), move_wait_ns=1_000_000)
            call(made[-1])
            torch.cuda.synchronize()
            ep.ep_set_test_hooks(ctx)
            assert layer.buf.device_status() == (ep.EP_ERR_TIMEOUT if held else ep.EP_OK)
            assert bool((ws[-256:-248] == 0).all()) and bool((ws[-248:] == 0xA5).all()), i
            assert held or torch.equal(out, want)
    finally:
        for s in made:
            assert rt.cudaStreamDestroy(ctypes.c_void_p(s.cuda_stream)) == 0


# N, H, I, E, K, fp8, SMs: the small form, the large one with 16 and with 64 columns a job, tokens laid out
FORMS = [(9, 264, 72, 8, 2, False, 0), (9, 256, 128, 8, 2, True, 0), (3, 2824, 1416, 40, 6, False, 0), (3, 2176, 1920, 20, 4, True, 0),
         (40, 264, 72, 8, 2, False, 0), (33, 1152, 256, 4, 3, True, 0), (60, 1152, 640, 4, 3, True, 16)]


@pytest.mark.parametrize("N,H,I,E,K,fp8,sms", FORMS)
@pytest.mark.parametrize("shared", ["x", "residual", "both"])
def test_the_output_may_be_what_is_read(N, H, I, E, K, fp8, sms, shared):
    """In each form, over and over: the output is x, the residual, or both of them."""
    layer = Layer(N, H, I, E, K, fp8=fp8, bias=True, residual=True, drop=0.1, seed=4, max_sms=sms)
    if shared == "both":
        layer.residual = layer.x
    want = layer.check()
    for _ in range(10):
        x = layer.x.clone()
        residual = x if shared == "both" else layer.residual.clone()
        out = residual if shared == "residual" else x
        got = layer.buf.expert_layer(x, layer.idx, layer.wts, layer.gu, layer.down, biases=layer.bias, residual=residual, out=out)
        assert got is out and layer.buf.device_status() == ep.EP_OK and torch.equal(out, want)
