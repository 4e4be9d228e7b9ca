"""GPU checks of the example's steps with biases, clipping and the whole layer: a run of the operators together, as
they are used."""
import os
import subprocess
import sys

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer, ep
from expert_reference import silu, weights
from test_gpu_example_step import example
from test_gpu_experts import _setup  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_step_with_biases_and_clipping(captured):
    """As the step without them: every gradient within 2^-6 in the 2-norm (eight bf16 roundings of 1.7e-3), the
    biases' among them, and then all scaled by one factor: the norm they are left with is the limit."""
    R, T, H, E, K, inner = 2, 45, 136, 6, 3, 72
    gen = torch.Generator("cuda").manual_seed(11)
    x = torch.randn(R, T, H, device="cuda", generator=gen).bfloat16()
    idx = torch.rand(R * T, E, device="cuda", generator=gen).topk(K).indices.view(R, T, K)
    idx[0, :7, 1] = -1
    idx[1, 3] = -1      # a token without an expert
    wts = torch.rand(R * T, K, device="cuda", generator=gen) * 2.0 - 0.5
    target = torch.randn(R * T, H, device="cuda", generator=gen).bfloat16()
    wgu, wd = weights(E, 2 * inner, H, 1), weights(E, H, inner, 2)
    biases = torch.randn(E, 2 * inner, device="cuda", generator=gen).bfloat16(), torch.randn(E, H, device="cuda", generator=gen)
    params = (wgu, wd, *biases)
    grads = [torch.zeros(t.shape, device="cuda") for t in params]
    buf = Buffer(R, T, H, E, K, low_latency_mode=False)
    h = buf.new_handle()

    def step():
        return example().train_step(buf, h, x, idx, wts, wgu, wd, tuple(grads[:2]), lambda name: None, loss_grad=lambda out: target,
                                    biases=biases, bias_grads=tuple(grads[2:]), max_norm=0.5)

    if captured:
        step()      # what is set up on first use
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = step()
        for g in grads:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
    else:
        got = step()
    assert buf.device_status() == ep.EP_OK

    args = [t.double().requires_grad_() for t in (x.view(R * T, H), wts, *params)]
    tok, w, a, b, ba, bb = args
    out, flat = 0.0, idx.view(R * T, K)
    for k in range(K):
        e = flat[:, k].clamp_min(0)
        v = torch.einsum("nh,nih->ni", tok, a[e]) + ba[e]
        y = torch.einsum("ni,nhi->nh", silu(v[:, :inner]) * v[:, inner:], b[e]) + bb[e]
        out = out + torch.where(flat[:, k:k + 1] < 0, 0.0, w[:, k:k + 1] * y)
    want = torch.autograd.grad((out * target.double()).sum(), args)
    for name, g, ref in (("out", got[0], out.detach()), ("x", got[1], want[0]), ("routing weights", got[2], want[1])):
        assert float((g.double() - ref).norm() / ref.norm()) < 2.0 ** -6, name
    norm = torch.stack([t.norm() for t in want[2:]]).norm()
    for g, ref in zip(grads, want[2:]):
        ref = ref * (0.5 / norm)
        assert float((g.double() - ref).norm() / ref.norm()) < 2.0 ** -6
    assert abs(float(torch.stack([g.double().norm() for g in grads]).norm()) - 0.5) <= 2.0 ** -19


@pytest.mark.parametrize("args", [["train", "--bias", "--clip", "1.0"], ["decode"], ["decode", "--bias", "--tokens", "1"]])
def test_example_runs(args):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    small = ["--ranks", "2", "--hidden", "256", "--experts", "8", "--topk", "2", "--inner", "128", "--steps", "2"]
    if "--tokens" not in args:
        small += ["--tokens", "8"]
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "expert_mlp.py"), *args, *small], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith(args[0])
