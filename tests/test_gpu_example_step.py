"""GPU check of the training example: its step's gradients against autograd in 64 bits."""
import importlib.util
import os

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer, ep
from expert_reference import silu, weights
from test_gpu_experts import _setup  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_mlp.py")
    spec = importlib.util.spec_from_file_location("expert_mlp_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("padded", [False, True])
def test_step_is_the_gradient_of_its_forward_pass(padded):
    """Tokens -> dispatch -> experts -> combine with routing weights (masked entries
    among them), for a loss sum(out * t): the gradients of the tokens, both weights
    and the routing weights.  The step keeps gu, h, y, dy, dh, dgu, dx and its result
    in bf16.  A bf16 rounding is 1.7e-3 in the 2-norm (2^-8 at most, over all
    mantissas): eight of them stay below 2^-6."""
    R, T, H, E, K, inner = 2, 45, 136, 6, 3, 72
    gen = torch.Generator("cuda").manual_seed(11)
    x = torch.randn(R, T, H, device="cuda", generator=gen).bfloat16()
    idx = torch.rand(R * T, E, device="cuda", generator=gen).topk(K).indices.view(R, T, K)
    idx[0, :7, 1] = -1
    idx[1, 3] = -1      # a token without an expert
    wts = torch.rand(R * T, K, device="cuda", generator=gen) * 2.0 - 0.5
    target = torch.randn(R * T, H, device="cuda", generator=gen).bfloat16()
    wgu, wd = weights(E, 2 * inner, H, 1), weights(E, H, inner, 2)
    grads = torch.zeros(wgu.shape, device="cuda"), torch.zeros(wd.shape, device="cuda")
    buf = Buffer(R, T, H, E, K, low_latency_mode=padded)
    got = example().train_step(buf, buf.new_handle(), x, idx, wts, wgu, wd, grads, lambda name: None,
                               loss_grad=lambda out: target)
    assert buf.device_status() == ep.EP_OK

    args = [t.double().requires_grad_() for t in (x.view(R * T, H), wts, wgu, wd)]
    tok, w, a, b = args
    out, flat = 0.0, idx.view(R * T, K)
    for k in range(K):
        e = flat[:, k].clamp_min(0)
        v = torch.einsum("nh,nih->ni", tok, a[e])
        y = torch.einsum("ni,nhi->nh", silu(v[:, :inner]) * v[:, inner:], b[e])
        out = out + torch.where(flat[:, k:k + 1] < 0, 0.0, w[:, k:k + 1] * y)
    want = torch.autograd.grad((out * target.double()).sum(), args)
    for name, g, ref in (("out", got[0], out.detach()), ("x", got[1], want[0]), ("routing weights", got[2], want[1]),
                         ("gate and up", grads[0], want[2]), ("down", grads[1], want[3])):
        assert float((g.double() - ref).norm() / ref.norm()) < 2.0 ** -6, name
    assert bool((got[2][flat < 0] == 0).all())
