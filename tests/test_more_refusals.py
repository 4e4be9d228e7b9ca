"""Refusals of the layer, linear and gradient calls that need no GPU: a NULL context is refused before any
CUDA call, and Buffer checks shapes before it calls the library."""
import ctypes

import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer, ep
from combine_get_dispatch_02_gb300 import build as epbuild

E = ep.EP_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    epbuild.build()
    return ep.lib()


def group(E=4, H=64, K=2, rows=16):
    """A Buffer without a context, for its checks of shapes alone."""
    b = object.__new__(Buffer)
    b.num_ranks, b.max_tokens_per_rank, b.hidden, b.num_experts, b.topk, b.rows, b._ctx = 1, 8, H, E, K, rows, None
    return b


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_layer_without_a_context(lib):
    n = ctypes.c_uint64(0)
    assert lib.ep_expert_layer(*[None] * 4, 1, 8, *[None] * 10) == E
    assert lib.ep_expert_layer_workspace(None, 1, 8, ctypes.byref(n)) == E


@pytest.mark.parametrize("change", [
    dict(x=bf(3, 64)), dict(x=bf(2, 32)), dict(topk_idx=torch.zeros(2, 3, dtype=torch.int64)), dict(topk_weights=torch.zeros(3, 2)),
    dict(w_gate_up=bf(3, 32, 64)), dict(w_gate_up=bf(4, 31, 64)), dict(w_gate_up=bf(4, 32, 72)), dict(w_down=bf(4, 64, 24)),
    dict(w_down=(bf(4, 64, 16), torch.zeros(4, 1, 1))), dict(biases=(bf(4, 30), None)), dict(biases=(None, bf(4, 63))),
    dict(residual=bf(3, 64)), dict(out=bf(3, 64)),
    dict(w_gate_up=(bf(4, 32, 64), torch.zeros(4, 2, 1)), w_down=(bf(4, 64, 16), torch.zeros(4, 1, 1)))])
def test_layer_shapes(change):
    args = dict(x=bf(2, 64), topk_idx=torch.zeros(2, 2, dtype=torch.int64), topk_weights=torch.zeros(2, 2), w_gate_up=bf(4, 32, 64),
                w_down=bf(4, 64, 16))
    with pytest.raises(ValueError):
        group().expert_layer(**{**args, **change})


def test_linear_and_gradients_without_a_context(lib):
    assert lib.ep_expert_linear(None, None, None, None, 8, 8, None, 0, 0, None, None, None, None) == E
    assert lib.ep_expert_linear_backward(None, None, None, None, 8, 0, 0, None, None, None) == E
    assert lib.ep_grad_norm(None, None, 0, None, None) == E
    assert lib.ep_grad_clip(None, None, 0, None, None, None, None) == E


@pytest.mark.parametrize("change", [
    dict(x=bf(16, 24)), dict(x=bf(15, 32)), dict(w=bf(3, 40, 32)), dict(bias=bf(4, 32)), dict(bias=bf(40)), dict(residual=bf(16, 32)),
    dict(z=bf(15, 40)), dict(out=bf(16, 48))])
def test_linear_shapes(change):
    args = dict(x=bf(16, 32), w=bf(4, 40, 32), handle=None)
    with pytest.raises(ValueError):
        group().expert_linear(**{**args, **change})


@pytest.mark.parametrize("change", [
    dict(dy=bf(15, 40)), dict(z=bf(16, 32)), dict(z=None), dict(out=bf(16, 32)), dict(dbias=torch.zeros(4, 32)), dict(accumulate=True)])
def test_linear_backward_shapes(change):
    args = dict(dy=bf(16, 40), z=bf(16, 40), handle=None, activation="relu")
    with pytest.raises(ValueError):
        group().expert_linear_backward(**{**args, **change})


def test_gradient_lists():
    for grads, out in (([torch.zeros(4)], None), ([torch.zeros(4)], []), ([bf(4)], [bf(4)])):
        with pytest.raises(ValueError):
            group().clip_grads(grads, 1.0, out=out)
