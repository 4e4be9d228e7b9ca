"""Gated experts between dispatch and combine, as a serving and as a training step.

serve: FP8 dispatch -> gate and up products, SwiGLU and cast -> down product -> combine
train: bf16 dispatch -> gate and up -> SwiGLU -> down -> combine, and back: the gradient of the
       combine is a dispatch whose rows take their entry's routing weight (and, for those weights, a
       product of each token's gradient with its experts' outputs), the experts' backward pass, the
       gradient of the dispatch is a combine

Usage: python examples/expert_mlp.py serve|train [--ranks R] [--tokens T] [--hidden H] [--experts E]
       [--topk K] [--inner I] [--padded] [--steps N]
Prints the mean time of a step and of its parts (CUDA events around each, L2 as the step leaves it).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_get_dispatch_02_gb300 import Buffer, ep  # noqa: E402


class Clock:
    """Times the parts of a step by CUDA events; reading waits for the GPU."""

    def __init__(self):
        self.marks = []

    def __call__(self, name):
        e = torch.cuda.Event(enable_timing=True)
        e.record()
        self.marks.append((name, e))

    def parts(self):
        torch.cuda.synchronize()
        return [(b[0], a[1].elapsed_time(b[1]) * 1e3) for a, b in zip(self.marks, self.marks[1:])]


def serve_step(buf, h, x, idx, wts, w_gate_up, w_down, clock):
    clock("start")
    recv, _, h = buf.low_latency_dispatch(x, idx, buf.max_tokens_per_rank, buf.num_experts, use_fp8=True, handle=h)
    clock("dispatch (FP8)")
    hidden = buf.expert_gate_fp8(recv, w_gate_up, h)
    clock("gate, up, SwiGLU, cast")
    y = buf.expert_gemm_fp8(hidden, w_down, h)
    clock("down")
    out = buf.low_latency_combine(y, idx, wts, h, buf.num_experts)
    clock("combine")
    return out


def combine_backward(buf, h, dout, y, wts):
    """Gradients of out[t] = sum_k wts[t, k] * y[row(t, k)]: (dy in the receive layout, dwts [N, K]);
    masked entries have none."""
    slot = h.tensors()["slot"].long()
    dy, _, _ = buf.low_latency_dispatch(dout, None, buf.max_tokens_per_rank, buf.num_experts, use_fp8=False, handle=h)
    # the weight of each row's entry; masked entries write behind the last row
    w = torch.zeros(buf.rows + 1, 1, device=dy.device)
    w[torch.where(slot < 0, buf.rows, slot).view(-1)] = wts.view(-1, 1)
    wide = dout.float()
    dw = torch.stack([(wide * y.index_select(0, s.clamp_min(0))).sum(1) for s in slot.unbind(1)], 1)
    return torch.mul(dy, w[:-1], out=dy), torch.where(slot < 0, 0.0, dw)


def train_step(buf, h, x, idx, wts, w_gate_up, w_down, grads, clock, loss_grad=lambda out: out):
    """Forward and backward of out = combine(experts(dispatch(x)), wts); loss_grad(out) [N, H] bf16 is the
    loss's gradient (the default: of half the sum of out's squares).  Adds the weights' gradients to
    ``grads``; returns (out, dx [N, H], dwts [N, K])."""
    clock("start")
    recv, _, h = buf.low_latency_dispatch(x, idx, buf.max_tokens_per_rank, buf.num_experts, use_fp8=False, handle=h)
    clock("dispatch")
    y, saved = buf.expert_mlp(recv, w_gate_up, w_down, h)
    clock("experts")
    out = buf.low_latency_combine(y, idx, wts, h, buf.num_experts)
    clock("combine")
    dy, dwts = combine_backward(buf, h, loss_grad(out), y, wts)
    clock("combine backward")
    dx, *_ = buf.expert_mlp_backward(dy, saved, w_gate_up, w_down, h, grads=grads)
    clock("experts backward")
    dtok = buf.low_latency_combine(dx, idx, None, h, buf.num_experts)
    clock("dispatch backward")
    return out, dtok, dwts


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("mode", choices=("serve", "train"))
    for name, value in (("ranks", 8), ("tokens", 512), ("hidden", 4096), ("experts", 64), ("topk", 6), ("inner", 1024),
                        ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--padded", action="store_true", help="fixed-size receive buffers (low-latency mode)")
    a = ap.parse_args()
    torch.manual_seed(0)
    dev = "cuda"
    buf = Buffer(a.ranks, a.tokens, a.hidden, a.experts, a.topk, low_latency_mode=a.padded)
    x = torch.randn(a.ranks, a.tokens, a.hidden, device=dev).bfloat16()
    logits = torch.randn(a.ranks * a.tokens, a.experts, device=dev)
    top = logits.topk(a.topk)
    idx, wts = top.indices.view(a.ranks, a.tokens, a.topk), torch.softmax(top.values, -1).contiguous()
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev).normal_(0.0, s[-1] ** -0.5)  # noqa: E731
    w_gate_up, w_down = bf(a.experts, 2 * a.inner, a.hidden), bf(a.experts, a.hidden, a.inner)
    h = buf.new_handle()
    if a.mode == "serve":
        qgu, qd = buf.cast_weights(w_gate_up), buf.cast_weights(w_down)
        step = lambda clock: (serve_step(buf, h, x, idx, wts, qgu, qd, clock),)  # noqa: E731
    else:
        grads = (torch.zeros(w_gate_up.shape, device=dev), torch.zeros(w_down.shape, device=dev))
        step = lambda clock: train_step(buf, h, x, idx, wts, w_gate_up, w_down, grads, clock)  # noqa: E731
    for _ in range(3):
        step(Clock())
    clocks = [Clock() for _ in range(a.steps)]
    for c in clocks:
        out = step(c)
    rows = [c.parts() for c in clocks]
    if buf.device_status() != ep.EP_OK or not all(bool(torch.isfinite(t.float()).all()) for t in out):
        raise SystemExit("the step failed")
    n = a.ranks * a.tokens
    total = sum(us for r in rows for _, us in r) / len(rows)
    print(f"{a.mode}: {n} tokens, top-{a.topk} of {a.experts}, hidden {a.hidden}, inner {a.inner}: {total:.1f} us a step "
          f"({n / total:.2f} M tokens/s)")
    for i, (name, _) in enumerate(rows[0]):
        print(f"  {name:24s} {sum(r[i][1] for r in rows) / len(rows):9.1f} us")


if __name__ == "__main__":
    main()
