"""Plain 64-bit references and error bounds for the expert operators.

Bounds.  A product of bf16 (or e4m3) values is exact in fp32, so a sum of k of
them in fp32, in any order and even if every addition truncates, is off by at
most (k + 32) * 2^-23 * S with S the sum of the products' magnitudes (the 32
covers the few extra fp32 roundings of scales and partial sums).  A bf16
rounding adds 2^-8 / 2 of the value, an e4m3 rounding 2^-4 of it (2^-10 in
units of the scale below 2^-6)."""
from __future__ import annotations

import torch

BF16 = 2.0 ** -8        # half of a bf16 step, relative (8 significand bits), and what the sum's error adds to it


def sum_bound(k: int, s: torch.Tensor) -> torch.Tensor:
    return (k + 32) * 2.0 ** -23 * s


def topk_for_counts(counts, ranks: int = 1, seed: int = 0) -> torch.Tensor:
    """topk_idx [R, T, 1] that gives expert e exactly counts[e] rows (masked
    entries fill up the last rank)."""
    ids = torch.cat([torch.full((c,), e, dtype=torch.int64) for e, c in enumerate(counts)] + [torch.empty(0, dtype=torch.int64)])
    pad = -len(ids) % ranks
    ids = torch.cat([ids, torch.full((max(pad, ranks if len(ids) == 0 else 0),), -1, dtype=torch.int64)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(seed))]
    return ids.view(ranks, -1, 1)


def groups(buf, handle):
    """[(base, count)] of the experts, on the host."""
    t = handle.tensors()
    return list(zip(t["base"].tolist(), t["tokens_per_expert"].tolist()))


def in_use(rows: int, grp) -> torch.Tensor:
    m = torch.zeros(rows, dtype=torch.bool)
    for b, c in grp:
        m[b:b + c] = True
    return m.cuda()


def receive(rows, width, grp, seed, scale=1.0, dtype=torch.bfloat16):
    """A receive buffer: N(0, scale) in the rows in use, NaN elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.full((rows, width), float("nan"), device="cuda", dtype=dtype)
    for b, c in grp:
        if c:
            x[b:b + c] = (torch.randn(c, width, generator=g, device="cuda") * scale).to(dtype)
    return x


def weights(E, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(E, n, k, generator=g, device="cuda") * k ** -0.5).bfloat16()


def cast_rows(x: torch.Tensor):
    """The dispatch's FP8 rule per 128 channels of a row (fp32 steps)."""
    t = x.float().view(x.shape[0], -1, 128)
    a = t.abs().amax(-1).clamp_min(1e-4)
    q = (t * (448.0 / a).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(x.shape), a / torch.full_like(a, 448.0)   # by a tensor: an IEEE division (by a number multiplies)


def cast_blocks(w: torch.Tensor):
    """The same rule per 128 x 128 block of w [E, n, k]."""
    E, n, k = w.shape
    nb = -(-n // 128)
    t = torch.nn.functional.pad(w.float(), (0, 0, 0, nb * 128 - n)).view(E, nb, 128, k // 128, 128)
    a = t.abs().amax((2, 4)).clamp_min(1e-4)
    q = (t * (448.0 / a)[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(E, nb * 128, k)[:, :n].contiguous(), a / torch.full_like(a, 448.0)


def wide_rows(q, s):
    return q.float().double() * s.double().repeat_interleave(128, 1)


def wide_block(q, s):
    return q.float().double() * s.double().repeat_interleave(128, 0)[: q.shape[0]].repeat_interleave(128, 1)


def silu(g):
    return g * torch.sigmoid(g)


def assert_close(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}: "
        f"{got[tuple(bad.nonzero()[0])].item()} for {want[tuple(bad.nonzero()[0])].item()}")


def assert_untouched(out, sentinel, used, what=""):
    """Rows not in use still hold the sentinel's bits."""
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[out.element_size()]
    assert bool((out.view(kind)[~used] == sentinel.view(kind)[~used]).all()), f"{what}: a row outside the groups was written"
