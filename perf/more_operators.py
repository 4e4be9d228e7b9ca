"""A layer of experts with biases at both ends of its use, as cases that can be timed and compared: the product with
bias, activation and residual of a training or prefill step and its backward pass, the norm and the clipping of
the gradients that end a training step, and the whole layer of a decode step.

A case is one operator with its sizes.  ``prepare`` makes what a user's program has in hand, ``run`` makes one pass:
with ``own`` through this repository's ``Buffer``, else in elementary torch operations in 32 bits.

Operators (rows of expert e: base[e] .. base[e] + count[e]; other rows are neither read nor written):
  layer       out[t] = residual[t] + sum_k w[t, k] (Wd[e] h[t, k] + bd[e]), e = idx[t, k] (-1: none),
              h = silu(g) u, [g; u] = Wgu[e] x[t] + bgu[e]
              x, residual bf16 [N, H], Wgu [E, 2 * inner, H], Wd [E, H, inner] bf16, or e4m3 with a scale per
              128 x 128 block, biases bf16 (or none)                                    -> out bf16 [N, H]
  linear      z = W[e] x[row] + b[e], y[row] = act(z) + residual[row]
              x bf16 [rows, k], W bf16 [E, n, k], b bf16 / fp32 [E, n], residual bf16   -> y bf16 [rows, n], z bf16
  linear_bwd  dz[row] = dy[row] act'(z[row]), db[e] = sum_row dy[row] act'(z[row])
              dy, z bf16 [rows, n]                                                      -> dz bf16, db fp32 [E, n]
  clip        norm = sqrt(sum of all tensors' squares), g * min(1, max_norm / norm)
              bf16 / fp32 tensors, to other buffers or in place                         -> norm fp32, the tensors
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def _layer(name, tokens, hidden, inner, experts, topk, dtype="bf16", bias=False, residual=False, routing="uniform", drop=0.0):
    return dict(name=name, op="layer", tokens=tokens, hidden=hidden, inner=inner, experts=experts, topk=topk, dtype=dtype,
                bias=bias, residual=residual, routing=routing, drop=drop)


def _rows(name, op, ranks, tokens, experts, topk, n, k, act, routing="uniform", layout="packed", drop=0.0, bias="bf16",
          residual=False, save=False):
    return dict(name=name, op=op, ranks=ranks, tokens=tokens, experts=experts, topk=topk, n=n, k=k, act=act, routing=routing,
                layout=layout, drop=drop, bias=bias, residual=residual, save=save)


def _clip(name, tensors, numel, dtype, clipped):
    return dict(name=name, op="clip", tensors=tensors, numel=numel, dtype=dtype, clipped=clipped)


def listed():
    return [
        # one token in the tiny group (top-4 of 32, hidden 1024): the smallest decode step, latency alone
        _layer("layer_one_token", 1, 1024, 512, 32, 4),
        # one token at the low-latency setting's sizes, FP8 weights: 8 experts' bytes
        _layer("layer_fp8_one_token", 1, 7168, 2048, 256, 8, dtype="fp8", residual=True),
        # a small batch over the example's experts, with biases, masked entries and the residual stream
        _layer("layer_batch", 32, 4096, 1024, 64, 6, bias=True, residual=True, drop=0.1),
        # the most tokens of a call at the low-latency setting: nearly every expert has a few
        _layer("layer_fp8_most_tokens", 128, 7168, 2048, 256, 8, dtype="fp8"),
        # one token per rank in the tiny group: the product's smallest call, everything in its epilogue
        _rows("linear_one_token", "linear", 4, 1, 32, 4, 1024, 1024, "gelu", layout="padded", residual=True),
        # decode in low-latency mode, 16 rows per expert: bias and a second branch's output added, no activation
        _rows("linear_decode", "linear", 32, 16, 256, 8, 7168, 2048, "none", layout="padded", residual=True, bias="fp32"),
        # a training step in normal mode, about 1000 rows per expert: the activation's input is kept
        _rows("linear_normal", "linear", 8, 4096, 256, 8, 2048, 7168, "silu", routing="group", save=True),
        # its backward pass
        _rows("linear_bwd_normal", "linear_bwd", 8, 4096, 256, 8, 2048, 0, "gelu_tanh", routing="group"),
        # skewed routing, rows with gaps between the experts, channels that no tile divides: 0 to thousands of rows each
        _rows("linear_bwd_skew_odd", "linear_bwd", 13, 391, 52, 6, 1416, 0, "gelu", routing="zipf", layout="padded", drop=0.1),
        # a few biases' and norms' gradients: latency alone
        _clip("clip_small", 12, 1024, "bf16", True),
        # the fp32 gradients of the example's experts, clipped on their way to the optimizer's buffers
        _clip("clip_experts", 2, 64 * 4096 * 2048, "fp32", True),
        # many tensors of uneven sizes in place, the norm below the limit: nothing is written
        _clip("clip_none_in_place", 300, 1 << 21, "mixed", False),
    ]


def _cost(c):
    """Rough work of the plain form."""
    if c["op"] == "layer":
        passes = min(c["tokens"] * c["topk"], c["experts"])
        size = 3.0 * c["hidden"] * c["inner"]
        return max(passes * size * (60.0 + 2.0 * c["tokens"]), 60.0 * c["experts"] * size / 4)
    if c["op"] == "clip":
        return 60.0 * c["tensors"] * c["numel"]
    tokens = c["ranks"] * c["tokens"]
    most = tokens if c["routing"] == "zipf" else min(tokens, tokens * c["topk"] * 1.5 / c["experts"] + 32)
    rows = c["experts"] * tokens if c["layout"] == "padded" else tokens * c["topk"]
    return max(2.0 * c["experts"] * most * c["n"] * max(c["k"], 30), 400.0 * c["experts"] * c["n"] * c["k"],
               800.0 * rows * (c["n"] + c["k"]))


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(("layer", "layer", "layer", "linear", "linear", "linear_bwd", "clip"))
        routing, drop = rng.choice(("uniform", "uniform", "zipf")), rng.choice((0.0, 0.0, 0.1))
        if op == "layer":
            experts = log(2, 256)
            fp8 = rng.random() < 0.5
            hidden, inner = (128 * log(2, 56), 128 * log(1, 16)) if fp8 else (8 * log(32, 896), 8 * log(8, 256))
            c = _layer("", log(1, 128), hidden, inner, experts, min(rng.randint(1, 8), experts), dtype="fp8" if fp8 else "bf16",
                       bias=rng.random() < 0.5, residual=rng.random() < 0.5, routing=routing, drop=drop)
        elif op == "clip":
            c = _clip("", log(1, 1500), log(1, 1 << 28), rng.choice(("bf16", "fp32", "mixed")), rng.random() < 0.7)
            if c["tensors"] * c["numel"] > 1.2e9:
                continue
        else:
            ranks = rng.choice((1, 2, 4, 8, 13, 16, 32))
            experts = ranks * max(1, log(8, 256) // ranks)
            n, k = (8 * log(32, 896) for _ in range(2))
            c = _rows("", op, ranks, log(1, 4096), experts, min(rng.randint(1, 8), experts), n, k if op == "linear" else 0,
                      rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), routing=routing,
                      layout=rng.choice(("packed", "packed", "padded")), drop=drop,
                      bias=rng.choice(("bf16", "fp32", "none")) if op == "linear" else "bf16",
                      residual=op == "linear" and rng.random() < 0.5, save=op == "linear" and rng.random() < 0.5)
        del c["name"]
        if _cost(c) < 6e12:
            return c


# ------------------------------------------------------------------ inputs

def _route(c, N, gen):
    """topk_idx [N, K] int64, -1 for a masked entry."""
    E, K = c["experts"], c["topk"]
    dev = "cuda"
    logits = torch.randn(N, E, generator=gen, device=dev)
    if c["routing"] == "group":     # the 4 of 8 groups of experts with the best member, then top-k inside them
        best = logits.view(N, 8, E // 8).amax(2)
        keep = torch.zeros(N, 8, device=dev, dtype=torch.bool).scatter_(1, best.topk(4, dim=1).indices, True)
        logits = logits.masked_fill(~keep.repeat_interleave(E // 8, dim=1), float("-inf"))
    elif c["routing"] == "zipf":    # popularity (i + 1)^-1.2 over shuffled experts, drawn without replacement
        pop = (torch.randperm(E, generator=gen, device=dev).double() + 1.0).pow(-1.2)
        u = torch.rand(N, E, generator=gen, device=dev, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
        logits = (pop.log() - (-u.log()).log()).float()
    top = logits.topk(K, dim=1)
    idx, wts = top.indices.clone(), torch.softmax(top.values, -1).contiguous()
    if c["drop"] > 0:
        idx[torch.rand(idx.shape, generator=gen, device=dev) < c["drop"]] = -1
    return idx, wts


def _normal(shape, std, gen, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _weights_fp8(E, n, k, gen):
    """e4m3 codes [E, n, k] and a scale per 128 x 128 block [E, ceil(n / 128), k / 128]."""
    nb = -(-n // 128)
    q = torch.empty(E, n, k, dtype=FP8, device="cuda")
    sc = torch.empty(E, nb, k // 128, device="cuda")
    for e in range(E):
        v = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
        b = torch.nn.functional.pad(v, (0, 0, 0, nb * 128 - n)).view(nb, 128, k // 128, 128)
        a = b.abs().amax((1, 3)).clamp_min(1e-4)
        q[e] = (b * (448.0 / a)[:, None, :, None]).clamp_(-448.0, 448.0).reshape(nb * 128, k)[:n].to(FP8)
        sc[e] = a / 448.0
    return q, sc


def _received(rows, live, width, gen):
    """A receive buffer: N(0, 1) in the rows in use, what was there before (NaN) in the others."""
    x = torch.full((rows, width), float("nan"), dtype=torch.bfloat16, device="cuda")
    for part in live.split(32768):
        x.index_copy_(0, part, _normal((part.numel(), width), 1.0, gen))
    return x


def _prepare_layer(c, gen):
    N, H, I, E = c["tokens"], c["hidden"], c["inner"], c["experts"]
    idx, wts = _route(c, N, gen)
    s = dict(op="layer", idx=idx, wts=wts, x=_normal((N, H), 1.0, gen), bias=None, residual=None, out=torch.empty(
        N, H, dtype=torch.bfloat16, device="cuda"))
    if c["dtype"] == "fp8":
        s.update(gate_up=_weights_fp8(E, 2 * I, H, gen), down=_weights_fp8(E, H, I, gen))
    else:
        s.update(gate_up=_normal((E, 2 * I, H), H ** -0.5, gen), down=_normal((E, H, I), I ** -0.5, gen))
    if c["bias"]:
        s["bias"] = _normal((E, 2 * I), 0.5, gen), _normal((E, H), 0.5, gen)
    if c["residual"]:
        s["residual"] = _normal((N, H), 1.0, gen)
    if own:
        from combine_get_dispatch_02_gb300 import Buffer
        s["buf"] = Buffer(1, N, H, E, c["topk"])
    return s


def _prepare_rows(c, gen):
    N, E, n, k = c["ranks"] * c["tokens"], c["experts"], c["n"], c["k"]
    idx, _ = _route(c, N, gen)
    flat = idx.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=E).cpu()
    padded = c["layout"] == "padded"
    rows = E * N if padded else N * c["topk"]
    base = torch.arange(E) * N if padded else counts.cumsum(0) - counts
    most = max(1, int(counts.max()))
    owner = torch.repeat_interleave(torch.arange(E), counts)
    within = torch.arange(owner.numel()) - (counts.cumsum(0) - counts)[owner]
    s = dict(op=c["op"], act=c["act"], E=E, most=most, counts=counts.tolist(), base=base.tolist(), owner=owner.cuda(),
             row=(base[owner] + within).cuda(), cell=(owner * most + within).cuda(), bias=None, residual=None, z=None)
    live = s["row"]

    def result():
        return torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")

    if c["op"] == "linear":
        s.update(x=_received(rows, live, k, gen), w=_normal((E, n, k), k ** -0.5, gen), y=result())
        if c["bias"] != "none":
            s["bias"] = _normal((E, n), 0.5, gen, torch.float32 if c["bias"] == "fp32" else torch.bfloat16)
        if c["residual"]:
            s["residual"] = _received(rows, live, n, gen)
        if c["save"]:
            s["z"] = result()
    else:
        s.update(dy=_received(rows, live, n, gen), z=_received(rows, live, n, gen), dz=result(),
                 db=torch.zeros(E, n, device="cuda"))
    if own:     # the group and the layout that dispatch left in its handle
        from combine_get_dispatch_02_gb300 import Buffer
        s["buf"] = Buffer(c["ranks"], c["tokens"], 128, E, c["topk"], low_latency_mode=padded)
        s["handle"] = s["buf"].get_dispatch_layout(idx.view(c["ranks"], c["tokens"], c["topk"]))[3]
    return s


def _clip_sizes(c):
    """Element counts of the tensors: the first whole, the others from it down to a ninth, odd ones among them."""
    return [max(1, c["numel"] // (1 + (5 * i) % 9) - (i & 3)) if i else c["numel"] for i in range(c["tensors"])]


def _prepare_clip(c, gen):
    """The tensors lie one behind the other in a buffer per type, as an optimizer keeps them."""
    sizes = _clip_sizes(c)
    wide = [c["dtype"] == "fp32" or (c["dtype"] == "mixed" and i % 3 == 1) for i in range(len(sizes))]
    flat = [torch.empty(sum(n for n, w in zip(sizes, wide) if w == f32), dtype=torch.float32 if f32 else torch.bfloat16,
                        device="cuda") for f32 in (False, True)]
    to = [torch.zeros_like(f) for f in flat] if c["clipped"] else flat
    grads, out, at = [], [], [0, 0]
    for i, (n, w) in enumerate(zip(sizes, wide)):
        grads.append(flat[w][at[w]:at[w] + n].normal_(0.0, 10.0 ** -(i % 5), generator=gen))
        out.append(to[w][at[w]:at[w] + n])
        at[w] += n
    size = math.sqrt(sum(n * 100.0 ** -(i % 5) for i, n in enumerate(sizes)))     # about the norm
    s = dict(op="clip", grads=grads, out=out, flat=flat, to=to, max_norm=0.25 * size if c["clipped"] else 4.0 * size + 16.0)
    if own:
        from combine_get_dispatch_02_gb300 import Buffer
        s["buf"] = Buffer(1, 1, 128, 1, 1)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    make = {"layer": _prepare_layer, "clip": _prepare_clip}.get(case["op"], _prepare_rows)
    s = make(dict(case), gen)
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        return _own(s)
    return {"layer": _plain_layer, "linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "clip": _plain_clip}[s["op"]](s)


def _own(s):
    buf = s["buf"]
    if s["op"] == "layer":
        return buf.expert_layer(s["x"], s["idx"], s["wts"], s["gate_up"], s["down"], biases=s["bias"], residual=s["residual"],
                                out=s["out"])
    if s["op"] == "linear":
        y = buf.expert_linear(s["x"], s["w"], s["handle"], bias=s["bias"], activation=s["act"], residual=s["residual"],
                              out=s["y"], z=s["z"])
        return y if s["z"] is None else (y, s["z"])
    if s["op"] == "linear_bwd":
        return buf.expert_linear_backward(s["dy"], s["z"], s["handle"], activation=s["act"], out=s["dz"], dbias=s["db"])
    norm = buf.clip_grads(s["grads"], s["max_norm"], out=None if s["to"] is s["flat"] else s["out"])
    return norm, s["to"]


def _wide(w, e):
    """The weights of the experts e (a tensor of one index) in 32 bits."""
    if not isinstance(w, tuple):
        return w.index_select(0, e)[0].float()
    q, sc = w[0].view(torch.uint8).index_select(0, e)[0].view(FP8).float(), w[1].index_select(0, e)[0]
    n, k = q.shape
    return q.view(n, k // 128, 128).mul_(sc.repeat_interleave(128, 0)[:n].unsqueeze(-1)).view(n, k)


def _plain_layer(s):
    """Entry by entry where there are fewer entries than experts, else expert by expert for all tokens."""
    x, idx, wts = s["x"].float(), s["idx"], s["wts"]
    N, K = idx.shape
    E = (s["gate_up"][0] if isinstance(s["gate_up"], tuple) else s["gate_up"]).shape[0]
    acc = torch.zeros_like(x)

    def experts(e, rows):
        gu = rows @ _wide(s["gate_up"], e).T
        if s["bias"] is not None:
            gu = gu + s["bias"][0].index_select(0, e).float()
        g, u = gu.chunk(2, dim=-1)
        y = (g / (1.0 + torch.exp(-g)) * u) @ _wide(s["down"], e).T
        return y if s["bias"] is None else y + s["bias"][1].index_select(0, e).float()

    if N * K < E:
        for t in range(N):
            for k in range(K):
                e = idx[t, k:k + 1]
                y = experts(e.clamp_min(0), x[t:t + 1])
                acc[t:t + 1] += torch.where(e.view(1, 1) >= 0, wts[t, k] * y, torch.zeros_like(y))
    else:
        every = torch.arange(E, device=x.device)
        for i in range(E):
            share = torch.where(idx == i, wts, torch.zeros_like(wts)).sum(1, keepdim=True)
            acc += share * experts(every[i:i + 1], x)
    if s["residual"] is not None:
        acc += s["residual"].float()
    s["out"].copy_(acc)
    return s["out"]


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _gather(s, v):
    """The rows in use, fp32, as [E, most, width]; zero where an expert has fewer."""
    g = torch.zeros(s["E"] * s["most"], v.shape[1], device=v.device)
    return g.index_copy_(0, s["cell"], v[s["row"]].float()).view(s["E"], s["most"], v.shape[1])


def _plain_linear(s):
    z = torch.bmm(_gather(s, s["x"]), s["w"].float().transpose(1, 2))
    if s["bias"] is not None:
        z += s["bias"].float().unsqueeze(1)
    z = z.view(-1, z.shape[-1])[s["cell"]]
    y = _act(z, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"][s["row"]].float()
    s["y"].index_copy_(0, s["row"], y.to(torch.bfloat16))
    if s["z"] is None:
        return s["y"]
    s["z"].index_copy_(0, s["row"], z.to(torch.bfloat16))
    return s["y"], s["z"]


def _plain_linear_bwd(s):
    d = s["dy"][s["row"]].float() * _slope(s["z"][s["row"]].float(), s["act"])
    s["dz"].index_copy_(0, s["row"], d.to(torch.bfloat16))
    wide = torch.zeros(s["E"] * s["most"], d.shape[1], device=d.device).index_copy_(0, s["cell"], d)
    s["db"].copy_(wide.view(s["E"], s["most"], -1).sum(1))
    return s["dz"], s["db"]


def _plain_clip(s):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = total.sqrt()
    coef = (s["max_norm"] / norm).clamp_max(1.0).float()
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * coef)
    return norm.float(), s["to"]


# ------------------------------------------------------------------ work and the definition in 64 bits

def work(case):
    c = case
    if c["op"] == "clip":
        sizes = _clip_sizes(c)
        total = sum(n * (4 if c["dtype"] == "fp32" or (c["dtype"] == "mixed" and i % 3 == 1) else 2) for i, n in enumerate(sizes))
        return dict(bytes=total * (2 if c["clipped"] else 1) + 4, flops=(3 if c["clipped"] else 2) * sum(sizes))
    E, K = c["experts"], c["topk"]
    N = c["tokens"] if c["op"] == "layer" else c["ranks"] * c["tokens"]
    rows = N * K * (1.0 - c["drop"])
    used = min(E * (1.0 - (1.0 - K * (1.0 - c["drop"]) / E) ** N), rows)      # experts with a row, for even routing
    if c["op"] == "layer":
        H, I = c["hidden"], c["inner"]
        size = 1 + 4 / 16384 if c["dtype"] == "fp8" else 2
        return dict(bytes=used * (3 * H * I * size + (2 * (2 * I + H) if c["bias"] else 0)) + N * H * (6 if c["residual"] else 4)
                    + 12 * N * K, flops=6 * rows * H * I)
    n, k = c["n"], c["k"]
    if c["op"] == "linear":
        bias = {"none": 0, "bf16": 2, "fp32": 4}[c["bias"]]
        return dict(bytes=2 * rows * (n + k + n * c["residual"] + n * c["save"]) + used * n * (2 * k + bias) + 16 * E,
                    flops=2 * rows * n * k)
    return dict(bytes=6 * rows * n + 4 * E * n + 16 * E, flops=12 * rows * n)


def exact(case, seed):
    if case["op"] == "linear" and 2.0 * case["ranks"] * case["tokens"] * case["topk"] * case["n"] * case["k"] > 1.2e13:
        return None
    s = prepare(case, seed)
    wide = lambda t: t.to(torch.float64)  # noqa: E731
    if s["op"] == "clip":
        squares = [sum(float(wide(part).square().sum()) for part in g.split(1 << 26)) for g in s["grads"]]
        norm = math.sqrt(math.fsum(squares))
        coef = min(1.0, s["max_norm"] / norm)
        return torch.tensor(norm, dtype=torch.float64, device="cuda"), [wide(f) * coef for f in s["flat"]]
    if s["op"] == "layer":
        out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda") if s["residual"] is None else wide(s["residual"])
        x, wts = wide(s["x"]), wide(s["wts"])

        def matrix(w, e):
            if not isinstance(w, tuple):
                return wide(w[e])
            m = wide(w[0][e].float())
            return m * wide(w[1][e]).repeat_interleave(128, 0)[: m.shape[0]].repeat_interleave(128, 1)

        for e in range(case["experts"]):
            t, k = (s["idx"] == e).nonzero(as_tuple=True)
            if t.numel() == 0:
                continue
            v = x[t] @ matrix(s["gate_up"], e).T
            if s["bias"] is not None:
                v = v + wide(s["bias"][0][e])
            half = v.shape[1] // 2
            y = (v[:, :half] * torch.sigmoid(v[:, :half]) * v[:, half:]) @ matrix(s["down"], e).T
            if s["bias"] is not None:
                y = y + wide(s["bias"][1][e])
            out.index_add_(0, t, wts[t, k].unsqueeze(1) * y)
        return out
    act = case["act"]

    def normal_cdf(v):
        return 0.5 * torch.special.erfc(-v / math.sqrt(2.0))

    def tanh_arg(v):
        return math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)

    if s["op"] == "linear":
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        zs = None if s["z"] is None else torch.zeros_like(y)
        for e in range(s["E"]):
            b, m = s["base"][e], s["counts"][e]
            if m == 0:
                continue
            z = wide(s["x"][b:b + m]) @ wide(s["w"][e]).T
            if s["bias"] is not None:
                z = z + wide(s["bias"][e])
            a = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "gelu": lambda v: v * normal_cdf(v),
                 "gelu_tanh": lambda v: v * torch.sigmoid(2 * tanh_arg(v)), "silu": lambda v: v * torch.sigmoid(v)}[act](z)
            y[b:b + m] = a if s["residual"] is None else a + wide(s["residual"][b:b + m])
            if zs is not None:
                zs[b:b + m] = z
        return y if zs is None else (y, zs)
    dz = torch.zeros(s["dz"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["db"].shape, dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        b, m = s["base"][e], s["counts"][e]
        if m == 0:
            continue
        z = wide(s["z"][b:b + m])
        if act == "none":
            d = torch.ones_like(z)
        elif act == "relu":
            d = (z > 0).double()
        elif act == "gelu":
            d = normal_cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        else:
            p = torch.sigmoid(z if act == "silu" else 2 * tanh_arg(z))
            inner = 1.0 if act == "silu" else 2 * math.sqrt(2.0 / math.pi) * (1 + 3 * 0.044715 * z * z)
            d = p + z * p * (1 - p) * inner
        dz[b:b + m] = wide(s["dy"][b:b + m]) * d
        db[e] = dz[b:b + m].sum(0)
    return dz, db
