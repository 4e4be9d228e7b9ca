"""Refusals of outputs that overlap what their call still reads, by one row or one number too: the host refuses them,
nothing runs.  What may be shared stays allowed."""
import pytest
import torch

from combine_get_dispatch_02_gb300 import Buffer
from combine_get_dispatch_02_gb300 import build as epbuild
from combine_get_dispatch_02_gb300 import ep
from expert_reference import receive, weights
from test_gpu_expert_layer import Layer
from test_gpu_expert_linear import group

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    epbuild.build()
    torch.cuda.set_device(0)


def refused(f, *args, **kw):
    with pytest.raises(ep.EPError) as e:
        f(*args, **kw)
    assert e.value.status == ep.EP_ERR_INVALID_ARG


def beside(t, after, numbers):
    """A tensor like t and one like `after`, which begins `numbers` numbers before the end of the first."""
    whole = torch.full((t.numel() + after.numel() - numbers,), 7.0, device="cuda", dtype=t.dtype)
    a, b = whole[:t.numel()].view(t.shape), whole[t.numel() - numbers:].view(after.shape)
    a.copy_(t)
    return a, b


def test_linear():
    buf, h, grp = group([3, 5, 33])
    n = k = 40
    x, w, res = receive(buf.rows, k, grp, 1), weights(3, n, k, 2), receive(buf.rows, n, grp, 3)
    like = torch.zeros(buf.rows, n, device="cuda", dtype=torch.bfloat16)
    z = torch.zeros_like(like)
    bias = torch.zeros(3, n, device="cuda", dtype=torch.bfloat16)
    for numbers in (8, 40, x.numel() - 8):      # whole pieces of 16 bytes: the alignment is right
        a, b = beside(x, like, numbers)
        refused(buf.expert_linear, a, w, h, out=b)
        refused(buf.expert_linear, a, w, h, out=like, z=b)
        b, a = beside(like, x, numbers)
        refused(buf.expert_linear, a, w, h, out=b)
        a, b = beside(res, like, numbers)
        refused(buf.expert_linear, x, w, h, residual=a, out=b)
        refused(buf.expert_linear, x, w, h, residual=a, out=like, z=b)
        a, b = beside(z, like, numbers)
        refused(buf.expert_linear, x, w, h, z=a, out=b)
    a, b = beside(w, like, 8)
    refused(buf.expert_linear, x, a, h, out=b)
    a, b = beside(bias, like, 8)
    refused(buf.expert_linear, x, w, h, bias=a, out=b)
    refused(buf.expert_linear, x, w, h, bias=a, out=like, z=b)
    torch.cuda.synchronize()
    assert bool((like == 0).all()) and bool((z == 0).all())
    # next to each other, and the residual as either output
    a, b = beside(x, like, 0)
    want, wz = buf.expert_linear(x, w, h, residual=res, activation="gelu", z=z).clone(), z.clone()
    live = slice(0, 41)
    assert torch.equal(buf.expert_linear(a, w, h, residual=res, activation="gelu", out=b)[live], want[live])
    r = res.clone()
    assert torch.equal(buf.expert_linear(x, w, h, residual=r, activation="gelu", out=r, z=z)[live], want[live])
    r = res.clone()
    assert torch.equal(buf.expert_linear(x, w, h, residual=r, activation="gelu", z=r)[live], want[live])
    assert torch.equal(r[live], wz[live]) and torch.equal(z[live], wz[live]) and buf.device_status() == ep.EP_OK


def test_linear_backward():
    buf, h, grp = group([3, 5, 33])
    dy, z = receive(buf.rows, 40, grp, 1), receive(buf.rows, 40, grp, 2)
    out, db = torch.zeros_like(dy), torch.zeros(3, 40, device="cuda")
    for numbers in (8, 40, dy.numel() - 8):
        a, b = beside(dy, out, numbers)
        refused(buf.expert_linear_backward, a, z, h, activation="gelu", out=b, dbias=db)
        a, b = beside(z, out, numbers)
        refused(buf.expert_linear_backward, dy, a, h, activation="gelu", out=b, dbias=db)
    for t, kw in ((dy, {"out": out}), (z, {"out": out}), (out, {})):
        whole = torch.zeros(t.numel() + 240, device="cuda", dtype=torch.bfloat16)
        a, b = whole[:t.numel()].view(t.shape), whole[t.numel() - 8:t.numel() + 232].view(torch.float32).view(3, 40)
        args = {"out": a} if t is out else kw
        refused(buf.expert_linear_backward, a if t is dy else dy, a if t is z else z, h, activation="gelu", dbias=b, **args)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((db == 0).all())
    # z is not read without an activation: it may lie anywhere
    a, b = beside(dy, out, 0)
    buf.expert_linear_backward(a, b, h, out=b, dbias=db)
    assert torch.equal(b[:41], dy[:41]) and buf.device_status() == ep.EP_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_layer(fp8):
    layer = Layer(9, 256, 128, 5, 2, fp8=fp8, bias=True, residual=True)
    want = layer.check()
    like = torch.zeros_like(want)
    N, H, I = 9, 256, 128
    (wgu, sgu), (wd, sd) = ((layer.gu, None), (layer.down, None)) if not fp8 else (layer.gu, layer.down)
    need = ep.ep_expert_layer_workspace(layer.buf.ctx, N, I)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    names = dict(x=layer.x, idx=layer.idx, wts=layer.wts, wgu=wgu, sgu=sgu, bgu=layer.bias[0], wd=wd, sd=sd, bd=layer.bias[1],
                 residual=layer.residual, ws=ws, out=like)

    def call(**kw):
        t = {**names, **kw}
        ep.ep_expert_layer(layer.buf.ctx, t["x"], t["idx"], t["wts"], N, I, t["wgu"], t["sgu"], t["bgu"], t["wd"], t["sd"], t["bd"],
                           t["residual"], t["ws"], t["out"])

    def shared(a, b, numbers):
        """Tensors like a and b in one piece of memory, the second from `numbers` bytes before the end of the first."""
        size = a.numel() * a.element_size()
        whole = torch.zeros(size + b.numel() * b.element_size(), dtype=torch.uint8, device="cuda")
        first, second = whole[:size].view(a.dtype).view(a.shape), whole[size - numbers:size - numbers + b.numel() * b.element_size()]
        first.copy_(a)
        return first, second.view(b.dtype).view(b.shape)

    for name, t in names.items():
        if t is None:
            continue
        if name != "out":
            a, b = shared(t, like, 16)
            refused(call, **{name: a, "out": b})
        if name != "ws":
            a, b = shared(t, ws, 16)
            refused(call, **{name: a, "ws": b})
    torch.cuda.synchronize()
    assert bool((like == 0).all()) and bool((ws == 0).all())
    a, b = shared(layer.x, like, 0)
    call(x=a, out=b)
    assert torch.equal(b, want) and layer.buf.device_status() == ep.EP_OK


def test_gradients():
    buf = Buffer(1, 1, 128, 1, 1)
    flat = torch.ones(2048, dtype=torch.float64, device="cuda")
    partials, last, first = flat[:1024], flat[1023:1030].view(torch.float32), flat[1024:1030].view(torch.float32)
    norm, other = torch.zeros(1, device="cuda"), torch.ones(64, device="cuda")
    refused(ep.ep_grad_norm, buf.ctx, ep.grad_list([other, last]), partials)
    refused(ep.ep_grad_clip, buf.ctx, ep.grad_list([other, last]), partials, 1.0, norm)
    refused(ep.ep_grad_clip, buf.ctx, ep.grad_list([first, other]), partials, 1.0, other[63:])
    refused(ep.ep_grad_clip, buf.ctx, ep.grad_list([first], [other[:12]]), partials, 1.0, other[5:6])
    torch.cuda.synchronize()
    assert bool((flat == 1).all()) and bool((other == 1).all())
    first.fill_(2.0)
    ep.ep_grad_norm(buf.ctx, ep.grad_list([first]), partials)
    ep.ep_grad_clip(buf.ctx, ep.grad_list([first], [other[:12]]), partials, 1e9, other[12:13])
    assert float(other[12]) == pytest.approx(48.0 ** 0.5, rel=1e-6) and bool((other[:12] == 2).all()) and bool((other[13:] == 1).all())
