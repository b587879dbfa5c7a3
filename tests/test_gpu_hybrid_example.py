"""A stack of ``examples/gdn_block.py``'s blocks with linear attention, window attention and the gated delta rule as their token
mixers against a 64-bit composition: a prompt, tokens one at a time from the states and the cache, gradients."""
from types import SimpleNamespace

import pytest
import torch

import test_gpu_block_example as one
from test_gpu_block_example import rel

pytestmark = pytest.mark.gpu
block = one.block
LAYERS = 3


class Rounded(torch.autograd.Function):
    """A value, and the gradient that comes back to it, stored in bf16."""
    @staticmethod
    def forward(ctx, x):
        return x.bfloat16().double()

    @staticmethod
    def backward(ctx, g):
        return g.bfloat16().double()


def delta_rule(q, k, v, g, beta):
    S, o = torch.zeros(*q.shape[:1], *q.shape[2:], 128, dtype=torch.float64), []
    for t in range(q.shape[1]):
        S = S * g[:, t].exp()[..., None, None]
        d = (v[:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t])) * beta[:, t, :, None]
        S = S + k[:, t, :, :, None] * d[..., None, :]
        o.append(torch.einsum("bhkv,bhk->bhv", S, q[:, t]) * 128 ** -0.5)
    return torch.stack(o, 1)


def plain(p, x, r):
    """A block in 64 bits (on the CPU), `r` over everything that the block's operators write in bf16."""
    c = {k: v.detach().double().cpu() if not v.requires_grad else v for k, v in vars(p).items() if torch.is_tensor(v)}
    B, T, D = x.shape

    def norm(t, w, eps=1e-6):
        return r(t * torch.rsqrt(t.square().mean(-1, keepdim=True) + eps) * w)

    n1 = norm(x, c["norm1"])
    q, k, v = (r(n1 @ c[w].t()).view(B, T, -1, 128) for w in ("wq", "wk", "wv"))
    if p.mixer != "window":
        q, k = (norm(t, c["unit"], 1e-12) for t in (q, k))
    i = torch.arange(T)
    back = i[:, None] - i[None]
    if p.mixer == "linear":
        w = torch.exp(c["decay"][:, None, None] * back.clamp(min=0)) * (back >= 0)
        o = torch.einsum("bhij,bjhd->bihd", r(torch.einsum("bihd,bjhd->bhij", q, k) * w), v) * 128 ** -0.5
    elif p.mixer == "window":
        sees = (back >= 0) & ((back < p.window) | (i[None] < p.sinks))
        k, v = (t.repeat_interleave(p.heads // t.shape[2], 2) for t in (k, v))
        z = (torch.einsum("bihd,bjhd->bhij", q, k) * 128 ** -0.5).masked_fill(~sees, -torch.inf)
        o = torch.einsum("bhij,bjhd->bihd", z.softmax(-1), v)
    else:
        a, b = (n1 @ c["wab"].t() + c["ab_bias"]).split(p.heads, -1)
        o = delta_rule(q, k, v, torch.nn.functional.logsigmoid(a), torch.sigmoid(b))
    on = norm(r(o), c["onorm"]).reshape(B, T, D)
    stream = r(on @ c["wo"].t() + x)
    gate, up = (norm(stream, c["norm2"]) @ c["wgu"].t()).split(c["wd"].shape[1], -1)
    return r(r(gate * torch.sigmoid(gate) * up) @ c["wd"].t() + stream)


def plain_stack(layers, x, r=lambda t: t):
    for p in layers:
        x = plain(p, x, r)
    return x


def setup(block, B, T):
    layers = block.make_stack(("linear", "window", "delta"), heads=2, ff=200, kv_heads=1, window=40, sinks=3)
    g = torch.Generator(device="cuda").manual_seed(7)
    return layers, torch.randn(B, T, 256, generator=g, device="cuda").bfloat16(), g


def derivative(layers, x, grads, up, r):
    """{"x" or (layer, weight): gradient} of the 64-bit composition"""
    moved, at = [SimpleNamespace(**vars(p)) for p in layers], x.double().cpu().requires_grad_()
    for p, d in zip(moved, grads):
        for n in d:
            setattr(p, n, getattr(p, n).double().cpu().requires_grad_())
    (plain_stack(moved, at, r) * up).sum().backward()
    return {"x": at.grad} | {(i, n): getattr(p, n).grad for i, (p, d) in enumerate(zip(moved, grads)) for n in d}


def test_stack_forward_and_decode(block):
    """One block is within 1.5 % (see its own test); the roundings of three are independent: the square root of three times that."""
    layers, x, _ = setup(block, 2, 150)
    y, states = block.forward_stack(layers, x)
    want = plain_stack(layers, x.double().cpu())
    bound = 1.5e-2 * LAYERS ** 0.5
    assert rel(y, want) < bound
    head, states = block.forward_stack(layers, x[:, :120].contiguous())
    parts = [head]
    for t in range(120, 150):
        got, again = block.forward_stack(layers, x[:, t:t + 1].contiguous(), states)
        assert all(a is b for a, b in zip(again, states))
        parts.append(got)
    assert rel(torch.cat(parts, 1), want) < bound
    assert rel(torch.cat(parts, 1)[:, 120:], want[:, 120:]) < bound
    with pytest.raises(ValueError, match="room"):  # (the window layer's cache is full)
        block.forward(layers[1], torch.zeros(2, block.ROOM - 29, 256, dtype=x.dtype, device="cuda"), states[1])


def test_stack_gradients_against_differences(block):
    """As for one block (3 % of the terms' root mean square sum), for three: the square root of three times that.  The differences' step
    is 1e-6: here the first tokens' o is within a few times the norm's root of eps, whose slope a step of 1e-4 does not follow (8 %; the
    64-bit composition's own derivative agrees with the smaller step), and 64 bits leave 1e-16 of the loss over the step, far below."""
    layers, x, g = setup(block, 1, 90)
    keeps = []
    y, _ = block.forward_stack(layers, x, keeps=keeps)
    dy = torch.randn(y.shape, generator=g, device="cuda").bfloat16()
    dx, grads = block.backward_stack(layers, keeps, dy)
    up, t = dy.double().cpu(), 1e-6
    assert "wab" in grads[2] and "wab" not in grads[0] and "wab" not in grads[1]
    # the composition's own derivative, and that with its roundings
    exact, rounded = (derivative(layers, x, grads, up, r) for r in (lambda t: t, Rounded.apply))
    bad = []
    for i, name, grad in [(0, "x", dx)] + [(i, n, d) for i in range(LAYERS) for n, d in grads[i].items()]:
        d = torch.randn(grad.shape, generator=g, device="cuda").double()
        d = d + 3 * grad.double() / grad.double().square().mean().sqrt()
        loss = []
        for s in (t, -t):
            q, at = [SimpleNamespace(**vars(p)) for p in layers], x.double().cpu()
            if name == "x":
                at = at + s * d.cpu()
            else:
                setattr(q[i], name, getattr(layers[i], name).double() + s * d)
            loss.append(float((plain_stack(q, at) * up).sum()))
        want, got = (loss[0] - loss[1]) / (2 * t), float((grad.double() * d).sum())
        scale = float((grad.double() * d).square().sum().sqrt()) + abs(want)
        if not abs(got - want) <= 3e-2 * LAYERS ** 0.5 * scale:
            bad.append((i, name, got, want))
        # as far from the exact gradient as the same roundings in 64 bits bring it, half as much again for the sums' order
        at = "x" if name == "x" else (i, name)
        if not rel(grad, exact[at]) <= 1.5 * float((rounded[at] - exact[at]).norm() / exact[at].norm()):
            bad.append((i, name, rel(grad, exact[at])))
    assert not bad, bad


def test_mixer_names(block):
    with pytest.raises(ValueError, match="mixer"):
        block.make_params(2, 64, mixer="other")
