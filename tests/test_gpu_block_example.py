"""The decoder block of ``examples/gdn_block.py`` (every operator of the library together) against a 64-bit
composition with the oracle's recurrence: forward, decoding from a state cache, 8-bit projections, gradients."""
import os
import sys
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from layer_reference import norm
from oracle import recurrence

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import gdn_block
    return gdn_block


def setup(block, B, T, heads=2, ff=200):
    p = block.make_params(heads, ff, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for n in ("norm1", "norm2"):
        setattr(p, n, 1 + 0.2 * torch.randn(heads * 128, generator=g, device="cuda"))
    return p, torch.randn(B, T, heads * 128, generator=g, device="cuda").bfloat16(), g


def plain(p, x):
    """The block in 64 bits (on the CPU)."""
    c = {k: v.detach().double().cpu() for k, v in vars(p).items() if torch.is_tensor(v)}
    x = x.double().cpu()
    B, T, D = x.shape
    n1 = norm(x, None, c["norm1"], 1e-6)[0]
    q, k, v = ((n1 @ c[w].t()).view(B, T, p.heads, 128) for w in ("wq", "wk", "wv"))
    a, b = (n1 @ c["wab"].t() + c["ab_bias"]).split(p.heads, -1)
    qn, kn = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
    o, ht = recurrence(qn.numpy(), kn.numpy(), v.numpy(), torch.nn.functional.logsigmoid(a).numpy(), torch.sigmoid(b).numpy(), 128 ** -0.5,
                       None, None, gate="scalar")
    on = norm(torch.from_numpy(o), None, c["onorm"], 1e-6)[0].reshape(B, T, D)
    stream = on @ c["wo"].t() + x
    n2 = norm(stream, None, c["norm2"], 1e-6)[0]
    gate, up = (n2 @ c["wgu"].t()).split(c["wd"].shape[1], -1)
    return (gate * torch.sigmoid(gate) * up) @ c["wd"].t() + stream, torch.from_numpy(ht)


def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


def test_forward_and_decode(block):
    """About ten roundings to bf16 lie on the way (2^-9 root mean square each, halved where the residual dominates):
    1.5 % in the 2-norm covers them; e4m3 operands (2^-5 root mean square each) 6 %."""
    p, x, _ = setup(block, 2, 150)
    y, state = block.forward(p, x)
    want, ht = plain(p, x)
    assert rel(y, want) < 1.5e-2 and rel(state, ht) < 1.5e-2
    y8, _ = block.forward(p, x, q8=block.quantise(p))
    assert 1e-4 < rel(y8, want) < 6e-2
    # a prefill of 120 tokens, then one at a time from the state cache
    head, cache = block.forward(p, x[:, :120].contiguous())
    parts = [head]
    for t in range(120, 150):
        got, same = block.forward(p, x[:, t:t + 1].contiguous(), cache)
        assert same is cache
        parts.append(got)
    assert rel(torch.cat(parts, 1), want) < 1.5e-2 and rel(cache, ht) < 1.5e-2


def test_gradients_against_differences(block):
    """Along a random direction of the input and of each weight: central differences of the 64-bit block (step 1e-4)
    against the gradients, whose operands are rounded to bf16 on the way: 3 % of the terms' root mean square sum."""
    p, x, g = setup(block, 1, 90)
    keep = SimpleNamespace()
    y, _ = block.forward(p, x, keep=keep)
    dy = torch.randn(y.shape, generator=g, device="cuda").bfloat16()
    dx, dw = block.backward(p, keep, dy)
    up, t = dy.double().cpu(), 1e-4
    for name, grad in {"x": dx, **dw}.items():
        d = torch.randn(grad.shape, generator=g, device="cuda").double()
        # the gradient's own direction has a large share, so that the comparison is not of noise
        d = d + 3 * grad.double() / grad.double().square().mean().sqrt()
        loss = []
        for s in (t, -t):
            q, xs = SimpleNamespace(**vars(p)), x.double()
            if name == "x":
                xs = xs + s * d
            else:
                setattr(q, name, getattr(p, name).double() + s * d)
            loss.append(float((plain(q, xs)[0] * up).sum()))
        want, got = (loss[0] - loss[1]) / (2 * t), float((grad.double() * d).sum())
        scale = float((grad.double() * d).square().sum().sqrt()) + abs(want)
        assert abs(got - want) <= 3e-2 * scale, (name, got, want)


def test_example_runs(block, capsys):
    block.make_params(2, 256)  # (the full sizes are the example's own run)
    assert np.isfinite(float(block.forward(*setup(block, 1, 70)[:2])[0].float().sum()))
