"""A gated-delta-rule decoder block out of the library's operators: prefill, decoding from a state cache (in bf16
or with 8-bit projections), and a training step's gradients.

    python examples/gdn_block.py            # on a GB300: runs each at a small size and prints what it took

The block (hidden width D = H * 128, feed-forward width F):

    n1     = rms_norm(x)                              q, k, v = n1 Wq^T, n1 Wk^T, n1 Wv^T;  a, b = n1 Wab^T (fp32)
    o      = delta rule of (q / |q|, k / |k|, v, logsigmoid(a), sigmoid(b)) per head
    stream = rms_norm_head(o) Wo^T + x                the residual's addition in the projection's epilogue
    y      = gated(rms_norm(stream)) Wd^T + stream    gated(n) = silu(n Wg^T) * (n Wu^T)
"""
from __future__ import annotations

import os
import sys
import time
from types import SimpleNamespace

import torch
import torch.nn.functional as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gated_deltanet_gb300 as gdn  # noqa: E402

HEAD = 128


def make_params(heads=16, ff=5504, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    D = heads * HEAD

    def w(rows, cols):
        return (torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5).bfloat16()

    return SimpleNamespace(
        heads=heads, norm1=torch.ones(D, device=device), wq=w(D, D), wk=w(D, D), wv=w(D, D), wab=w(2 * heads, D),
        ab_bias=torch.cat([torch.full((heads,), 3.0), torch.zeros(heads)]).to(device),
        unit=torch.full((HEAD,), HEAD ** -0.5, device=device),  # rms_norm with this weight divides by the L2 norm
        onorm=torch.ones(HEAD, device=device), wo=w(D, D), norm2=torch.ones(D, device=device), wgu=w(2 * ff, D), wd=w(D, ff))


def quantise(p):
    """The projections that follow a norm, in e4m3 with a scale per output row (laid out once)."""
    names = ("wq", "wk", "wv", "wgu")
    return SimpleNamespace(**{n: gdn.quantize_rows(getattr(p, n)) for n in names})


def _heads(t, p):
    return t.view(*t.shape[:-1], p.heads, HEAD)


def forward(p, x, state=None, keep=None, q8=None):
    """The block on x [B, T, D]: returns (y, final state [B, H, 128, 128] fp32).

    ``state``: the state to continue from; a single token updates it in place (decoding).  ``keep``: a namespace that
    receives what :func:`backward` needs.  ``q8``: :func:`quantise`'s weights: the projections after the norms run in 8
    bits."""
    if q8 is None:
        n1, _ = gdn.rms_norm(x, p.norm1)
        q, k, v = (gdn.linear(n1, w) for w in (p.wq, p.wk, p.wv))
    else:
        (n8, s8, _), (n1, _) = gdn.rms_norm_quant(x, p.norm1), gdn.rms_norm(x, p.norm1)
        q, k, v = (gdn.linear(n8, w, x_scale=s8, weight_scale=s) for w, s in (q8.wq, q8.wk, q8.wv))
    ab = gdn.linear(n1, p.wab, p.ab_bias, out_dtype=torch.float32)
    a, b = ab[..., :p.heads], ab[..., p.heads:]
    qn, _ = gdn.rms_norm(_heads(q, p), p.unit, eps=1e-12)
    kn, _ = gdn.rms_norm(_heads(k, p), p.unit, eps=1e-12)
    g, beta = F.logsigmoid(a).contiguous(), torch.sigmoid(b).contiguous()
    v = _heads(v, p)
    if x.shape[1] == 1 and state is not None:
        o, state = gdn.fused_recurrent_gated_delta_rule(qn, kn, v, g, beta, initial_state=state, output_final_state=True,
                                                        final_state=state)
    else:
        o, state = gdn.chunk_gated_delta_rule(qn, kn, v, g, beta, initial_state=state, output_final_state=True,
                                              keys_unit_norm=True)
    on, _ = gdn.rms_norm(o, p.onorm)
    on = on.view(x.shape)
    stream = gdn.linear(on, p.wo, residual=x)
    if q8 is None:
        n2, _ = gdn.rms_norm(stream, p.norm2)
        h = gdn.gated_linear(n2, p.wgu)
    else:
        n2, s2, _ = gdn.rms_norm_quant(stream, p.norm2)
        h = gdn.gated_linear(n2, q8.wgu[0], x_scale=s2, weight_scale=q8.wgu[1])
    y = gdn.linear(h, p.wd, residual=stream)
    if keep is not None:
        vars(keep).update(x=x, n1=n1, q=q, k=k, a=a, beta=beta, qn=qn, kn=kn, v=v, g=g, o=o, on=on, stream=stream, n2=n2, h=h)
    return y, state


def backward(p, s, dy):
    """Gradients of a :func:`forward` from zero state that kept ``s``: (dx, {weight name: gradient})."""
    d = {}
    dh, d["wd"], _ = gdn.linear_bwd(dy, s.h, p.wd)
    dn2, d["wgu"] = gdn.gated_linear_bwd(dh, s.n2, p.wgu)
    dstream, d["norm2"] = gdn.rms_norm_bwd(dn2, s.stream, p.norm2, dy)  # joins the residual's gradient
    don, d["wo"], _ = gdn.linear_bwd(dstream, s.on, p.wo)
    do, d["onorm"] = gdn.rms_norm_bwd(_heads(don, p), s.o, p.onorm)
    dqn, dkn, dv, dbeta, dg, _ = gdn.chunk_gated_delta_rule_bwd(s.qn, s.kn, s.v, s.g, s.beta, do)
    dq, _ = gdn.rms_norm_bwd(dqn.bfloat16(), _heads(s.q, p), p.unit, eps=1e-12)
    dk, _ = gdn.rms_norm_bwd(dkn.bfloat16(), _heads(s.k, p), p.unit, eps=1e-12)
    dab = torch.cat([dg * torch.sigmoid(-s.a), dbeta * s.beta * (1 - s.beta)], -1).bfloat16()
    dn1 = None
    for name, grad in (("wq", dq), ("wk", dk), ("wv", dv.bfloat16()), ("wab", dab)):
        one, d[name], _ = gdn.linear_bwd(grad.reshape(*s.x.shape[:-1], -1), s.n1, getattr(p, name))
        dn1 = one if dn1 is None else dn1 + one
    dx, d["norm1"] = gdn.rms_norm_bwd(dn1, s.x, p.norm1, dstream)
    return dx, d


def main():
    p = make_params()
    q8 = quantise(p)
    D = p.heads * HEAD
    x = torch.randn(4, 4096, D, device="cuda").bfloat16()
    token = torch.randn(64, 1, D, device="cuda").bfloat16()
    cache = torch.zeros(64, p.heads, HEAD, HEAD, device="cuda")

    def train():
        keep = SimpleNamespace()
        y, _ = forward(p, x, keep=keep)
        backward(p, keep, y)

    for name, f in (("prefill 4 x 4096", lambda: forward(p, x)), ("prefill 4 x 4096, 8-bit projections", lambda: forward(p, x, q8=q8)),
                    ("decode 64 x 1", lambda: forward(p, token, cache)), ("decode 64 x 1, 8-bit projections", lambda: forward(p, token, cache, q8=q8)),
                    ("forward and backward 4 x 4096", train)):
        for _ in range(3):
            f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(10):
            f()
        torch.cuda.synchronize()
        print(f"{name}: {(time.perf_counter() - t) * 100:.3f} ms")
    assert gdn.read_layer_status() == 0 and gdn.read_device_status() == 0


if __name__ == "__main__":
    main()
