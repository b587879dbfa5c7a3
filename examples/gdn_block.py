"""A decoder block out of the library's operators, with the gated delta rule, linear attention or window attention as its
token mixer, and a stack of such blocks: prefill, decoding from a state or a cache of keys and values (in bf16 or with
8-bit projections), and a training step's gradients.

    python examples/gdn_block.py            # on a GB300: runs each at a small size and prints what it took

The block (hidden width D = H * 128, feed-forward width F):

    n1     = rms_norm(x)                              q, k, v = n1 Wq^T, n1 Wk^T, n1 Wv^T;  a, b = n1 Wab^T (fp32)
    o      = delta rule of (q / |q|, k / |k|, v, logsigmoid(a), sigmoid(b)) per head
    stream = rms_norm_head(o) Wo^T + x                the residual's addition in the projection's epilogue
    y      = gated(rms_norm(stream)) Wd^T + stream    gated(n) = silu(n Wg^T) * (n Wu^T)

With linear attention o is that of (q / |q|, k / |k|, v) with a constant decay per head; with window attention that of
(q, k, v), several query heads to a key head, over the last tokens and the first ones.
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
ROOM = 256  # slots of a window layer's cache behind its prompt


def make_params(heads=16, ff=5504, seed=0, device="cuda", mixer="delta", kv_heads=None, window=1024, sinks=4):
    """Weights of a block.  ``mixer``: "delta", "linear" or "window" (which takes ``kv_heads``, ``window`` and ``sinks``)."""
    if mixer not in ("delta", "linear", "window"):
        raise ValueError(f"mixer must be delta, linear or window, not {mixer!r}")
    kv = kv_heads if mixer == "window" and kv_heads else heads
    g = torch.Generator(device=device).manual_seed(seed)
    D = heads * HEAD

    def w(rows, cols):
        return (torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5).bfloat16()

    return SimpleNamespace(
        mixer=mixer, window=window, sinks=sinks, decay=-torch.exp2(-5.0 - torch.arange(heads, device=device) * (7.0 / heads)),
        heads=heads, norm1=torch.ones(D, device=device), wq=w(D, D), wk=w(kv * HEAD, D), wv=w(kv * HEAD, D), wab=w(2 * heads, D),
        ab_bias=torch.cat([torch.full((heads,), 3.0), torch.zeros(heads)]).to(device),
        unit=torch.full((HEAD,), HEAD ** -0.5, device=device),  # rms_norm with this weight divides by the L2 norm
        onorm=torch.ones(HEAD, device=device), wo=w(D, D), norm2=torch.ones(D, device=device), wgu=w(2 * ff, D), wd=w(D, ff))


def quantise(p):
    """The projections that follow a norm, in e4m3 with a scale per output row (laid out once)."""
    names = ("wq", "wk", "wv", "wgu")
    return SimpleNamespace(**{n: gdn.quantize_rows(getattr(p, n)) for n in names})


def _heads(t):
    return t.view(*t.shape[:-1], -1, HEAD)


def _delta(p, s, state):
    ab = gdn.linear(s.n1, p.wab, p.ab_bias, out_dtype=torch.float32)
    s.a, b = ab[..., :p.heads], ab[..., p.heads:]
    s.g, s.beta = F.logsigmoid(s.a).contiguous(), torch.sigmoid(b).contiguous()
    if s.x.shape[1] == 1 and state is not None:
        return gdn.fused_recurrent_gated_delta_rule(s.qn, s.kn, s.v, s.g, s.beta, initial_state=state, output_final_state=True,
                                                    final_state=state)
    return gdn.chunk_gated_delta_rule(s.qn, s.kn, s.v, s.g, s.beta, initial_state=state, output_final_state=True,
                                      keys_unit_norm=True)


def _linear(p, s, state):
    if s.x.shape[1] == 1 and state is not None:
        return gdn.fused_recurrent_linear_attention(s.qn, s.kn, s.v, p.decay, initial_state=state, output_final_state=True,
                                                    final_state=state)
    return gdn.chunk_linear_attention(s.qn, s.kn, s.v, p.decay, initial_state=state, output_final_state=True)


def _window(p, s, cache):
    B, T = s.x.shape[:2]
    if cache is None:  # a prompt: its keys and values begin the cache
        o, s.lse = gdn.window_attention(s.qh, s.kh, s.v, p.window, p.sinks, return_lse=True)
        room = torch.zeros(B, ROOM, *s.v.shape[2:], dtype=s.v.dtype, device=s.v.device)
        return o, SimpleNamespace(k=torch.cat([s.kh, room], 1), v=torch.cat([s.v, room], 1),
                                  lengths=torch.full((B,), T, dtype=torch.int32, device=s.v.device), room=ROOM)
    if T > cache.room:
        raise ValueError(f"the cache has room for {cache.room} more tokens, not {T}")
    cache.room -= T
    rows, at = torch.arange(B, device=s.v.device)[:, None], cache.lengths[:, None] + torch.arange(T, device=s.v.device)
    cache.k[rows, at], cache.v[rows, at] = s.kh, s.v
    cache.lengths += T
    return gdn.window_attention_decode(s.qh, cache.k, cache.v, cache.lengths, p.window, p.sinks), cache


MIXERS = {"delta": _delta, "linear": _linear, "window": _window}


def forward(p, x, state=None, keep=None, q8=None):
    """The block on x [B, T, D]: returns (y, final state [B, H, 128, 128] fp32, or a window layer's cache).

    ``state``: the state to continue from; a single token updates it in place (decoding), a cache takes all new tokens.
    ``keep``: a namespace that receives what :func:`backward` needs.  ``q8``: :func:`quantise`'s weights: the projections
    after the norms run in 8 bits."""
    if q8 is None:
        n1, _ = gdn.rms_norm(x, p.norm1)
        q, k, v = (gdn.linear(n1, w) for w in (p.wq, p.wk, p.wv))
    else:
        (n8, s8, _), (n1, _) = gdn.rms_norm_quant(x, p.norm1), gdn.rms_norm(x, p.norm1)
        q, k, v = (gdn.linear(n8, w, x_scale=s8, weight_scale=s) for w, s in (q8.wq, q8.wk, q8.wv))
    s = keep if keep is not None else SimpleNamespace()
    vars(s).update(x=x, n1=n1, qh=_heads(q), kh=_heads(k), v=_heads(v))
    if p.mixer != "window":
        s.qn, _ = gdn.rms_norm(s.qh, p.unit, eps=1e-12)
        s.kn, _ = gdn.rms_norm(s.kh, p.unit, eps=1e-12)
    s.o, state = MIXERS[p.mixer](p, s, state)
    on, _ = gdn.rms_norm(s.o, p.onorm)
    s.on = on.view(x.shape)
    s.stream = gdn.linear(s.on, p.wo, residual=x)
    if q8 is None:
        s.n2, _ = gdn.rms_norm(s.stream, p.norm2)
        s.h = gdn.gated_linear(s.n2, p.wgu)
    else:
        s.n2, s2, _ = gdn.rms_norm_quant(s.stream, p.norm2)
        s.h = gdn.gated_linear(s.n2, q8.wgu[0], x_scale=s2, weight_scale=q8.wgu[1])
    return gdn.linear(s.h, p.wd, residual=s.stream), state


def backward(p, s, dy):
    """Gradients of a :func:`forward` from zero state that kept ``s``: (dx, {weight name: gradient})."""
    d = {}
    dh, d["wd"], _ = gdn.linear_bwd(dy, s.h, p.wd)
    dn2, d["wgu"] = gdn.gated_linear_bwd(dh, s.n2, p.wgu)
    dstream, d["norm2"] = gdn.rms_norm_bwd(dn2, s.stream, p.norm2, dy)  # joins the residual's gradient
    don, d["wo"], _ = gdn.linear_bwd(dstream, s.on, p.wo)
    do, d["onorm"] = gdn.rms_norm_bwd(_heads(don), s.o, p.onorm)
    grads = {}
    if p.mixer == "window":
        dq, dk, dv = gdn.window_attention_bwd(do, s.qh, s.kh, s.v, s.o, s.lse, p.window, p.sinks)
    else:
        if p.mixer == "linear":
            dqn, dkn, dv, _ = gdn.chunk_linear_attention_bwd(s.qn, s.kn, s.v, p.decay, do)
        else:
            dqn, dkn, dv, dbeta, dg, _ = gdn.chunk_gated_delta_rule_bwd(s.qn, s.kn, s.v, s.g, s.beta, do)
            grads["wab"] = torch.cat([dg * torch.sigmoid(-s.a), dbeta * s.beta * (1 - s.beta)], -1).bfloat16()
        dq, _ = gdn.rms_norm_bwd(dqn.bfloat16(), s.qh, p.unit, eps=1e-12)
        dk, _ = gdn.rms_norm_bwd(dkn.bfloat16(), s.kh, p.unit, eps=1e-12)
    grads.update(wq=dq, wk=dk, wv=dv.bfloat16())
    dn1 = None
    for name, grad in grads.items():
        one, d[name], _ = gdn.linear_bwd(grad.reshape(*s.x.shape[:-1], -1), s.n1, getattr(p, name))
        dn1 = one if dn1 is None else dn1 + one
    dx, d["norm1"] = gdn.rms_norm_bwd(dn1, s.x, p.norm1, dstream)
    return dx, d


def make_stack(mixers=("linear", "linear", "linear", "window"), **kw):
    """A block of each mixer, one behind the other."""
    return [make_params(seed=i, mixer=m, **kw) for i, m in enumerate(mixers)]


def forward_stack(layers, x, states=None, keeps=None):
    """The stack on x: (y, each layer's state or cache).  ``keeps``: a list that receives a namespace for each layer."""
    out = []
    for i, p in enumerate(layers):
        keep = None if keeps is None else SimpleNamespace()
        x, state = forward(p, x, None if states is None else states[i], keep)
        out.append(state)
        if keeps is not None:
            keeps.append(keep)
    return x, out


def backward_stack(layers, keeps, dy):
    """(dx, each layer's weight gradients)"""
    grads = []
    for p, s in zip(reversed(layers), reversed(keeps)):
        dy, d = backward(p, s, dy)
        grads.insert(0, d)
    return dy, grads


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

    stack = make_stack(kv_heads=4)
    prompt = torch.randn(64, 1024, D, device="cuda").bfloat16()
    _, states = forward_stack(stack, prompt)  # (the states and the cache that the tokens continue)

    def train_stack():
        keeps = []
        y, _ = forward_stack(stack, x, keeps=keeps)
        backward_stack(stack, keeps, y)

    for name, f in (("prefill 4 x 4096", lambda: forward(p, x)), ("prefill 4 x 4096, 8-bit projections", lambda: forward(p, x, q8=q8)),
                    ("decode 64 x 1", lambda: forward(p, token, cache)), ("decode 64 x 1, 8-bit projections", lambda: forward(p, token, cache, q8=q8)),
                    ("forward and backward 4 x 4096", train),
                    ("three linear layers and a window layer, prefill 4 x 4096", lambda: forward_stack(stack, x)),
                    ("those, decode 64 x 1 behind 1024", lambda: forward_stack(stack, token, states)),
                    ("those, forward and backward 4 x 4096", train_stack)):
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
