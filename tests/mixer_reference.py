"""Plain 64-bit forms of the token mixers beside the gated delta rule (linear attention with a decay per head, attention with a
sliding window and sinks), with bounds on what their kernels may be off, counted in roundings.

Everything is written out per sequence and head as full matrices over the tokens.  Bounds: `SUM` is half a step of fp32; a kernel's
fp32 sum of n terms is off by at most n SUM of the sum of the terms' sizes; `half(dtype)` is half a step of a rounding to dtype.
Operands of the tensor cores are rounded to bf16 once more (`half(bfloat16)` of each)."""
import torch

SUM = 2.0 ** -24
BF = torch.bfloat16


def half(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, want, bound, what=""):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: not finite at other places"
    f = torch.isfinite(want)
    assert torch.equal(got[~f], want[~f]), what
    off = (got - want).abs()[f] - (bound.expand_as(want)[f] + 1e-30)
    assert off.numel() == 0 or off.max() <= 0, f"{what}: off by {float(off.max()):.3g} more than allowed, at {int(off.argmax())} of {off.numel()}"


def check_norm(got, want, rel, what=""):
    """Roundings are not all to one side: the 2-norm sees a wrong term that an element's bound lets through."""
    f = torch.isfinite(want)
    off = float((got.double() - want)[f].norm()) / max(1e-30, float(want[f].norm()))
    assert off <= rel, f"{what}: 2-norm off by {off:.3g} of its value"


def sequences(t, cu):
    """[B, T, h, d] as a list of [h, tokens, d] in 64 bits."""
    x = t.double().transpose(1, 2)
    return list(x) if cu is None else [x[0][:, a:b] for a, b in zip(cu.tolist(), cu.tolist()[1:])]


def joined(parts, like, cu):
    """The reverse of sequences."""
    if cu is None:
        return torch.stack(parts).transpose(1, 2)
    out = torch.zeros(like.shape[0], parts[0].shape[0], like.shape[1], parts[0].shape[2], dtype=torch.float64, device=like.device)
    for p, a, b in zip(parts, cu.tolist(), cu.tolist()[1:]):
        out[0][:, a:b] = p
    return out.transpose(1, 2)


def powers(decay, n):
    """exp(decay n) per head with 0 steps leaving everything, for a decay of minus infinity too"""
    return torch.where(n == 0, 1.0, torch.exp(decay[:, None, None] * n.clamp_min(1)))


# ---------------------------------------------------------------- linear attention
def linear(q, k, v, decay, scale, h0, cu):
    """o, ht and the same with every factor's size (what bounds sums and roundings)."""
    HV, V, r = v.shape[2], v.shape[3], v.shape[2] // q.shape[2]
    d = torch.zeros(HV, dtype=torch.float64, device=q.device) if decay is None else decay.double()
    got = []
    for size in (False, True):
        os, hs = [], []
        for n, (qs, ks, vs) in enumerate(zip(*(sequences(t, cu) for t in (q, k, v)))):
            s0 = torch.zeros(HV, q.shape[3], V, dtype=torch.float64, device=q.device) if h0 is None else h0[n].double()
            qs, ks = qs.repeat_interleave(r, 0), ks.repeat_interleave(r, 0)
            if size:
                qs, ks, vs, s0 = qs.abs(), ks.abs(), vs.abs(), s0.abs()
            T = qs.shape[1]
            i = torch.arange(T, device=q.device)
            gap = i[:, None] - i
            w = torch.where(gap >= 0, powers(d, gap.clamp_min(0)[None].expand(HV, -1, -1)), 0.0)
            o = ((qs @ ks.mT) * w) @ vs + powers(d, (i + 1)[None, :, None]) * (qs @ s0)
            os.append(abs(scale) * o if size else scale * o)
            t = torch.full((1, 1, 1), T, device=q.device)
            hs.append((ks * powers(d, (T - 1 - i)[None, :, None])).mT @ vs + powers(d, t) * s0)
        got += [joined(os, q, cu), torch.stack(hs) if hs else torch.zeros(0, HV, q.shape[3], V, dtype=torch.float64, device=q.device)]
    return got


def linear_bwd(q, k, v, decay, do, scale, h0, dht, cu):
    """dq, dk, dv, dh0 by autograd of the plain form in 64 bits (dh0 None without h0), and their sizes."""
    HV, r = v.shape[2], v.shape[2] // q.shape[2]
    x = [t.double().detach().requires_grad_() for t in (q, k, v)] + [None if h0 is None else h0.double().detach().requires_grad_()]
    o, ht, _, _ = linear(x[0], x[1], x[2], decay, scale, x[3], cu)
    loss = (o * do.double()).sum() + (0 if dht is None else (ht * dht.double()).sum())
    grads = torch.autograd.grad(loss, [t for t in x if t is not None], allow_unused=True)
    grads = [torch.zeros_like(t) if g is None else g for g, t in zip(grads, [t for t in x if t is not None])]
    a = [t.double().abs().detach().requires_grad_() for t in (q, k, v)] + [None if h0 is None else h0.double().abs().detach().requires_grad_()]
    o, ht, _, _ = linear(a[0], a[1], a[2], decay, abs(scale), a[3], cu)
    loss = (o * do.double().abs()).sum() + (0 if dht is None else (ht * dht.double().abs()).sum())
    sizes = torch.autograd.grad(loss, [t for t in a if t is not None], allow_unused=True)
    sizes = [torch.zeros_like(t) if g is None else g for g, t in zip(sizes, [t for t in a if t is not None])]
    if h0 is None:
        grads.append(None)
        sizes.append(None)
    return grads, sizes


def linear_bound(value, size, terms, dtype):
    """An output of dtype: its own rounding, the fp32 sums, and in bf16 the rounding of the operands of two products in a row
    (decayed products of q and k, the state; `size` bounds what each of them contributes)."""
    b = half(dtype) * value.abs() + terms * SUM * size
    return b + 1.01 * half(BF) * size if dtype == BF else b


def state_bound(size, terms, dtype):
    """States are fp32: the sums, and in bf16 the split of the decayed values into two bf16 parts (2^-16 of them)."""
    return (terms * SUM + (2.0 ** -16 if dtype == BF else 0)) * size


# ---------------------------------------------------------------- window attention
def seen(Lq, Lk, window, sinks, device):
    p = torch.arange(Lq, device=device)[:, None] + Lk - Lq
    j = torch.arange(Lk, device=device)
    return (j <= p) & ((p - j < window) | (j < sinks))


def _heads(q, k, v, cu, cu_k):
    G = q.shape[2] // k.shape[2]
    for qs, ks, vs in zip(sequences(q, cu), sequences(k, cu_k), sequences(v, cu_k)):
        yield qs, ks.repeat_interleave(G, 0), vs.repeat_interleave(G, 0)


def window(q, k, v, w, sinks, scale, cu=None, cu_k=None):
    """o, lse, and the bounds of both."""
    cu_k = cu if cu_k is None else cu_k
    D, dtype = q.shape[3], q.dtype
    parts = [[], [], [], []]
    for qs, ks, vs in _heads(q, k, v, cu, cu_k):
        m = seen(qs.shape[1], ks.shape[1], w, sinks, q.device)
        z = torch.where(m, scale * (qs @ ks.mT), -torch.inf)
        lse = torch.logsumexp(z, -1, keepdim=True) if ks.shape[1] else torch.full((*qs.shape[:2], 1), -torch.inf, dtype=torch.float64, device=q.device)
        p = torch.where(m, torch.exp(z - torch.where(torch.isfinite(lse), lse, 0.0)), 0.0)
        o = p @ vs
        # a score is off by its sum's roundings and by those of the exponent (2^-21 of a weight by the fast exponential)
        dz = torch.where(m, (D + 4) * SUM * abs(scale) * (qs.abs() @ ks.mT.abs()) + 4 * SUM * (z.abs() + lse.abs()) + 2.0 ** -21, 0.0)
        dz = torch.where(torch.isfinite(dz), dz, 0.0)
        worst = dz.amax(-1, keepdim=True) if ks.shape[1] else torch.zeros_like(lse)
        n = ks.shape[1] + 8
        bo = half(dtype) * o.abs() + ((2 * worst + n * SUM) + (1.01 * half(BF) if dtype == BF else 0)) * (p @ vs.abs())
        bl = worst + n * SUM + 4 * SUM * torch.where(torch.isfinite(lse), lse.abs(), 0.0)
        for a, b in zip(parts, (o, lse, bo, bl)):
            a.append(b)
    o, lse, bo, bl = (joined(p, q, cu) for p in parts)
    return o, lse[..., 0].transpose(1, 2), bo, bl[..., 0].transpose(1, 2)


def window_bwd(do, q, k, v, o, w, sinks, scale, cu=None, cu_k=None):
    """(dq, dk, dv) and their bounds; `o` is the forward's rounded output, which delta is taken from."""
    cu_k = cu if cu_k is None else cu_k
    D, G, dtype = q.shape[3], q.shape[2] // k.shape[2], q.dtype
    eo, r = half(dtype), half(BF) if dtype == BF else 0
    out = [[] for _ in range(6)]
    for (qs, ks, vs), g, ro in zip(_heads(q, k, v, cu, cu_k), sequences(do, cu), sequences(o, cu)):
        m = seen(qs.shape[1], ks.shape[1], w, sinks, q.device)
        z = torch.where(m, scale * (qs @ ks.mT), -torch.inf)
        lse = torch.logsumexp(z, -1, keepdim=True) if ks.shape[1] else torch.full((*qs.shape[:2], 1), -torch.inf, dtype=torch.float64, device=q.device)
        p = torch.where(m, torch.exp(z - torch.where(torch.isfinite(lse), lse, 0.0)), 0.0)
        dp = g @ vs.mT
        delta = (p * dp).sum(-1, keepdim=True)
        dz = p * (dp - delta) * scale
        n = max(qs.shape[1] * G, ks.shape[1]) + D + 16
        # what p, dp and delta may be off
        ep = p * (2 * (D + 4) * SUM * abs(scale) * (qs.abs() @ ks.mT.abs()) + 2.0 ** -20 + 8 * SUM * torch.where(m, z.abs(), 0.0) + 8 * SUM * torch.where(torch.isfinite(lse), lse.abs(), 0.0))
        ed = (D + 4) * SUM * (g.abs() @ vs.mT.abs()) + eo * 1.01 * (g.abs() * ro.abs()).sum(-1, keepdim=True) + n * SUM * (p * dp.abs()).sum(-1, keepdim=True)
        if dtype == BF:  # (o's own error beside its rounding: the weights' in bf16)
            ed = ed + 1.02 * r * (g.abs() * (p @ vs.abs())).sum(-1, keepdim=True)
        ez = abs(scale) * (ep * (dp - delta).abs() + p * ed) * 1.02 + (r + 4 * SUM) * dz.abs()
        epv = ep + r * p
        fold = lambda t: t.reshape(k.shape[2], G, *t.shape[1:]).sum(1)  # noqa: E731
        grads = dz @ ks, fold(dz.mT @ qs), fold(p.mT @ g)
        sums = (ez + n * SUM * dz.abs()) @ ks.abs(), fold((ez + n * SUM * dz.abs()).mT @ qs.abs()), fold((epv + n * SUM * p).mT @ g.abs())
        for i in range(3):
            out[i].append(grads[i])
            out[3 + i].append(eo * grads[i].abs() + 1.02 * sums[i])
    got = [joined(out[i], t, c) for i, t, c in ((0, q, cu), (1, k, cu_k), (2, v, cu_k), (3, q, cu), (4, k, cu_k), (5, v, cu_k))]
    return got[:3], got[3:]


def window_step(q, k, v, lengths, w, sinks, scale):
    """o and its bound: the last T tokens of each filled cache."""
    os, bs = [], []
    for n in range(q.shape[0]):
        L = max(0, min(int(lengths[n]), k.shape[1]))
        o, _, b, _ = window(q[n:n + 1], k[n:n + 1, :L], v[n:n + 1, :L], w, sinks, scale)
        os.append(o[0])
        bs.append(b[0])
    return torch.stack(os), torch.stack(bs)
