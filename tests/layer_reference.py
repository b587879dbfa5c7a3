"""Plain 64-bit forms of the decoder-block operators and bounds on what correct kernels may be off by.

A bound counts, element by element: one rounding of the output (half a step: `eps / 2` of its type), the fp32
sums of the products (each of K terms off by at most 2^-23 of the sum of the terms' magnitudes: the worst case of
any order, with a factor of two for hardware that truncates), the roundings of intermediate operands where the
operator documents one (dz of the backward passes), and 2^-19 of a factor for the activations' fast exponential.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}
EXP = 2.0 ** -19
SUM = 2.0 ** -23
E4M3_MAX, SCALE_MIN = 448.0, 2.0 ** -126
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid")


def act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "relu":
        return z.clamp_min(0)
    if name == "sigmoid":
        return torch.sigmoid(z)
    return z


def slope(z, name):
    with torch.enable_grad():
        v = z.detach().clone().requires_grad_(True)
        return torch.autograd.grad(act(v, name).sum(), v)[0]


def off(bound, got, want):
    """Whether got is within the bound of want everywhere (64-bit comparison), and the worst ratio."""
    d = (got.double() - want).abs()
    ratio = float((d / bound.clamp_min(1e-300)).max()) if d.numel() else 0.0
    return not bool(torch.isfinite(got.double()).all() & (d <= bound).all()), ratio


def check(got, want, bound, what=""):
    bad, ratio = off(bound, got, want)
    assert not bad, f"{what}: {ratio:.3g} times the bound"


# ---------------------------------------------------------------- norm
def norm(x, r, w, eps):
    h = x.double() + (r.double() if r is not None else 0)
    n = (h.square().mean(-1, keepdim=True) + eps).sqrt()
    y = h / n * (w.double() if w is not None else 1)
    return y, h


def norm_bound(y, h, D, dtype):
    # the mean of D squares, the root, the division and two products: a few fp32 roundings beside the sum's
    rel = D * SUM + 8 * 2.0 ** -24
    return HALF[dtype] * y.abs() + rel * y.abs() + 2.0 ** -133, HALF[dtype] * h.abs() + 2.0 ** -24 * h.abs()


def norm_bwd(dy, h, w, dh, eps):
    dy, h = dy.double(), h.double()
    w = w.double() if w is not None else torch.ones(h.shape[-1], dtype=torch.float64, device=h.device)
    n = (h.square().mean(-1, keepdim=True) + eps).sqrt()
    inner = (w * dy * h).mean(-1, keepdim=True)
    dx = (w * dy - h * inner / n ** 2) / n + (dh.double() if dh is not None else 0)
    return dx, (dy * h / n).sum(0)


def norm_bwd_bound(dy, h, w, dh, eps, dx, dtype):
    M, D = h.shape
    dy, h = dy.double().abs(), h.double().abs()
    w = w.double().abs() if w is not None else 1.0
    n = (h.square().mean(-1, keepdim=True) + eps).sqrt()
    rel = D * SUM + 16 * 2.0 ** -24
    parts = (w * dy + 2 * h * (w * dy * h).mean(-1, keepdim=True) / n ** 2) / n + (dh.double().abs() if dh is not None else 0)
    return HALF[dtype] * dx.abs() + rel * parts, (M * SUM + rel) * (dy * h / n).sum(0)


# ---------------------------------------------------------------- products
def scaled(x, s):
    return x.double() if s is None else x.double() * s.double()[:, None]


def product(x, w):
    """z and the bound on its fp32 sum."""
    K = x.shape[1]
    return x @ w.t(), (2 * K + 4) * SUM * (x.abs() @ w.abs().t())


def linear(x, w, b, name, r, dtype, xs=None, ws=None):
    z, e = product(scaled(x, xs), scaled(w, ws))
    if b is not None:
        z = z + b.double()
        e = e + SUM * z.abs()
    y = act(z, name)
    bound = 1.2 * e + (EXP * y.abs() if name != "none" else 0)
    if r is not None:
        y = y + r.double()
    return y, bound + HALF[dtype] * (y.abs() + bound) + 2.0 ** -133


def dact_bound(z, e, dy, name):
    # |act''| <= 1.13 for every activation here (relu: its kink, where z may fall on either side)
    d = slope(z, name)
    bend = torch.where(z.abs() <= e, 1.0, 0.0).double() if name == "relu" else 1.2 * e
    return dy.double() * d, dy.double().abs() * (bend + (EXP * (1 + z.abs()) if name not in ("none", "relu") else 0))


def linear_bwd(dy, x, w, b, name, dtype):
    """dx, dw, db and their bounds."""
    M, N = dy.shape
    xd, wd = x.double(), w.double()
    z, e = product(xd, wd)
    if b is not None:
        z, e = z + b.double(), e + SUM * z.abs()
    dz, ez = dact_bound(z, e, dy, name)
    kept = ez + (HALF[dtype] * (dz.abs() + ez) if name != "none" else 0)
    dx, dw = dz @ wd, dz.t() @ xd
    bx = kept @ wd.abs() + (2 * N + 4) * SUM * ((dz.abs() + kept) @ wd.abs())
    bw = kept.t() @ xd.abs() + (2 * M + 4) * SUM * ((dz.abs() + kept).t() @ xd.abs())
    bb = ez.sum(0) + M * SUM * (dz.abs() + ez).sum(0)
    return (dx, dw, dz.sum(0)), (bx + HALF[dtype] * (dx.abs() + bx), bw + HALF[dtype] * (dw.abs() + bw), bb + 2.0 ** -140)


def gated(x, w, name, dtype, xs=None, ws=None):
    F = w.shape[0] // 2
    z, e = product(scaled(x, xs), scaled(w, ws))
    g, u, eg, eu = z[:, :F], z[:, F:], e[:, :F], e[:, F:]
    a = act(g, name)
    ea = 1.2 * eg + (EXP * a.abs() if name != "none" else 0)
    y = a * u
    bound = ea * (u.abs() + eu) + a.abs() * eu + SUM * y.abs()
    return y, bound + HALF[dtype] * (y.abs() + bound) + 2.0 ** -133


def gated_bwd(dy, x, w, name, dtype):
    M, F = dy.shape
    xd, wd, dyd = x.double(), w.double(), dy.double()
    z, e = product(xd, wd)
    g, u, eg, eu = z[:, :F], z[:, F:], e[:, :F], e[:, F:]
    a = act(g, name)
    ea = 1.2 * eg + (EXP * a.abs() if name != "none" else 0)
    ds, es = dact_bound(g, eg, dyd.abs(), name)
    ds = slope(g, name)
    dz = torch.cat([dyd * u * ds, dyd * a], 1)
    ez = torch.cat([es * (u.abs() + eu) + dyd.abs() * eu * ds.abs() + SUM * (dyd * u * ds).abs(), dyd.abs() * ea], 1)
    kept = ez + HALF[dtype] * (dz.abs() + ez)
    dx, dw = dz @ wd, dz.t() @ xd
    bx = kept @ wd.abs() + (4 * F + 4) * SUM * ((dz.abs() + kept) @ wd.abs())
    bw = kept.t() @ xd.abs() + (2 * M + 4) * SUM * ((dz.abs() + kept).t() @ xd.abs())
    return (dx, dw), (bx + HALF[dtype] * (dx.abs() + bx), bw + HALF[dtype] * (dw.abs() + bw))
