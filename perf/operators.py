"""The decoder-block operators around the gated delta rule: the cases they are measured on, their plain forms and
their values in 64 bits.

* the root-mean-square norm with the residual's addition, a bf16/fp32 or e4m3 output, and its gradients
  (``rms_norm``, ``rms_norm_quant``, ``rms_norm_bwd``),
* the linear layer with scales, bias, activation and residual in its epilogue, and its gradients
  (``linear``, ``linear_bwd``),
* the gated linear unit ``act(x Wg^T) * (x Wu^T)`` of a feed-forward block, and its gradients
  (``gated_linear``, ``gated_linear_bwd``).

Sizes: 16 heads of 128 make a hidden width of 2048; 4 sequences of 4096 tokens a batch of 16384 rows; 64 sequences
decoding together 64 rows; 5504 is 8/3 of 2048 rounded up to a multiple of 128.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # 64 sequences decoding together: the norm before the quantised projections of one layer
        {"name": "norm_quant_decode", "op": "norm", "M": 64, "D": 2048, "dtype": "bf16", "residual": True, "quant": True},
        # a prefill of 4 x 4096 tokens: the norm between token mixer and feed-forward block
        {"name": "norm_prefill", "op": "norm", "M": 16384, "D": 2048, "dtype": "bf16", "residual": True, "quant": False},
        # an fp32 run of an odd batch and an odd width: rows that are not 16-byte aligned
        {"name": "norm_f32_odd", "op": "norm", "M": 1777, "D": 1001, "dtype": "f32", "residual": False, "quant": False},
        # the gradients of the norm in a training step of 4 x 4096 tokens
        {"name": "norm_bwd_train", "op": "norm_bwd", "M": 16384, "D": 2048, "dtype": "bf16"},
        # a single token: the feed-forward block's output projection onto the residual stream
        {"name": "linear_one_token", "op": "linear", "M": 1, "K": 5504, "N": 2048, "dtype": "bf16", "bias": False, "act": "none", "residual": True},
        # 64 tokens decoding: the joint q, k, v projection in 8 bits
        {"name": "linear_quant_decode", "op": "linear", "M": 64, "K": 2048, "N": 6144, "dtype": "e4m3", "bias": False, "act": "none", "residual": False},
        # prefill: the output projection of the token mixer onto the residual stream
        {"name": "linear_prefill", "op": "linear", "M": 16384, "K": 2048, "N": 2048, "dtype": "bf16", "bias": True, "act": "none", "residual": True},
        # training on a ragged packed batch: the gradients of a layer with bias and activation
        {"name": "linear_bwd_ragged", "op": "linear_bwd", "M": 3001, "K": 2048, "N": 2048, "dtype": "bf16", "bias": True, "act": "gelu"},
        # 64 tokens decoding: the feed-forward block's gated half
        {"name": "gated_decode", "op": "gated", "M": 64, "K": 2048, "F": 5504, "dtype": "bf16", "act": "silu"},
        # a ragged prefill in bf16
        {"name": "gated_prefill_ragged", "op": "gated", "M": 8191, "K": 2048, "F": 5504, "dtype": "bf16", "act": "silu"},
        # prefill in 8 bits
        {"name": "gated_quant_prefill", "op": "gated", "M": 16384, "K": 2048, "F": 5504, "dtype": "e4m3", "act": "silu"},
        # the largest: the gradients of the gated half in a training step of 4 x 4096 tokens
        {"name": "gated_bwd_train", "op": "gated_bwd", "M": 16384, "K": 2048, "F": 5504, "dtype": "bf16", "act": "silu"},
    ]


MOST_FLOPS = 12 * 16384 * 2048 * 5504
MOST_BYTES = 4 * 16384 * 2048 * 2


def _size(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of `step`."""
    size = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))
    return size + step if size == 3072 else size


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd"])
    M = _size(rng, 1, 16384)
    if op in ("norm", "norm_bwd"):
        D = _size(rng, 64, 8192, rng.choice([1, 8, 128]))
        M = max(1, min(M, MOST_BYTES // (8 * D)))
        c = {"op": op, "M": M, "D": D, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "norm":
            c |= {"residual": rng.random() < 0.7, "quant": rng.random() < 0.4}
        return c
    # widths: multiples of 128 and of 16 as models have them, now and then an odd one
    K = _size(rng, 128, 8192, rng.choice([128, 128, 16]))
    N = _size(rng, 128, 8192, rng.choice([128, 128, 16]))
    if rng.random() < 0.15:
        K, N = _size(rng, 65, 2049) | 1, _size(rng, 65, 2049) | 1
    grad = op.endswith("_bwd")
    dtype = rng.choice(["bf16"] * 5 + ["f32"]) if grad else rng.choice(["bf16", "bf16", "bf16", "e4m3", "e4m3", "f32"])
    if dtype == "e4m3":
        K = max(16, K // 16 * 16)
    times = {"linear": 2, "linear_bwd": 6, "gated": 4, "gated_bwd": 12}[op]
    M = max(1, min(M, MOST_FLOPS // (times * K * N)))
    if op.startswith("linear"):
        c = {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "bias": rng.random() < 0.5, "act": rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "relu"])}
        if op == "linear":
            c["residual"] = rng.random() < 0.5
        return c
    return {"op": op, "M": M, "K": K, "F": N, "dtype": dtype, "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "sigmoid"])}


def _quantised(t):
    """What a program keeps of a matrix in 8 bits: e4m3 values and one fp32 scale per row."""
    scale = (t.abs().amax(dim=1) / E4M3_MAX).clamp_min(SCALE_MIN)
    return (t / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    M = case["M"]
    if case["op"] in ("norm", "norm_bwd"):
        D, dt = case["D"], DTYPES[case["dtype"]]
        # a residual stream: a few channels much larger than the others
        big = 1.0 + 9.0 * (torch.rand(D, generator=g, device="cuda") < 0.01)
        s["x"] = (n(M, D) * big).to(dt)
        s["weight"] = 1.0 + 0.2 * n(D)
        s["eps"] = 1e-6
        if case["op"] == "norm":
            s["r"] = (2.0 * n(M, D) * big).to(dt) if case["residual"] else None
        else:
            s["dy"], s["dh"] = n(M, D).to(dt), n(M, D).to(dt)
        return s
    K = case["K"]
    rows = case["N"] if case["op"].startswith("linear") else 2 * case["F"]
    x, w = n(M, K), n(rows, K) / math.sqrt(K)
    if case["dtype"] == "e4m3":
        s["x"], s["xs"] = _quantised(x)
        s["w"], s["ws"] = _quantised(w)
        out = torch.bfloat16
    else:
        out = DTYPES[case["dtype"]]
        s["x"], s["w"], s["xs"], s["ws"] = x.to(out), w.to(out), None, None
    if case["op"].startswith("linear"):
        s["b"] = 0.1 * n(rows) if case["bias"] else None
        if case["op"] == "linear":
            s["r"] = n(M, rows).to(out) if case["residual"] else None
        else:
            s["dy"] = n(M, rows).to(out)
    elif case["op"] == "gated_bwd":
        s["dh"] = n(M, case["F"]).to(out)
    return s


# ---------------------------------------------------------------- the plain forms, in 32 bits


def _act(z, name):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "relu":
        return z.clamp_min(0)
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    return z


def _act_slope(z, name):
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 - p)
    return torch.ones_like(z)


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + s["eps"]) * s["weight"]
        dt = s["x"].dtype
        kept = None if s["r"] is None else h.to(dt)
        if not s["quant"]:
            return y.to(dt), kept
        scale = (y.abs().amax(dim=1) / E4M3_MAX).clamp_min(SCALE_MIN)
        q = (y * (1 / scale)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return q, scale, kept
    if op == "norm_bwd":
        h, dy, w = s["x"].float(), s["dy"].float(), s["weight"]
        rstd = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + s["eps"])
        xh, dxh = h * rstd, dy * w
        dx = s["dh"].float() + rstd * (dxh - xh * (dxh * xh).mean(dim=1, keepdim=True))
        return dx.to(s["x"].dtype), (dy * xh).sum(dim=0)
    x, w = s["x"].float(), s["w"].float()
    if s["xs"] is not None:
        x, w = x * s["xs"][:, None], w * s["ws"][:, None]
    z = x @ w.t()
    out = torch.bfloat16 if s["dtype"] == "e4m3" else s["x"].dtype
    if op == "linear":
        y = _act(z if s["b"] is None else z + s["b"], s["act"])
        return (y if s["r"] is None else y + s["r"].float()).to(out)
    if op == "linear_bwd":
        dz = s["dy"].float() * _act_slope(z if s["b"] is None else z + s["b"], s["act"])
        return (dz @ w).to(out), (dz.t() @ x).to(out), None if s["b"] is None else dz.sum(dim=0)
    F = s["F"]
    gate, up = z[:, :F], z[:, F:]
    if op == "gated":
        return (_act(gate, s["act"]) * up).to(out)
    dh = s["dh"].float()
    dz = torch.cat([dh * up * _act_slope(gate, s["act"]), dh * _act(gate, s["act"])], dim=1)
    return (dz @ w).to(out), (dz.t() @ x).to(out)


def run(s):
    if not own:
        return _plain(s)
    import gated_deltanet_gb300 as gdn

    op = s["op"]
    if op == "norm":
        if s["quant"]:
            return gdn.rms_norm_quant(s["x"], s["weight"], s["r"], s["eps"])
        return gdn.rms_norm(s["x"], s["weight"], s["r"], s["eps"])
    if op == "norm_bwd":
        return gdn.rms_norm_bwd(s["dy"], s["x"], s["weight"], s["dh"], s["eps"])
    act = None if s["act"] == "none" else s["act"]
    if op == "linear":
        return gdn.linear(s["x"], s["w"], s["b"], act, s["r"], x_scale=s["xs"], weight_scale=s["ws"])
    if op == "linear_bwd":
        return gdn.linear_bwd(s["dy"], s["x"], s["w"], s["b"], act)
    if op == "gated":
        return gdn.gated_linear(s["x"], s["w"], act, x_scale=s["xs"], weight_scale=s["ws"])
    return gdn.gated_linear_bwd(s["dh"], s["x"], s["w"], act)


def work(case):
    M, op, e = case["M"], case["op"], {"bf16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]
    if op == "norm":
        D = case["D"]
        read = M * D * e * (2 if case["residual"] else 1) + 4 * D
        write = M * D * (e if case["residual"] else 0) + (M * D + 4 * M if case["quant"] else M * D * e)
        return {"bytes": read + write, "flops": 4 * M * D}
    if op == "norm_bwd":
        return {"bytes": 4 * M * case["D"] * e + 8 * case["D"], "flops": 10 * M * case["D"]}
    K, eo = case["K"], max(e, 2)
    rows = case["N"] if op.startswith("linear") else 2 * case["F"]
    scales = 4 * (M + rows) if e == 1 else 0
    if op == "linear":
        return {"bytes": (M + rows) * K * e + scales + M * rows * eo * (2 if case["residual"] else 1) + (4 * rows if case["bias"] else 0), "flops": 2 * M * rows * K}
    if op == "linear_bwd":
        again = case["act"] != "none"
        return {"bytes": 2 * (M + rows) * K * e + M * rows * e + (8 * rows if case["bias"] else 0), "flops": (6 if again else 4) * M * rows * K}
    if op == "gated":
        return {"bytes": (M + rows) * K * e + scales + M * case["F"] * eo, "flops": 2 * M * rows * K}
    return {"bytes": 2 * (M + rows) * K * e + M * case["F"] * e, "flops": 6 * M * rows * K}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    op = case["op"]
    if op == "norm":
        h = d["x"] + d["r"] if case["residual"] else d["x"]
        y = torch.einsum("md,m,d->md", h, 1 / (torch.linalg.vector_norm(h, dim=1) ** 2 / case["D"] + s["eps"]).sqrt(), d["weight"])
        kept = h if case["residual"] else None
        if not case["quant"]:
            return y, kept
        scale = torch.maximum(y.max(dim=1).values, (-y).max(dim=1).values) / E4M3_MAX
        scale = torch.where(scale < SCALE_MIN, SCALE_MIN, scale)
        return torch.div(y, scale[:, None]).to(torch.float8_e4m3fn).double(), scale, kept
    if op == "norm_bwd":
        # y_j = w_j h_j / n with n = sqrt(|h|^2 / D + eps), so dn/dh_i = h_i / (D n)
        h, norm = d["x"], (torch.linalg.vector_norm(d["x"], dim=1, keepdim=True) ** 2 / case["D"] + s["eps"]).sqrt()
        inner = torch.einsum("md,md,d->m", d["dy"], h, d["weight"])[:, None]
        return d["dh"] + d["dy"] * d["weight"] / norm - h * inner / (case["D"] * norm ** 3), torch.einsum("md,md->d", d["dy"], h / norm)
    x, w = d["x"], d["w"]
    if "xs" in d:
        x, w = torch.einsum("m,mk->mk", d["xs"], x), torch.einsum("n,nk->nk", d["ws"], w)
    z = torch.einsum("mk,nk->mn", x, w)
    f = {"none": (lambda t: t, lambda t: torch.ones_like(t)),
         "relu": (lambda t: torch.where(t > 0, t, 0.0), lambda t: torch.where(t > 0, 1.0, 0.0).double()),
         "sigmoid": (torch.special.expit, lambda t: torch.special.expit(t) * torch.special.expit(-t)),
         "silu": (lambda t: t * torch.special.expit(t), lambda t: torch.special.expit(t) + t * torch.special.expit(t) * torch.special.expit(-t)),
         # Phi and its density
         "gelu": (lambda t: t * torch.special.ndtr(t), lambda t: torch.special.ndtr(t) + t * torch.exp(-t * t / 2) * (2 * math.pi) ** -0.5)}
    # 0.5 (1 + tanh(u)) is the logistic function of 2 u, here with 2 u = a t + b t^3
    a = 2 * math.sqrt(2 / math.pi)
    b = a * 0.044715
    f["gelu_tanh"] = (lambda t: t * torch.special.expit(a * t + b * t ** 3),
                      lambda t: torch.special.expit(a * t + b * t ** 3) * (1 + t * (a + 3 * b * t ** 2) * torch.special.expit(-a * t - b * t ** 3)))
    act, slope = f[case["act"]]
    if op.startswith("linear"):
        if case["bias"]:
            z = z + d["b"]
        if op == "linear":
            return act(z) + (d["r"] if case["residual"] else 0)
        dz = d["dy"] * slope(z)
        return torch.einsum("mn,nk->mk", dz, w), torch.einsum("mn,mk->nk", dz, x), torch.einsum("mn->n", dz) if case["bias"] else None
    gate, up = z.split(case["F"], dim=1)
    if op == "gated":
        return act(gate) * up
    dg, du = d["dh"] * slope(gate) * up, act(gate) * d["dh"]
    wg, wu = w.split(case["F"], dim=0)
    return torch.einsum("mf,fk->mk", dg, wg) + torch.einsum("mf,fk->mk", du, wu), torch.cat([torch.einsum("mf,mk->fk", dg, x), torch.einsum("mf,mk->fk", du, x)])
