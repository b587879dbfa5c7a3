"""Token mixers beside the gated delta rule: the cases they are measured on, their plain forms and their values in 64 bits.

* linear attention with a decay for each head, ``S_t = exp(decay_h) S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t``: the chunked
  form for prompts, the recurrent form for single tokens, and the gradients
  (``chunk_linear_attention``, ``fused_recurrent_linear_attention``, ``chunk_linear_attention_bwd``),
* softmax attention with a sliding window and a few first tokens that stay visible (sinks): for prompts, for single tokens over
  a cache, and the gradients (``window_attention``, ``window_attention_decode``, ``window_attention_bwd``).

Sizes: heads of 128 (or 64), 16 of them in a layer of width 2048; 4 sequences of 4096 tokens a training batch; 65536 tokens a long
prompt; 64 sequences decoding together; a window of 1024 to 4096 tokens and 4 sinks.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a prefill of 4 x 4096 tokens from a cached state
        {"name": "linear_prefill", "op": "linear", "N": 4, "T": 16384, "ragged": False, "H": 16, "HV": 16, "K": 128, "V": 128, "dtype": "bf16", "state": True},
        # one long prompt with few heads
        {"name": "linear_long", "op": "linear", "N": 1, "T": 65536, "ragged": False, "H": 8, "HV": 8, "K": 128, "V": 128, "dtype": "bf16", "state": False},
        # one token for one sequence: latency
        {"name": "linear_one_token", "op": "linear_step", "N": 1, "T": 1, "ragged": False, "H": 8, "HV": 8, "K": 128, "V": 128, "dtype": "bf16", "state": True},
        # 64 sequences decoding together
        {"name": "linear_decode", "op": "linear_step", "N": 64, "T": 64, "ragged": False, "H": 16, "HV": 16, "K": 128, "V": 128, "dtype": "bf16", "state": True},
        # the gradients in a training step of 4 x 4096 tokens
        {"name": "linear_bwd_train", "op": "linear_bwd", "N": 4, "T": 16384, "ragged": False, "H": 16, "HV": 16, "K": 128, "V": 128, "dtype": "bf16", "state": False},
        # the gradients of a packed batch of sequences of any length, two value heads to a key head
        {"name": "linear_bwd_packed", "op": "linear_bwd", "N": 13, "T": 8191, "ragged": True, "H": 4, "HV": 8, "K": 128, "V": 128, "dtype": "bf16", "state": True},
        # a prefill of 4 x 4096 tokens, four query heads to a key head
        {"name": "window_prefill", "op": "window", "N": 4, "T": 16384, "ragged": False, "H": 16, "HK": 4, "D": 128, "window": 1024, "sinks": 4, "dtype": "bf16", "lse": False},
        # a packed batch of prompts of any length, an odd window
        {"name": "window_packed", "op": "window", "N": 9, "T": 9001, "ragged": True, "H": 16, "HK": 16, "D": 128, "window": 777, "sinks": 1, "dtype": "bf16", "lse": True},
        # one token for one sequence with a long cache: latency
        {"name": "window_one_token", "op": "window_step", "N": 1, "S": 16384, "H": 16, "HK": 4, "D": 128, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # 64 sequences decoding together
        {"name": "window_decode", "op": "window_step", "N": 64, "S": 8192, "H": 16, "HK": 4, "D": 128, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # the gradients in a training step of 4 x 4096 tokens
        {"name": "window_bwd_train", "op": "window_bwd", "N": 4, "T": 16384, "ragged": False, "H": 16, "HK": 4, "D": 128, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # the gradients of an odd batch in fp32
        {"name": "window_bwd_f32", "op": "window_bwd", "N": 3, "T": 1503, "ragged": True, "H": 4, "HK": 2, "D": 64, "window": 100, "sinks": 2, "dtype": "f32"},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_LINEAR = 16384 * 16        # tokens x value heads of the linear forms
MOST_WINDOW = 16384 * 16 * 1024  # query tokens x heads x keys seen of the window forms


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_step", "linear_bwd", "window", "window", "window_step", "window_bwd"])
    dtype = rng.choice(["bf16"] * 4 + ["f32"])
    if op.startswith("linear"):
        H = rng.choice([1, 2, 4, 5, 8, 16, 32])
        HV = H * rng.choice([1, 1, 1, 2, 4])
        K, V = rng.choice([(128, 128), (128, 128), (64, 64)]) if dtype == "bf16" else rng.choice([(128, 128), (64, 64), (64, 96), (32, 20)])
        state = rng.random() < 0.6
        if op == "linear_step":
            N = max(1, min(_size(rng, 1, 256), 64 * 16 * 128 * 128 * 2 // (HV * K * V)))
            return {"op": op, "N": N, "T": N * rng.choice([1, 1, 1, 2, 3, 5]), "ragged": False, "H": H, "HV": HV, "K": K, "V": V, "dtype": dtype, "state": state}
        N = _size(rng, 1, 40)
        most = MOST_LINEAR // HV if dtype == "bf16" else MOST_LINEAR // HV // 8
        ragged = rng.random() < 0.5
        T = max(N, min(most, _size(rng, 1, 65536)))
        return {"op": op, "N": N, "T": T if ragged else T // N * N, "ragged": ragged, "H": H, "HV": HV, "K": K, "V": V, "dtype": dtype, "state": state}
    HK = rng.choice([1, 2, 3, 4, 8])
    H = HK * rng.choice([1, 2, 4, 8])
    D = rng.choice([128, 128, 64]) if dtype == "bf16" else rng.choice([128, 64, 40])
    window, sinks = _size(rng, 1, 4096), rng.choice([0, 0, 1, 4, 4, 16, 130])
    if op == "window_step":
        N = _size(rng, 1, 128)
        S = max(1, min(_size(rng, 64, 32768), 64 * 8192 * 4 * 2 // (N * HK)))
        return {"op": op, "N": N, "S": S, "H": H, "HK": HK, "D": D, "window": window, "sinks": sinks, "dtype": dtype}
    N = _size(rng, 1, 24)
    most = MOST_WINDOW // H // (1 if dtype == "bf16" else 16)
    T = max(N, min(_size(rng, 1, 32768), most // min(window + sinks, 4096)))
    ragged = rng.random() < 0.5
    c = {"op": op, "N": N, "T": T if ragged else T // N * N, "ragged": ragged, "H": H, "HK": HK, "D": D, "window": window, "sinks": sinks, "dtype": dtype}
    return c | {"lse": rng.random() < 0.5} if op == "window" else c


def _lengths(case):
    """Tokens of each sequence: cuts at random places (the same for every seed), or all alike."""
    N, T = case["N"], case["T"]
    if not case["ragged"]:
        return [T // N] * N
    cuts = sorted(random.Random(1000 * N + T).randint(0, T) for _ in range(N - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _filled(case):
    """Tokens in each sequence's cache, between half of it and all."""
    r = random.Random(case["N"] + case["S"])
    return [r.randint((case["S"] + 1) // 2, case["S"]) for _ in range(case["N"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    n = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    N = case["N"]
    if case["op"] == "window_step":
        H, HK, D, S = case["H"], case["HK"], case["D"], case["S"]
        s["q"], s["k"], s["v"] = n(N, 1, H, D).to(dt), n(N, S, HK, D).to(dt), n(N, S, HK, D).to(dt)
        s["lengths"] = torch.tensor(_filled(case), dtype=torch.int32, device="cuda")
        return s
    lens = _lengths(case)
    B, T = (1, case["T"]) if case["ragged"] else (N, case["T"] // N)
    s["lens"] = lens
    s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0) if case["ragged"] else None
    if case["op"].startswith("linear"):
        H, HV, K, V = case["H"], case["HV"], case["K"], case["V"]
        act = torch.nn.functional.silu  # as the short convolutions before such a layer end
        s["q"], s["k"], s["v"] = act(n(B, T, H, K)).to(dt), act(n(B, T, H, K)).to(dt), n(B, T, HV, V).to(dt)
        s["decay"] = -torch.exp2(-8.0 * torch.arange(1, HV + 1, device="cuda") / HV)
        s["h0"] = n(N, HV, K, V) if case["state"] else None
        if case["op"] == "linear_bwd":
            s["do"] = n(B, T, HV, V).to(dt)
            s["dht"] = n(N, HV, K, V) if case["state"] else None
        return s
    H, HK, D = case["H"], case["HK"], case["D"]
    s["q"], s["k"], s["v"] = n(B, T, H, D).to(dt), n(B, T, HK, D).to(dt), n(B, T, HK, D).to(dt)
    if case["op"] == "window_bwd":  # a training step keeps the forward's output and its softmax statistics
        s["do"] = n(B, T, H, D).to(dt)
        s["o"], s["lse"] = _window(s)
    return s


# ---------------------------------------------------------------- the plain forms, in 32 bits


def _padded(s, *tensors):
    """Packed tensors [1, T, ...] as [N, longest, ...] with zeros behind each sequence's end; batched ones as they are."""
    if s["cu"] is None:
        return [t.float() for t in tensors]
    at, inside = _places(s)
    return [torch.where(inside.reshape(*inside.shape, *[1] * (t.dim() - 2)), t[0].float()[at.clamp(max=t.shape[1] - 1)], 0.0) for t in tensors]


def _places(s):
    i = torch.arange(max(s["lens"]), device="cuda")
    return s["cu"][:-1, None] + i, i < (s["cu"][1:] - s["cu"][:-1])[:, None]


def _packed(s, t):
    """The reverse of _padded for [N, longest, ...]."""
    return t if s["cu"] is None else t[_places(s)[1]][None]


def _seq_lengths(s):
    n = s["q"].shape[1]
    return (s["cu"][1:] - s["cu"][:-1]) if s["cu"] is not None else torch.full((s["N"],), n, device="cuda")


def _mix(a, b, c, decay, start, lens, C, late=None):
    """``out_t = sum_{u <= t} exp(decay (t - u)) (a_t . b_u) c_u + exp(decay (t + 1)) a_t start`` per head and the state
    ``X = sum_u exp(decay (len - 1 - u)) b_u c_u^T + exp(decay len) start``, chunks of C tokens at once.  a, b [N, H, T, K], c [N, H, T, V],
    rows behind the length zero.  ``late``: `start` stands one token later (it enters out_t with exp(decay t))."""
    N, H, T, K = a.shape
    n, V = -(-T // C), c.shape[-1]
    a, b, c = (torch.nn.functional.pad(t, (0, 0, 0, n * C - T)).reshape(N, H, n, C, -1) for t in (a, b, c))
    d, i, z = decay.double()[:, None, None], torch.arange(C, device="cuda"), 0 if late is None else 1
    gap = i[:, None] - i
    inside = torch.where(gap >= 0, torch.exp(d * gap.clamp_min(0)), 0.0).float()  # [H, C, C]
    y = ((a @ b.mT) * inside[:, None]) @ c
    each = (b * torch.exp(d * (C - 1 - i)[:, None]).float()[:, None]).mT @ c  # [N, H, n, K, V]
    m = torch.arange(n + 1, device="cuda")
    hops = m[:, None] - 1 - m[:n]
    carry = torch.where(hops >= 0, torch.exp(d * C * hops.clamp_min(0)), 0.0).float()  # [H, n + 1, n]
    X = (carry @ each.reshape(N, H, n, K * V)).reshape(N, H, n + 1, K, V)
    if start is not None:
        X = X + torch.exp(d * (C * m[:, None] - z).clamp_min(-z)).float()[..., None] * start[:, :, None]
    y = y + (a @ X[:, :, :n]) * torch.exp(d * (i + 1)[:, None]).float()[:, None]
    # zero rows behind the end left the sums alone, but each of them decayed the state: it is taken at the chunk before the end
    last = lens // C
    rest = lens - last * C
    w = torch.arange(N, device="cuda")
    Xl = X[w, :, last]  # [N, H, K, V]
    full = torch.cat([b, torch.zeros_like(b[:, :, :1])], 2)[w, :, last], torch.cat([c, torch.zeros_like(c[:, :, :1])], 2)[w, :, last]
    left = (rest[:, None] - 1 - i)[:, None, :, None]
    g = torch.where(left >= 0, torch.exp(decay.double()[:, None, None] * left.clamp_min(0)), 0.0).float()
    Xe = Xl * torch.exp(decay.double() * rest[:, None]).float()[..., None, None] + (full[0] * g).mT @ full[1]
    return y.reshape(N, H, n * C, V)[:, :, :T], Xe


def _linear(s):
    q, k, v = (t.transpose(1, 2) for t in _padded(s, s["q"], s["k"], s["v"]))
    r, dt = s["HV"] // s["H"], s["q"].dtype
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    o, ht = _mix(q, k, v, s["decay"], s["h0"], _seq_lengths(s), min(128, q.shape[2]))
    return _packed(s, (o * s["K"] ** -0.5).transpose(1, 2)).to(dt), ht


def _linear_step(s):
    q, k, v = (t.float().transpose(1, 2) for t in (s["q"], s["k"], s["v"]))
    r, T, d = s["HV"] // s["H"], q.shape[2], s["decay"].double()[:, None]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    i = torch.arange(T, device="cuda")
    gap = i[:, None] - i
    o = ((q @ k.mT) * torch.where(gap >= 0, torch.exp(d[..., None] * gap.clamp_min(0)), 0.0).float()) @ v
    ht = (k * torch.exp(d * (T - 1 - i)).float()[..., None]).mT @ v
    if s["h0"] is not None:
        o = o + (q @ s["h0"]) * torch.exp(d * (i + 1)).float()[..., None]
        ht = ht + s["h0"] * torch.exp(d * T).float()[..., None]
    return (o * s["K"] ** -0.5).transpose(1, 2).to(s["q"].dtype), ht


def _flipped(s, t):
    """[N, H, T, D] with each sequence's tokens in reverse order (zeros stay behind)."""
    at = _seq_lengths(s)[:, None] - 1 - torch.arange(t.shape[2], device="cuda")
    got = t.gather(2, at.clamp_min(0)[:, None, :, None].expand_as(t))
    return torch.where((at >= 0)[:, None, :, None], got, 0.0)


def _linear_bwd(s):
    q, k, v, do = (t.transpose(1, 2) for t in _padded(s, s["q"], s["k"], s["v"], s["do"]))
    r, dt, lens, scale = s["HV"] // s["H"], s["q"].dtype, _seq_lengths(s), s["K"] ** -0.5
    q, k, C = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1), min(128, q.shape[2])
    dq = scale * _mix(do, v, k, s["decay"], None if s["h0"] is None else s["h0"].mT, lens, C)[0]
    # the state's gradient runs backward in time: R_t = exp(decay) R_{t+1} + scale q_t do_t^T, with dht joining at the last token
    q, k, v, do = (_flipped(s, t) for t in (q, k, v, do))
    late = None if s["dht"] is None else s["dht"] * torch.exp(-s["decay"].double()).float()[:, None, None]
    dk = _mix(v, do, scale * q, s["decay"], None if late is None else late.mT, lens, C)[0]
    dv, R = _mix(k, scale * q, do, s["decay"], late, lens, C)
    dh0 = None if s["h0"] is None else R * torch.exp(s["decay"].double()).float()[:, None, None]
    N, HV, T, K = dk.shape
    dq, dk = (t.reshape(N, s["H"], r, T, K).sum(2) for t in (dq, _flipped(s, dk)))
    return [_packed(s, t.transpose(1, 2)).to(dt) for t in (dq, dk, _flipped(s, dv))] + [dh0]


def _band(s, T, lens):
    """Blocks of queries and the keys that each may see: the query positions [n, C], the key positions [n, W] and what is seen [N, n, C, W]."""
    w, sinks = s["window"], s["sinks"]
    C = T if w >= T // 2 else max(64, min(w, 1024))
    n = -(-T // C)
    qi = torch.arange(n * C, device="cuda").reshape(n, C)
    if n == 1:
        ki = torch.arange(T, device="cuda")[None]
    else:
        near = qi[:, :1] - (w - 1) + torch.arange(C + w - 1, device="cuda")
        first = torch.arange(min(sinks, T), device="cuda").expand(n, -1)
        ki = torch.cat([torch.where(first < near[:, :1], first, -1), near], 1)
    gap = qi[:, :, None] - ki[:, None]
    seen = (ki[:, None] >= 0) & (gap >= 0) & ((gap < w) | (ki[:, None] < sinks))
    return qi, ki, seen[None] & (qi[:, :, None] < lens[:, None, None, None])


def _scores(s):
    q, k, v = _padded(s, s["q"], s["k"], s["v"])
    N, T, H, D = q.shape
    HK = s["HK"]
    qi, ki, seen = _band(s, T, _seq_lengths(s))
    n, C = qi.shape
    blocks = lambda t: torch.nn.functional.pad(t, (0, 0, 0, 0, 0, n * C - T)).reshape(N, n, C, HK, H // HK, -1).permute(0, 3, 4, 1, 2, 5)  # noqa: E731
    kb, vb = (t[:, ki.clamp(0, T - 1)].permute(0, 3, 1, 2, 4)[:, :, None] for t in (k, v))  # [N, HK, 1, n, W, D]
    qb = blocks(q)
    z = torch.where(seen[:, None, None], (qb @ kb.mT) * D ** -0.5, -math.inf)
    return z, qb, kb, vb, ki, blocks


def _unblocked(s, t, T):
    N, HK, G, n, C, D = t.shape
    return t.permute(0, 3, 4, 1, 2, 5).reshape(N, n * C, HK * G, D)[:, :T]


def _window(s):
    z, _, _, vb, _, _ = _scores(s)
    T = max(s["lens"])
    top = z.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    o = (e @ vb) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top
    o, lse = _packed(s, _unblocked(s, o, T)), _packed(s, _unblocked(s, lse, T))
    return o.to(s["q"].dtype), lse[..., 0].transpose(1, 2).contiguous()


def _window_bwd(s):
    z, qb, kb, vb, ki, blocks = _scores(s)
    N, T, H, D, HK = s["N"], max(s["lens"]), s["H"], s["D"], s["HK"]
    do, o, lse = _padded(s, s["do"], s["o"], s["lse"].transpose(1, 2)[..., None].contiguous())
    dob, lseb = blocks(do), blocks(lse)
    p = torch.exp(z - torch.where(torch.isfinite(lseb), lseb, 0.0))
    dz = p * (dob @ vb.mT - (dob * blocks(o)).sum(-1, keepdim=True)) * D ** -0.5
    dq = _unblocked(s, dz @ kb, T)
    at = ki.clamp(0, T - 1).reshape(-1)

    def gathered(t):  # sums over the query heads of a key head, and of the blocks that share a key
        return torch.zeros(N, T, HK, D, device="cuda").index_add_(1, at, t.sum(2).permute(0, 2, 3, 1, 4).reshape(N, -1, HK, D))

    return [_packed(s, t).to(s["q"].dtype) for t in (dq, gathered(dz.mT @ qb), gathered(p.mT @ dob))]


def _window_step(s):
    N, S, HK, D = s["k"].shape
    w, lens = min(s["window"], S), s["lengths"].long()[:, None]
    near = lens - w + torch.arange(w, device="cuda")
    first = torch.arange(min(s["sinks"], S), device="cuda").expand(N, -1)
    ki = torch.cat([torch.where(first < near[:, :1], first, -1), near], 1)
    row = torch.arange(N, device="cuda")[:, None]
    k, v = (t[row, ki.clamp(0, S - 1)].float().transpose(1, 2) for t in (s["k"], s["v"]))  # [N, HK, W, D]
    q = s["q"].float().reshape(N, HK, s["H"] // HK, D)
    z = torch.where(((ki >= 0) & (ki < lens))[:, None, None], (q @ k.mT) * D ** -0.5, -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return ((e @ v) / e.sum(-1, keepdim=True)).reshape(N, 1, s["H"], D).to(s["q"].dtype)


def run(s):
    op = s["op"]
    if not own:
        if op == "linear":
            return _linear(s)
        if op == "linear_step":
            return _linear_step(s)
        if op == "linear_bwd":
            return _linear_bwd(s)
        if op == "window":
            return _window(s) if s["lse"] else _window(s)[0]
        return _window_bwd(s) if op == "window_bwd" else _window_step(s)
    import gated_deltanet_gb300 as gdn

    if op == "linear":
        return gdn.chunk_linear_attention(s["q"], s["k"], s["v"], s["decay"], initial_state=s["h0"], output_final_state=True, cu_seqlens=s["cu"])
    if op == "linear_step":
        return gdn.fused_recurrent_linear_attention(s["q"], s["k"], s["v"], s["decay"], initial_state=s["h0"], output_final_state=True, cu_seqlens=s["cu"])
    if op == "linear_bwd":
        return list(gdn.chunk_linear_attention_bwd(s["q"], s["k"], s["v"], s["decay"], s["do"], initial_state=s["h0"], dht=s["dht"], cu_seqlens=s["cu"]))
    if op == "window":
        return gdn.window_attention(s["q"], s["k"], s["v"], s["window"], s["sinks"], cu_seqlens=s["cu"], return_lse=s["lse"])
    if op == "window_step":
        return gdn.window_attention_decode(s["q"], s["k"], s["v"], s["lengths"], s["window"], s["sinks"])
    return list(gdn.window_attention_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["window"], s["sinks"], cu_seqlens=s["cu"]))


def work(case):
    e, op, N = {"bf16": 2, "f32": 4}[case["dtype"]], case["op"], case["N"]
    if op.startswith("linear"):
        H, HV, K, V, T = (case[k] for k in ("H", "HV", "K", "V", "T"))
        state, qk, vo = 4 * N * HV * K * V, T * H * K * e, T * HV * V * e
        if op == "linear_bwd":  # q, k, v, do and dq, dk, dv; h0, dht and dh0
            return {"bytes": 4 * qk + 3 * vo + (3 * state if case["state"] else 0), "flops": 10 * T * HV * K * V}
        return {"bytes": 2 * qk + 2 * vo + (2 if case["state"] else 1) * state, "flops": 4 * T * HV * K * V}
    H, HK, D, w, sinks = (case[k] for k in ("H", "HK", "D", "window", "sinks"))
    if op == "window_step":
        keys = sum(min(n, w + sinks) for n in _filled(case))
        return {"bytes": 2 * keys * HK * D * e + 2 * N * H * D * e, "flops": 4 * keys * H * D}
    pairs = 0
    for n in _lengths(case):  # a token at position p sees min(p + 1, w + sinks) keys
        full = min(n, w + sinks)
        pairs += full * (full + 1) // 2 + (n - full) * (w + sinks)
    q, k, stats = case["T"] * H * D * e, case["T"] * HK * D * e, 4 * case["T"] * H
    if op == "window":
        return {"bytes": 2 * q + 2 * k + (stats if case["lse"] else 0), "flops": 4 * pairs * H * D}
    return {"bytes": 4 * q + 4 * k + stats, "flops": 10 * pairs * H * D}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    x = {k: t.double() for k, t in s.items() if torch.is_tensor(t)}
    op, N = case["op"], case["N"]
    if op == "window_step":
        out = []
        for b, n in enumerate(_filled(case)):
            seen = [j for j in range(n) if j >= n - case["window"] or j < case["sinks"]]
            k, v = (t[b, seen].repeat_interleave(case["H"] // case["HK"], 1) for t in (x["k"], x["v"]))
            p = torch.softmax(torch.einsum("hd,khd->hk", x["q"][b, 0], k) / math.sqrt(case["D"]), 1)
            out.append(torch.einsum("hk,khd->hd", p, v))
        return torch.stack(out)[:, None]
    lens = s["lens"]
    starts = [sum(lens[:i]) for i in range(N)]
    flat = {k: x[k].reshape(case["T"], *x[k].shape[2:]) for k in ("q", "k", "v", "do") if k in x}
    shaped = lambda t: t.reshape(*s["q"].shape[:2], *t.shape[1:])  # noqa: E731
    if op.startswith("linear"):
        r, lam, scale = case["HV"] // case["H"], torch.exp(x["decay"])[None, :, None, None], 1 / math.sqrt(case["K"])
        flat["q"], flat["k"] = flat["q"].repeat_interleave(r, 1), flat["k"].repeat_interleave(r, 1)
        zero = torch.zeros(N, case["HV"], case["K"], case["V"], dtype=torch.float64, device="cuda")
        S = x["h0"].clone() if case["state"] else zero.clone()
        o, dq = torch.zeros_like(flat["v"]), torch.zeros_like(flat["q"])
        order = sorted(range(N), key=lambda i: -lens[i])  # longest first: those still running are the first m
        place = torch.tensor([starts[i] for i in order], device="cuda")
        end = torch.tensor([starts[i] + lens[i] for i in order], device="cuda")
        back = torch.tensor(order, device="cuda").argsort()
        S, m = S[order], N
        for t in range(max(lens)):
            while lens[order[m - 1]] <= t:
                m -= 1
            at = place[:m] + t
            S[:m] = lam * S[:m] + flat["k"][at][..., :, None] * flat["v"][at][..., None, :]
            if op == "linear_bwd":
                dq[at] = scale * (S[:m] @ flat["do"][at][..., None])[..., 0]
            else:
                o[at] = scale * (flat["q"][at][..., None, :] @ S[:m])[..., 0, :]
        if op != "linear_bwd":
            return shaped(o), S[back]
        dk, dv, m = torch.zeros_like(dq), torch.zeros_like(o), N
        R = (x["dht"] if case["state"] else zero)[order] / lam  # what stands one token after the last
        for t in range(max(lens)):
            while lens[order[m - 1]] <= t:
                m -= 1
            at = end[:m] - 1 - t
            R[:m] = lam * R[:m] + scale * flat["q"][at][..., :, None] * flat["do"][at][..., None, :]
            dk[at] = (R[:m] @ flat["v"][at][..., None])[..., 0]
            dv[at] = (flat["k"][at][..., None, :] @ R[:m])[..., 0, :]
        dq, dk = (t.unflatten(1, (case["H"], r)).sum(2) for t in (dq, dk))
        return [shaped(dq), shaped(dk), shaped(dv), (lam * R)[back] if case["state"] else None]
    H, HK, G = case["H"], case["HK"], case["H"] // case["HK"]
    got = {k: torch.zeros_like(flat[v]) for k, v in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "k"))}
    lse = torch.zeros(H, case["T"], dtype=torch.float64, device="cuda")
    for a, n in zip(starts, lens):
        for i in range(0, n, 512):
            j = min(n, i + 512)
            lo = max(0, i - case["window"] + 1)
            cols = list(range(min(case["sinks"], lo))) + list(range(lo, j))
            cols = torch.tensor(cols, device="cuda")
            gap = torch.arange(i, j, device="cuda")[:, None] - cols
            hidden = (gap < 0) | ((gap >= case["window"]) & (cols >= case["sinks"]))
            q, k, v = flat["q"][a + i:a + j], flat["k"][a + cols], flat["v"][a + cols]
            z = torch.einsum("ihgd,jhd->hgij", q.unflatten(1, (HK, G)), k) / math.sqrt(case["D"])
            z = z.masked_fill(hidden, -math.inf)
            l = torch.logsumexp(z, -1)
            p = torch.exp(z - l[..., None])
            o = torch.einsum("hgij,jhd->ihgd", p, v)
            lse[:, a + i:a + j] = l.flatten(0, 1)
            got["o"][a + i:a + j] = o.flatten(1, 2)
            if op == "window_bwd":
                do = flat["do"][a + i:a + j].unflatten(1, (HK, G))
                dp = torch.einsum("ihgd,jhd->hgij", do, v)
                dz = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(case["D"])
                got["dq"][a + i:a + j] = torch.einsum("hgij,jhd->ihgd", dz, k).flatten(1, 2)
                got["dk"][a + cols] += torch.einsum("hgij,ihgd->jhd", dz, q.unflatten(1, (HK, G)))
                got["dv"][a + cols] += torch.einsum("hgij,ihgd->jhd", p, do)
    if op == "window_bwd":
        return [shaped(got[k]) for k in ("dq", "dk", "dv")]
    o = shaped(got["o"])
    B, T = o.shape[:2]
    return (o, lse.reshape(H, B, T).transpose(0, 1)) if case["lse"] else o
