"""Linear attention with a decay per head and attention with a sliding window and sinks on the GPU against their 64-bit forms
(``mixer_reference``), element by element within bounds that count roundings, at the sizes where kernels go wrong: one token, tiles that
end inside, sequences of any length next to each other, empty ones, shared heads, strided and unaligned inputs, rows that see nothing."""
import ctypes

import pytest
import torch

import layer_c
import mixer_reference as ref
import test_mixers_host as host

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import gated_deltanet_gb300 as g
    g.load_library()
    yield g
    assert g.read_layer_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def offsets(lens):
    return None if lens is None else torch.tensor([0] + lens, device="cuda").cumsum(0)


# ---------------------------------------------------------------- linear attention
# (B, T or lengths, H, HV, K, V)
LINEAR = [
    (1, 1, 1, 1, 128, 128), (2, 127, 2, 2, 128, 128), (1, 128, 1, 2, 128, 128), (3, 129, 2, 2, 128, 128), (1, 600, 2, 4, 128, 128),
    (2, 300, 1, 1, 64, 64), (1, 65, 2, 6, 64, 64), (1, 257, 1, 1, 128, 64), (1, 100, 2, 2, 32, 20), (2, 70, 1, 1, 256, 256), (1, 40, 1, 1, 7, 1),
    (1, [1, 0, 127, 128, 200, 3], 2, 2, 128, 128), (1, [0, 0, 5], 1, 3, 64, 64), (1, [130, 1, 1, 64], 2, 2, 33, 65),
]
LINEAR_STEEP = [(1, 300, 4, 4, 128, 128), (1, [200, 90], 4, 4, 64, 64)]


def linear_inputs(case, dtype, state, seed=0):
    B, T, H, HV, K, V = case
    cu = offsets(T) if isinstance(T, list) else None
    n, T = (len(T), sum(T)) if isinstance(T, list) else (B, T)
    g = gen(seed + T * 7 + K + HV)
    q, k, v = randn(g, B, T, H, K, dtype=dtype), randn(g, B, T, H, K, dtype=dtype), randn(g, B, T, HV, V, dtype=dtype)
    decay = -torch.exp2(-6.0 * torch.rand(HV, generator=g, device="cuda"))
    h0 = randn(g, n, HV, K, V) if state else None
    return q, k, v, decay, h0, cu, g


def longest(case):
    return max(case[1]) if isinstance(case[1], list) else case[1]


def check_linear(got, q, k, v, decay, scale, h0, cu, T):
    o, ht, so, sh = ref.linear(q, k, v, decay, scale, h0, cu)
    n = q.shape[3] + 2 * T + 16
    ref.check(got[0], o, ref.linear_bound(o, so, n, q.dtype), "o")
    ref.check(got[1], ht, ref.state_bound(sh, n, q.dtype), "state")
    if q.dtype == BF:  # three roundings of 2^-8 / sqrt(3) root mean square at most
        ref.check_norm(got[0], o, 2.0 ** -8, "o")
    ref.check_norm(got[1], ht, 1e-5, "state")


@pytest.mark.parametrize("case", LINEAR, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("state", [False, True])
def test_linear(gdn, case, dtype, state):
    q, k, v, decay, h0, cu, _ = linear_inputs(case, dtype, state)
    got = gdn.chunk_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    check_linear(got, q, k, v, decay, q.shape[3] ** -0.5, h0, cu, longest(case))
    assert got[0].dtype == dtype and got[1].dtype == F32


@pytest.mark.parametrize("case", LINEAR, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_recurrent(gdn, case, dtype):
    q, k, v, decay, h0, cu, _ = linear_inputs(case, dtype, True, 1)
    got = gdn.fused_recurrent_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    o, ht, so, sh = ref.linear(q, k, v, decay, q.shape[3] ** -0.5, h0, cu)
    n = q.shape[3] + 2 * longest(case) + 16
    ref.check(got[0], o, ref.half(dtype) * o.abs() + n * ref.SUM * so, "o")
    ref.check(got[1], ht, n * ref.SUM * sh, "state")


@pytest.mark.parametrize("case", LINEAR_STEEP, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_decays(gdn, case, dtype):
    """Nothing decays, everything at once (a factor of zero), too steep for a chunk's range, and almost nothing."""
    q, k, v, _, h0, cu, g = linear_inputs(case, dtype, True, 2)
    decay = torch.tensor([0.0, -torch.inf, -30.0, -1e-5], device="cuda")
    for f in (gdn.chunk_linear_attention, gdn.fused_recurrent_linear_attention):
        got = f(q, k, v, decay, 0.3, initial_state=h0, output_final_state=True, cu_seqlens=cu)
        check_linear(got, q, k, v, decay, 0.3, h0, cu, longest(case))
        none = f(q, k, v, None, 0.3, initial_state=h0, output_final_state=True, cu_seqlens=cu)
        check_linear(none, q, k, v, None, 0.3, h0, cu, longest(case))
    do, dht = randn(g, *v.shape, dtype=dtype), randn(g, *h0.shape)
    check_linear_bwd(gdn, q, k, v, decay, do, 0.3, h0, dht, cu, longest(case))
    check_linear_bwd(gdn, q, k, v, None, do, 0.3, h0, dht, cu, longest(case))


def check_linear_bwd(gdn, q, k, v, decay, do, scale, h0, dht, cu, T):
    got = gdn.chunk_linear_attention_bwd(q, k, v, decay, do, scale, h0, dht, cu)
    want, size = ref.linear_bwd(q, k, v, decay, do, scale, h0, dht, cu)
    n = max(q.shape[3], v.shape[3]) + 2 * T + 16 + v.shape[2]
    for name, a, b, s in zip(("dq", "dk", "dv"), got, want, size):
        ref.check(a, b, ref.linear_bound(b, s, n, q.dtype), name)
        if q.dtype == BF:
            ref.check_norm(a, b, 2.0 ** -8, name)
    assert (got[3] is None) == (h0 is None)
    if h0 is not None:
        ref.check(got[3], want[3], ref.state_bound(size[3], n, q.dtype), "dh0")


@pytest.mark.parametrize("case", LINEAR, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("state", [False, True])
def test_linear_bwd(gdn, case, dtype, state):
    q, k, v, decay, h0, cu, g = linear_inputs(case, dtype, state, 3)
    dht = randn(g, *((1 if cu is None else 0) * q.shape[0] + (0 if cu is None else len(cu) - 1), v.shape[2], q.shape[3], v.shape[3])) if state else None
    check_linear_bwd(gdn, q, k, v, decay, randn(g, *v.shape, dtype=dtype), q.shape[3] ** -0.5, h0, dht, cu, longest(case))


def test_linear_bwd_against_differences(gdn):
    """fp32: the slope of sum(o do) + sum(ht dht) along a direction, from the forward kernel at both sides.  The function is
    trilinear in (q, k, v), so that a central difference with step e is off by e^2 of a third-order term and by the sums' rounding
    over e: with e = 2^-5 both are below 1e-3 of the gradients' size here."""
    q, k, v, decay, h0, _, g = linear_inputs((1, 90, 2, 2, 64, 64), F32, True, 4)
    do, dht = randn(g, *v.shape), randn(g, *h0.shape)
    grads = gdn.chunk_linear_attention_bwd(q, k, v, decay, do, None, h0, dht)
    along = [randn(g, *t.shape) for t in (q, k, v, h0)]
    e = 2.0 ** -5

    def f(s):
        x = [t + s * u for t, u in zip((q, k, v, h0), along)]
        o, ht = gdn.chunk_linear_attention(x[0], x[1], x[2], decay, initial_state=x[3], output_final_state=True)
        return (o.double() * do).sum() + (ht.double() * dht).sum()

    slope = (f(e) - f(-e)) / (2 * e)
    third = (f(2 * e) - 2 * f(e) + 2 * f(-e) - f(-2 * e)) / (2 * e ** 3)  # of a cubic: exact but for rounding
    want = sum((a.double() * u).sum() for a, u in zip(grads, along))
    size = sum((a.double() * u).abs().sum() for a, u in zip(grads, along))
    assert abs(slope - e ** 2 / 6 * third - want) <= 1e-3 * size


def test_linear_long(gdn):
    """Many chunks and few heads (split along the sequence), against the recurrent form's fp32 states and the plain form of a piece."""
    for T in (3000, 20011):
        q, k, v, decay, h0, _, g = linear_inputs((1, T, 1, 1, 128, 128), BF, True, 5)
        decay = torch.tensor([-2e-4], device="cuda")
        o, ht = gdn.chunk_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True)
        o2, ht2 = gdn.fused_recurrent_linear_attention(q.float(), k.float(), v.float(), decay, initial_state=h0, output_final_state=True)
        ref.check_norm(o, o2.double(), 2.0 ** -8, "o")
        ref.check_norm(ht, ht2.double(), 2e-5, "state")
        do, dht = randn(g, *v.shape, dtype=BF), randn(g, *h0.shape)
        got = gdn.chunk_linear_attention_bwd(q, k, v, decay, do, None, h0, dht)
        want = gdn.chunk_linear_attention_bwd(q.float(), k.float(), v.float(), decay, do.float(), None, h0, dht)
        for name, a, b in zip(("dq", "dk", "dv", "dh0"), got, want):
            ref.check_norm(a, b.double(), 2e-5 if name == "dh0" else 2.0 ** -8, name)


@pytest.mark.parametrize("case", [(2, 4096, 2, 2, 128, 128), (1, 5000, 1, 2, 64, 64), (1, [700, 0, 3000, 129], 2, 2, 128, 128), (4, 127, 1, 1, 128, 128)], ids=str)
@pytest.mark.parametrize("slow", [False, True])
def test_linear_state_is_fp32(gdn, case, slow):
    """Final states and the initial state's gradient are returned in fp32 and are as good from bf16 inputs on the tensor cores: their 2-norm is off by
    what fp32 products may be (4e-7) and two units of the decays' exponentials (2^-22)."""
    q, k, v, decay, h0, cu, g = linear_inputs(case, BF, True, 9)
    if slow:
        decay = -torch.linspace(1e-5, 1e-3, v.shape[2], device="cuda")
    _, ht = gdn.chunk_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    do, dht = randn(g, *v.shape, dtype=BF), randn(g, *h0.shape)
    dh0 = gdn.chunk_linear_attention_bwd(q, k, v, decay, do, None, h0, dht, cu)[3]
    ref.check_norm(ht, ref.linear(q, k, v, decay, q.shape[3] ** -0.5, h0, cu)[1], 4e-7 + 2.0 ** -22, "state")
    ref.check_norm(dh0, ref.linear_bwd(q, k, v, decay, do, q.shape[3] ** -0.5, h0, dht, cu)[0][3], 4e-7 + 2.0 ** -22, "dh0")


@pytest.mark.parametrize("T", [1, 3])
def test_linear_state_in_place(gdn, T):
    q, k, v, decay, h0, _, _ = linear_inputs((3, T, 2, 4, 128, 128), BF, True, 6)
    o, ht = gdn.fused_recurrent_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True)
    cache = h0.clone()
    o2, ht2 = gdn.fused_recurrent_linear_attention(q, k, v, decay, initial_state=cache, output_final_state=True, final_state=cache)
    assert ht2.data_ptr() == cache.data_ptr() and torch.equal(ht, cache) and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_linear_strided(gdn, dtype, off):
    """Slices of one fused projection, on 16-byte boundaries and off them, and a transposed layout."""
    g = gen(9)
    B, T, H, D = 2, 150, 2, 64
    fused = randn(g, B, T, 3 * H * D + 16, dtype=dtype)[..., off:]
    q, k, v = (fused[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    decay = -torch.rand(H, generator=g, device="cuda")
    got = gdn.chunk_linear_attention(q, k, v, decay, output_final_state=True)
    check_linear(got, q, k, v, decay, D ** -0.5, None, None, T)
    turned = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    again = gdn.chunk_linear_attention(*turned, decay, output_final_state=True)
    check_linear(again, q, k, v, decay, D ** -0.5, None, None, T)
    do = randn(g, B, T, H * D + 8, dtype=dtype)[..., off and 1:][..., :H * D].unflatten(-1, (H, D))
    check_linear_bwd(gdn, q, k, v, decay, do, 0.2, None, None, None, T)
    one = gdn.fused_recurrent_linear_attention(q, k, v, decay, output_final_state=True)
    check_linear(one, q, k, v, decay, D ** -0.5, None, None, T)


# ---------------------------------------------------------------- window attention
# (B, Tq or lengths, Tk or lengths or None, H, HK, D, window, sinks)
WINDOW = [
    (1, 1, None, 1, 1, 128, 1, 0), (2, 127, None, 2, 1, 128, 64, 0), (1, 128, None, 2, 2, 128, 1000, 0), (1, 300, None, 4, 2, 128, 100, 4),
    (2, 129, None, 2, 2, 64, 1, 0), (1, 257, None, 2, 1, 64, 130, 1), (1, 260, None, 1, 1, 128, 7, 140), (1, 200, None, 2, 1, 40, 33, 2),
    (1, 90, None, 1, 1, 256, 20, 3), (1, 33, None, 1, 1, 1, 5, 1), (1, 513, None, 2, 1, 128, 128, 0), (1, 700, None, 8, 1, 64, 256, 300),
    # queries that continue a cache, and queries before the first key (rows that see nothing)
    (1, 100, 333, 2, 1, 128, 150, 4), (2, 1, 200, 2, 2, 128, 64, 2), (1, 300, 100, 2, 1, 128, 50, 3), (2, 150, 20, 1, 1, 64, 500, 0), (1, 5, 0, 1, 1, 128, 3, 1),
    # packed
    (1, [1, 0, 127, 128, 300, 3], None, 2, 1, 128, 100, 4), (1, [200, 64, 1], None, 3, 3, 64, 31, 0), (1, [0, 0, 77], None, 1, 1, 96, 10, 1),
    (1, [5, 0, 130, 40], [200, 3, 130, 7], 2, 1, 128, 60, 5),
]


def window_inputs(case, dtype, seed=0):
    B, Tq, Tk, H, HK, D, w, sinks = case
    cu = offsets(Tq) if isinstance(Tq, list) else None
    cu_k = offsets(Tk) if isinstance(Tk, list) else None
    tq = sum(Tq) if isinstance(Tq, list) else Tq
    tk = tq if Tk is None else sum(Tk) if isinstance(Tk, list) else Tk
    g = gen(seed + tq * 5 + D + w)
    q, k, v = randn(g, B, tq, H, D, dtype=dtype), randn(g, B, tk, HK, D, dtype=dtype), randn(g, B, tk, HK, D, dtype=dtype)
    return q, k, v, w, sinks, cu, cu_k, g


@pytest.mark.parametrize("case", WINDOW, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_window(gdn, case, dtype):
    q, k, v, w, sinks, cu, cu_k, _ = window_inputs(case, dtype)
    o, lse = gdn.window_attention(q, k, v, w, sinks, cu_seqlens=cu, cu_seqlens_k=cu_k, return_lse=True)
    eo, el, bo, bl = ref.window(q, k, v, w, sinks, q.shape[3] ** -0.5, cu, cu_k)
    ref.check(o, eo, bo, "o")
    ref.check(lse, el, bl, "lse")
    assert torch.equal(gdn.window_attention(q, k, v, w, sinks, cu_seqlens=cu, cu_seqlens_k=cu_k), o)


def check_window_bwd(gdn, q, k, v, do, w, sinks, scale, cu, cu_k):
    o, lse = gdn.window_attention(q, k, v, w, sinks, scale, cu, cu_k, return_lse=True)
    got = gdn.window_attention_bwd(do, q, k, v, o, lse, w, sinks, scale, cu, cu_k)
    want, bound = ref.window_bwd(do, q, k, v, o, w, sinks, scale, cu, cu_k)
    for name, a, b, e in zip(("dq", "dk", "dv"), got, want, bound):
        ref.check(a, b, e, name)
        if q.dtype == BF and b.norm() > 0:
            # the output's rounding, the operand's, and delta's from a rounded o: below 2^-8 together in the root mean square
            ref.check_norm(a, b, 2.0 ** -7 if name != "dv" else 2.0 ** -8, name)


@pytest.mark.parametrize("case", WINDOW, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_bwd(gdn, case, dtype):
    q, k, v, w, sinks, cu, cu_k, g = window_inputs(case, dtype, 1)
    check_window_bwd(gdn, q, k, v, randn(g, *q.shape, dtype=dtype), w, sinks, q.shape[3] ** -0.5, cu, cu_k)


@pytest.mark.parametrize("case", [
    # several runs of far queries to a tile of sinks, one tile of them and more
    (2, 2600, None, 2, 1, 128, 100, 4), (1, 3000, None, 2, 2, 64, 100, 300), (1, 2500, None, 2, 1, 128, 1, 512), (2, 1200, 2300, 2, 1, 64, 333, 130),
    # sequences of several runs next to short and empty ones, keys packed otherwise than queries
    (1, [1100, 2300, 0, 40, 1500], None, 2, 1, 128, 100, 4), (1, [1100, 40, 2300, 5], [1500, 900, 1200, 0], 2, 1, 64, 60, 130), (1, [3, 0, 1500, 7], [900, 1300, 2600, 2], 1, 1, 128, 90, 2),
    # lengths next to those from which on sinks are dealt out: window, sinks in tiles of 32, 64 or 128, in large batches half a run of 256 or 1024
    (1, [131, 132, 133, 163, 164, 165, 227, 228, 229, 357], None, 2, 1, 64, 100, 4), (1, [259, 260, 261, 291, 292, 293, 355, 356, 357, 500], None, 1, 1, 128, 100, 130),
    (1, [740, 739, 741, 260, 259, 261, 291, 292, 293, 60] * 5, None, 4, 4, 64, 100, 4),
], ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_bwd_far_queries(gdn, case, dtype):
    q, k, v, w, sinks, cu, cu_k, g = window_inputs(case, dtype, 5)
    check_window_bwd(gdn, q, k, v, randn(g, *q.shape, dtype=dtype), w, sinks, q.shape[3] ** -0.5, cu, cu_k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("long", [[], [1900], [1300, 0, 300, 2200]])
def test_window_many_sequences(gdn, dtype, long):
    """Hundreds of short and empty sequences, and between them none, one or a few that are longer than the window and the sinks."""
    short = [int(x) for x in torch.randint(0, 40, (200,), generator=torch.Generator().manual_seed(len(long)))]
    at = {20 + 50 * i: x for i, x in enumerate(long)}
    lens = [at.get(i, x) for i, x in enumerate(short)]
    q, k, v, w, sinks, cu, _, g = window_inputs((1, lens, None, 2, 1, 64, 50, 3), dtype, 6)
    o, lse = gdn.window_attention(q, k, v, w, sinks, cu_seqlens=cu, return_lse=True)
    eo, el, bo, bl = ref.window(q, k, v, w, sinks, 0.125, cu)
    ref.check(o, eo, bo, "o")
    ref.check(lse, el, bl, "lse")
    check_window_bwd(gdn, q, k, v, randn(g, *q.shape, dtype=dtype), w, sinks, 0.125, cu, None)


def test_window_bwd_against_differences(gdn):
    """fp32: the slope of sum(o do) along a direction.  Step 2^-7: the second-order term is below 1e-3 of the gradients' size, the
    sums' rounding over the step too."""
    q, k, v, w, sinks, _, _, g = window_inputs((1, 120, None, 4, 2, 64, 40, 3), F32, 2)
    do = randn(g, *q.shape)
    o, lse = gdn.window_attention(q, k, v, w, sinks, return_lse=True)
    grads = gdn.window_attention_bwd(do, q, k, v, o, lse, w, sinks)
    along = [randn(g, *t.shape) for t in (q, k, v)]
    e = 2.0 ** -7

    def f(s):
        return (gdn.window_attention(*(t + s * u for t, u in zip((q, k, v), along)), w, sinks).double() * do).sum()

    slope = (8 * (f(e) - f(-e)) - (f(2 * e) - f(-2 * e))) / (12 * e)
    want = sum((a.double() * u).sum() for a, u in zip(grads, along))
    size = sum((a.double() * u).abs().sum() for a, u in zip(grads, along))
    assert abs(slope - want) <= 1e-3 * size


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_window_strided(gdn, dtype, off):
    g = gen(19)
    B, T, H, D = 2, 200, 2, 64
    fused = randn(g, B, T, 3 * H * D + 16, dtype=dtype)[..., off:]
    q, k, v = (fused[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    o = gdn.window_attention(q, k, v, 70, 2)
    eo, _, bo, _ = ref.window(q, k, v, 70, 2, D ** -0.5)
    ref.check(o, eo, bo)
    turned = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    ref.check(gdn.window_attention(*turned, 70, 2), eo, bo)
    do = randn(g, B, T, H * D + 8, dtype=dtype)[..., off and 1:][..., :H * D].unflatten(-1, (H, D))
    check_window_bwd(gdn, q, k, v, do, 70, 2, 0.2, None, None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_large_scores(gdn, dtype):
    """Scores far apart from tile to tile (the running maximum moves by hundreds) and far below zero."""
    g = gen(23)
    T, D = 400, 128
    q, k, v = randn(g, 1, T, 1, D, dtype=dtype), randn(g, 1, T, 1, D), randn(g, 1, T, 1, D, dtype=dtype)
    k = (k * torch.linspace(0.1, 40, T, device="cuda")[None, :, None, None] - q.float() * 3).to(dtype)
    o, lse = gdn.window_attention(q, k, v, 250, 4, return_lse=True)
    eo, el, bo, bl = ref.window(q, k, v, 250, 4, D ** -0.5)
    ref.check(o, eo, bo, "o")
    ref.check(lse, el, bl, "lse")
    check_window_bwd(gdn, q, k, v, randn(g, 1, T, 1, D, dtype=dtype), 250, 4, D ** -0.5, None, None)


@pytest.mark.parametrize("H,HK", [(4, 2), (3, 3)])  # (a CTA's two tiles: two heads, neighbouring rows)
@pytest.mark.parametrize("D", [64, 128])
def test_window_tiles_without_keys(gdn, H, HK, D):
    """Tiles of queries that see no key at all write zeros over the place where their queries land: many of them, while copies on
    another stream slow the loads down."""
    g = gen(27)
    B, Tq, Tk = 4, 2300, 40
    q, k, v = randn(g, B, Tq, H, D, dtype=BF), randn(g, B, Tk, HK, D, dtype=BF), randn(g, B, Tk, HK, D, dtype=BF)
    cu, cu_k = offsets([700, 3, 1597]), offsets([0, 0, 37])
    side, src = torch.cuda.Stream(), torch.empty(2 ** 27, device="cuda", dtype=torch.uint8)
    dst = torch.empty_like(src)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            dst.copy_(src)
        o, lse = gdn.window_attention(q, k, v, 50, 3, return_lse=True)
        assert not o[:, :Tq - Tk].any() and (lse[..., :Tq - Tk] == -torch.inf).all()
        assert torch.isfinite(lse[..., Tq - Tk:]).all()
        o, lse = gdn.window_attention(q[:1], k[:1, :37], v[:1, :37], 50, 3, cu_seqlens=cu, cu_seqlens_k=cu_k, return_lse=True)
        assert not o[:, :Tq - 37].any() and (lse[..., :Tq - 37] == -torch.inf).all()
        assert torch.isfinite(lse[..., Tq - 37:]).all()
    side.synchronize()


# (N, T, S, H, HK, D, window, sinks, lengths)
STEP = [
    (1, 1, 64, 4, 1, 128, 16, 2, [40]), (3, 1, 300, 8, 2, 128, 100, 4, [300, 1, 0]), (2, 1, 1000, 2, 2, 64, 2000, 0, [999, 513]),
    (2, 3, 200, 4, 2, 128, 50, 5, [200, 2]), (1, 1, 4096, 32, 2, 128, 4096, 0, [4096]), (1, 1, 5000, 16, 1, 64, 700, 130, [4097]),
    (2, 2, 90, 3, 3, 40, 7, 1, [90, 61]), (1, 5, 40, 2, 1, 256, 12, 2, [33]), (1, 1, 20, 1, 1, 8, 1, 0, [20]), (2, 17, 257, 8, 1, 128, 64, 3, [257, 20]),
    (4, 1, 130, 24, 2, 96, 128, 1, [129, 130, 128, 7]),
]


@pytest.mark.parametrize("case", STEP, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_step(gdn, case, dtype):
    N, T, S, H, HK, D, w, sinks, lens = case
    g = gen(S + D)
    q, k, v = randn(g, N, T, H, D, dtype=dtype), randn(g, N, S, HK, D, dtype=dtype), randn(g, N, S, HK, D, dtype=dtype)
    for n, L in enumerate(lens):  # what was never written
        k[n, L:], v[n, L:] = torch.nan, torch.nan
    eo, bo = ref.window_step(q, k, v, lens, w, sinks, D ** -0.5)
    for t in (torch.int32, torch.int64):
        ref.check(gdn.window_attention_decode(q, k, v, torch.tensor(lens, dtype=t, device="cuda"), w, sinks), eo, bo)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_step_strided(gdn, dtype):
    """A cache with heads first, one that is a slice of a larger one off 16 bytes, lengths past its ends."""
    g = gen(31)
    N, S, H, HK, D = 2, 150, 4, 2, 64
    q = randn(g, N, 1, H, D, dtype=dtype)
    lens = torch.tensor([S + 7, -3], device="cuda")
    for k, v in ((randn(g, N, HK, S, D, dtype=dtype).transpose(1, 2), randn(g, N, S, HK, 2 * D, dtype=dtype)[..., D:]),
                 (randn(g, N, S, HK, D + 3, dtype=dtype)[..., 3:], randn(g, N, S, HK, D + 1, dtype=dtype)[..., 1:])):
        eo, bo = ref.window_step(q, k, v, [S, 0], 60, 2, 0.1)
        ref.check(gdn.window_attention_decode(q, k, v, lens, 60, 2, 0.1), eo, bo)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_step_in_turn(gdn, dtype):
    """A cache of window + sinks slots whose window is overwritten in turn, called with a window of all slots: as over all tokens."""
    g = gen(33)
    N, T, H, HK, D, w, sinks = 2, 75, 4, 2, 64, 24, 3
    q, k, v = randn(g, N, T, H, D, dtype=dtype), randn(g, N, T, HK, D, dtype=dtype), randn(g, N, T, HK, D, dtype=dtype)
    eo, _, bo, _ = ref.window(q, k, v, w, sinks, D ** -0.5)
    kept = [torch.full((N, w + sinks, HK, D), torch.nan, device="cuda", dtype=dtype) for _ in range(2)]
    for t in range(T):
        at = t if t < w + sinks else sinks + (t - sinks) % w
        kept[0][:, at], kept[1][:, at] = k[:, t], v[:, t]
        lens = torch.full((N,), min(t + 1, w + sinks), dtype=torch.int32, device="cuda")
        if t < w + sinks:  # (until it is full slots are positions)
            got = gdn.window_attention_decode(q[:, t:t + 1], *kept, lens, w, sinks)
        else:
            got = gdn.window_attention_decode(q[:, t:t + 1], *kept, lens, w + sinks)
        ref.check(got, eo[:, t:t + 1], bo[:, t:t + 1], t)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("at", [30, 1000])
def test_untouched_rows(gdn, at):
    """Tokens in front of the first sequence and behind the last stay as they were (outputs given by the caller) and reach nothing, whatever they hold."""
    g = gen(40)
    T, H, D = 470 + at, 2, 128
    cu = torch.tensor([at, 170 + at, 303 + at], device="cuda")
    q, k, v = (randn(g, 1, T, H, D, dtype=BF) for _ in range(3))
    for t in (q, k, v):
        t[:, :at], t[:, at + 303:] = torch.nan, torch.inf
    cut = [t[:, at:at + 303].contiguous() for t in (q, k, v)]
    decay = torch.tensor([-0.1, -0.01], device="cuda")
    out = torch.full_like(q, 7.0)
    gdn.chunk_linear_attention(q, k, v, decay, cu_seqlens=cu, out=out)
    want, _ = gdn.chunk_linear_attention(*cut, decay, cu_seqlens=cu - at)
    assert torch.equal(out[:, at:at + 303], want) and (out[:, :at] == 7).all() and (out[:, at + 303:] == 7).all()
    out.fill_(7.0)
    gdn.window_attention(q, k, v, 50, 3, cu_seqlens=cu, out=out)
    want = gdn.window_attention(*cut, 50, 3, cu_seqlens=cu - at)
    assert torch.equal(out[:, at:at + 303], want) and (out[:, :at] == 7).all() and (out[:, at + 303:] == 7).all()
    o, lse = gdn.window_attention(q, k, v, 50, 3, cu_seqlens=cu, return_lse=True)
    do = torch.randn_like(q)
    got = gdn.window_attention_bwd(do, q, k, v, o, lse, 50, 3, cu_seqlens=cu)
    want = gdn.window_attention_bwd(do[:, at:at + 303].contiguous(), *cut, o[:, at:at + 303].contiguous(), lse[:, :, at:at + 303].contiguous(), 50, 3, cu_seqlens=cu - at)
    for a, b in zip(got, want):
        assert torch.equal(a[:, at:at + 303], b)
    got = gdn.chunk_linear_attention_bwd(q, k, v, decay, do, cu_seqlens=cu)
    want = gdn.chunk_linear_attention_bwd(*cut, decay, do[:, at:at + 303].contiguous(), cu_seqlens=cu - at)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a[:, at:at + 303], b)


def test_neighbours_stay_apart(gdn):
    """A NaN or an infinity in one sequence of a packed batch reaches no other."""
    g = gen(41)
    lens, H, D = [70, 300, 129, 90], 2, 128
    cu = offsets(lens)
    q, k, v = (randn(g, 1, sum(lens), H, D, dtype=BF) for _ in range(3))
    do, decay = randn(g, 1, sum(lens), H, D, dtype=BF), torch.tensor([-0.1, -0.01], device="cuda")

    def everything():
        o, lse = gdn.window_attention(q, k, v, 60, 3, cu_seqlens=cu, return_lse=True)
        a, _ = gdn.chunk_linear_attention(q, k, v, decay, cu_seqlens=cu)
        return [o, a, *gdn.window_attention_bwd(do, q, k, v, o, lse, 60, 3, cu_seqlens=cu), *gdn.chunk_linear_attention_bwd(q, k, v, decay, do, cu_seqlens=cu)[:3]]

    clean = everything()
    for t in (q, k, v, do):
        t[:, 70:370] = torch.nan
        t[:, 200:300] = torch.inf
    for a, b in zip(everything(), clean):
        assert torch.equal(a[:, :70], b[:, :70]) and torch.equal(a[:, 370:], b[:, 370:])


def test_streams_and_graphs(gdn):
    """A run of them together (prompt, then tokens, then gradients) on a side stream and captured, replayed on new values."""
    g = gen(42)
    B, T, H, D = 2, 200, 2, 128
    q, k, v, do = (randn(g, B, T, H, D, dtype=BF) for _ in range(4))
    decay = torch.tensor([-0.1, -0.01], device="cuda")
    h0 = randn(g, B, H, D, D)
    lens = torch.tensor([T, 50], device="cuda")

    def all_of_them():
        o, ht = gdn.chunk_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True)
        o1, ht = gdn.fused_recurrent_linear_attention(q[:, :1], k[:, :1], v[:, :1], decay, initial_state=ht, output_final_state=True, final_state=ht)
        d = gdn.chunk_linear_attention_bwd(q, k, v, decay, do, None, h0)
        w, lse = gdn.window_attention(q, k, v, 64, 4, return_lse=True)
        w1 = gdn.window_attention_decode(q[:, -1:], k, v, lens, 64, 4)
        return [o, o1, ht, *d, w, lse, w1, *gdn.window_attention_bwd(do, q, k, v, w, lse, 64, 4)]

    want = all_of_them()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_of_them()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = all_of_them()
    for seed in (1, 2):
        new = [randn(gen(seed), *t.shape, dtype=BF) for t in (q, k, v, do)]
        for t, n in zip((q, k, v, do), new):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, all_of_them()):
            assert torch.equal(a, b)


def test_empty(gdn):
    q = torch.empty(0, 5, 2, 64, device="cuda", dtype=BF)
    o, ht = gdn.chunk_linear_attention(q, q, q, None, output_final_state=True)
    assert o.shape == q.shape and ht.shape == (0, 2, 64, 64)
    assert gdn.window_attention(q, q, q, 3).shape == q.shape
    z = torch.empty(2, 0, 2, 64, device="cuda", dtype=BF)
    h0 = torch.randn(2, 2, 64, 64, device="cuda")
    for f in (gdn.chunk_linear_attention, gdn.fused_recurrent_linear_attention):
        o, ht = f(z, z, z, None, initial_state=h0, output_final_state=True)
        assert torch.equal(ht, h0) and o.numel() == 0
        assert not f(z, z, z, None, output_final_state=True)[1].any()
    assert torch.equal(gdn.chunk_linear_attention_bwd(z, z, z, None, z, None, h0, h0)[3], h0)
    assert gdn.window_attention(z, z, z, 3).shape == z.shape
    k = torch.randn(2, 9, 2, 64, device="cuda").to(BF)
    lse = torch.empty(2, 2, 0, device="cuda")
    dq, dk, dv = gdn.window_attention_bwd(z, z, k, k, z, lse, 3)
    assert dq.numel() == 0 and not dk.any() and not dv.any()
    assert gdn.window_attention_decode(z, k, k, torch.tensor([9, 3], device="cuda"), 3).shape == z.shape


# ---------------------------------------------------------------- one sequence that holds up the others
@pytest.mark.parametrize("H,HV,D", [(1, 1, 128), (1, 2, 128), (2, 2, 64)])
def test_linear_packed_split(gdn, H, HV, D):
    """Of a packed batch only the sequences longer than a segment are split; the others, short and empty ones, keep their places."""
    lens = [0, 3, 9000, 1, 0, 200, 5000, 129]
    q, k, v, decay, h0, cu, g = linear_inputs((1, lens, H, HV, D, D), BF, True, 6)
    decay = -torch.linspace(2e-4, 2e-2, HV, device="cuda")
    o, ht = gdn.chunk_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    do, dht = randn(g, *v.shape, dtype=BF), randn(g, *h0.shape)
    got = gdn.chunk_linear_attention_bwd(q, k, v, decay, do, None, h0, dht, cu)
    o2, ht2 = gdn.fused_recurrent_linear_attention(q.float(), k.float(), v.float(), decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    want = gdn.chunk_linear_attention_bwd(q.float(), k.float(), v.float(), decay, do.float(), None, h0, dht, cu)
    at = 0
    for n, length in enumerate(lens):
        piece = slice(at, at + length)
        at += length
        ref.check_norm(ht[n], ht2[n].double(), 2e-5, "state")
        ref.check_norm(got[3][n], want[3][n].double(), 2e-5, "dh0")
        if length:
            ref.check_norm(o[:, piece], o2[:, piece].double(), 2.0 ** -8, "o")
            for name, a, b in zip(("dq", "dk", "dv"), got, want):
                ref.check_norm(a[:, piece], b[:, piece].double(), 2.0 ** -8, name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("long", [[], [1900], [1500, 0, 700, 2600]])
def test_linear_many_sequences(gdn, dtype, long):
    """Hundreds of short and empty sequences, and between them none, one or a few that are longer than a segment."""
    short = [int(x) for x in torch.randint(0, 40, (300,), generator=torch.Generator().manual_seed(len(long)))]
    at = {40 + 80 * i: x for i, x in enumerate(long)}
    lens = [at.get(i, x) for i, x in enumerate(short)]
    case = (1, lens, 1, 2, 64, 64)
    q, k, v, decay, h0, cu, g = linear_inputs(case, dtype, True, 7)
    got = gdn.chunk_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    check_linear(got, q, k, v, decay, 0.125, h0, cu, longest(case))
    do, dht = randn(g, *v.shape, dtype=dtype), randn(g, *h0.shape)
    check_linear_bwd(gdn, q, k, v, decay, do, 0.125, h0, dht, cu, longest(case))


@pytest.mark.parametrize("lens", [[2000, 1700, 3, 0, 1500], [900] * 8, [70] * 8], ids=str)
def test_linear_packed_rule(gdn, lens):
    """fp32, heads enough that several packed sequences' segment is chosen from their lengths: longer than what one sequence of all tokens would be
    cut into (the forward of the first), none (its gradients, equal lengths)."""
    case = (1, lens, 2, 24, 64, 64)
    q, k, v, decay, h0, cu, g = linear_inputs(case, F32, True, 8)
    got = gdn.chunk_linear_attention(q, k, v, decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    check_linear(got, q, k, v, decay, 0.125, h0, cu, longest(case))
    do, dht = randn(g, *v.shape), randn(g, *h0.shape)
    check_linear_bwd(gdn, q, k, v, decay, do, 0.125, h0, dht, cu, longest(case))


@pytest.mark.parametrize("window,sinks", [(100, 600), (2 ** 31 - 1, 2 ** 31 - 1), (2000, 0), (1, 1499)])
def test_window_many_sinks(gdn, window, sinks):
    """More sinks than are dealt out to CTAs of their own, and windows longer than the sequence."""
    q, k, v, _, _, _, _, g = window_inputs((1, 1500, None, 2, 1, 64, 1, 0), BF, 3)
    o, lse = gdn.window_attention(q, k, v, window, sinks, return_lse=True)
    eo, el, bo, bl = ref.window(q, k, v, window, sinks, 0.125)
    ref.check(o, eo, bo, "o")
    ref.check(lse, el, bl, "lse")
    check_window_bwd(gdn, q, k, v, randn(g, *q.shape, dtype=BF), window, sinks, 0.125, None, None)


def test_tables_are_clamped(gdn):
    """Offsets outside the tensor are taken as its ends."""
    g = gen(43)
    q, k, v, do = (randn(g, 1, 300, 2, 128, dtype=BF) for _ in range(4))
    decay, wild, cu = torch.tensor([-0.1, -0.01], device="cuda"), torch.tensor([-3, 170, 2 ** 40], device="cuda"), torch.tensor([0, 170, 300], device="cuda")

    def everything(cu):
        o, lse = gdn.window_attention(q, k, v, 60, 3, cu_seqlens=cu, return_lse=True)
        return [o, lse, *gdn.window_attention_bwd(do, q, k, v, o, lse, 60, 3, cu_seqlens=cu),
                *gdn.chunk_linear_attention(q, k, v, decay, output_final_state=True, cu_seqlens=cu),
                *gdn.fused_recurrent_linear_attention(q, k, v, decay, output_final_state=True, cu_seqlens=cu),
                *gdn.chunk_linear_attention_bwd(q, k, v, decay, do, cu_seqlens=cu)[:3]]

    for a, b in zip(everything(wild), everything(cu)):
        assert torch.equal(a, b)
    lens = torch.tensor([2 ** 40, -7], device="cuda")
    two = [t.view(2, 150, 2, 128) for t in (k, v)]
    got = gdn.window_attention_decode(q[:, :2].view(2, 1, 2, 128), *two, lens, 60, 3)
    assert torch.equal(got, gdn.window_attention_decode(q[:, :2].view(2, 1, 2, 128), *two, torch.tensor([150, 0], device="cuda"), 60, 3))


def test_offsets_past_32_bits(gdn):
    """2^24 + 1000 tokens of 128: the last rows, whose elements lie behind the 2^31st, against the plain forms of the last 700 tokens
    (what lies further back is outside the window, or has decayed by e^-150 and more)."""
    T, D, last, skip = 2 ** 24 + 1000, 128, 700, 300
    q, k, v, do = (torch.empty(1, T, 1, D, device="cuda", dtype=BF).normal_(generator=gen(44 + i)) for i in range(4))
    cut = [t[:, -last:].contiguous() for t in (q, k, v, do)]
    o, lse = gdn.window_attention(q, k, v, 64, 0, return_lse=True)
    eo, el, bo, bl = ref.window(*cut[:3], 64, 0, D ** -0.5)
    ref.check(o[:, -last + skip:], eo[:, skip:], bo[:, skip:], "o")
    ref.check(lse[..., -last + skip:], el[..., skip:], bl[..., skip:], "lse")
    got = gdn.window_attention_bwd(do, q, k, v, o, lse, 64, 0)
    want, bound = ref.window_bwd(cut[3], *cut[:3], o[:, -last:], 64, 0, D ** -0.5)
    for name, a, b, e in zip(("dq", "dk", "dv"), got, want, bound):
        ref.check(a[:, -last + skip:], b[:, skip:], e[:, skip:], name)
    del got, o, lse
    decay = torch.tensor([-0.5], device="cuda")
    o, ht = gdn.chunk_linear_attention(q, k, v, decay, output_final_state=True)
    eo, eh, so, sh = ref.linear(*cut[:3], decay, D ** -0.5, None, None)
    n = D + 2 * last + 16
    ref.check(o[:, -last + skip:], eo[:, skip:], ref.linear_bound(eo, so, n, BF)[:, skip:], "o")
    ref.check(ht, eh, ref.state_bound(sh, n, BF), "state")
    got = gdn.chunk_linear_attention_bwd(q, k, v, decay, do)
    want, size = ref.linear_bwd(*cut[:3], decay, cut[3], D ** -0.5, None, None, None)
    for name, a, b, s in zip(("dq", "dk", "dv"), got, want, size):
        ref.check(a[:, -last + skip:], b[:, skip:], ref.linear_bound(b, s, n + D, BF)[:, skip:], name)
    del got, o
    # one sequence's cache of as many slots: its newest and its first
    lens = torch.tensor([T], device="cuda")
    near = [torch.cat([t[:, :4], t[:, -64:]], 1) for t in (k, v)]
    got = gdn.window_attention_decode(q[:, -1:], k, v, lens, 64, 4)
    eo, bo = ref.window_step(q[:, -1:], *near, [68], 64, 4, D ** -0.5)
    ref.check(got, eo, bo, "o")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_bwd_o_by_strides(gdn, dtype):
    """The forward's output as it lies: heads in front of tokens, a slice, elements apart, one value for all heads."""
    for B, cu in ((2, None), (1, offsets([130, 0, 70]))):
        q, k, v, w, sinks, _, _, g = window_inputs((B, 200, None, 4, 2, 64, 40, 3), dtype, 4)
        do = randn(g, *q.shape, dtype=dtype)
        o, lse = gdn.window_attention(q, k, v, w, sinks, cu_seqlens=cu, return_lse=True)
        want = gdn.window_attention_bwd(do, q, k, v, o, lse, w, sinks, cu_seqlens=cu)
        wide = torch.zeros(B, 200, 4, 72, device="cuda", dtype=dtype)
        odd = torch.zeros(B, 200, 4, 65, device="cuda", dtype=dtype)
        wide[..., :64], odd[..., 1:] = o, o
        for p in (o.transpose(1, 2).contiguous().transpose(1, 2), o.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3), wide[..., :64], odd[..., 1:],
                  o.transpose(2, 3).contiguous().transpose(2, 3)):
            for a, b in zip(gdn.window_attention_bwd(do, q, k, v, p, lse, w, sinks, cu_seqlens=cu), want):
                assert torch.equal(a, b)
        one = o[:, :, :1].expand(-1, -1, 4, -1)
        for a, b in zip(gdn.window_attention_bwd(do, q, k, v, one, lse, w, sinks, cu_seqlens=cu),
                        gdn.window_attention_bwd(do, q, k, v, one.contiguous(), lse, w, sinks, cu_seqlens=cu)):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- calls of the C entries, at once, and cut short
def linear_call(lib, q, k, v, decay, do=None, stream=0):
    """(run, outputs): gdn_linear_attn, or its gradients, with the library's own workspace."""
    B, T, H, D = q.shape
    HV = v.shape[2]
    out = [torch.empty_like(v)] if do is None else [torch.empty_like(t) for t in (q, k, v)]
    named = dict(o=out[0]) if do is None else dict(zip(("dq", "dk", "dv"), out), dout=do)
    a = host.GdnLinearAttnArgs(**layer_c.pointers(B=B, T=T, H=H, HV=HV, K=D, V=D, num_seqs=B, dtype=1, scale=0.1, q=q, k=k, v=v, ldq=H * D, ldk=H * D,
                                                  ldv=HV * D, decay=decay, ld_dout=HV * D, **named))
    f = lib.gdn_linear_attn if do is None else lib.gdn_linear_attn_bwd
    return lambda kept=(q, k, v, decay, do): f(ctypes.byref(a), None, 0, stream), out  # (the block holds addresses alone)


def window_call(lib, q, k, v, o, lse, do=None, stream=0):
    B, T, H, D = q.shape
    HK = k.shape[2]
    grads = [] if do is None else [torch.empty_like(t) for t in (q, k, v)]
    a = host.GdnWindowAttnArgs(**layer_c.pointers(B=B, Tq=T, Tk=T, H=H, HK=HK, D=D, num_seqs=B, dtype=1, window=200, sinks=4, scale=0.1, q=q, k=k, v=v, ldq=H * D,
                                                  ldk=HK * D, ldv=HK * D, o=o, lse=lse, ld_dout=H * D, dout=do, **dict(zip(("dq", "dk", "dv"), grads))))
    f = lib.gdn_window_attn if do is None else lib.gdn_window_attn_bwd
    return lambda kept=(q, k, v, o, lse, do): f(ctypes.byref(a), None, 0, stream), grads or [o, lse]


L = host.L


def calls_and_results(gdn, lib, seed, stream=0):
    """Calls that take workspaces of the library's, in the order of a training step, their outputs, and what the binding gives."""
    g = gen(seed)
    q, k = (randn(g, 1, 3000, 1, 128, dtype=BF) for _ in range(2))
    v, do = (randn(g, 1, 3000, 2, 128, dtype=BF) for _ in range(2))
    decay = torch.tensor([-0.1, -1e-3], device="cuda")
    o, lse = torch.empty_like(v), torch.empty(1, 2, 3000, device="cuda")
    calls = [linear_call(lib, q, k, v, decay, None, stream), linear_call(lib, q, k, v, decay, do, stream), window_call(lib, v, q, k, o, lse, None, stream),
             window_call(lib, v, q, k, o, lse, do, stream)]
    w, l = gdn.window_attention(v, q, k, 200, 4, 0.1, return_lse=True)
    want = [[gdn.chunk_linear_attention(q, k, v, decay, 0.1)[0]], gdn.chunk_linear_attention_bwd(q, k, v, decay, do, 0.1)[:3], [w, l],
            gdn.window_attention_bwd(do, v, q, k, w, l, 200, 4, 0.1)]
    return calls, want


def test_library_workspace(gdn, L):
    """Without a workspace of the caller's, on two streams at once: as with one each."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [calls_and_results(gdn, L, 50 + i, s.cuda_stream) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for _ in range(3):
        for steps in zip(*(calls for calls, _ in both)):
            for run, _ in steps:
                assert run() == 0
    torch.cuda.synchronize()
    for calls, want in both:
        for (_, out), w in zip(calls, want):
            for a, b in zip(out, w):
                assert torch.equal(a, b)


def test_two_graphs_at_once(gdn):
    """Two captured runs, with the binding's workspaces, replayed on two streams at once."""
    g = gen(45)
    runs = []
    for _ in range(2):
        q, k = (randn(g, 1, 3000, 1, 128, dtype=BF) for _ in range(2))
        v, do = (randn(g, 1, 3000, 2, 128, dtype=BF) for _ in range(2))
        decay = torch.tensor([-0.1, -1e-3], device="cuda")

        def run(q=q, k=k, v=v, do=do, decay=decay):
            o, ht = gdn.chunk_linear_attention(q, k, v, decay, output_final_state=True)
            w, lse = gdn.window_attention(v, q, k, 200, 4, return_lse=True)
            return [o, ht, w, lse, *gdn.chunk_linear_attention_bwd(q, k, v, decay, do)[:3], *gdn.window_attention_bwd(do, v, q, k, w, lse, 200, 4)]
        want = run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        runs.append((graph, got, want, torch.cuda.Stream(), run))  # (run: a graph does not keep the tensors that were there before it)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, _, _, stream, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, want, _, _ in runs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_waits_that_run_out(gdn, L):
    """Calls whose kernels load nothing, so that their waits run out after 5 ms: reported once, and the next call is right."""
    L.gdn_layer_test_withhold.argtypes, L.gdn_layer_test_withhold.restype = [ctypes.c_int], None
    calls, want = calls_and_results(gdn, L, 52)
    torch.cuda.synchronize()
    assert gdn.read_layer_status() == 0
    for (run, out), w in zip(calls, want):
        L.gdn_layer_test_withhold(1)
        try:
            assert run() == 0
        finally:
            L.gdn_layer_test_withhold(0)
        torch.cuda.synchronize()
        assert gdn.read_layer_status() == -4 and gdn.read_layer_status() == 0
        assert run() == 0
        torch.cuda.synchronize()
        for a, b in zip(out, w):
            assert torch.equal(a, b)
