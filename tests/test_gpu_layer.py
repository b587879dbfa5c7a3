"""The decoder-block operators on the GPU against their 64-bit forms (``layer_reference``), element by element
within bounds that count roundings, at the sizes where kernels go wrong: one row, odd widths, rows that are not
16-byte aligned, strided inputs, partial tiles in every direction, empty batches."""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


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


# ---------------------------------------------------------------- norm
NORM_SIZES = [(1, 1), (3, 7), (5, 64), (257, 128), (2, 100), (33, 1001), (64, 2048), (3, 4104), (2, 8192), (3, 8193), (2, 20000),
              (700, 16), (1, 513)]


@pytest.mark.parametrize("M,D", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(gdn, M, D, dtype, residual):
    g = gen(M * 31 + D)
    x = randn(g, M, D, dtype=dtype)
    r = 3 * randn(g, M, D) if residual else None
    r = r.to(dtype) if residual else None
    w = [None, 1 + 0.3 * randn(g, D), (1 + 0.3 * randn(g, D)).to(BF)][(M + D) % 3]
    y, h = gdn.rms_norm(x, w, r, 1e-5)
    ey, eh = ref.norm(x, r, w, 1e-5)
    by, bh = ref.norm_bound(ey, eh, D, dtype)
    ref.check(y, ey, by, "y")
    assert (h is None) == (r is None)
    if r is not None:
        ref.check(h, eh, bh, "h")
    q, s, h2 = gdn.rms_norm_quant(x, w, r, 1e-5)
    check_quant(q, s, ey, D)
    if r is not None:
        assert torch.equal(h2, h)


def check_quant(q, s, y, D):
    want = (y.abs().amax(-1) / ref.E4M3_MAX).clamp_min(ref.SCALE_MIN)
    rel = (D + 16) * ref.SUM
    ref.check(s, want, want * rel, "scale")
    # half a step of e4m3 (2^-10 below its smallest normal value 2^-6), on top of the statistics' error
    units = y / want[..., None]
    ref.check(q, units, 2 ** -4 * units.abs().clamp_min(2 ** -6) + 2 * rel * units.abs(), "q")
    assert q.float().abs().max() <= 448
    if y.numel():
        assert (q.float().abs().amax(-1)[want > ref.SCALE_MIN] == 448).all()


@pytest.mark.parametrize("M,D", [(5, 64), (33, 1001), (3, 8193)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_rows(gdn, M, D, dtype):
    x = randn(gen(D), M, D, dtype=dtype) * torch.logspace(-3, 3, M, device="cuda")[:, None].to(dtype)
    x[0] = 0
    q, s = gdn.quantize_rows(x)
    check_quant(q, s, x.double(), D)
    assert s[0] == ref.SCALE_MIN and not q[0].float().any()


@pytest.mark.parametrize("M,D", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_bwd(gdn, M, D, dtype):
    g = gen(M * 17 + D)
    h, dy = randn(g, M, D, dtype=dtype), randn(g, M, D, dtype=dtype)
    dh = randn(g, M, D, dtype=dtype) if (M + D) % 2 else None
    w = 1 + 0.3 * randn(g, D)
    dx, dw = gdn.rms_norm_bwd(dy, h, w, dh, 1e-5)
    ex, ew = ref.norm_bwd(dy, h, w, dh, 1e-5)
    bx, bw = ref.norm_bwd_bound(dy, h, w, dh, 1e-5, ex, dtype)
    ref.check(dx, ex, bx, "dx")
    ref.check(dw, ew, bw, "dw")
    dx2, dw2 = gdn.rms_norm_bwd(dy, h, None, dh, 1e-5)
    ex, ew = ref.norm_bwd(dy, h, None, dh, 1e-5)
    ref.check(dx2, ex, ref.norm_bwd_bound(dy, h, None, dh, 1e-5, ex, dtype)[0], "dx without a weight")
    assert dw2 is None


def test_norm_many_rows(gdn):
    """More rows than a grid holds at once, several rows per block, and sums over all of them."""
    g = gen(5)
    M, D = 30001, 128
    h, dy, w = randn(g, M, D, dtype=BF), randn(g, M, D, dtype=BF), 1 + 0.3 * randn(g, D)
    y, _ = gdn.rms_norm(h, w)
    ey, eh = ref.norm(h, None, w, 1e-6)
    ref.check(y, ey, ref.norm_bound(ey, eh, D, BF)[0])
    dx, dw = gdn.rms_norm_bwd(dy, h, w)
    ex, ew = ref.norm_bwd(dy, h, w, None, 1e-6)
    bx, bw = ref.norm_bwd_bound(dy, h, w, None, 1e-6, ex, BF)
    ref.check(dx, ex, bx)
    ref.check(dw, ew, bw)
    again = gdn.rms_norm_bwd(dy, h, w)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # a fixed order of sums


def test_norm_rows_with_infinities_and_nan(gdn):
    """A row with a NaN or an infinity spoils itself and no other; a zero row stays finite."""
    g = gen(6)
    x = randn(g, 6, 256, dtype=BF)
    x[1, 3], x[2, 4], x[3] = float("nan"), float("inf"), 0
    y, _ = gdn.rms_norm(x, None)
    good = [0, 3, 4, 5]
    ey, eh = ref.norm(x, None, None, 1e-6)
    ref.check(y[good], ey[good], ref.norm_bound(ey[good], eh[good], 256, BF)[0])
    assert y[1].isnan().all() and y[2, 4].isnan()
    q, s, _ = gdn.rms_norm_quant(x, None)
    assert s[1].isnan() and s[2].isnan() and s[good].isfinite().all() and q[good].float().isfinite().all()
    assert q[1].float().isnan().all() and not q[3].float().any()


def test_norm_strides_and_shapes(gdn):
    g = gen(7)
    fused = randn(g, 4, 9, 3 * 128, dtype=BF)
    x, r = fused[..., 128:256], fused[..., 256:]
    y, h = gdn.rms_norm(x, None, r)
    y2, h2 = gdn.rms_norm(x.contiguous(), None, r.contiguous())
    assert y.shape == x.shape and torch.equal(y, y2) and torch.equal(h, h2)
    odd = randn(g, 5 * 129 + 1, dtype=BF)[1:].view(5, 129)[:, :128]  # rows on odd elements
    ey, eh = ref.norm(odd, None, None, 1e-6)
    ref.check(gdn.rms_norm(odd)[0], ey, ref.norm_bound(ey, eh, 128, BF)[0])
    # the residual stream updated in place
    stream = r.contiguous()
    y3, h3 = gdn.rms_norm(x, None, stream, residual_out=stream)
    assert h3 is stream and torch.equal(stream, h2) and torch.equal(y3, y2)
    wide = randn(g, 3, 9000, dtype=BF)
    stream = randn(g, 3, 9000, dtype=BF)
    y4, h4 = gdn.rms_norm(wide, None, stream.clone())
    y5, h5 = gdn.rms_norm(wide, None, stream, residual_out=stream)
    assert torch.equal(y4, y5) and torch.equal(h4, stream)


# ---------------------------------------------------------------- products
SIZES = [(1, 1, 1), (1, 128, 64), (3, 17, 33), (1, 2048, 1000), (16, 256, 128), (64, 640, 520), (65, 129, 4096), (127, 130, 72),
         (257, 384, 192), (300, 1000, 520), (1025, 640, 704), (2000, 264, 48)]
COMBOS = [("none", False, False), ("silu", True, True), ("gelu", True, False), ("gelu_tanh", False, True), ("relu", True, True),
          ("sigmoid", False, False), ("none", True, True)]


def operands(g, M, N, K, dtype):
    x, w = randn(g, M, K), randn(g, N, K) / K ** 0.5
    if dtype != E4:
        return x.to(dtype), w.to(dtype), None, None
    xs, ws = 0.5 + torch.rand(M, generator=g, device="cuda"), 0.5 + torch.rand(N, generator=g, device="cuda")
    return (x * 16).to(E4), (w * 16).to(E4), xs / 16, ws / 16


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32, E4])
def test_linear(gdn, M, N, K, dtype):
    name, has_bias, has_res = COMBOS[(M + N + K) % len(COMBOS)]
    g = gen(M + 3 * N + 7 * K)
    x, w, xs, ws = operands(g, M, N, K, dtype)
    b = randn(g, N) if has_bias else None
    for out in ((F32,) if dtype == F32 else (BF, F32)):
        r = randn(g, M, N, dtype=out) if has_res else None
        y = gdn.linear(x, w, b, name, r, x_scale=xs, weight_scale=ws, out_dtype=out)
        want, bound = ref.linear(x, w, b, name, r, out, xs, ws)
        assert y.dtype == out and y.shape == (M, N)
        ref.check(y, want, bound, f"{name} {out}")


@pytest.mark.parametrize("name,has_bias,has_res", [(a, b, r) for a in ref.ACTS for b in (False, True) for r in (False, True)])
@pytest.mark.parametrize("M", [5, 300])
def test_linear_epilogues(gdn, name, has_bias, has_res, M):
    g = gen(11)
    x, w = randn(g, M, 192, dtype=BF), (randn(g, 272, 192) / 5).to(BF)
    b = randn(g, 272) if has_bias else None
    r = randn(g, M, 272, dtype=BF) if has_res else None
    y = gdn.linear(x, w, b, name, r)
    want, bound = ref.linear(x, w, b, name, r, BF)
    ref.check(y, want, bound)
    if has_res:
        stream = r.clone()
        assert gdn.linear(x, w, b, name, stream, out=stream) is stream and torch.equal(stream, y)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_bwd(gdn, M, N, K, dtype):
    name, has_bias, _ = COMBOS[(M + N + 2 * K) % len(COMBOS)]
    g = gen(M + 5 * N + 7 * K)
    x, w, _, _ = operands(g, M, N, K, dtype)
    b = randn(g, N) if has_bias else None
    dy = randn(g, M, N, dtype=dtype)
    got = gdn.linear_bwd(dy, x, w, b, name)
    want, bound = ref.linear_bwd(dy, x, w, b, name, dtype)
    for n, a, e, t in zip(("dx", "dw", "db"), got, want, bound):
        if a is not None:
            ref.check(a, e, t, f"{name} {n}")
    assert (got[2] is None) == (b is None)
    only = gdn.linear_bwd(dy, x, w, b, name, need_dx=False)
    assert only[0] is None and torch.equal(only[1], got[1])
    only = gdn.linear_bwd(dy, x, w, b, name, need_dweight=False)
    assert only[1] is None and torch.equal(only[0], got[0])


@pytest.mark.parametrize("M,F,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32, E4])
def test_gated(gdn, M, F, K, dtype):
    name = ref.ACTS[(M + F + K) % len(ref.ACTS)]
    g = gen(M + 3 * F + 5 * K)
    x, w, xs, ws = operands(g, M, 2 * F, K, dtype)
    y = gdn.gated_linear(x, w, name, x_scale=xs, weight_scale=ws)
    want, bound = ref.gated(x, w, name, y.dtype, xs, ws)
    assert y.shape == (M, F)
    ref.check(y, want, bound, name)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("M", [5, 300])
def test_gated_activations(gdn, name, M):
    g = gen(13)
    x, w = randn(g, M, 192, dtype=BF), (randn(g, 2 * 136, 192) / 5).to(BF)
    ref.check(gdn.gated_linear(x, w, name), *ref.gated(x, w, name, BF))
    dy = randn(g, M, 136, dtype=BF)
    got, (want, bound) = gdn.gated_linear_bwd(dy, x, w, name), ref.gated_bwd(dy, x, w, name, BF)
    for a, e, t in zip(got, want, bound):
        ref.check(a, e, t)


@pytest.mark.parametrize("M,F,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gated_bwd(gdn, M, F, K, dtype):
    name = ("silu", "gelu", "gelu_tanh", "sigmoid")[(M + F + K) % 4]
    g = gen(M + 3 * F + 11 * K)
    x, w, _, _ = operands(g, M, 2 * F, K, dtype)
    dy = randn(g, M, F, dtype=dtype)
    dx, dw, y = gdn.gated_linear_bwd(dy, x, w, name, return_output=True)
    want, bound = ref.gated_bwd(dy, x, w, name, dtype)
    ref.check(dx, want[0], bound[0], f"{name} dx")
    ref.check(dw, want[1], bound[1], f"{name} dw")
    ref.check(y, *ref.gated(x, w, name, dtype), f"{name} y")


# contractions long enough, and outputs few enough, for several pairs of SMs to share a tile; the least rows of the tiles
# of 256; a weight's gradient over many rows
LONG = [(128, 130, 1600), (129, 72, 1600), (129, 200, 3216), (257, 330, 3200), (520, 129, 6416), (4100, 72, 104)]


@pytest.mark.parametrize("M,N,K", LONG)
@pytest.mark.parametrize("dtype", [BF, F32, E4])
def test_long_contractions(gdn, M, N, K, dtype):
    g = gen(M + N + K)
    x, w, xs, ws = operands(g, M, N, K, dtype)
    b = randn(g, N)
    for out in ((F32,) if dtype == F32 else (BF, F32)):
        r = randn(g, M, N, dtype=out)
        y = gdn.linear(x, w, b, "gelu", r, x_scale=xs, weight_scale=ws, out_dtype=out)
        want, bound = ref.linear(x, w, b, "gelu", r, out, xs, ws)
        ref.check(y, want, bound, f"{out}")
        assert torch.equal(y, gdn.linear(x, w, b, "gelu", r, x_scale=xs, weight_scale=ws, out_dtype=out))
    x, w, xs, ws = operands(g, M, 2 * N, K, dtype)
    h = gdn.gated_linear(x, w, "silu", x_scale=xs, weight_scale=ws)
    want, bound = ref.gated(x, w, "silu", F32 if dtype == F32 else BF, xs, ws)
    ref.check(h, want, bound, "gated")


@pytest.mark.parametrize("M,N,K", LONG)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_contractions_bwd(gdn, M, N, K, dtype):
    g = gen(M + N + K)
    x, w, _, _ = operands(g, M, N, K, dtype)
    b, dy = randn(g, N), randn(g, M, N, dtype=dtype)
    want, bound = ref.linear_bwd(dy, x, w, b, "silu", dtype)
    got = gdn.linear_bwd(dy, x, w, b, "silu")
    for n, a, e, t in zip(("dx", "dw", "db"), got, want, bound):
        ref.check(a, e, t, n)
    assert all(torch.equal(a, c) for a, c in zip(got, gdn.linear_bwd(dy, x, w, b, "silu")))
    w = operands(g, M, 2 * N, K, dtype)[1]
    got, (want, bound) = gdn.gated_linear_bwd(dy, x, w, "gelu"), ref.gated_bwd(dy, x, w, "gelu", dtype)
    for n, a, e, t in zip(("dx", "dw"), got, want, bound):
        ref.check(a, e, t, f"gated {n}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_against_differences(gdn, dtype):
    """Central differences of the 64-bit forward along random directions."""
    g = gen(17)
    M, N, K, t = 70, 96, 136, 1e-4
    x, w, _, _ = operands(g, M, 2 * N, K, dtype)
    b, dy, dy2 = randn(g, 2 * N), randn(g, M, 2 * N, dtype=dtype), randn(g, M, N, dtype=dtype)

    def along(f, args, i, d, up):
        vals = []
        for s in (t, -t):
            a = [v.double() for v in args]
            a[i] = a[i] + s * d
            vals.append((f(*a) * up.double()).sum())
        return (vals[0] - vals[1]) / (2 * t)

    cases = [(lambda x, w, b: ref.linear(x, w, b, "silu", None, dtype)[0], (x, w, b), dy, gdn.linear_bwd(dy, x, w, b, "silu"),
              ref.linear_bwd(dy, x, w, b, "silu", dtype)[1]),
             (lambda x, w: ref.gated(x, w, "gelu", dtype)[0], (x, w), dy2, gdn.gated_linear_bwd(dy2, x, w, "gelu"),
              ref.gated_bwd(dy2, x, w, "gelu", dtype)[1])]
    nw = 1 + 0.3 * randn(g, K)
    dyn = randn(g, M, K, dtype=dtype)
    got = gdn.rms_norm_bwd(dyn, x, nw)
    bounds = ref.norm_bwd_bound(dyn, x, nw, None, 1e-6, ref.norm_bwd(dyn, x, nw, None, 1e-6)[0], dtype)
    cases.append((lambda h, w: ref.norm(h, None, w, 1e-6)[0], (x, nw), dyn, got, bounds))
    for f, args, up, grads, bound in cases:
        for i, (grad, bnd) in enumerate(zip(grads, bound)):
            d = torch.randn(grad.shape, generator=g, device="cuda").double()
            want, have = along(f, args, i, d, up), (grad.double() * d).sum()
            # the elements' bounds, and the differences' own error of order t^2
            assert (have - want).abs() <= (bnd * d.abs()).sum() + 1e-5 * want.abs() + 1e-5, (i, float(have), float(want))


def test_products_take_strided_and_unaligned_rows(gdn):
    g = gen(19)
    fused = randn(g, 3, 50, 3 * 128, dtype=BF)
    x = fused[..., 128:256]
    w = (randn(g, 200, 300) / 11).to(BF)[:, 100:228]
    r = randn(g, 150, 410, dtype=BF)[:, 3:203]
    y = gdn.linear(x, w, None, None, r)
    want, bound = ref.linear(x.reshape(150, 128), w, None, "none", r, BF)
    assert y.shape == (3, 50, 200)
    ref.check(y.view(150, 200), want, bound)
    flat = randn(g, 70 * 130 + 1, dtype=BF)[1:]
    xo = flat.view(70, 130)[:, :128]  # rows on odd elements
    wo = (randn(g, 96 * 129 + 3) / 11).to(BF)[3:].view(96, 129)[:, :128]
    ref.check(gdn.linear(xo, wo), *ref.linear(xo, wo, None, "none", None, BF))
    ref.check(gdn.gated_linear(xo, wo), *ref.gated(xo, wo, "silu", BF))
    dy = randn(g, 70 * 49, dtype=BF).view(70, 49)[:, 1:]
    for a, e, t in zip(gdn.gated_linear_bwd(dy, xo, wo), *ref.gated_bwd(dy, xo, wo, "silu", BF)):
        ref.check(a, e, t)
    dy = randn(g, 70 * 97, dtype=BF).view(70, 97)[:, 1:]
    for a, e, t in zip(gdn.linear_bwd(dy, xo, wo), *ref.linear_bwd(dy, xo, wo, None, "none", BF)):
        if a is not None:
            ref.check(a, e, t)


@pytest.mark.parametrize("first", [0, 1])
def test_offsets_past_32_bits(gdn, first):
    """Rows of a buffer whose elements lie more than 2^32 apart, on and off 16-byte boundaries."""
    g = gen(31 + first)
    room = torch.empty(9 << 29, dtype=BF, device="cuda")
    ld = room.numel() // 300 // 8 * 8
    x = room[first:].as_strided((299, 72), (ld, 1), first)
    x.copy_(randn(g, 299, 72))
    assert 298 * ld > 1 << 32
    near, w = x.contiguous(), (randn(g, 144, 72) / 8).to(BF)
    assert torch.equal(gdn.linear(x, w, None, "silu"), gdn.linear(near, w, None, "silu"))
    assert torch.equal(gdn.gated_linear(x, w), gdn.gated_linear(near, w))
    dy = randn(g, 299, 144, dtype=BF)
    for a, b in zip(gdn.linear_bwd(dy, x, w, None, "silu"), gdn.linear_bwd(dy, near, w, None, "silu")):
        assert a is b is None or torch.equal(a, b)
    y, _ = gdn.rms_norm(x, None)
    want = near.double() * torch.rsqrt(near.double().square().mean(1, keepdim=True) + 1e-6)
    assert ((y.double() - want).abs() <= want.abs() * (2 ** -8 + 2 ** -18) + 2 ** -133).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_rows(gdn, dtype):
    x, w, b = torch.zeros(0, 64, device="cuda", dtype=dtype), torch.ones(32, 64, device="cuda", dtype=dtype), torch.ones(32, device="cuda")
    assert gdn.rms_norm(x, None, x)[0].shape == (0, 64)
    assert gdn.rms_norm_quant(x)[1].shape == (0,)
    dx, dw = gdn.rms_norm_bwd(x, x, torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()
    assert gdn.linear(x, w, b, "silu").shape == (0, 32)
    assert gdn.gated_linear(x, w).shape == (0, 16)
    dx, dw, db = gdn.linear_bwd(x[:, :32], x, w, b, "silu")
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    dx, dw = gdn.gated_linear_bwd(x[:, :16], x, w)
    assert dx.shape == (0, 64) and not dw.any()


def test_infinities_stay_in_their_rows(gdn):
    """What is beyond a partial tile never reaches the result, and a spoilt row spoils only itself."""
    g = gen(23)
    x, w = randn(g, 70, 72, dtype=BF), (randn(g, 136, 72) / 8).to(BF)
    x[3, 5], x[69, 71] = float("inf"), float("nan")
    y = gdn.linear(x, w)
    good = [i for i in range(70) if i not in (3, 69)]
    want, bound = ref.linear(x[good], w, None, "none", None, BF)
    ref.check(y[good], want, bound)
    assert not y[3].isfinite().any() and y[69].isnan().all()
    h = gdn.gated_linear(x, w)
    want, bound = ref.gated(x[good], w, "silu", BF)
    ref.check(h[good], want, bound)


@pytest.mark.parametrize("rows", [10, 70])
def test_fp32_infinities_and_largest_values(gdn, rows):
    """An infinity times a weight is an infinity of its sign, and values between bf16's and fp32's largest are finite."""
    g = gen(27)
    x, w = randn(g, rows, 200), randn(g, 136, 200) / 8
    w[:, 9] = 1e-6 * (1 + torch.rand(136, generator=g, device="cuda"))
    w[:, 5] = torch.where(w[:, 5].abs() < 1e-3, 0.5, w[:, 5])
    w[17, 5] = 0
    x[3, 5], x[5, 150], x[7, 9] = -float("inf"), float("nan"), 3.4e38
    y = gdn.linear(x, w)
    good = [i for i in range(rows) if i not in (3, 5)]
    want, bound = ref.linear(x[good], w, None, "none", None, torch.float32)
    ref.check(y[good], want, bound)
    assert y[5].isnan().all() and y[3, 17].isnan()
    rest = torch.arange(136, device="cuda") != 17
    assert torch.equal(y[3][rest], -float("inf") * w[rest, 5].sign())


def test_other_stream_and_graph(gdn):
    g = gen(29)
    M, K, F = 200, 256, 320
    x, w, dy = randn(g, M, K, dtype=BF), (randn(g, 2 * F, K) / 16).to(BF), randn(g, M, F, dtype=BF)
    down, nw = (randn(g, K, F) / 18).to(BF), 1 + 0.1 * randn(g, K)

    def step():
        n, h = gdn.rms_norm(x, nw, x)
        y = gdn.gated_linear(n, w)
        out = gdn.linear(y, down, None, None, h)
        dx, dw = gdn.gated_linear_bwd(dy, n, w)
        dn, dnw = gdn.rms_norm_bwd(dx, h, nw)
        return out, dx, dw, dn, dnw, *gdn.linear_bwd(out, y, down, None, "gelu")[:2]

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.copy_(randn(g, M, K, dtype=BF))
    graph.replay()
    for a, b in zip(held, step()):
        assert torch.equal(a, b)


def test_refusals(gdn):
    x, w = torch.zeros(4, 64, device="cuda", dtype=BF), torch.zeros(32, 64, device="cuda", dtype=BF)
    for err, f in [
        (TypeError, lambda: gdn.rms_norm(x.half())), (TypeError, lambda: gdn.rms_norm(x, None, x.float())),
        (ValueError, lambda: gdn.rms_norm(x, torch.ones(63, device="cuda"))), (ValueError, lambda: gdn.rms_norm(x, None, x[:2])),
        (TypeError, lambda: gdn.rms_norm(x, torch.ones(64, device="cuda").double())), (gdn.GdnError, lambda: gdn.rms_norm(x, eps=-1.0)),
        (TypeError, lambda: gdn.linear(x, w.float())), (TypeError, lambda: gdn.linear(x.half(), w.half())),
        (ValueError, lambda: gdn.linear(x, w[:, :32])), (ValueError, lambda: gdn.linear(x, w, activation="tanh")),
        (ValueError, lambda: gdn.linear(x, w, torch.zeros(31, device="cuda"))), (TypeError, lambda: gdn.linear(x, w, x[0, :32])),
        (TypeError, lambda: gdn.linear(x, w, residual=torch.zeros(4, 32, device="cuda"))),
        (ValueError, lambda: gdn.linear(x, w, x_scale=torch.ones(4, device="cuda"))),
        (TypeError, lambda: gdn.linear(x, w, x_scale=torch.ones(4, device="cuda"), weight_scale=torch.ones(32, device="cuda"))),
        (TypeError, lambda: gdn.linear(x.float(), w.float(), out_dtype=BF)), (ValueError, lambda: gdn.linear(x, w, out=x)),
        (ValueError, lambda: gdn.gated_linear(x, w[:31])), (ValueError, lambda: gdn.linear(x, w.cpu())),
        (TypeError, lambda: gdn.linear_bwd(x.to(E4), x.to(E4), w.to(E4))), (ValueError, lambda: gdn.linear_bwd(x, x, w)),
        (ValueError, lambda: gdn.gated_linear_bwd(x[:2, :16], x, w)),
    ]:
        with pytest.raises(err):
            f()
