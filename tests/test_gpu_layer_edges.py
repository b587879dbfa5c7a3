"""The decoder-block operators on the GPU at their edges: outputs in the place of inputs, eps of zero, arguments far out,
workspaces under capture, waits that run out.  Bounds as in ``layer_reference``."""
import pytest
import torch

import layer_c
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


@pytest.fixture(scope="module")
def lib(gdn):
    return layer_c.library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def here():
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("D", [101, 1001, 2048, 8193, 16384])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("place", ["dy", "dh"])
def test_norm_bwd_in_place(gdn, lib, D, dtype, place):
    """dx in the place of dy or of dh: the gradients of a call with a dx of its own, bit for bit."""
    g = gen(D)
    M = 37
    h, dy, dh = (randn(g, M, D, dtype=dtype) for _ in range(3))
    w = 1 + 0.3 * randn(g, D)
    want = gdn.rms_norm_bwd(dy, h, w, dh, 1e-5)
    given = {"dy": dy.clone(), "dh": dh.clone()}
    dw = torch.empty(D, device="cuda")
    a = layer_c.norm_bwd_args(given["dy"], h, w, given["dh"], given[place], dw, 1e-5)
    need = lib.gdn_rms_norm_bwd_workspace_size(a)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert lib.gdn_rms_norm_bwd(a, ws.data_ptr(), need, here()) == 0
    assert torch.equal(given[place], want[0]) and torch.equal(dw, want[1])
    ex, ew = ref.norm_bwd(dy, h, w, dh, 1e-5)
    bx, bw = ref.norm_bwd_bound(dy, h, w, dh, 1e-5, ex, dtype)
    ref.check(given[place], ex, bx, "dx")
    ref.check(dw, ew, bw, "dw")


@pytest.mark.parametrize("D", [101, 2048, 9000])
def test_norm_stream_in_the_place_of_x(gdn, lib, D):
    """h in the place of x (x + residual replaces x)."""
    g = gen(D)
    x, r, y = randn(g, 37, D, dtype=BF), randn(g, 37, D, dtype=BF), torch.empty(37, D, dtype=BF, device="cuda")
    want = gdn.rms_norm(x, None, r, 1e-5)
    a = layer_c.GdnNormArgs(**layer_c.pointers(rows=37, width=D, dtype=1, w_dtype=0, out_dtype=1, eps=1e-5, x=x, ldx=D, residual=r,
                                               ld_residual=D, y=y, h=x))
    assert lib.gdn_rms_norm(a, here()) == 0
    assert torch.equal(y, want[0]) and torch.equal(x, want[1])


@pytest.mark.parametrize("M,D", [(1, 5), (3, 101), (3, 104), (9, 33), (5, 512), (130, 257), (2, 513), (3, 9000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_bwd_without_eps(gdn, M, D, dtype):
    """eps = 0 with rows that are not zero is an ordinary call, also where the rows do not fill a block."""
    g = gen(M + D)
    h, dy, w = randn(g, M, D, dtype=dtype), randn(g, M, D, dtype=dtype), 1 + 0.3 * randn(g, D)
    dx, dw = gdn.rms_norm_bwd(dy, h, w, None, 0.0)
    ex, ew = ref.norm_bwd(dy, h, w, None, 0.0)
    bx, bw = ref.norm_bwd_bound(dy, h, w, None, 0.0, ex, dtype)
    ref.check(dx, ex, bx, "dx")
    ref.check(dw, ew, bw, "dw")


# ---------------------------------------------------------------- the library-managed workspace
def product_args(x, w, **kw):
    code = layer_c.code(x)
    return layer_c.GdnLinearArgs(**layer_c.pointers(rows=x.shape[0], out_features=w.shape[0], in_features=x.shape[1], dtype=code, out_dtype=code,
                                                    x=x, ldx=x.shape[1], w=w, ldw=w.shape[1], **kw))


def gradient_call(lib, g, M, N, K):
    """A gelu layer's gradients by the C entry without a workspace, what they write, and the same by the Python call."""
    x, w, dy = randn(g, M, K, dtype=BF), (randn(g, N, K) / K ** 0.5).to(BF), randn(g, M, N, dtype=BF)
    out = torch.zeros_like(x), torch.zeros_like(w)
    a = product_args(x, w, act=2, dy=dy, ld_dy=N, dx=out[0], dw=out[1])
    assert lib.gdn_linear_bwd_workspace_size(a) > 0
    return (lambda: lib.gdn_linear_bwd(a, None, 0, here())), out, (dy, x, w, None, "gelu"), a


def test_no_workspace_given(gdn, lib):
    """workspace NULL: every entry that needs one, on a stream that had none."""
    g = gen(41)
    x, w, dy = randn(g, 70, 129, dtype=BF), (randn(g, 64, 129) / 11).to(BF), randn(g, 70, 64, dtype=BF)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        y, h = torch.empty(70, 64, dtype=BF, device="cuda"), torch.empty(70, 32, dtype=BF, device="cuda")
        assert lib.gdn_linear(product_args(x, w, y=y, ldy=64), None, 0, here()) == 0
        a = product_args(x, w, act=1, y=h, ldy=32)
        a.out_features = 32
        assert lib.gdn_gated_linear(a, None, 0, here()) == 0
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        assert lib.gdn_linear_bwd(product_args(x, w, act=1, dy=dy, ld_dy=64, dx=dx, dw=dw), None, 0, here()) == 0
        gx, gw = torch.empty_like(x), torch.empty_like(w)
        a = product_args(x, w, act=1, dy=dy, ld_dy=64, dx=gx, dw=gw)
        a.out_features = 32
        assert lib.gdn_gated_linear_bwd(a, None, 0, here()) == 0
        nx, nw = torch.empty_like(dy), torch.empty(64, device="cuda")
        assert lib.gdn_rms_norm_bwd(layer_c.norm_bwd_args(dy, y, torch.ones(64, device="cuda"), None, nx, nw, 1e-5), None, 0, here()) == 0
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(y, gdn.linear(x, w)) and torch.equal(h, gdn.gated_linear(x, w))
    for got, want in (((dx, dw), gdn.linear_bwd(dy, x, w, None, "silu")), ((gx, gw), gdn.gated_linear_bwd(dy[:, :32], x, w)),
                      ((nx, nw), gdn.rms_norm_bwd(dy, y, torch.ones(64, device="cuda"), None, 1e-5))):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_graphs_keep_the_library_managed_workspace(gdn, lib):
    """A captured call's buffer outlives the workspace's growth; growth under capture is refused and enqueues nothing."""
    g = gen(43)
    small, out, args, _ = gradient_call(lib, g, 200, 64, 72)
    large, out2, args2, a2 = gradient_call(lib, g, 3000, 640, 72)
    assert lib.gdn_linear_bwd_workspace_size(a2) > 2 << 20
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        assert small() == 0
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            assert small() == 0
            assert large() == -5
        assert large() == 0  # the workspace grows
        for t in out:
            t.zero_()
        graph.replay()
        graph.replay()
    stream.synchronize()
    for have, a in ((out, args), (out2, args2)):
        want = gdn.linear_bwd(*a)
        assert torch.equal(have[0], want[0]) and torch.equal(have[1], want[1])


def test_token_mixer_in_graphs(gdn):
    """The delta rule and its gradients captured on a stream that had no workspace: replays give what eager calls give, before and after
    larger calls on that stream and a second graph's capture there."""
    g = gen(47)

    def inputs(T):
        q, k, v = (randn(g, 1, T, 2, 128, dtype=BF) for _ in range(3))
        k = torch.nn.functional.normalize(k.float(), dim=-1).to(BF)
        gate, beta = -torch.rand(1, T, 2, generator=g, device="cuda") / 10, torch.rand(1, T, 2, generator=g, device="cuda")
        return q, k, v, gate, beta

    def step(x, do):
        o, ht = gdn.chunk_gated_delta_rule(*x, output_final_state=True)
        return o, ht, gdn.chunk_gated_delta_rule_bwd(*x, do)

    x, big = inputs(200), inputs(1500)
    do, do2 = torch.ones_like(x[2]), torch.ones_like(big[2])
    want, want2 = step(x, do), step(big, do2)
    stream, graph, second = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        got = step(x, do)
    with torch.cuda.stream(stream):
        graph.replay()
        got2 = step(big, do2)
        graph.replay()
    stream.synchronize()
    with torch.cuda.graph(second, stream=stream):
        again = step(x, do)
    with torch.cuda.stream(stream):
        second.replay()
        graph.replay()
        assert gdn.read_device_status() == 0
    stream.synchronize()

    def near(a, b):
        # (the gradients' sums over tiles are atomic: their order may change)
        for s, t in zip([*a[:2], *a[2]], [*b[:2], *b[2]]):
            assert (s is None and t is None) or ((s.float() - t.float()).norm() <= 1e-5 * t.float().norm()).item()
    near(got, want)
    near(again, want)
    near(got2, want2)


# ---------------------------------------------------------------- waits that run out
@pytest.fixture
def withheld(lib):
    """Calls whose kernels load nothing: their waits run out after 5 ms."""
    def call(f):
        lib.gdn_layer_test_withhold(1)
        try:
            f()
        finally:
            lib.gdn_layer_test_withhold(0)
        torch.cuda.synchronize()
    return call


# rows, outputs, contraction: few rows with a contraction in one piece and split; many rows in one tile with its contraction split,
# in one tile without, in several tiles
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (16, 200, 2048), (200, 130, 2048), (200, 64, 72), (2000, 640, 200)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_waits_that_run_out(gdn, withheld, M, N, K, dtype):
    """A timeout is reported once, and the next call on the stream is right."""
    if dtype == F32 and M <= 64:
        pytest.skip("nothing waits there")
    g = gen(M)
    x, w = randn(g, M, K, dtype=dtype), randn(g, N, K, dtype=dtype)
    want = gdn.linear(x, w)
    assert gdn.read_layer_status() == 0
    withheld(lambda: gdn.linear(x, w))
    assert gdn.read_layer_status() == -4 and gdn.read_layer_status() == 0
    assert torch.equal(gdn.linear(x, w), want)


def test_one_read_clears_every_kernel_s_status(gdn, withheld):
    """Timeouts in products of many and of few rows: one read reports and clears both."""
    w = randn(gen(4), 64, 72, dtype=BF)
    for order in ((5, 300), (300, 5)):
        for M in order:
            withheld(lambda: gdn.linear(randn(gen(M), M, 72, dtype=BF), w))
        assert gdn.read_layer_status() == -4 and gdn.read_layer_status() == 0


# ---------------------------------------------------------------- activations far out
def one_column(z):
    """x and weight whose product is z itself (one term, a factor of one)."""
    return z[:, None].contiguous(), torch.ones(1, 1, dtype=z.dtype, device="cuda")


@pytest.mark.parametrize("rows", [60, 120, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sigmoid_slope_keeps_its_digits(gdn, rows, dtype):
    """The slope of the logistic function falls like exp(-|z|) on both sides and is relative in its error on both.  fp32:
    the exponential (2 units of 2^-23), 1 + e, the reciprocal, two products: below 2^-20.  bf16: the exponent's rounding, |z| 2^-23, and the
    approximate exponential and reciprocal beside the rounding of dz."""
    z = torch.linspace(-70, 70, rows, device="cuda").to(dtype)
    x, w = one_column(z)
    dx = gdn.linear_bwd(torch.ones_like(x), x, w, None, "sigmoid")[0][:, 0]
    want = torch.special.expit(z.double()) * torch.special.expit(-z.double())
    rel = 2.0 ** -20 if dtype == F32 else ref.HALF[BF] + 2.0 ** -19 + z.double().abs() * 2.0 ** -22
    ref.check(dx, want, rel * want)
    both = gdn.gated_linear_bwd(torch.ones_like(x), x, torch.ones(2, 1, dtype=dtype, device="cuda"), "sigmoid")[0][:, 0]
    p = torch.special.expit(z.double())
    # z sigmoid'(z) + sigmoid(z): each of the two terms rounded by itself
    parts = (z.double() * want).abs() + p
    ref.check(both, z.double() * want + p, (2 * rel + ref.HALF[dtype]) * parts)


@pytest.mark.parametrize("rows", [8, 72, 264])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
def test_slopes_far_out(gdn, rows, dtype, name):
    """Arguments whose squares pass fp32's range: the slopes have their limits, 1 or 0."""
    z = torch.tensor([1e18, 3e19, 1e25, 3e38, -1e18, -3e19, -1e25, -3e38], device="cuda").repeat(rows // 8).to(dtype)
    x, w = one_column(z)
    dx = gdn.linear_bwd(torch.ones_like(x), x, w, None, name)[0][:, 0]
    assert torch.equal(dx, torch.zeros_like(z) if name == "sigmoid" else (z > 0).to(dtype))


@pytest.mark.parametrize("D", [64, 129, 9000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantised_infinities(gdn, D, dtype):
    """A row that holds an infinity or a NaN has a NaN for its scale, with the norm and without."""
    x = randn(gen(D), 5, D, dtype=dtype)
    x[1, 3], x[2, D - 1], x[3, 0] = float("inf"), -float("inf"), float("nan")
    for q, s in (gdn.quantize_rows(x), gdn.rms_norm_quant(x, None)[:2]):
        assert s[1:4].isnan().all() and s[[0, 4]].isfinite().all()
        assert q[[0, 4]].float().isfinite().all()


def test_bias_gradient_of_many_columns(gdn):
    """More columns than a grid has rows of blocks of 128."""
    N = (1 << 23) + 5
    g = gen(1)
    x, w, b, dy = randn(g, 40, 1, dtype=BF), randn(g, N, 1, dtype=BF), randn(g, N), randn(g, 40, N, dtype=BF)
    db = gdn.linear_bwd(dy, x, w, b, None, need_dx=False, need_dweight=False)[2]
    ref.check(db, dy.double().sum(0), 40 * ref.SUM * dy.double().abs().sum(0))


# ---------------------------------------------------------------- outputs and operands
@pytest.mark.parametrize("M", [5, 300])
def test_outputs_over_operands_are_refused(gdn, M):
    """A product reads its operands while it writes: y in their place is refused, in the residual's place it is not."""
    x, w = randn(gen(M), M, 64, dtype=BF), randn(gen(2), 64, 64, dtype=BF)
    before = x.clone()
    for f in (lambda: gdn.linear(x, w, out=x), lambda: gdn.gated_linear(x, w.repeat(2, 1), out=x),
              lambda: gdn.linear(x[:, :64], w, None, None, x, out=x), lambda: gdn.linear(w, w, out=w)):
        with pytest.raises(gdn.GdnError):
            f()
    shifted = torch.empty(M * 64 + 8, dtype=BF, device="cuda")
    with pytest.raises(gdn.GdnError):
        gdn.linear(x, w, residual=shifted[8:].view(M, 64), out=shifted[:-8].view(M, 64))
    assert torch.equal(x, before)
    stream = before.clone()
    assert torch.equal(gdn.linear(x, w, residual=stream, out=stream), gdn.linear(x, w, residual=before))


@pytest.mark.parametrize("M", [1, 5, 300])
def test_slices_of_one_buffer(gdn, lib, M):
    """x, the residual and y as columns side by side in the rows of one buffer share no element: an ordinary call."""
    g = gen(M)
    rows, w = randn(g, M, 192, dtype=BF), randn(g, 64, 64, dtype=BF)
    want = gdn.linear(rows[:, :64], w, residual=rows[:, 64:128])
    a = layer_c.GdnLinearArgs(**layer_c.pointers(rows=M, out_features=64, in_features=64, dtype=1, out_dtype=1, x=rows, ldx=192, w=w, ldw=64,
                                                 residual=rows[:, 64:], ld_residual=192, y=rows[:, 128:], ldy=192))
    assert lib.gdn_linear(a, None, 0, here()) == 0
    assert torch.equal(rows[:, 128:], want)


@pytest.mark.parametrize("rows", [60, 300])
@pytest.mark.parametrize("name", ["silu", "sigmoid"])
def test_far_tails_in_bf16(gdn, rows, name):
    """bf16 outputs of arguments from 16 to 90: the exponent's rounding makes exp(-z) off by |z| 2^-23 of itself, beside the approximate exponential and
    reciprocal (2^-21) and the output's rounding; a logistic function below the smallest normal fp32 number may be zero."""
    z = torch.linspace(16, 90, rows // 2, device="cuda")
    z = torch.cat([z, -z]).to(BF)
    x, w = one_column(z)
    y = gdn.linear(x, w, None, name)[:, 0]
    zd = z.double()
    want = ref.act(zd, name)
    lost = 2.0 ** -126 * (zd.abs() if name == "silu" else 1)
    ref.check(y, want, want.abs() * (ref.HALF[BF] + 2.0 ** -20 + zd.abs() * 2.0 ** -23 * 1.01) + lost)


# ---------------------------------------------------------------- fp32 products
def norm_off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("M,N,K", [(5, 72, 48), (64, 129, 2048), (70, 136, 48), (129, 72, 1600), (257, 330, 3200), (520, 129, 6416), (300, 520, 2048)])
def test_fp32_products_to_the_last_bits(gdn, M, N, K):
    """The relative 2-norm of the error, which sees every plane of an operand and every product of planes (two planes instead of
    three: 3.5e-6).  On the tensor cores: sums of 128 in 8 truncated steps, at most 4.3 units of 2^-24 off in the mean; their sum in fp32, sqrt(K / 128)
    / 2.4 units; the output's rounding; below 4e-7 together.  On the CUDA cores (64 rows and fewer): a sum of K terms of random signs in order, sqrt(K)
    / 2.4 units, and the rounding."""
    g = gen(M + K)
    tol = 4e-7 if M > 64 else 2.0 ** -24 * (1 + K ** 0.5 / 2.4)
    x, w, dy = randn(g, M, K), randn(g, N, K) / K ** 0.5, randn(g, M, N)
    assert norm_off(gdn.linear(x, w), x.double() @ w.double().t()) < tol
    dx, dw, _ = gdn.linear_bwd(dy, x, w)
    assert norm_off(dx, dy.double() @ w.double()) < (4e-7 if M > 64 else 2.0 ** -24 * (1 + N ** 0.5 / 2.4))
    assert norm_off(dw, dy.double().t() @ x.double()) < 4e-7
    w = randn(g, 2 * N, K) / K ** 0.5
    gate, up = (x.double() @ w.double().t()).split(N, 1)
    # a product of two such sums
    assert norm_off(gdn.gated_linear(x, w, None), gate * up) < 2.5 * tol
