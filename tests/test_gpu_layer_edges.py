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
