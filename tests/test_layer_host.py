"""Argument checks of the decoder-block operators, on the CPU: what the C entry points refuse before
anything is enqueued, and what the binding refuses.  No pointer here is ever dereferenced."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import gated_deltanet_gb300 as g
    g.load_library()
    return g


INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -6
P = 4096  # an aligned address that nothing reads


I64, INT, VP = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p


class GdnNormArgs(ctypes.Structure):
    _fields_ = [("rows", I64), ("width", INT), ("dtype", INT), ("w_dtype", INT), ("out_dtype", INT),
                ("eps", ctypes.c_float), ("x", VP), ("ldx", I64), ("residual", VP), ("ld_residual", I64),
                ("weight", VP), ("y", VP), ("scale", VP), ("h", VP), ("dy", VP), ("ld_dy", I64), ("dh", VP),
                ("ld_dh", I64), ("dx", VP), ("dweight", VP)]


class GdnLinearArgs(ctypes.Structure):
    _fields_ = [("rows", I64), ("out_features", INT), ("in_features", INT), ("dtype", INT), ("out_dtype", INT),
                ("act", INT), ("x", VP), ("ldx", I64), ("w", VP), ("ldw", I64), ("x_scale", VP), ("w_scale", VP),
                ("bias", VP), ("residual", VP), ("ld_residual", I64), ("y", VP), ("ldy", I64), ("dy", VP),
                ("ld_dy", I64), ("dx", VP), ("dw", VP), ("dbias", VP)]


@pytest.fixture(scope="module")
def L(gdn):
    lib = ctypes.CDLL(gdn.build.lib_path())
    np_, lp = ctypes.POINTER(GdnNormArgs), ctypes.POINTER(GdnLinearArgs)
    for f in (lib.gdn_rms_norm, lib.gdn_quantize_rows):
        f.argtypes, f.restype = [np_, VP], INT
    for n, t in (("gdn_rms_norm_bwd", np_), ("gdn_linear", lp), ("gdn_linear_bwd", lp), ("gdn_gated_linear", lp),
                 ("gdn_gated_linear_bwd", lp)):
        f, w = getattr(lib, n), getattr(lib, n + "_workspace_size")
        f.argtypes, f.restype = [t, VP, ctypes.c_size_t, VP], INT
        w.argtypes, w.restype = [t], ctypes.c_size_t
    return lib


def norm_args(**kw):
    d = dict(rows=4, width=64, dtype=1, w_dtype=0, out_dtype=1, eps=1e-6, x=P, ldx=64, weight=P, y=P)
    d.update(kw)
    return GdnNormArgs(**d)


def linear_args(**kw):
    d = dict(rows=4, out_features=64, in_features=32, dtype=1, out_dtype=1, act=0, x=P, ldx=32, w=P, ldw=32, y=P, ldy=64)
    d.update(kw)
    return GdnLinearArgs(**d)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(width=0), dict(dtype=2), dict(dtype=9), dict(w_dtype=2), dict(out_dtype=0),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(x=P + 1), dict(y=None),
                                dict(ldx=63), dict(out_dtype=2), dict(residual=P, ld_residual=8), dict(h=P + 1)])
def test_norm_refuses(L, kw):
    assert L.gdn_rms_norm(ctypes.byref(norm_args(**kw)), None) == INVALID


def test_norm_null_struct(L):
    assert L.gdn_rms_norm(None, None) == INVALID
    assert L.gdn_quantize_rows(None, None) == INVALID
    assert L.gdn_rms_norm_bwd(None, None, 0, None) == INVALID
    assert L.gdn_rms_norm_bwd_workspace_size(None) == 0
    for n in ("gdn_linear", "gdn_linear_bwd", "gdn_gated_linear", "gdn_gated_linear_bwd"):
        assert getattr(L, n)(None, None, 0, None) == INVALID
        assert getattr(L, n + "_workspace_size")(None) == 0


def test_quantize_needs_the_8_bit_type(L):
    assert L.gdn_quantize_rows(ctypes.byref(norm_args(scale=P)), None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None, dx=P), INVALID), (dict(dy=P, ld_dy=64, dx=None), INVALID), (dict(dy=P, ld_dy=3, dx=P), INVALID),
    (dict(dy=P, ld_dy=64, dx=P, dh=P, ld_dh=5), INVALID), (dict(dy=P, ld_dy=64, dx=P, dweight=P + 2), INVALID),
])
def test_norm_bwd_refuses(L, kw, code):
    assert L.gdn_rms_norm_bwd(ctypes.byref(norm_args(**kw)), P, 1 << 30, None) == code


def test_norm_bwd_small_workspace(L):
    a = norm_args(dy=P, ld_dy=64, dx=P, dweight=P)
    need = L.gdn_rms_norm_bwd_workspace_size(ctypes.byref(a))
    assert need >= 64 * 4
    assert L.gdn_rms_norm_bwd(ctypes.byref(a), P, need - 1, None) == WORKSPACE
    assert L.gdn_rms_norm_bwd(ctypes.byref(a), P + 128, need, None) == INVALID


@pytest.mark.parametrize("call", ["gdn_linear", "gdn_gated_linear"])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(out_features=0), INVALID), (dict(in_features=0), INVALID), (dict(dtype=3), INVALID),
    (dict(out_dtype=2), INVALID), (dict(dtype=0, out_dtype=1), UNSUPPORTED), (dict(act=6), INVALID), (dict(act=-1), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(ldx=31), INVALID), (dict(ldw=31), INVALID),
    (dict(ldy=63), INVALID), (dict(x=P + 1), INVALID), (dict(y=P + 1), INVALID), (dict(x_scale=P), INVALID),
    (dict(x_scale=P, w_scale=P), INVALID), (dict(dtype=2, w_scale=P), INVALID), (dict(dtype=2, x_scale=P + 2, w_scale=P), INVALID),
])
def test_linear_refuses(L, call, kw, code):
    assert getattr(L, call)(ctypes.byref(linear_args(**kw)), None, 0, None) == code


def test_gated_takes_no_bias_residual_or_other_output(L):
    for kw in (dict(bias=P), dict(residual=P, ld_residual=64), dict(dbias=P)):
        assert L.gdn_gated_linear(ctypes.byref(linear_args(**kw)), None, 0, None) == INVALID
    assert L.gdn_gated_linear(ctypes.byref(linear_args(out_dtype=0)), None, 0, None) == UNSUPPORTED


@pytest.mark.parametrize("call", ["gdn_linear_bwd", "gdn_gated_linear_bwd"])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUPPORTED), (dict(out_dtype=0), UNSUPPORTED), (dict(dy=None), INVALID), (dict(ld_dy=63), INVALID),
    (dict(dx=P + 1), INVALID), (dict(dw=P + 1), INVALID), (dict(dbias=P + 1), INVALID),
])
def test_linear_bwd_refuses(L, call, kw, code):
    d = dict(dy=P, ld_dy=64, dx=P, dw=P, y=None)
    d.update(kw)
    assert getattr(L, call)(ctypes.byref(linear_args(**d)), P, 1 << 30, None) == code


def test_bwd_small_workspace(L):
    for call in ("gdn_linear_bwd", "gdn_gated_linear_bwd"):
        a = linear_args(act=1, dy=P, ld_dy=64, dx=P, dw=P, y=None)
        need = getattr(L, call + "_workspace_size")(ctypes.byref(a))
        assert need >= 4 * 64 * 2
        assert getattr(L, call)(ctypes.byref(a), P, need - 1, None) == WORKSPACE
        assert getattr(L, call)(ctypes.byref(a), P + 8, need, None) == INVALID


def test_binding_refuses_host_tensors(gdn):
    x, w = torch.zeros(4, 8), torch.zeros(16, 8)
    for f in (lambda: gdn.rms_norm(x), lambda: gdn.rms_norm_quant(x), lambda: gdn.quantize_rows(x), lambda: gdn.rms_norm_bwd(x, x),
              lambda: gdn.linear(x, w), lambda: gdn.linear_bwd(x, x, w), lambda: gdn.gated_linear(x, w),
              lambda: gdn.gated_linear_bwd(x, x, w)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


def test_row_views(gdn):
    """Which layouts are taken as they are, and which are copied."""
    view = gdn.layer._load().row_view
    t = torch.arange(2 * 3 * 12, dtype=torch.float32).reshape(2, 3, 12)
    v, n, ld = view(t, 12)
    assert (n, ld) == (6, 12) and v.data_ptr() == t.data_ptr()
    s = t[..., 4:8]  # a slice of a fused projection: rows 12 apart
    v, n, ld = view(s, 4)
    assert (n, ld) == (6, 12) and v.data_ptr() == s.data_ptr()
    for v in (t[:, ::2, :], t.transpose(0, 1), t[..., ::2], t[0, 0].expand(5, 12), t[:1, :, :4], t[:, :1], t[:1, :1, 2:]):
        c, n, ld = view(v, v.shape[-1])
        assert n == v.numel() // v.shape[-1]
        assert torch.equal(torch.as_strided(c, (n, v.shape[-1]), (ld, 1), c.storage_offset()), v.reshape(n, -1))
    assert view(torch.zeros(0, 12), 12)[1] == 0
    assert view(torch.zeros(12), 12)[1:] == (1, 12)
    with pytest.raises(ValueError, match="columns"):
        view(t, 11)
    with pytest.raises(ValueError, match="columns"):
        view(torch.tensor(1.0), 1)


def test_binding_refuses_what_is_no_tensor(gdn):
    with pytest.raises(TypeError, match="tensor"):
        gdn.rms_norm([1.0, 2.0])
    with pytest.raises(TypeError, match="tensor"):
        gdn.linear(torch.zeros(2, 8), "w")
    with pytest.raises(ValueError, match="activation"):
        gdn.linear(torch.zeros(2, 8), torch.zeros(2, 8), activation="tanh")
    with pytest.raises(TypeError, match="out_dtype"):
        gdn.linear(torch.zeros(2, 8), torch.zeros(2, 8), out_dtype=torch.float16)
