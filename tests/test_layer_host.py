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


def norm_args(**kw):
    from gated_deltanet_gb300.layer import GdnNormArgs
    d = dict(rows=4, width=64, dtype=1, w_dtype=0, out_dtype=1, eps=1e-6, x=P, ldx=64, weight=P, y=P)
    d.update(kw)
    return GdnNormArgs(**d)


def linear_args(**kw):
    from gated_deltanet_gb300.layer import GdnLinearArgs
    d = dict(rows=4, out_features=64, in_features=32, dtype=1, out_dtype=1, act=0, x=P, ldx=32, w=P, ldw=32, y=P, ldy=64)
    d.update(kw)
    return GdnLinearArgs(**d)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(width=0), dict(dtype=2), dict(dtype=9), dict(w_dtype=2), dict(out_dtype=0),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(x=P + 1), dict(y=None),
                                dict(ldx=63), dict(out_dtype=2), dict(residual=P, ld_residual=8), dict(h=P + 1)])
def test_norm_refuses(gdn, kw):
    from gated_deltanet_gb300.layer import _library
    assert _library().gdn_rms_norm(ctypes.byref(norm_args(**kw)), None) == INVALID


def test_norm_null_struct(gdn):
    from gated_deltanet_gb300.layer import _library
    L = _library()
    assert L.gdn_rms_norm(None, None) == INVALID
    assert L.gdn_quantize_rows(None, None) == INVALID
    assert L.gdn_rms_norm_bwd(None, None, 0, None) == INVALID
    assert L.gdn_rms_norm_bwd_workspace_size(None) == 0
    for n in ("gdn_linear", "gdn_linear_bwd", "gdn_gated_linear", "gdn_gated_linear_bwd"):
        assert getattr(L, n)(None, None, 0, None) == INVALID
        assert getattr(L, n + "_workspace_size")(None) == 0


def test_quantize_needs_the_8_bit_type(gdn):
    from gated_deltanet_gb300.layer import _library
    assert _library().gdn_quantize_rows(ctypes.byref(norm_args(scale=P)), None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None, dx=P), INVALID), (dict(dy=P, ld_dy=64, dx=None), INVALID), (dict(dy=P, ld_dy=3, dx=P), INVALID),
    (dict(dy=P, ld_dy=64, dx=P, dh=P, ld_dh=5), INVALID), (dict(dy=P, ld_dy=64, dx=P, dweight=P + 2), INVALID),
])
def test_norm_bwd_refuses(gdn, kw, code):
    from gated_deltanet_gb300.layer import _library
    assert _library().gdn_rms_norm_bwd(ctypes.byref(norm_args(**kw)), P, 1 << 30, None) == code


def test_norm_bwd_small_workspace(gdn):
    from gated_deltanet_gb300.layer import _library
    a = norm_args(dy=P, ld_dy=64, dx=P, dweight=P)
    need = _library().gdn_rms_norm_bwd_workspace_size(ctypes.byref(a))
    assert need >= 64 * 4
    assert _library().gdn_rms_norm_bwd(ctypes.byref(a), P, need - 1, None) == WORKSPACE
    assert _library().gdn_rms_norm_bwd(ctypes.byref(a), P + 128, need, None) == INVALID


@pytest.mark.parametrize("call", ["gdn_linear", "gdn_gated_linear"])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(out_features=0), INVALID), (dict(in_features=0), INVALID), (dict(dtype=3), INVALID),
    (dict(out_dtype=2), INVALID), (dict(dtype=0, out_dtype=1), UNSUPPORTED), (dict(act=6), INVALID), (dict(act=-1), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(ldx=31), INVALID), (dict(ldw=31), INVALID),
    (dict(ldy=63), INVALID), (dict(x=P + 1), INVALID), (dict(y=P + 1), INVALID), (dict(x_scale=P), INVALID),
    (dict(x_scale=P, w_scale=P), INVALID), (dict(dtype=2, w_scale=P), INVALID), (dict(dtype=2, x_scale=P + 2, w_scale=P), INVALID),
])
def test_linear_refuses(gdn, call, kw, code):
    from gated_deltanet_gb300.layer import _library
    assert getattr(_library(), call)(ctypes.byref(linear_args(**kw)), None, 0, None) == code


def test_gated_takes_no_bias_residual_or_other_output(gdn):
    from gated_deltanet_gb300.layer import _library
    L = _library()
    for kw in (dict(bias=P), dict(residual=P, ld_residual=64), dict(dbias=P)):
        assert L.gdn_gated_linear(ctypes.byref(linear_args(**kw)), None, 0, None) == INVALID
    assert L.gdn_gated_linear(ctypes.byref(linear_args(out_dtype=0)), None, 0, None) == UNSUPPORTED


@pytest.mark.parametrize("call", ["gdn_linear_bwd", "gdn_gated_linear_bwd"])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUPPORTED), (dict(out_dtype=0), UNSUPPORTED), (dict(dy=None), INVALID), (dict(ld_dy=63), INVALID),
    (dict(dx=P + 1), INVALID), (dict(dw=P + 1), INVALID), (dict(dbias=P + 1), INVALID),
])
def test_linear_bwd_refuses(gdn, call, kw, code):
    from gated_deltanet_gb300.layer import _library
    d = dict(dy=P, ld_dy=64, dx=P, dw=P, y=None)
    d.update(kw)
    assert getattr(_library(), call)(ctypes.byref(linear_args(**d)), P, 1 << 30, None) == code


def test_bwd_small_workspace(gdn):
    from gated_deltanet_gb300.layer import _library
    L = _library()
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


def test_row_views():
    """Which layouts are taken as they are, and which are copied."""
    from gated_deltanet_gb300.layer import _rows
    t = torch.arange(2 * 3 * 12, dtype=torch.float32).reshape(2, 3, 12)
    assert _rows("t", t, 12)[1:] == (6, 12) and _rows("t", t, 12)[0] is t
    s = t[..., 4:8]  # a slice of a fused projection: rows 12 apart
    assert _rows("s", s, 4)[1:] == (6, 12) and _rows("s", s, 4)[0] is s
    for v in (t[:, ::2, :], t.transpose(0, 1), t[..., ::2], t[0, 0].expand(5, 12)):
        c, n, ld = _rows("v", v, v.shape[-1])
        assert n == v.numel() // v.shape[-1]
        assert torch.equal(torch.as_strided(c, (n, v.shape[-1]), (ld, 1), c.storage_offset()), v.reshape(n, -1))
    assert _rows("e", torch.zeros(0, 12), 12)[1] == 0
    assert _rows("one", torch.zeros(12), 12)[1:] == (1, 12)
    with pytest.raises(ValueError, match="columns"):
        _rows("t", t, 11)
    with pytest.raises(ValueError, match="rows"):
        _rows("t", t, 12, 5)
