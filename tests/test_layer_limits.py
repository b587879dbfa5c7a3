"""Sizes, overlaps and builds that the decoder-block operators refuse, on the CPU.  No pointer here is ever dereferenced."""
import ctypes

import pytest
import torch

import layer_c
from test_layer_host import INVALID, UNSUPPORTED, P, linear_args


@pytest.fixture(scope="module")
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import gated_deltanet_gb300 as g
    g.load_library()
    return g


@pytest.fixture(scope="module")
def L(gdn):
    return layer_c.library()


MOST = (1 << 31) - 256


@pytest.mark.parametrize("call", ["gdn_linear", "gdn_gated_linear", "gdn_linear_bwd", "gdn_gated_linear_bwd"])
def test_rows_past_32_bits_are_refused(L, call):
    """A tile's row coordinate has 31 bits."""
    d = dict(act=1, dy=P, ld_dy=64, dx=P, dw=P, y=None) if call.endswith("bwd") else {}
    size = getattr(L, call + "_workspace_size")
    for rows in (MOST + 1, 1 << 31, 1 << 40):
        a = linear_args(rows=rows, **d)
        assert size(ctypes.byref(a)) == 0
        assert getattr(L, call)(ctypes.byref(a), P, 1 << 60, None) == UNSUPPORTED
    if d:
        assert size(ctypes.byref(linear_args(rows=MOST, **d))) >= MOST * 64 * 2


@pytest.mark.parametrize("call", ["gdn_linear", "gdn_gated_linear"])
@pytest.mark.parametrize("kw", [
    dict(x=P, y=P), dict(x=P, y=P + 64 * 3 + 62), dict(x=P, y=1 << 20, w=(1 << 20) + 32), dict(y=1 << 20, w=(1 << 20) + 4 * 128 - 16),
    # slices of rows of one buffer that share a column
    dict(x=P, ldx=200, y=P + 62, ldy=200), dict(x=P + 126, ldx=200, y=P, ldy=200), dict(x=P + 400 * 3, ldx=200, y=P, ldy=200),
])
def test_outputs_over_operands_are_refused(L, call, kw):
    d = dict(x=1 << 24, w=1 << 25, **{k: v for k, v in kw.items() if k not in ("x", "w")})
    d.update(kw)
    assert getattr(L, call)(ctypes.byref(linear_args(**d)), P, 1 << 30, None) == INVALID


@pytest.mark.parametrize("kw", [dict(residual=P + 16, ld_residual=64), dict(residual=P, ld_residual=72), dict(residual=P + 128, ld_residual=64),
                                dict(bias=P), dict(bias=P + 4 * 128 - 4)])
def test_outputs_over_other_inputs_are_refused(L, kw):
    """y may be the residual, row for row, and lie over no other input."""
    a = linear_args(x=1 << 24, w=1 << 25, y=P, **kw)
    assert L.gdn_linear(ctypes.byref(a), P, 1 << 30, None) == INVALID


def test_binding_built_for_another_pytorch_is_not_loaded(gdn, monkeypatch):
    """The compiled binding holds for the PyTorch and Python whose headers it was compiled with: with others it counts as not built,
    and is refused where nobody built it again."""
    assert not gdn.build.needs_build()
    gdn.layer._load()
    monkeypatch.setattr(gdn.build, "running", lambda: "torch 0.0, python 3.0")
    assert gdn.build.needs_build()
    monkeypatch.setattr(gdn.layer, "_module", None)
    with pytest.raises(ImportError, match="built for torch .* torch 0.0"):
        gdn.layer._load()


def test_library_builds_without_pytorch(gdn, monkeypatch, tmp_path):
    """Users of the C library alone: without PyTorch no binding is wanted, and one that fails to compile does not cost the library."""
    monkeypatch.setattr(gdn.build, "running", lambda: None)
    monkeypatch.setattr(gdn.build, "BINDING", str(tmp_path / "_layer.so"))
    assert not gdn.build.needs_build()
    monkeypatch.undo()
    monkeypatch.setattr(gdn.build, "BINDING", str(tmp_path / "_layer.so"))
    monkeypatch.setenv("CXX", "false")
    before = gdn.build.os.path.getmtime(gdn.build.LIB)
    assert gdn.build.needs_build()
    with pytest.raises(RuntimeError, match="false"):
        gdn.build.build()
    assert gdn.build.os.path.getmtime(gdn.build.LIB) == before


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_quant"])
def test_a_place_for_the_stream_goes_with_a_residual(gdn, name):
    """Without a residual there is no sum to write: the buffer would be left as it was."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="residual_out"):
        getattr(gdn, name)(x, residual_out=torch.zeros(4, 8))
