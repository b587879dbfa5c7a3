"""Sizes, overlaps and builds that the decoder-block operators refuse, on the CPU.  No pointer here is ever dereferenced."""
import ctypes

import pytest

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
