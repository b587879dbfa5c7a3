"""The C entries of the decoder-block operators through ctypes, for what the Python binding never passes: outputs in the
place of inputs, no workspace of the caller's."""
import ctypes

from test_layer_host import INT, VP, GdnLinearArgs, GdnNormArgs

CODES = {"torch.float32": 0, "torch.bfloat16": 1, "torch.float8_e4m3fn": 2}


def library():
    import gated_deltanet_gb300 as gdn
    lib = ctypes.CDLL(gdn.build.lib_path())
    np_, lp = ctypes.POINTER(GdnNormArgs), ctypes.POINTER(GdnLinearArgs)
    for f in (lib.gdn_rms_norm, lib.gdn_quantize_rows):
        f.argtypes, f.restype = [np_, VP], INT
    for n, t in (("gdn_rms_norm_bwd", np_), ("gdn_linear", lp), ("gdn_linear_bwd", lp), ("gdn_gated_linear", lp),
                 ("gdn_gated_linear_bwd", lp)):
        f, w = getattr(lib, n), getattr(lib, n + "_workspace_size")
        f.argtypes, f.restype = [t, VP, ctypes.c_size_t, VP], INT
        w.argtypes, w.restype = [t], ctypes.c_size_t
    lib.gdn_layer_test_withhold.argtypes, lib.gdn_layer_test_withhold.restype = [INT], None
    return lib


def code(t):
    return CODES[str(t.dtype)]


def pointers(**kw):
    """Tensors as their addresses, everything else as it is."""
    return {k: v.data_ptr() if hasattr(v, "data_ptr") else v for k, v in kw.items()}


def norm_bwd_args(dy, h, w, dh, dx, dw, eps):
    M, D = h.shape
    return GdnNormArgs(**pointers(rows=M, width=D, dtype=code(h), w_dtype=0, out_dtype=code(h), eps=eps, x=h, ldx=D, weight=w, dy=dy, ld_dy=D,
                                  dh=dh, ld_dh=D, dx=dx, dweight=dw))
