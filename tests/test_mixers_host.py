"""Argument checks of the token mixers beside the gated delta rule, on the CPU: what the C entry points refuse before anything is
enqueued, and what the binding refuses.  No pointer here is ever dereferenced.  And the plain forms that the GPU tests compare with,
against differences and a second formulation."""
import ctypes

import pytest
import torch

import mixer_reference as ref

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -6
I64, INT, VP, F = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float


class GdnLinearAttnArgs(ctypes.Structure):
    _fields_ = [(n, INT) for n in ("B", "T", "H", "HV", "K", "V", "num_seqs", "dtype")] + [("scale", F), ("q", VP), ("k", VP), ("v", VP)] + [
        (n, I64) for n in ("ldq", "ldk", "ldv")] + [(n, VP) for n in ("decay", "h0", "cu_seqlens", "o", "ht", "dout")] + [("ld_dout", I64)] + [
        (n, VP) for n in ("dht", "dq", "dk", "dv", "dh0")]


class GdnWindowAttnArgs(ctypes.Structure):
    _fields_ = [(n, INT) for n in ("B", "Tq", "Tk", "H", "HK", "D", "num_seqs", "dtype", "window", "sinks")] + [("scale", F)] + [
        (n, VP) for n in ("q", "k", "v")] + [(n, I64) for n in ("ldq", "ldk", "ldv")] + [
        (n, VP) for n in ("cu_seqlens_q", "cu_seqlens_k", "o", "lse", "dout")] + [("ld_dout", I64)] + [(n, VP) for n in ("dq", "dk", "dv")] + [
        (n, I64) for n in ("o_seq", "o_tok", "o_head")]


class GdnWindowDecodeArgs(ctypes.Structure):
    _fields_ = [(n, INT) for n in ("N", "T", "S", "H", "HK", "D", "dtype", "window", "sinks")] + [("scale", F), ("q", VP), ("ldq", I64), ("k", VP),
                ("v", VP)] + [(n, I64) for n in ("k_seq", "k_tok", "k_head", "v_seq", "v_tok", "v_head")] + [("lengths", VP), ("lengths_64", INT), ("o", VP)]


@pytest.fixture(scope="module")
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import gated_deltanet_gb300 as g
    g.load_library()
    return g


@pytest.fixture(scope="module")
def L(gdn):
    lib = ctypes.CDLL(gdn.build.lib_path())
    for n, t in (("linear_attn", GdnLinearAttnArgs), ("linear_attn_bwd", GdnLinearAttnArgs), ("window_attn", GdnWindowAttnArgs),
                 ("window_attn_bwd", GdnWindowAttnArgs), ("window_attn_decode", GdnWindowDecodeArgs)):
        f, w = getattr(lib, "gdn_" + n), getattr(lib, "gdn_" + n + "_workspace_size")
        f.argtypes, f.restype = [ctypes.POINTER(t), VP, ctypes.c_size_t, VP], INT
        w.argtypes, w.restype = [ctypes.POINTER(t)], ctypes.c_size_t
    lib.gdn_linear_attn_recurrent.argtypes, lib.gdn_linear_attn_recurrent.restype = [ctypes.POINTER(GdnLinearAttnArgs), VP], INT
    return lib


def at(i):
    """The i-th of addresses 2^28 apart that nothing reads."""
    return (i + 1) << 28


def linear_args(**kw):
    d = dict(B=2, T=8, H=2, HV=4, K=64, V=64, num_seqs=2, dtype=1, scale=0.1, q=at(0), k=at(1), v=at(2), ldq=128, ldk=128, ldv=256, decay=at(3), o=at(4),
             ht=at(5), dout=at(6), ld_dout=256, dq=at(7), dk=at(8), dv=at(9), dh0=at(10), dht=at(11), h0=at(12))
    return GdnLinearAttnArgs(**(d | kw))


def window_args(**kw):
    d = dict(B=2, Tq=8, Tk=8, H=4, HK=2, D=64, num_seqs=2, dtype=1, window=4, sinks=1, scale=0.1, q=at(0), k=at(1), v=at(2), ldq=256, ldk=128, ldv=128,
             o=at(3), lse=at(4), dout=at(5), ld_dout=256, dq=at(6), dk=at(7), dv=at(8))
    return GdnWindowAttnArgs(**(d | kw))


def decode_args(**kw):
    d = dict(N=2, T=1, S=16, H=4, HK=2, D=64, dtype=1, window=4, sinks=1, scale=0.1, q=at(0), ldq=256, k=at(1), v=at(2), k_seq=2048, k_tok=128, k_head=64,
             v_seq=2048, v_tok=128, v_head=64, lengths=at(3), lengths_64=0, o=at(4))
    return GdnWindowDecodeArgs(**(d | kw))


NAN, INF = float("nan"), float("inf")
LINEAR_BAD = [dict(B=-1), dict(T=-1), dict(H=0), dict(HV=3), dict(K=0), dict(V=0), dict(num_seqs=3), dict(dtype=2), dict(dtype=9), dict(scale=NAN), dict(scale=INF),
              dict(q=None), dict(k=None), dict(v=None), dict(q=at(0) + 1), dict(ldq=127), dict(ldv=255), dict(decay=at(3) + 2), dict(h0=at(12) + 1),
              dict(cu_seqlens=at(20)), dict(cu_seqlens=at(20) + 4, B=1)]


@pytest.mark.parametrize("kw", LINEAR_BAD + [dict(o=None), dict(o=at(4) + 1), dict(ht=at(5) + 2), dict(o=at(0)), dict(o=at(2) + 256), dict(ht=at(4)), dict(ht=at(12)),
                                             dict(o=at(12)), dict(ht=at(3))])
def test_linear_refuses(L, kw):
    a = linear_args(**kw)
    assert L.gdn_linear_attn(ctypes.byref(a), None, 0, None) == INVALID
    assert L.gdn_linear_attn_workspace_size(ctypes.byref(a)) == 0
    if kw != dict(ht=at(12)):  # (a state updated in place is the recurrent form's)
        assert L.gdn_linear_attn_recurrent(ctypes.byref(a), None) == INVALID


@pytest.mark.parametrize("kw", LINEAR_BAD + [dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(ld_dout=255), dict(dq=at(0)), dict(dk=at(7)), dict(dv=at(6)),
                                             dict(dh0=at(11)), dict(dht=at(11) + 1)])
def test_linear_bwd_refuses(L, kw):
    a = linear_args(**kw)
    assert L.gdn_linear_attn_bwd(ctypes.byref(a), None, 0, None) == INVALID
    assert L.gdn_linear_attn_bwd_workspace_size(ctypes.byref(a)) == 0


WINDOW_BAD = [dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(H=0), dict(H=3), dict(HK=0), dict(D=0), dict(num_seqs=1), dict(dtype=2), dict(window=0), dict(sinks=-1),
              dict(scale=NAN), dict(q=None), dict(k=None), dict(v=None), dict(v=at(2) + 1), dict(ldq=255), dict(ldk=127), dict(cu_seqlens_q=at(20), B=1),
              dict(cu_seqlens_q=at(20), cu_seqlens_k=at(21)), dict(o=None), dict(o=at(3) + 1), dict(lse=at(4) + 2)]


@pytest.mark.parametrize("kw", WINDOW_BAD + [dict(o=at(0)), dict(o=at(1) + 512), dict(lse=at(3))])
def test_window_refuses(L, kw):
    assert L.gdn_window_attn(ctypes.byref(window_args(**kw)), None, 0, None) == INVALID


@pytest.mark.parametrize("kw", WINDOW_BAD + [dict(lse=None), dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(ld_dout=255), dict(dq=at(5)), dict(dk=at(6)),
                                             dict(dv=at(3)), dict(dq=at(4)), dict(o_tok=-64), dict(o_seq=1 << 29, o_tok=64, o_head=512)])
def test_window_bwd_refuses(L, kw):
    a = window_args(**kw)
    assert L.gdn_window_attn_bwd(ctypes.byref(a), None, 0, None) == INVALID
    assert L.gdn_window_attn_bwd_workspace_size(ctypes.byref(a)) == 0


@pytest.mark.parametrize("kw", [dict(N=-1), dict(T=-1), dict(S=-1), dict(H=3), dict(HK=0), dict(D=0), dict(dtype=2), dict(window=0), dict(sinks=-1), dict(scale=INF), dict(q=None),
                                dict(k=None), dict(v=None), dict(o=None), dict(lengths=None), dict(lengths=at(3) + 4, lengths_64=1), dict(ldq=255), dict(k_tok=-1), dict(v_seq=-8),
                                dict(o=at(0)), dict(o=at(1) + 4096), dict(k=at(1) + 1)])
def test_decode_refuses(L, kw):
    assert L.gdn_window_attn_decode(ctypes.byref(decode_args(**kw)), None, 0, None) == INVALID


def test_sizes_that_are_not_built(L):
    assert L.gdn_linear_attn(ctypes.byref(linear_args(K=257, ldq=514, ldk=514)), None, 0, None) == UNSUPPORTED
    assert L.gdn_linear_attn_recurrent(ctypes.byref(linear_args(V=300, ldv=1200)), None) == UNSUPPORTED
    assert L.gdn_window_attn(ctypes.byref(window_args(D=257, ldq=1028, ldk=514, ldv=514)), None, 0, None) == UNSUPPORTED
    assert L.gdn_window_attn_decode(ctypes.byref(decode_args(D=257, ldq=1028)), None, 0, None) == UNSUPPORTED


def test_null_structs(L):
    for n in ("linear_attn", "linear_attn_bwd", "window_attn", "window_attn_bwd", "window_attn_decode"):
        assert getattr(L, "gdn_" + n)(None, None, 0, None) == INVALID
        assert getattr(L, f"gdn_{n}_workspace_size")(None) == 0
    assert L.gdn_linear_attn_recurrent(None, None) == INVALID


def test_nothing_to_do(L):
    """No sequences, no tokens to attend from: nothing is enqueued."""
    assert L.gdn_linear_attn(ctypes.byref(linear_args(B=0, num_seqs=0)), None, 0, None) == 0
    assert L.gdn_linear_attn_recurrent(ctypes.byref(linear_args(B=0, num_seqs=0)), None) == 0
    assert L.gdn_linear_attn_bwd(ctypes.byref(linear_args(B=0, num_seqs=0)), None, 0, None) == 0
    assert L.gdn_window_attn(ctypes.byref(window_args(B=0, num_seqs=0)), None, 0, None) == 0
    assert L.gdn_window_attn(ctypes.byref(window_args(Tq=0)), None, 0, None) == 0
    assert L.gdn_window_attn_bwd(ctypes.byref(window_args(B=0, num_seqs=0)), None, 0, None) == 0
    assert L.gdn_window_attn_decode(ctypes.byref(decode_args(N=0)), None, 0, None) == 0
    assert L.gdn_window_attn_decode(ctypes.byref(decode_args(T=0)), None, 0, None) == 0


def test_workspaces(L):
    a = linear_args(dv=at(9))
    need = L.gdn_linear_attn_bwd_workspace_size(ctypes.byref(a))
    assert need >= 2 * 16 * 4 * 64 * 4  # two value heads to a key head: fp32 parts of dq and dk
    assert L.gdn_linear_attn_bwd(ctypes.byref(a), at(30), need - 1, None) == WORKSPACE
    assert L.gdn_linear_attn_bwd(ctypes.byref(a), at(30) + 64, need, None) == INVALID
    w = window_args()
    need = L.gdn_window_attn_bwd_workspace_size(ctypes.byref(w))
    assert need >= 16 * 4 * 4
    assert L.gdn_window_attn_bwd(ctypes.byref(w), at(30), need - 1, None) == WORKSPACE


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("heads", [1, 32])
def test_linear_workspace_of_many_sequences(L, dtype, backward, heads):
    """States are held for the segments of sequences that are cut: of T tokens, whatever the lengths, at most twice as many as one sequence of
    all tokens has."""
    size = L.gdn_linear_attn_bwd_workspace_size if backward else L.gdn_linear_attn_workspace_size

    def need(n):
        return size(ctypes.byref(linear_args(B=1, T=65536, H=heads, HV=heads, K=128, V=128, num_seqs=n, dtype=dtype, cu_seqlens=at(20000), ldq=heads * 128,
                                             ldk=heads * 128, ldv=heads * 128, ld_dout=heads * 128,
                                             **{k: at(1000 * i) for i, k in enumerate(("q", "k", "v", "o", "dout", "dq", "dk", "dv", "h0", "ht", "dht", "dh0", "decay"))})))

    one = need(1)
    assert one > 0 or heads > 1  # (many heads fill the GPU with whole sequences)
    for n in (1024, 4096, 65536):
        assert (need(n) > 0) == (one > 0) and need(n) <= 2 * one + 256


@pytest.mark.parametrize("dtype,most", [(0, 4), (1, 2.5)])
@pytest.mark.parametrize("window", [1, 128, 1024])
@pytest.mark.parametrize("sinks", [4, 300, 512])
def test_window_workspace_of_many_sequences(L, dtype, most, window, sinks):
    """fp32 parts of the sinks' gradients: of T tokens, whatever the lengths, two for each long sequence's sinks and one for each run of its queries
    (256 on the CUDA cores, 1024 on the tensor cores), to 512 sinks at most: 2 + 512 / 256 or 2 + 512 / 1024 times dK and dV in fp32."""
    T, heads, D = 65536, 16, 128

    def need(n):
        return L.gdn_window_attn_bwd_workspace_size(ctypes.byref(window_args(
            B=1, Tq=T, Tk=T, H=heads, HK=heads, D=D, num_seqs=n, dtype=dtype, window=window, sinks=sinks, cu_seqlens_q=at(200), cu_seqlens_k=at(201), ldq=heads * D,
            ldk=heads * D, ldv=heads * D, ld_dout=heads * D, **{k: at(10 * i) for i, k in enumerate(("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv"))})))

    for n in (1, 1024, 4096, 65536):
        assert 0 < need(n) <= T * heads * 4 + most * 2 * T * heads * D * 4


def test_binding_refuses_host_tensors(gdn):
    t, s, n = torch.zeros(1, 4, 2, 64), torch.zeros(1, 2, 64, 64), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: gdn.chunk_linear_attention(t, t, t), lambda: gdn.fused_recurrent_linear_attention(t, t, t, initial_state=s),
                 lambda: gdn.chunk_linear_attention_bwd(t, t, t, None, t), lambda: gdn.window_attention(t, t, t, 3),
                 lambda: gdn.window_attention_bwd(t, t, t, t, t, torch.zeros(1, 2, 4), 3), lambda: gdn.window_attention_decode(t, t, t, n, 3)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError, match="must be a tensor"):
        gdn.window_attention(t.numpy(), t, t, 3)


# ---------------------------------------------------------------- the plain forms themselves
def test_linear_reference_is_the_recurrence():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, h0, decay = r(1, 7, 1, 3), r(1, 7, 1, 3), r(1, 7, 2, 4), r(2, 2, 3, 4), torch.tensor([-0.3, -torch.inf], dtype=torch.float64)
    cu = torch.tensor([0, 5, 7])
    o, ht, _, _ = ref.linear(q, k, v, decay, 0.5, h0, cu)
    for n, (a, b) in enumerate(((0, 5), (5, 7))):
        S = h0[n].clone()
        for t in range(a, b):
            S = torch.exp(decay)[:, None, None] * S + k[0, t, 0][None, :, None] * v[0, t][:, None, :]
            assert torch.allclose(o[0, t], 0.5 * torch.einsum("d,hdv->hv", q[0, t, 0], S), atol=1e-12)
        assert torch.allclose(ht[n], S, atol=1e-12)


def test_window_reference_gradients_are_differences():
    """Along a direction, in 64 bits: the central difference with step 1e-5 is off by about 1e-10 of the values, its rounding by 1e-11."""
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = r(1, 9, 4, 5), r(1, 12, 2, 5), r(1, 12, 2, 5), r(1, 9, 4, 5)
    cu, cu_k = torch.tensor([0, 4, 9]), torch.tensor([0, 3, 12])
    f = lambda *x: (ref.window(*x, 3, 2, 0.4, cu, cu_k)[0] * do).sum()  # noqa: E731
    o = ref.window(q, k, v, 3, 2, 0.4, cu, cu_k)[0]
    grads, _ = ref.window_bwd(do, q, k, v, o, 3, 2, 0.4, cu, cu_k)
    for i in range(3):
        u = r(*(q, k, v)[i].shape)
        x, y = [q, k, v], [q, k, v]
        x[i], y[i] = x[i] + 1e-5 * u, y[i] - 1e-5 * u
        assert abs((f(*x) - f(*y)) / 2e-5 - (grads[i] * u).sum()) < 1e-7
    # a sequence of four queries over three keys: its first query sees nothing
    assert not o[0, 0].any() and not grads[0][0, 0].any()
