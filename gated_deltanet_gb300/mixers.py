"""Token mixers beside the gated delta rule: linear attention with a decay for each head, and softmax attention with a sliding
window and a few first tokens that stay visible (``gdn_linear_attn``, ``gdn_window_attn``, their forms for single tokens and their
gradients in ``include/gdn.h``).

Layouts are the delta rule's: CUDA tensors [B, T, heads, size] in float32 or bfloat16, heads that share a key head are neighbours,
``cu_seqlens`` (int64, on the device) for packed input.  The work runs on the current stream and gradients are explicit calls.
Slices of a fused projection (consecutive heads, any distance between tokens) are taken as they are, other strides are made
contiguous first.  Outputs and temporary buffers come from PyTorch's allocator, so the calls can be captured into a CUDA graph.
bfloat16 heads of 64 and 128 run on the tensor cores, everything else (to 256) on the CUDA cores.  Inputs are finite: a NaN or an
infinity reaches, besides what depends on it, other tokens of its sequence nearby (hidden behind a mask it does too), but no other
sequence.  Outputs of packed input hold nothing where no sequence has tokens.
"""
from __future__ import annotations

from . import layer


def _m():
    return layer._module or layer._load()


def chunk_linear_attention(q, k, v, decay=None, scale=None, initial_state=None, output_final_state=False, cu_seqlens=None, *, out=None,
                           final_state=None):
    """Linear attention with a decay for each value head, in chunks (prompts, training):
    ``S_t = exp(decay) S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t``.

    q, k [B, T, H, K]; v [B, T, HV, V] (float32 or bfloat16, same dtype, HV a multiple of H); decay [HV] float32, the natural
    logarithm of what a token leaves of the state (None: 0, nothing decays), a constant of the layer; scale defaults to
    ``K ** -0.5``; initial_state [N, HV, K, V] float32 or None; cu_seqlens [N + 1] for packed input (B == 1).  Returns
    ``(o, final_state)``, the state None unless requested, float32 and summed as such (for bfloat16 heads of 64 and 128 the call then
    takes about a sixth longer).  ``out`` and ``final_state`` overlap no input."""
    return _m().linear_attn(q, k, v, decay, scale, initial_state, output_final_state, cu_seqlens, out, final_state, False)


def fused_recurrent_linear_attention(q, k, v, decay=None, scale=None, initial_state=None, output_final_state=False, cu_seqlens=None, *,
                                     out=None, final_state=None):
    """:func:`chunk_linear_attention` token by token (decoding, short continuations).  ``final_state`` may be ``initial_state``
    itself, which is then updated in place."""
    return _m().linear_attn(q, k, v, decay, scale, initial_state, output_final_state, cu_seqlens, out, final_state, True)


def chunk_linear_attention_bwd(q, k, v, decay, do, scale=None, initial_state=None, dht=None, cu_seqlens=None):
    """Gradients of :func:`chunk_linear_attention`: ``do`` with respect to o (its shape and dtype), ``dht`` [N, HV, K, V] float32
    (or None) with respect to the final state.  Returns ``(dq, dk, dv, dh0)`` in the dtypes of q, k, v and float32 (dh0 None
    without an initial state)."""
    return _m().linear_attn_bwd(q, k, v, decay, do, scale, initial_state, dht, cu_seqlens)


def window_attention(q, k, v, window, sinks=0, scale=None, cu_seqlens=None, cu_seqlens_k=None, *, return_lse=False, out=None):
    """Causal softmax attention with a sliding window and sinks: query i of a sequence with Lq queries and Lk keys stands at
    position ``p = i + Lk - Lq`` and sees key j when ``j <= p`` and (``p - j < window`` or ``j < sinks``).

    q [B, Tq, H, D]; k, v [B, Tk, HK, D] (float32 or bfloat16, same dtype, H a multiple of HK); window >= 1 (as long as the
    sequence: plain causal attention); scale defaults to ``D ** -0.5``; cu_seqlens [N + 1] for packed input (B == 1), with
    cu_seqlens_k where the keys are packed otherwise (a prompt continuing a cache).  Returns o in q's dtype, with ``return_lse``
    ``(o, lse)``, lse [B, H, Tq] float32 = log sum exp(scale q k).  A row that sees no key gives zeros and -inf."""
    o, lse = _m().window_attn(q, k, v, window, sinks, scale, cu_seqlens, cu_seqlens_k, return_lse, out)
    return (o, lse) if return_lse else o


def window_attention_decode(q, k_cache, v_cache, lengths, window, sinks=0, scale=None, *, out=None):
    """:func:`window_attention` of a few new tokens over a cache: q [B, T, H, D] (T = 1 when decoding), k_cache and v_cache
    [B, S, HK, D] at any strides between slots, heads and sequences, lengths [B] (int32 or int64, on the device): the slots filled,
    the T new tokens' among them.  Slots from lengths on and those that no new token sees are not read.  Slots are positions; a cache of
    ``window + sinks`` slots whose window is overwritten in turn serves single tokens once it is full, with a window of all its slots
    (the softmax does not depend on their order)."""
    return _m().window_attn_decode(q, k_cache, v_cache, lengths, window, sinks, scale, out)


def window_attention_bwd(do, q, k, v, o, lse, window, sinks=0, scale=None, cu_seqlens=None, cu_seqlens_k=None):
    """Gradients of :func:`window_attention` from its inputs, its outputs o and lse, and ``do``: returns ``(dq, dk, dv)`` in the
    inputs' dtype."""
    return _m().window_attn_bwd(do, q, k, v, o, lse, window, sinks, scale, cu_seqlens, cu_seqlens_k)
