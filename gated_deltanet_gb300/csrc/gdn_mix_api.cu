// C-ABI layer of the token mixers beside the gated delta rule: argument checks, workspace layout and the launches of each call.
#include <cmath>

#include "gdn_mix.cuh"

using namespace gdn;

namespace {

constexpr int kMaxHead = 256;

size_t esize(gdn_dtype t) { return t == GDN_F32 ? 4 : 2; }
bool real(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
bool on(const void *p, size_t e) { return ((uintptr_t)p & (e - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// The bytes of `tokens` rows of `width` elements of size e, `ld` elements apart
struct Span {
    uintptr_t lo, hi;
    Span(const void *p, int64_t tokens, int64_t width, int64_t ld, size_t e)
        : lo((uintptr_t)p), hi(p && tokens > 0 && width > 0 ? lo + (uintptr_t)((tokens - 1) * ld + width) * e : lo) {}
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi && lo < hi && o.lo < o.hi; }
};
template <int OUT, int IN>
bool apart(const Span (&out)[OUT], const Span (&in)[IN])
{
    for (int i = 0; i < OUT; ++i) {
        for (int j = 0; j < IN; ++j)
            if (out[i].meets(in[j])) return false;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return false;
    }
    return true;
}

// ---------------------------------------------------------------- linear attention
gdn_status check_lin(const gdn_linear_attn_args *a, bool backward, bool recurrent)
{
    if (!a || a->B < 0 || a->T < 0 || a->num_seqs < 0 || a->H < 1 || a->HV < 1 || a->HV % a->H || a->K < 1 || a->V < 1) return GDN_ERR_INVALID;
    if (!real(a->dtype) || !std::isfinite(a->scale)) return GDN_ERR_INVALID;
    if (a->K > kMaxHead || a->V > kMaxHead) return GDN_ERR_UNSUPPORTED;
    if (a->cu_seqlens ? a->B != 1 : a->num_seqs != a->B) return GDN_ERR_INVALID;
    const int64_t tokens = (int64_t)a->B * a->T, qk = (int64_t)a->H * a->K, vo = (int64_t)a->HV * a->V;
    if (qk > INT32_MAX || vo > INT32_MAX || a->T > INT32_MAX / 2 || (int64_t)a->num_seqs * a->HV > INT32_MAX / 8) return GDN_ERR_UNSUPPORTED;
    const size_t e = esize(a->dtype);
    if (tokens > 0 && (!a->q || !a->k || !a->v)) return GDN_ERR_INVALID;
    if (tokens > 1 && (a->ldq < qk || a->ldk < qk || a->ldv < vo)) return GDN_ERR_INVALID;
    if (!on(a->q, e) || !on(a->k, e) || !on(a->v, e) || !on(a->decay, 4) || !on(a->h0, 4) || !on(a->cu_seqlens, 8)) return GDN_ERR_INVALID;
    const int64_t state = (int64_t)a->num_seqs * a->HV * a->K * a->V;
    const Span q(a->q, tokens, qk, a->ldq, e), k(a->k, tokens, qk, a->ldk, e), v(a->v, tokens, vo, a->ldv, e), h0(a->h0, 1, state, state, 4),
        decay(a->decay, 1, a->HV, a->HV, 4), cu(a->cu_seqlens, 1, a->num_seqs + 1, 1, 8), none(nullptr, 0, 0, 0, 1);
    if (!backward) {
        if (tokens > 0 && !a->o) return GDN_ERR_INVALID;
        if (!on(a->o, e) || !on(a->ht, 4)) return GDN_ERR_INVALID;
        const Span out[] = {Span(a->o, tokens, vo, vo, e), Span(a->ht, 1, state, state, 4)};
        const Span in[] = {q, k, v, decay, cu, recurrent && a->ht == a->h0 ? none : h0};
        return apart(out, in) && !out[0].meets(h0) ? GDN_OK : GDN_ERR_INVALID;
    }
    if (tokens > 0 && (!a->dout || !a->dq || !a->dk || !a->dv)) return GDN_ERR_INVALID;
    if (tokens > 1 && a->ld_dout < vo) return GDN_ERR_INVALID;
    if (!on(a->dout, e) || !on(a->dht, 4) || !on(a->dq, e) || !on(a->dk, e) || !on(a->dv, e) || !on(a->dh0, 4)) return GDN_ERR_INVALID;
    const Span out[] = {Span(a->dq, tokens, qk, qk, e), Span(a->dk, tokens, qk, qk, e), Span(a->dv, tokens, vo, vo, e), Span(a->dh0, 1, state, state, 4)};
    const Span in[] = {q, k, v, decay, cu, h0, Span(a->dout, tokens, vo, a->ld_dout, e), Span(a->dht, 1, state, state, 4)};
    return apart(out, in) ? GDN_OK : GDN_ERR_INVALID;
}

LinArgs lin_args(const gdn_linear_attn_args *a)
{
    LinArgs l{};
    l.decay = a->decay;
    l.cu = a->cu_seqlens;
    l.T = a->T;
    l.N = a->num_seqs;
    l.HV = a->HV;
    return l;
}
LinArgs lin_forward(const gdn_linear_attn_args *a)
{
    LinArgs l = lin_args(a);
    const int r = a->HV / a->H;
    l.passes = 1;
    l.pass[0] = {a->q, a->k, a->v, a->ldq, a->ldk, a->ldv, r, r, 1, a->o, a->h0, a->ht, 1.f, a->scale, a->K, a->V, 0, 0, 0};
    return l;
}
// dq and dk of shared heads: fp32 parts of every value head first (`part`: both, one after the other)
LinArgs lin_backward(const gdn_linear_attn_args *a, float *part)
{
    LinArgs l = lin_args(a);
    const int r = a->HV / a->H;
    const int64_t n = (int64_t)a->B * a->T * a->HV * a->K;
    l.passes = 3;
    l.pass[0] = {a->dout, a->v, a->k, a->ld_dout, a->ldv, a->ldk, 1, 1, r, part ? (void *)part : a->dq, a->h0, nullptr, 1.f, a->scale, a->V, a->K, part != nullptr, 1, 0};
    l.pass[1] = {a->v, a->dout, a->q, a->ldv, a->ld_dout, a->ldq, 1, 1, r, part ? (void *)(part + n) : a->dk, a->dht, nullptr, a->scale, 1.f, a->V, a->K, part != nullptr, 1, 1};
    l.pass[2] = {a->k, a->q, a->dout, a->ldk, a->ldq, a->ld_dout, r, r, 1, a->dv, a->dht, a->dh0, a->scale, 1.f, a->K, a->V, 0, 0, 1};
    return l;
}
bool lin_on_tc(const gdn_linear_attn_args *a, const LinArgs &l) { return a->dtype == GDN_BF16 && lin_tc_ok(l, (int64_t)a->B * a->T); }
size_t lin_split_bytes(const gdn_linear_attn_args *a, const LinArgs &l) { return up256(lin_on_tc(a, l) ? lin_tc_plan(l, a->K).bytes : lin_simt_plan(l).bytes); }
cudaError_t run_lin(const gdn_linear_attn_args *a, const LinArgs &l, void *ws, cudaStream_t st)
{
    return lin_on_tc(a, l) ? launch_lin_tc(l, ws, (int64_t)a->B * a->T, st) : launch_lin_simt(l, a->dtype, ws, st);
}
size_t lin_part_bytes(const gdn_linear_attn_args *a)
{
    return a->HV == a->H ? 0 : up256((size_t)a->B * a->T * a->HV * a->K * 2 * sizeof(float));
}

// ---------------------------------------------------------------- window attention
gdn_status check_win(const gdn_window_attn_args *a, bool backward)
{
    if (!a || a->B < 0 || a->Tq < 0 || a->Tk < 0 || a->num_seqs < 0 || a->H < 1 || a->HK < 1 || a->H % a->HK || a->D < 1) return GDN_ERR_INVALID;
    if (!real(a->dtype) || !std::isfinite(a->scale) || a->window < 1 || a->sinks < 0) return GDN_ERR_INVALID;
    if (a->D > kMaxHead || a->H > 65535) return GDN_ERR_UNSUPPORTED;
    if ((a->cu_seqlens_q != nullptr) != (a->cu_seqlens_k != nullptr)) return GDN_ERR_INVALID;
    if (a->cu_seqlens_q ? a->B != 1 : a->num_seqs != a->B) return GDN_ERR_INVALID;
    const int64_t tq = (int64_t)a->B * a->Tq, tk = (int64_t)a->B * a->Tk, wq = (int64_t)a->H * a->D, wk = (int64_t)a->HK * a->D;
    if (wq > INT32_MAX || a->Tq > INT32_MAX / 2 || a->Tk > INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
    const size_t e = esize(a->dtype);
    if ((tq > 0 && !a->q) || (tk > 0 && (!a->k || !a->v))) return GDN_ERR_INVALID;
    if ((tq > 1 && a->ldq < wq) || (tk > 1 && (a->ldk < wk || a->ldv < wk))) return GDN_ERR_INVALID;
    if (!on(a->q, e) || !on(a->k, e) || !on(a->v, e) || !on(a->cu_seqlens_q, 8) || !on(a->cu_seqlens_k, 8)) return GDN_ERR_INVALID;
    if (!on(a->o, e) || !on(a->lse, 4) || (tq > 0 && !a->o)) return GDN_ERR_INVALID;
    const Span q(a->q, tq, wq, a->ldq, e), k(a->k, tk, wk, a->ldk, e), v(a->v, tk, wk, a->ldv, e), o(a->o, tq, wq, wq, e),
        lse(a->lse, 1, tq * a->H, 1, 4), cq(a->cu_seqlens_q, 1, a->num_seqs + 1, 1, 8), ck(a->cu_seqlens_k, 1, a->num_seqs + 1, 1, 8);
    if (!backward) {
        const Span out[] = {o, lse}, in[] = {q, k, v, cq, ck};
        return apart(out, in) ? GDN_OK : GDN_ERR_INVALID;
    }
    if (tq > 0 && (!a->lse || !a->dout || !a->dq)) return GDN_ERR_INVALID;
    if (tk > 0 && (!a->dk || !a->dv)) return GDN_ERR_INVALID;
    if (tq > 1 && a->ld_dout < wq) return GDN_ERR_INVALID;
    if (!on(a->dout, e) || !on(a->dq, e) || !on(a->dk, e) || !on(a->dv, e)) return GDN_ERR_INVALID;
    if (a->o_seq < 0 || a->o_tok < 0 || a->o_head < 0) return GDN_ERR_INVALID;
    const bool strided = a->o_seq || a->o_tok || a->o_head;
    const Span kept = strided ? Span(a->o, tq > 0, (a->B - 1) * a->o_seq + (a->Tq - 1) * a->o_tok + (a->H - 1) * a->o_head + a->D, 1, e) : o;
    const Span out[] = {Span(a->dq, tq, wq, wq, e), Span(a->dk, tk, wk, wk, e), Span(a->dv, tk, wk, wk, e)};
    const Span in[] = {q, k, v, cq, ck, kept, lse, Span(a->dout, tq, wq, a->ld_dout, e)};
    return apart(out, in) ? GDN_OK : GDN_ERR_INVALID;
}
WinArgs win_args(const gdn_window_attn_args *a)
{
    WinArgs w{};
    w.q = a->q; w.k = a->k; w.v = a->v;
    w.ldq = a->ldq; w.ldk = a->ldk; w.ldv = a->ldv;
    w.cu_q = a->cu_seqlens_q; w.cu_k = a->cu_seqlens_k;
    w.Tq = a->Tq; w.Tk = a->Tk; w.N = a->num_seqs;
    w.H = a->H; w.HK = a->HK; w.D = a->D;
    w.window = std::max(1, std::min(a->window, a->Tk));  // (no sequence is longer: the same keys, and sums that fit 32 bits)
    w.sinks = std::min(a->sinks, a->Tk);
    w.scale = a->scale;
    w.o = a->o;
    w.lse = a->lse;
    const bool strided = a->o_seq || a->o_tok || a->o_head;
    w.o_head = strided ? a->o_head : a->D;
    w.o_tok = strided ? a->o_tok : (int64_t)a->H * a->D;
    w.o_seq = strided ? a->o_seq : a->Tq * ((int64_t)a->H * a->D);
    w.dout = a->dout; w.ld_dout = a->ld_dout;
    w.dq = a->dq; w.dk = a->dk; w.dv = a->dv;
    return w;
}

size_t win_delta_bytes(const gdn_window_attn_args *a) { return up256((size_t)a->B * a->Tq * a->H * sizeof(float)); }
bool win_bwd_on_tc(const gdn_window_attn_args *a)
{
    return a->dtype == GDN_BF16 && win_bwd_tc_ok(win_args(a), (int64_t)a->B * a->Tq, (int64_t)a->B * a->Tk);
}

gdn_status check_step(const gdn_window_decode_args *a)
{
    if (!a || a->N < 0 || a->T < 0 || a->S < 0 || a->H < 1 || a->HK < 1 || a->H % a->HK || a->D < 1) return GDN_ERR_INVALID;
    if (!real(a->dtype) || !std::isfinite(a->scale) || a->window < 1 || a->sinks < 0) return GDN_ERR_INVALID;
    if (a->D > kMaxHead) return GDN_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)a->N * a->T, w = (int64_t)a->H * a->D;
    if (w > INT32_MAX || rows * a->H > INT32_MAX || a->S > INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
    const size_t e = esize(a->dtype);
    if (rows == 0) return GDN_OK;
    if (!a->q || !a->o || !a->lengths || (a->S > 0 && (!a->k || !a->v))) return GDN_ERR_INVALID;
    if (rows > 1 && a->ldq < w) return GDN_ERR_INVALID;
    if (!on(a->q, e) || !on(a->k, e) || !on(a->v, e) || !on(a->o, e) || !on(a->lengths, a->lengths_64 ? 8 : 4)) return GDN_ERR_INVALID;
    for (int64_t s : {a->k_seq, a->k_tok, a->k_head, a->v_seq, a->v_tok, a->v_head})
        if (s < 0) return GDN_ERR_INVALID;
    auto cache = [&](const void *p, int64_t seq, int64_t tok, int64_t head) {
        return Span(p, a->S > 0 ? 1 : 0, (a->N - 1) * seq + (a->S - 1) * tok + (a->HK - 1) * head + a->D, 1, e);
    };
    const Span out[] = {Span(a->o, rows, w, w, e)};
    const Span in[] = {Span(a->q, rows, w, a->ldq, e), cache(a->k, a->k_seq, a->k_tok, a->k_head), cache(a->v, a->v_seq, a->v_tok, a->v_head),
                       Span(a->lengths, 1, a->N, 1, a->lengths_64 ? 8 : 4)};
    return apart(out, in) ? GDN_OK : GDN_ERR_INVALID;
}

gdn_status of(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

}  // namespace

extern "C" {

size_t gdn_linear_attn_workspace_size(const gdn_linear_attn_args *a)
{
    return check_lin(a, false, false) == GDN_OK && a->num_seqs > 0 ? lin_split_bytes(a, lin_forward(a)) : 0;
}

gdn_status gdn_linear_attn(const gdn_linear_attn_args *a, void *ws, size_t ws_bytes, gdn_stream_t stream)
{
    gdn_status s = check_lin(a, false, false);
    if (s != GDN_OK || a->num_seqs == 0) return s;
    const LinArgs l = lin_forward(a);
    char *base = nullptr;
    if ((s = take_workspace(lin_split_bytes(a, l), ws, ws_bytes, stream, &base)) != GDN_OK) return s;
    return of(run_lin(a, l, base, stream));
}

gdn_status gdn_linear_attn_recurrent(const gdn_linear_attn_args *a, gdn_stream_t stream)
{
    const gdn_status s = check_lin(a, false, true);
    if (s != GDN_OK || a->num_seqs == 0) return s;
    LinStepArgs l{};
    l.q = a->q; l.k = a->k; l.v = a->v;
    l.ldq = a->ldq; l.ldk = a->ldk; l.ldv = a->ldv;
    l.decay = a->decay; l.h0 = a->h0; l.cu = a->cu_seqlens;
    l.o = a->o; l.ht = a->ht;
    l.T = a->T; l.N = a->num_seqs; l.H = a->H; l.HV = a->HV; l.K = a->K; l.V = a->V;
    l.scale = a->scale;
    return of(launch_lin_step(l, a->dtype, stream));
}

size_t gdn_linear_attn_bwd_workspace_size(const gdn_linear_attn_args *a)
{
    if (check_lin(a, true, false) != GDN_OK || a->num_seqs == 0) return 0;
    const size_t parts = lin_part_bytes(a);
    return parts + lin_split_bytes(a, lin_backward(a, parts ? (float *)256 : nullptr));  // (parts are aligned wherever they lie)
}

gdn_status gdn_linear_attn_bwd(const gdn_linear_attn_args *a, void *ws, size_t ws_bytes, gdn_stream_t stream)
{
    gdn_status s = check_lin(a, true, false);
    if (s != GDN_OK || a->num_seqs == 0) return s;
    char *base = nullptr;
    if ((s = take_workspace(gdn_linear_attn_bwd_workspace_size(a), ws, ws_bytes, stream, &base)) != GDN_OK) return s;
    const size_t parts = lin_part_bytes(a);
    float *const part = parts ? (float *)base : nullptr;
    const LinArgs l = lin_backward(a, part);
    cudaError_t e = run_lin(a, l, base + parts, stream);
    if (part && e == cudaSuccess) {
        const int64_t tokens = (int64_t)a->B * a->T;
        const int r = a->HV / a->H;
        e = launch_lin_heads(part, l, tokens, a->H, r, a->K, a->dq, a->dk, a->dtype, stream);
    }
    return of(e);
}

size_t gdn_window_attn_workspace_size(const gdn_window_attn_args *a)
{
    (void)a;
    return 0;
}

gdn_status gdn_window_attn(const gdn_window_attn_args *a, void *, size_t, gdn_stream_t stream)
{
    const gdn_status s = check_win(a, false);
    if (s != GDN_OK || a->num_seqs == 0 || a->Tq == 0) return s;
    const WinArgs w = win_args(a);
    const int64_t tq = (int64_t)a->B * a->Tq, tk = (int64_t)a->B * a->Tk;
    if (tq == 0) return GDN_OK;
    return of(a->dtype == GDN_BF16 && win_tc_ok(w, tq, tk) ? launch_win_tc(w, tq, tk, stream) : launch_win_simt(w, a->dtype, stream));
}

size_t gdn_window_attn_bwd_workspace_size(const gdn_window_attn_args *a)
{
    if (check_win(a, true) != GDN_OK || a->num_seqs == 0) return 0;
    return win_delta_bytes(a) + (win_bwd_on_tc(a) ? win_bwd_tc_bytes(win_args(a)) : win_dkv_simt_bytes(win_args(a)));
}

gdn_status gdn_window_attn_bwd(const gdn_window_attn_args *a, void *ws, size_t ws_bytes, gdn_stream_t stream)
{
    gdn_status s = check_win(a, true);
    if (s != GDN_OK || a->num_seqs == 0) return s;
    char *base = nullptr;
    if ((s = take_workspace(gdn_window_attn_bwd_workspace_size(a), ws, ws_bytes, stream, &base)) != GDN_OK) return s;
    WinArgs w = win_args(a);
    float *const delta = (float *)base;
    w.delta = delta;
    const int64_t tq = (int64_t)a->B * a->Tq, tk = (int64_t)a->B * a->Tk;
    if (win_bwd_on_tc(a)) return of(launch_win_bwd_tc(w, tq, tk, delta, base + win_delta_bytes(a), stream));
    cudaError_t e = cudaSuccess;
    if (tq > 0) e = launch_win_delta(w, a->dtype, delta, stream);
    if (e == cudaSuccess && tq > 0) e = launch_win_dq_simt(w, a->dtype, stream);
    if (e == cudaSuccess && tk > 0) e = launch_win_dkv_simt(w, a->dtype, base + win_delta_bytes(a), stream);
    return of(e);
}

size_t gdn_window_attn_decode_workspace_size(const gdn_window_decode_args *a)
{
    (void)a;
    return 0;
}

gdn_status gdn_window_attn_decode(const gdn_window_decode_args *a, void *, size_t, gdn_stream_t stream)
{
    const gdn_status s = check_step(a);
    if (s != GDN_OK || a->N == 0 || a->T == 0) return s;
    WinStepArgs w{};
    w.q = a->q; w.ldq = a->ldq;
    w.k = a->k; w.v = a->v;
    w.k_seq = a->k_seq; w.k_tok = a->k_tok; w.k_head = a->k_head;
    w.v_seq = a->v_seq; w.v_tok = a->v_tok; w.v_head = a->v_head;
    w.lengths = a->lengths; w.lengths_64 = a->lengths_64;
    w.N = a->N; w.T = a->T; w.S = a->S; w.H = a->H; w.HK = a->HK; w.D = a->D;
    w.window = std::max(1, std::min(a->window, a->S));
    w.sinks = std::min(a->sinks, a->S);
    w.scale = a->scale;
    w.o = a->o;
    return of(launch_win_step(w, a->dtype, stream));
}

}  // extern "C"
