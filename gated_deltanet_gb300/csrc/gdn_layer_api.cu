// C-ABI layer of the decoder-block operators: argument checks, workspace layout and the launches of
// each call.
#include <cmath>

#include "gdn_mix.cuh"

using namespace gdn;

gdn_status gdn::take_workspace(size_t need, void *ws, size_t bytes, cudaStream_t st, char **out)
{
    *out = nullptr;
    if (need == 0) return GDN_OK;
    if (ws) {
        if (bytes < need) return GDN_ERR_WORKSPACE;
        if ((uintptr_t)ws & 255) return GDN_ERR_INVALID;
        *out = (char *)ws;
        return GDN_OK;
    }
    need += 256;  // past the status word of the library-managed workspace
    if (!managed_workspace_holds(need, st)) {
        cudaStreamCaptureStatus cs;
        if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) return GDN_ERR_CUDA;
        if (cs != cudaStreamCaptureStatusNone) return GDN_ERR_NOMEM;
    }
    void *p = nullptr;
    size_t got = 0;
    const gdn_status s = managed_workspace(need, st, &p, &got);
    if (s == GDN_OK) *out = (char *)p + 256;
    return s;
}

namespace {

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t esize(gdn_dtype t) { return t == GDN_F32 ? 4 : t == GDN_BF16 ? 2 : 1; }

bool real(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
bool on_element(const void *p, gdn_dtype t) { return ((uintptr_t)p & (esize(t) - 1)) == 0; }

// ---------------------------------------------------------------- norm
gdn_status check_norm(const gdn_norm_args *a)
{
    if (!a || a->rows < 0 || a->width < 1) return GDN_ERR_INVALID;
    if (!real(a->dtype) || !real(a->w_dtype)) return GDN_ERR_INVALID;
    if (!(a->eps >= 0.f) || std::isinf(a->eps)) return GDN_ERR_INVALID;
    if (a->rows > 0 && !a->x) return GDN_ERR_INVALID;
    if (a->rows > 1 && a->ldx < a->width) return GDN_ERR_INVALID;
    if (!on_element(a->x, a->dtype) || !on_element(a->weight, a->w_dtype)) return GDN_ERR_INVALID;
    return GDN_OK;
}

gdn_status run_norm(const gdn_norm_args *a, bool normalise, cudaStream_t st)
{
    gdn_status s = check_norm(a);
    if (s != GDN_OK) return s;
    if (a->out_dtype != a->dtype && a->out_dtype != GDN_E4M3) return GDN_ERR_INVALID;
    if (a->rows == 0) return GDN_OK;
    if (!a->y || (a->out_dtype == GDN_E4M3 && !a->scale)) return GDN_ERR_INVALID;
    if (!on_element(a->residual, a->dtype) || !on_element(a->y, a->out_dtype) || !on_element(a->h, a->dtype) ||
        ((uintptr_t)a->scale & 3))
        return GDN_ERR_INVALID;
    NormArgs n{};
    n.M = a->rows; n.D = a->width;
    n.dt = a->dtype; n.w_dt = a->w_dtype; n.out_dt = a->out_dtype;
    n.x = a->x; n.ldx = a->ldx; n.eps = a->eps;
    n.y = a->y; n.scale = a->scale;
    n.normalise = normalise;
    if (normalise) {
        if (a->residual && a->rows > 1 && a->ld_residual < a->width) return GDN_ERR_INVALID;
        n.r = a->residual; n.ldr = a->ld_residual;
        n.w = a->weight;
        n.h = a->h;
    }
    return launch_norm(n, st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// ---------------------------------------------------------------- products
struct Carve {  // offsets into a workspace
    size_t at = 0;
    size_t take(size_t bytes)
    {
        const size_t o = at;
        at = up256(at + bytes);
        return o;
    }
};

// fp32 rows to this many go to the CUDA cores as they are; more are worth their splitting into bf16 planes for the
// tensor cores (at 2048 x 2048: 64 rows take 28 us on the CUDA cores, the splitting of w alone about 10; 1024 rows take
// 389 us there and 46 on the tensor cores)
constexpr int64_t kF32Rows = 64;

cudaError_t launch_product(const GemmArgs &g, Epi epi, cudaStream_t st)
{
    return g.in == GDN_F32 && !g.a_plane ? launch_gemm_simt(g, epi, st) : launch_gemm_tc(g, epi, st);
}

// An operand of the tensor cores: as it is, or a copy in the workspace: padded where its rows do not start on 16-byte
// boundaries (one more read and write of it; its odd rows could only be loaded element by element), in bf16 planes where
// it is fp32.
struct Operand {
    const void *p;
    int64_t ld, rows, cols, plane;
    bool copy;
    size_t off;
    void plan(const void *ptr, int64_t stride, int64_t r, int64_t c, gdn_dtype t, bool planes, Carve &ws)
    {
        p = ptr; ld = stride; rows = r; cols = c;
        off = 0;
        plane = 0;
        copy = planes || (t != GDN_F32 && r > 0 && !tma_ok(ptr, stride, r, esize(t)));
        if (copy) {
            const size_t e = planes ? 2 : esize(t);
            const int64_t q = 16 / (int64_t)e;
            ld = (c + q - 1) / q * q;
            if (planes) plane = r * ld;
            off = ws.take((size_t)r * ld * e * (planes ? 3 : 1));
        }
    }
    cudaError_t make(int64_t stride, gdn_dtype t, char *base, cudaStream_t st)
    {
        if (!copy) return cudaSuccess;
        const void *src = p;
        p = base + off;
        return plane ? launch_split((const float *)src, stride, rows, cols, base + off, ld, plane, st)
                     : launch_copy_rows(src, t, stride, rows, cols, base + off, ld, st);
    }
};

// A tensor that the epilogue of a product of many rows reads or writes: as it is, or, where its rows do not start on
// 16-byte boundaries, by a copy in the workspace that has such rows (8071 x 955 x 571 with a residual: 84 us with an
// epilogue that goes by elements, 43 with the copies).
struct Rows16 {
    int64_t ld, cols;
    bool copy;
    size_t off;
    void plan(const void *ptr, int64_t stride, int64_t r, int64_t c, gdn_dtype t, bool many, Carve &ws)
    {
        ld = stride; cols = c;
        off = 0;
        copy = many && ptr && r > 0 && !tma_ok(ptr, stride, r, esize(t));
        if (copy) {
            const int64_t q = 16 / (int64_t)esize(t);
            ld = (c + q - 1) / q * q;
            off = ws.take((size_t)r * ld * esize(t));
        }
    }
};

// (the coordinates of a tile of 256 rows are 32-bit integers)
constexpr int64_t kMostRows = INT32_MAX - 255;

gdn_status check_linear(const gdn_linear_args *a, bool gated, bool backward)
{
    if (!a || a->rows < 0 || a->out_features < 1 || a->in_features < 1) return GDN_ERR_INVALID;
    if (gated && a->out_features > (1 << 30)) return GDN_ERR_INVALID;
    if (a->dtype != GDN_F32 && a->dtype != GDN_BF16 && a->dtype != GDN_E4M3) return GDN_ERR_INVALID;
    if (a->act < GDN_ACT_NONE || a->act > GDN_ACT_SIGMOID) return GDN_ERR_INVALID;
    if (backward && a->dtype == GDN_E4M3) return GDN_ERR_UNSUPPORTED;
    const gdn_dtype plain_out = a->dtype == GDN_F32 ? GDN_F32 : GDN_BF16;
    if (!real(a->out_dtype)) return GDN_ERR_INVALID;
    if (a->out_dtype != plain_out && (gated || backward || a->dtype == GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if ((a->x_scale != nullptr) != (a->w_scale != nullptr)) return GDN_ERR_INVALID;
    if (a->x_scale && a->dtype != GDN_E4M3) return GDN_ERR_INVALID;
    if (gated && (a->bias || a->residual || a->dbias)) return GDN_ERR_INVALID;
    const int64_t K = a->in_features, N = a->out_features;
    if ((a->rows > 1 && a->ldx < K) || a->ldw < K) return GDN_ERR_INVALID;
    if (!a->w || (a->rows > 0 && !a->x)) return GDN_ERR_INVALID;
    if (!on_element(a->x, a->dtype) || !on_element(a->w, a->dtype) || ((uintptr_t)a->bias & 3) ||
        ((uintptr_t)a->x_scale & 3) || ((uintptr_t)a->w_scale & 3))
        return GDN_ERR_INVALID;
    if (backward) {
        if (a->rows > 0 && !a->dy) return GDN_ERR_INVALID;
        if (a->rows > 1 && a->ld_dy < N) return GDN_ERR_INVALID;
        if (!on_element(a->dy, a->dtype) || !on_element(a->dx, a->dtype) || !on_element(a->dw, a->dtype) ||
            ((uintptr_t)a->dbias & 3))
            return GDN_ERR_INVALID;
        if (gated && a->y && (!on_element(a->y, a->dtype) || (a->rows > 1 && a->ldy < N))) return GDN_ERR_INVALID;
    } else {
        if (a->rows > 0 && !a->y) return GDN_ERR_INVALID;
        if (a->rows > 1 && a->ldy < N) return GDN_ERR_INVALID;
        if (a->residual && a->rows > 1 && a->ld_residual < N) return GDN_ERR_INVALID;
        if (!on_element(a->y, a->out_dtype) || !on_element(a->residual, a->out_dtype)) return GDN_ERR_INVALID;
    }
    return a->rows <= kMostRows ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// Rows of `cols` bytes, `ld` bytes apart
struct Block {
    uintptr_t at;
    int64_t rows, cols, ld;
    Block(const void *p, int64_t r, int64_t c, int64_t stride, size_t e)
        : at((uintptr_t)p), rows(p ? r : 0), cols(c * (int64_t)e), ld(r > 1 ? stride * (int64_t)e : c * (int64_t)e) {}
    uintptr_t end() const { return at + (rows - 1) * ld + cols; }
    // one run of memory against rows: the first row that ends past it starts before its end
    bool meets(uintptr_t lo, uintptr_t hi) const
    {
        const int64_t r = lo < at + cols ? 0 : (int64_t)(lo - at - cols) / ld + 1;
        return r < rows && at + r * ld < hi;
    }
};
// Whether two blocks share a byte.  (Rows with gaps at different strides on both sides count as apart.)
bool share(const Block &a, const Block &b)
{
    if (a.rows <= 0 || b.rows <= 0 || a.at >= b.end() || b.at >= a.end()) return false;
    if (a.ld == a.cols) return b.meets(a.at, a.end());
    if (b.ld == b.cols) return a.meets(b.at, b.end());
    if (a.ld != b.ld) return false;
    const Block &lo = a.at <= b.at ? a : b, &hi = a.at <= b.at ? b : a;
    const int64_t off = (int64_t)(hi.at - lo.at) % lo.ld;  // of hi's rows within lo's
    return off < lo.cols || off + hi.cols > lo.ld;
}

// The kernels read operands while they write outputs: y lies over no input but, row for row, the residual.
bool output_apart(const gdn_linear_args *a, bool gated)
{
    const int64_t M = a->rows, N = a->out_features, K = a->in_features, wrows = gated ? 2 * N : N;
    const size_t e = esize(a->dtype), eo = esize(a->out_dtype);
    const Block y(a->y, M, N, a->ldy, eo), r(a->residual, M, N, a->ld_residual, eo);
    const bool same = a->y == a->residual && (M <= 1 || a->ldy == a->ld_residual);
    return !share(y, Block(a->x, M, K, a->ldx, e)) && !share(y, Block(a->w, wrows, K, a->ldw, e)) && (same || !share(y, r)) &&
           !share(y, Block(a->bias, 1, N, N, 4)) && !share(y, Block(a->x_scale, 1, M, M, 4)) && !share(y, Block(a->w_scale, 1, wrows, wrows, 4));
}

// A call's workspace: padded copies of operands and of what the epilogues read and write; backward: dz (its rows padded
// to 16 bytes) and the column sums of groups of rows
struct LinearPlan {
    Operand x, w, dz;  // dz: dy itself without an activation
    Rows16 extra, y, dx, dw;
    int64_t dz_cols, dz_ld, parts;
    size_t off_dz, off_part, bytes;
    bool own_dz, planes;
};
GemmArgs forward_product(const gdn_linear_args *a, const LinearPlan &p)
{
    GemmArgs g{};
    g.M = a->rows; g.N = a->out_features; g.K = a->in_features;
    g.in = a->dtype; g.out_dt = a->out_dtype;
    g.a = p.x.p; g.lda = p.x.ld; g.a_plane = p.x.plane;
    g.b = p.w.p; g.ldb = p.w.ld; g.b_plane = p.w.plane;
    g.x_scale = a->x_scale; g.w_scale = a->w_scale;
    g.bias = a->bias;
    g.act = a->act;
    return g;
}

// a product whose epilogue's tensors pass by their copies where there are such
cudaError_t launch_by_rows(GemmArgs g, Epi epi, const Rows16 &extra, const Rows16 &out, char *base, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    if (extra.copy) {
        e = launch_copy_rows(g.extra, g.out_dt, g.ld_extra, g.M, extra.cols, base + extra.off, extra.ld, st);
        g.extra = base + extra.off;
        g.ld_extra = extra.ld;
    }
    void *const dst = g.out;
    const int64_t ld = g.ldo;
    if (out.copy) {
        g.out = base + out.off;
        g.ldo = out.ld;
    }
    if (e == cudaSuccess) e = launch_product(g, epi, st);
    return e == cudaSuccess && out.copy ? launch_copy_rows(g.out, g.out_dt, out.ld, g.M, out.cols, dst, ld, st) : e;
}

LinearPlan plan_linear(const gdn_linear_args *a, bool gated, bool backward)
{
    LinearPlan p{};
    Carve c;
    const int64_t wrows = (gated ? 2 : 1) * (int64_t)a->out_features;
    p.planes = a->dtype == GDN_F32 && a->rows > kF32Rows;
    p.x.plan(a->x, a->ldx, a->rows, a->in_features, a->dtype, p.planes, c);
    p.w.plan(a->w, a->ldw, a->rows > 0 ? wrows : 0, a->in_features, a->dtype, p.planes, c);
    const bool many = p.planes || (a->dtype != GDN_F32 && a->rows > kFewRows);
    if (!backward) {
        p.extra.plan(gated ? nullptr : a->residual, a->ld_residual, a->rows, a->out_features, a->out_dtype, many, c);
        // (a gated product reads nothing by elements beside it, so that the copy of its output repays its launch only past a
        // round of tiles: 4000 x 255 x 576 9.3 us without and 10.5 with it, 3001 x 955 x 512 17.9 and 13.4)
        const bool round = (a->rows + 255) / 256 * ((a->out_features + 127) / 128) > device_sm_count() / 2;
        p.y.plan(a->y, a->ldy, a->rows, a->out_features, a->out_dtype, many && (!gated || round), c);
    } else {
        const int64_t q = 16 / (int64_t)esize(a->dtype);
        p.dz_cols = wrows;
        p.own_dz = gated || a->act != GDN_ACT_NONE;
        p.parts = (a->rows + 31) / 32;
        const void *dz = a->dy;
        p.dz_ld = a->ld_dy;
        if (p.own_dz) {
            if (a->dbias && a->rows > 0) p.parts = gemm_colparts(forward_product(a, p), kEpiDact);
            dz = nullptr;  // (in the workspace)
            p.dz_ld = (p.dz_cols + q - 1) / q * q;
            p.off_dz = c.take((size_t)a->rows * p.dz_ld * esize(a->dtype));
            p.extra.plan(a->dy, a->ld_dy, a->rows, a->out_features, a->dtype, many, c);
        }
        p.dx.plan(a->dx, a->in_features, a->rows, a->in_features, a->dtype, many, c);
        p.dw.plan(a->rows > 0 ? a->dw : nullptr, a->in_features, wrows, a->in_features, a->dtype, p.planes || a->dtype != GDN_F32, c);
        p.dz.plan(dz, p.dz_ld, a->rows, p.dz_cols, a->dtype, p.planes && (a->dx || a->dw), c);
        p.off_part = c.take(a->dbias ? (size_t)p.parts * a->out_features * sizeof(float) : 0);
    }
    p.bytes = c.at;
    return p;
}

gdn_status run_bwd(const gdn_linear_args *a, bool gated, void *ws, size_t ws_bytes, cudaStream_t st)
{
    gdn_status s = check_linear(a, gated, true);
    if (s != GDN_OK) return s;
    const int64_t M = a->rows, N = a->out_features, K = a->in_features;
    LinearPlan p = plan_linear(a, gated, true);
    if (M == 0) {
        if (a->dw && cudaMemsetAsync(a->dw, 0, (size_t)p.dz_cols * K * esize(a->dtype), st) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (a->dbias && cudaMemsetAsync(a->dbias, 0, (size_t)N * sizeof(float), st) != cudaSuccess) return GDN_ERR_CUDA;
        return GDN_OK;
    }
    char *base = nullptr;
    if ((s = take_workspace(p.bytes, ws, ws_bytes, st, &base)) != GDN_OK) return s;
    if (p.x.make(a->ldx, a->dtype, base, st) != cudaSuccess || p.w.make(a->ldw, a->dtype, base, st) != cudaSuccess)
        return GDN_ERR_CUDA;
    float *part = a->dbias ? (float *)(base + p.off_part) : nullptr;
    if (p.own_dz) {
        GemmArgs g = forward_product(a, p);
        g.extra = a->dy; g.ld_extra = a->ld_dy;
        g.out = base + p.off_dz; g.ldo = p.dz_ld;
        g.out2 = gated ? a->y : nullptr;
        g.ldo2 = a->ldy;
        g.colpart = part;
        p.dz.p = g.out;
        if (launch_by_rows(g, gated ? kEpiGatedBwd : kEpiDact, p.extra, Rows16{}, base, st) != cudaSuccess) return GDN_ERR_CUDA;
    } else if (part && launch_colsum_rows(a->dy, a->dtype, M, N, a->ld_dy, part, st) != cudaSuccess) {
        return GDN_ERR_CUDA;
    }
    if ((a->dx || a->dw) && p.dz.make(p.dz_ld, a->dtype, base, st) != cudaSuccess) return GDN_ERR_CUDA;
    if (part && launch_colsum_finish(part, p.parts, N, a->dbias, st) != cudaSuccess) return GDN_ERR_CUDA;
    GemmArgs g{};
    g.in = a->dtype; g.out_dt = a->dtype;
    g.a = p.dz.p; g.lda = p.dz.ld; g.a_plane = p.dz.plane;
    g.act = GDN_ACT_NONE;
    g.b_t = 1;
    if (a->dx) {  // dx[m][k] = sum_n dz[m][n] w[n][k]
        GemmArgs d = g;
        d.M = M; d.N = K; d.K = p.dz_cols;
        d.b = p.w.p; d.ldb = p.w.ld; d.b_plane = p.w.plane;
        d.out = a->dx; d.ldo = K;
        if (launch_by_rows(d, kEpiLinear, Rows16{}, p.dx, base, st) != cudaSuccess) return GDN_ERR_CUDA;
    }
    if (a->dw) {  // dw[n][k] = sum_m dz[m][n] x[m][k]
        GemmArgs d = g;
        d.M = p.dz_cols; d.N = K; d.K = M;
        d.a_t = 1;
        d.b = p.x.p; d.ldb = p.x.ld; d.b_plane = p.x.plane;
        d.out = a->dw; d.ldo = K;
        if (launch_by_rows(d, kEpiLinear, Rows16{}, p.dw, base, st) != cudaSuccess) return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

gdn_status run_fwd(const gdn_linear_args *a, bool gated, void *ws, size_t ws_bytes, cudaStream_t st)
{
    gdn_status s = check_linear(a, gated, false);
    if (s != GDN_OK) return s;
    if (a->rows == 0) return GDN_OK;
    if (!output_apart(a, gated)) return GDN_ERR_INVALID;
    LinearPlan p = plan_linear(a, gated, false);
    char *base = nullptr;
    if ((s = take_workspace(p.bytes, ws, ws_bytes, st, &base)) != GDN_OK) return s;
    if (p.x.make(a->ldx, a->dtype, base, st) != cudaSuccess || p.w.make(a->ldw, a->dtype, base, st) != cudaSuccess)
        return GDN_ERR_CUDA;
    GemmArgs g = forward_product(a, p);
    g.extra = a->residual; g.ld_extra = a->ld_residual;
    g.out = a->y; g.ldo = a->ldy;
    return launch_by_rows(g, gated ? kEpiGated : kEpiLinear, p.extra, p.y, base, st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t linear_workspace(const gdn_linear_args *a, bool gated, bool backward)
{
    return check_linear(a, gated, backward) == GDN_OK ? plan_linear(a, gated, backward).bytes : 0;
}

}  // namespace

bool &gdn::withhold_loads()
{
    static thread_local bool on = false;
    return on;
}

extern "C" {

gdn_status gdn_rms_norm(const gdn_norm_args *a, gdn_stream_t stream) { return run_norm(a, true, (cudaStream_t)stream); }

gdn_status gdn_quantize_rows(const gdn_norm_args *a, gdn_stream_t stream)
{
    if (!a || a->out_dtype != GDN_E4M3) return GDN_ERR_INVALID;
    return run_norm(a, false, (cudaStream_t)stream);
}

size_t gdn_rms_norm_bwd_workspace_size(const gdn_norm_args *a)
{
    if (check_norm(a) != GDN_OK || a->rows == 0 || !a->dweight) return 0;
    Carve c;
    c.take((size_t)norm_bwd_parts(a->rows, a->width, a->dtype, device_sm_count()) * a->width * sizeof(float));
    if (norm_bwd_wide(a->width)) c.take((size_t)a->rows * sizeof(float));
    return c.at;
}

gdn_status gdn_rms_norm_bwd(const gdn_norm_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream)
{
    cudaStream_t st = (cudaStream_t)stream;
    gdn_status s = check_norm(a);
    if (s != GDN_OK) return s;
    if (a->rows > 0 && (!a->dy || !a->dx)) return GDN_ERR_INVALID;
    if (a->rows > 1 && (a->ld_dy < a->width || (a->dh && a->ld_dh < a->width))) return GDN_ERR_INVALID;
    if (!on_element(a->dy, a->dtype) || !on_element(a->dh, a->dtype) || !on_element(a->dx, a->dtype) ||
        ((uintptr_t)a->dweight & 3))
        return GDN_ERR_INVALID;
    char *base = nullptr;
    if ((s = take_workspace(gdn_rms_norm_bwd_workspace_size(a), workspace, ws_bytes, st, &base)) != GDN_OK) return s;
    const int sms = device_sm_count();
    NormBwdArgs n{};
    n.M = a->rows; n.D = a->width;
    n.dt = a->dtype; n.w_dt = a->w_dtype;
    n.dy = a->dy; n.ld_dy = a->ld_dy;
    n.h = a->x; n.ld_h = a->ldx;
    n.dh = a->dh; n.ld_dh = a->ld_dh;
    n.w = a->weight; n.eps = a->eps;
    n.dx = a->dx; n.dw = a->dweight;
    if (base) {
        n.part = (float *)base;
        if (norm_bwd_wide(a->width))
            n.rstd = (float *)(base + up256((size_t)norm_bwd_parts(a->rows, a->width, a->dtype, sms) * a->width * sizeof(float)));
    }
    return launch_norm_bwd(n, sms, st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_linear_workspace_size(const gdn_linear_args *a)
{
    return linear_workspace(a, false, false);
}

gdn_status gdn_linear(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream)
{
    return run_fwd(a, false, workspace, ws_bytes, (cudaStream_t)stream);
}

size_t gdn_linear_bwd_workspace_size(const gdn_linear_args *a)
{
    return linear_workspace(a, false, true);
}

gdn_status gdn_linear_bwd(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream)
{
    return run_bwd(a, false, workspace, ws_bytes, (cudaStream_t)stream);
}

size_t gdn_gated_linear_workspace_size(const gdn_linear_args *a)
{
    return linear_workspace(a, true, false);
}

gdn_status gdn_gated_linear(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream)
{
    return run_fwd(a, true, workspace, ws_bytes, (cudaStream_t)stream);
}

size_t gdn_gated_linear_bwd_workspace_size(const gdn_linear_args *a)
{
    return linear_workspace(a, true, true);
}

gdn_status gdn_gated_linear_bwd(const gdn_linear_args *a, void *workspace, size_t ws_bytes, gdn_stream_t stream)
{
    return run_bwd(a, true, workspace, ws_bytes, (cudaStream_t)stream);
}

gdn_status gdn_read_layer_status(gdn_stream_t stream)
{
    // (each reads and clears its own)
    const gdn_status all[] = {read_tc_status((cudaStream_t)stream), read_small_status((cudaStream_t)stream), read_lin_status((cudaStream_t)stream),
                              read_win_status((cudaStream_t)stream), read_win_bwd_status((cudaStream_t)stream)};
    for (const gdn_status s : all)
        if (s != GDN_OK) return s;
    return GDN_OK;
}

void gdn_layer_test_withhold(int on) { withhold_loads() = on != 0; }

}  // extern "C"
