// Python binding of the decoder-block operators (gdn_rms_norm, gdn_linear, gdn_gated_linear and their
// gradients) and of the token mixers beside the gated delta rule (gdn_linear_attn, gdn_window_attn, theirs):
// checks and marshals PyTorch tensors.
//
// The calls of a decoding step run for a few microseconds on the GPU, and marshalling twenty fields from Python
// cost more than that (10 to 19 us a call through ctypes), so this part of the binding is compiled.  Outputs
// and workspaces come from PyTorch's allocator; the work runs on the current stream of the input's device.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <string>

#include "../../include/gdn.h"

namespace {

using at::Tensor;

PyObject *g_error;  // GdnError(code, what)

// A refusal: the Python exception is already set
struct Refused {};

[[noreturn]] void refuse(PyObject *type, const std::string &why)
{
    PyErr_SetString(type, why.c_str());
    throw Refused();
}
[[noreturn]] void bad_value(const std::string &why) { refuse(PyExc_ValueError, why); }
[[noreturn]] void bad_type(const std::string &why) { refuse(PyExc_TypeError, why); }

std::string shape_of(const Tensor &t)
{
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

const Tensor *tensor(const char *name, PyObject *o, bool optional = false)
{
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

void cuda(const char *name, const Tensor &t, const Tensor *with = nullptr)
{
    if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
    if (with && t.device() != with->device()) bad_value(std::string(name) + " is on another device than the input");
}

gdn_dtype code_of(const Tensor &t)
{
    return t.scalar_type() == at::kFloat ? GDN_F32 : t.scalar_type() == at::kBFloat16 ? GDN_BF16 : GDN_E4M3;
}
bool real(const Tensor &t) { return t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16; }
void need_real(const char *name, const Tensor &t)
{
    if (!real(t)) bad_type(std::string(name) + " must be float32 or bfloat16");
}

// A tensor as a matrix of `width` columns: as it is when its rows are contiguous and evenly spaced, else a
// contiguous copy.
struct Rows {
    Tensor t;
    int64_t n, ld;
    void *ptr() const { return t.data_ptr(); }
};
Rows rows(const char *name, const Tensor &t, int64_t width, int64_t expected = -1)
{
    const int64_t d = t.dim();
    if (d == 0 || t.size(d - 1) != width)
        bad_value(std::string(name) + " must have " + std::to_string(width) + " columns, got shape " + shape_of(t));
    const int64_t n = t.numel() / width;
    if (expected >= 0 && n != expected)
        bad_value(std::string(name) + " has " + std::to_string(n) + " rows, expected " + std::to_string(expected));
    if (t.is_contiguous()) return {t, n, width};
    bool even = d >= 2 && t.stride(d - 1) == 1 && t.stride(d - 2) >= width;
    for (int64_t i = 0; even && i + 2 < d; ++i) even = t.stride(i) == t.stride(i + 1) * t.size(i + 1);
    if (even) return {t, n, t.stride(d - 2)};
    return {t.contiguous(), n, width};
}

// A vector of n elements, contiguous
Tensor vec(const char *name, const Tensor &t, int64_t n, const Tensor &with, bool bf16_too)
{
    cuda(name, t, &with);
    if (t.scalar_type() != at::kFloat && !(bf16_too && t.scalar_type() == at::kBFloat16))
        bad_type(std::string(name) + (bf16_too ? " must be float32 or bfloat16" : " must be float32"));
    if (t.numel() != n)
        bad_value(std::string(name) + " must have " + std::to_string(n) + " elements, got " + std::to_string(t.numel()));
    return t.contiguous();
}

// (straight to the allocator: by the dispatcher, at::empty, a tensor takes 0.4 us longer, of a call's 4 to 8)
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor &on)
{
    return at::detail::empty_cuda(shape, type, on.device(), std::nullopt);
}

Tensor output(const char *name, const Tensor *given, at::IntArrayRef shape, at::ScalarType type, const Tensor &like)
{
    if (!given) return fresh(shape, type, like);
    if (given->sizes() != shape || given->scalar_type() != type || given->device() != like.device() || !given->is_contiguous())
        bad_value(std::string(name) + " must be a contiguous tensor of the output's shape, dtype and device");
    return *given;
}

int64_t width_of(const char *name, const Tensor &t)
{
    if (t.dim() == 0 || t.size(t.dim() - 1) < 1) bad_value(std::string(name) + " must have at least one column");
    return t.size(t.dim() - 1);
}

gdn_stream_t stream_of(const Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

void checked(gdn_status code, const char *what)
{
    if (code == GDN_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)code, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}

// a call with a workspace of the size it asks for
template <typename Args>
void launch(gdn_status (*call)(const Args *, void *, size_t, gdn_stream_t), size_t (*size)(const Args *), const Args &a,
            const Tensor &on, const char *what)
{
    const size_t need = size(&a);
    if (!need) return checked(call(&a, nullptr, 0, stream_of(on)), what);
    const Tensor ws = fresh({(int64_t)need}, at::kByte, on);
    checked(call(&a, ws.data_ptr(), need, stream_of(on)), what);
}

PyObject *wrap(const Tensor &t)
{
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <typename... T>
PyObject *tuple_of(const T &...t)
{
    PyObject *parts[] = {wrap(t)...};
    PyObject *out = PyTuple_New(sizeof...(T));
    for (size_t i = 0; i < sizeof...(T); ++i) {
        if (!out || !parts[i]) throw python_error();
        PyTuple_SET_ITEM(out, i, parts[i]);
    }
    return out;
}

void arity(Py_ssize_t have, Py_ssize_t want)
{
    if (have != want) bad_type("expected " + std::to_string(want) + " arguments");
}
bool truth(PyObject *o)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw python_error();
    return t;
}
double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int64_t integer(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

// ---------------------------------------------------------------- norm
gdn_norm_args norm_args(const Rows &x, int64_t width)
{
    gdn_norm_args a{};
    a.rows = x.n;
    a.width = (int)width;
    a.dtype = a.out_dtype = code_of(x.t);
    a.w_dtype = GDN_F32;
    a.x = x.ptr();
    a.ldx = x.ld;
    return a;
}

void columns_fit(int64_t width)
{
    if (width > INT32_MAX) bad_value("too many columns");
}

// (x, weight, residual, eps, quant, out, residual_out) -> (y, scale, h)
PyObject *rms_norm(PyObject *const *p)
{
    const Tensor &x = *tensor("x", p[0]);
    const Tensor *w = tensor("weight", p[1], true), *r = tensor("residual", p[2], true);
    const bool quant = truth(p[4]);
    if (!r && p[6] != Py_None) bad_value("residual_out goes with a residual");
    cuda("x", x);
    need_real("x", x);
    const int64_t width = width_of("x", x);
    columns_fit(width);
    const c10::cuda::CUDAGuard guard(x.device());
    const Rows xr = rows("x", x, width);
    gdn_norm_args a = norm_args(xr, width);
    a.eps = (float)number(p[3]);
    Tensor wv, h, scale;
    Rows rr;
    if (w) {
        wv = vec("weight", *w, width, x, true);
        a.weight = wv.data_ptr();
        a.w_dtype = code_of(wv);
    }
    if (r) {
        cuda("residual", *r, &x);
        if (r->scalar_type() != x.scalar_type()) bad_type("x and residual must share a dtype");
        if (r->sizes() != x.sizes()) bad_value("x and residual must share a shape");
        rr = rows("residual", *r, width, xr.n);
        a.residual = rr.ptr();
        a.ld_residual = rr.ld;
        h = output("residual_out", tensor("residual_out", p[6], true), x.sizes(), x.scalar_type(), x);
        a.h = h.data_ptr();
    }
    const Tensor y = output("out", tensor("out", p[5], true), x.sizes(), quant ? at::kFloat8_e4m3fn : x.scalar_type(), x);
    a.y = y.data_ptr();
    if (quant) {
        scale = fresh(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
        a.out_dtype = GDN_E4M3;
        a.scale = scale.data_ptr<float>();
    }
    checked(gdn_rms_norm(&a, stream_of(x)), "gdn_rms_norm");
    return tuple_of(y, scale, h);
}

// (x, out) -> (q, scale)
PyObject *quantize_rows(PyObject *const *p)
{
    const Tensor &x = *tensor("x", p[0]);
    cuda("x", x);
    need_real("x", x);
    const int64_t width = width_of("x", x);
    columns_fit(width);
    const c10::cuda::CUDAGuard guard(x.device());
    const Rows xr = rows("x", x, width);
    gdn_norm_args a = norm_args(xr, width);
    const Tensor q = output("out", tensor("out", p[1], true), x.sizes(), at::kFloat8_e4m3fn, x);
    const Tensor scale = fresh(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
    a.out_dtype = GDN_E4M3;
    a.y = q.data_ptr();
    a.scale = scale.data_ptr<float>();
    checked(gdn_quantize_rows(&a, stream_of(x)), "gdn_quantize_rows");
    return tuple_of(q, scale);
}

// (dy, h, weight, dh, eps) -> (dx, dweight)
PyObject *rms_norm_bwd(PyObject *const *p)
{
    const Tensor &dy = *tensor("dy", p[0]), &h = *tensor("h", p[1]);
    const Tensor *w = tensor("weight", p[2], true), *dh = tensor("dh", p[3], true);
    cuda("h", h);
    need_real("h", h);
    const int64_t width = width_of("h", h);
    columns_fit(width);
    for (const auto &n : {std::make_pair("dy", &dy), std::make_pair("dh", dh)}) {
        if (!n.second) continue;
        cuda(n.first, *n.second, &h);
        if (n.second->scalar_type() != h.scalar_type() || n.second->sizes() != h.sizes())
            bad_value(std::string(n.first) + " must share h's dtype and shape");
    }
    const c10::cuda::CUDAGuard guard(h.device());
    const Rows hr = rows("h", h, width), yr = rows("dy", dy, width, hr.n);
    gdn_norm_args a = norm_args(hr, width);
    a.eps = (float)number(p[4]);
    a.dy = yr.ptr();
    a.ld_dy = yr.ld;
    Rows dr;
    if (dh) {
        dr = rows("dh", *dh, width, hr.n);
        a.dh = dr.ptr();
        a.ld_dh = dr.ld;
    }
    const Tensor dx = fresh(h.sizes(), h.scalar_type(), h);
    a.dx = dx.data_ptr();
    Tensor wv, dw;
    if (w) {
        wv = vec("weight", *w, width, h, true);
        a.weight = wv.data_ptr();
        a.w_dtype = code_of(wv);
        dw = fresh({width}, at::kFloat, h);
        a.dweight = dw.data_ptr<float>();
    }
    launch(gdn_rms_norm_bwd, gdn_rms_norm_bwd_workspace_size, a, h, "gdn_rms_norm_bwd");
    return tuple_of(dx, dw);
}

// ---------------------------------------------------------------- products
struct Operands {
    gdn_linear_args a{};
    Rows x, w;
    Tensor xs, ws, b;
    int64_t N, K;  // columns of one half of the weight's rows; columns of x
};

void operands(Operands &o, const Tensor &x, const Tensor &w, int64_t act, const Tensor *xs, const Tensor *ws, int64_t halves)
{
    cuda("x", x);
    cuda("weight", w, &x);
    if (!real(x) && x.scalar_type() != at::kFloat8_e4m3fn) bad_type("x must be float32, bfloat16 or float8_e4m3fn");
    if (w.scalar_type() != x.scalar_type()) bad_type("x and weight must share a dtype");
    if (w.dim() != 2 || w.size(0) < 1 || w.size(1) < 1 || w.size(0) % halves)
        bad_value(std::string("weight must be ") + (halves == 2 ? "[2 F, K]" : "[N, K]") + ", got shape " + shape_of(w));
    o.N = w.size(0) / halves;
    o.K = w.size(1);
    columns_fit(o.N);
    columns_fit(o.K);
    o.x = rows("x", x, o.K);
    o.w = rows("weight", w, o.K);
    gdn_linear_args &a = o.a;
    a.rows = o.x.n;
    a.out_features = (int)o.N;
    a.in_features = (int)o.K;
    a.dtype = code_of(x);
    a.out_dtype = a.dtype == GDN_F32 ? GDN_F32 : GDN_BF16;
    a.act = (gdn_activation)act;
    a.x = o.x.ptr();
    a.ldx = o.x.ld;
    a.w = o.w.ptr();
    a.ldw = o.w.ld;
    if (!xs != !ws) bad_value("x_scale and weight_scale go together");
    if (xs) {
        if (a.dtype != GDN_E4M3) bad_type("scales go with float8_e4m3fn inputs");
        o.xs = vec("x_scale", *xs, a.rows, x, false);
        o.ws = vec("weight_scale", *ws, w.size(0), x, false);
        a.x_scale = o.xs.data_ptr<float>();
        a.w_scale = o.ws.data_ptr<float>();
    }
}

c10::SmallVector<int64_t, 6> like_rows(const Tensor &x, int64_t cols)
{
    c10::SmallVector<int64_t, 6> s(x.sizes().begin(), x.sizes().end());
    s.back() = cols;
    return s;
}

at::ScalarType plain_out(const Operands &o) { return o.a.dtype == GDN_F32 ? at::kFloat : at::kBFloat16; }

// (x, weight, bias, act, residual, x_scale, weight_scale, out_f32, out) -> y;  out_f32: True, False or None
PyObject *linear(PyObject *const *p)
{
    const Tensor &x = *tensor("x", p[0]), &w = *tensor("weight", p[1]);
    const Tensor *b = tensor("bias", p[2], true), *r = tensor("residual", p[4], true), *out = tensor("out", p[8], true);
    cuda("x", x);
    const c10::cuda::CUDAGuard guard(x.device());
    Operands o;
    operands(o, x, w, integer(p[3]), tensor("x_scale", p[5], true), tensor("weight_scale", p[6], true), 1);
    at::ScalarType type = plain_out(o);
    if (p[7] != Py_None) type = truth(p[7]) ? at::kFloat : at::kBFloat16;
    else if (out && real(*out)) type = out->scalar_type();
    if (o.a.dtype == GDN_F32 && type != at::kFloat) bad_type("float32 inputs give a float32 output");
    o.a.out_dtype = type == at::kFloat ? GDN_F32 : GDN_BF16;
    if (b) {
        o.b = vec("bias", *b, o.N, x, false);
        o.a.bias = o.b.data_ptr<float>();
    }
    Rows rr;
    if (r) {
        cuda("residual", *r, &x);
        if (r->scalar_type() != type) bad_type("residual must have the output's dtype");
        rr = rows("residual", *r, o.N, o.a.rows);
        o.a.residual = rr.ptr();
        o.a.ld_residual = rr.ld;
    }
    const Tensor y = output("out", out, like_rows(x, o.N), type, x);
    o.a.y = y.data_ptr();
    o.a.ldy = o.N;
    launch(gdn_linear, gdn_linear_workspace_size, o.a, x, "gdn_linear");
    return wrap(y);
}

// (x, weight, act, x_scale, weight_scale, out) -> y
PyObject *gated_linear(PyObject *const *p)
{
    const Tensor &x = *tensor("x", p[0]), &w = *tensor("weight", p[1]);
    cuda("x", x);
    const c10::cuda::CUDAGuard guard(x.device());
    Operands o;
    operands(o, x, w, integer(p[2]), tensor("x_scale", p[3], true), tensor("weight_scale", p[4], true), 2);
    const Tensor y = output("out", tensor("out", p[5], true), like_rows(x, o.N), plain_out(o), x);
    o.a.y = y.data_ptr();
    o.a.ldy = o.N;
    launch(gdn_gated_linear, gdn_gated_linear_workspace_size, o.a, x, "gdn_gated_linear");
    return wrap(y);
}

// the gradients' outputs and dy
void gradients(Operands &o, const Tensor &dy, const Tensor &x, const Tensor &w, bool need_dx, bool need_dw, Rows &dyr, Tensor &dx,
               Tensor &dw)
{
    cuda("dy", dy, &x);
    if (dy.scalar_type() != x.scalar_type()) bad_type("dy and x must share a dtype");
    dyr = rows("dy", dy, o.N, o.a.rows);
    o.a.dy = dyr.ptr();
    o.a.ld_dy = dyr.ld;
    if (need_dx) {
        dx = fresh(x.sizes(), x.scalar_type(), x);
        o.a.dx = dx.data_ptr();
    }
    if (need_dw) {
        dw = fresh(w.sizes(), x.scalar_type(), x);
        o.a.dw = dw.data_ptr();
    }
}

// (dy, x, weight, bias, act, need_dx, need_dweight) -> (dx, dweight, dbias)
PyObject *linear_bwd(PyObject *const *p)
{
    const Tensor &dy = *tensor("dy", p[0]), &x = *tensor("x", p[1]), &w = *tensor("weight", p[2]);
    const Tensor *b = tensor("bias", p[3], true);
    cuda("x", x);
    need_real("x", x);
    const c10::cuda::CUDAGuard guard(x.device());
    Operands o;
    operands(o, x, w, integer(p[4]), nullptr, nullptr, 1);
    Rows dyr;
    Tensor dx, dw, db;
    gradients(o, dy, x, w, truth(p[5]), truth(p[6]), dyr, dx, dw);
    if (b) {
        o.b = vec("bias", *b, o.N, x, false);
        o.a.bias = o.b.data_ptr<float>();
        db = fresh({o.N}, at::kFloat, x);
        o.a.dbias = db.data_ptr<float>();
    }
    launch(gdn_linear_bwd, gdn_linear_bwd_workspace_size, o.a, x, "gdn_linear_bwd");
    return tuple_of(dx, dw, db);
}

// (dy, x, weight, act, need_dx, need_dweight, return_output) -> (dx, dweight, output)
PyObject *gated_linear_bwd(PyObject *const *p)
{
    const Tensor &dy = *tensor("dy", p[0]), &x = *tensor("x", p[1]), &w = *tensor("weight", p[2]);
    cuda("x", x);
    need_real("x", x);
    const c10::cuda::CUDAGuard guard(x.device());
    Operands o;
    operands(o, x, w, integer(p[3]), nullptr, nullptr, 2);
    Rows dyr;
    Tensor dx, dw, y;
    gradients(o, dy, x, w, truth(p[4]), truth(p[5]), dyr, dx, dw);
    if (truth(p[6])) {
        y = fresh(like_rows(x, o.N), x.scalar_type(), x);
        o.a.y = y.data_ptr();
        o.a.ldy = o.N;
    }
    launch(gdn_gated_linear_bwd, gdn_gated_linear_bwd_workspace_size, o.a, x, "gdn_gated_linear_bwd");
    return tuple_of(dx, dw, y);
}

// ---------------------------------------------------------------- token mixers
// A tensor [B, T, heads, size] whose tokens are evenly spaced with consecutive heads and elements (a slice of a fused
// projection), else a contiguous copy; ld: elements from a token to the next.
struct Tokens {
    Tensor t;
    int64_t ld = 0;
    void *ptr() const { return t.data_ptr(); }
};
Tokens tokens(const Tensor &t)
{
    const int64_t B = t.size(0), T = t.size(1), h = t.size(2), d = t.size(3);
    if (t.is_contiguous()) return {t, h * d};
    const int64_t ld = T > 1 ? t.stride(1) : B > 1 ? t.stride(0) : h * d;
    if ((d == 1 || t.stride(3) == 1) && (h == 1 || t.stride(2) == d) && ld >= h * d && (B == 1 || t.stride(0) == T * ld)) return {t, ld};
    return {t.contiguous(), h * d};
}

void four(const char *name, const Tensor &t, const Tensor *with = nullptr)
{
    cuda(name, t, with);
    if (with && t.scalar_type() != with->scalar_type()) bad_type(std::string(name) + " and q must share a dtype");
    if (t.dim() != 4) bad_value(std::string(name) + " must have four dimensions, got shape " + shape_of(t));
    if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || t.size(2) > INT32_MAX || t.size(3) > INT32_MAX) bad_value(std::string(name) + " is too large");
}
void same_shape(const char *name, const Tensor &t, at::IntArrayRef shape)
{
    if (t.sizes() != shape) bad_value(std::string(name) + " has an unexpected shape " + shape_of(t));
}

// [N + 1] offsets of packed sequences
Tensor offsets(const char *name, const Tensor &t, const Tensor &with, int64_t batch)
{
    cuda(name, t, &with);
    if (t.scalar_type() != at::kLong) bad_type(std::string(name) + " must be int64");
    if (t.dim() != 1 || t.size(0) < 1) bad_value(std::string(name) + " must be [N + 1]");
    if (t.size(0) - 1 > INT32_MAX) bad_value(std::string(name) + " is too long");
    if (batch != 1) bad_value("packed input has a batch of 1");
    return t.contiguous();
}

struct Linear {
    gdn_linear_attn_args a{};
    Tokens q, k, v;
    Tensor decay, h0, cu;
};
// (a state [N, HV, K, V]; `out`: to be written, so as it is)
Tensor state(const char *name, const Tensor &t, const Tensor &with, at::IntArrayRef shape, bool out = false)
{
    cuda(name, t, &with);
    if (t.scalar_type() != at::kFloat) bad_type(std::string(name) + " must be float32");
    if (t.sizes() != shape) bad_value(std::string(name) + " must be [N, HV, K, V], got shape " + shape_of(t));
    if (out && !t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
    return t.contiguous();
}
std::array<int64_t, 4> state_shape(const gdn_linear_attn_args &a) { return {a.num_seqs, a.HV, a.K, a.V}; }

void linear_inputs(Linear &l, const Tensor &q, const Tensor &k, const Tensor &v, const Tensor *decay, PyObject *scale, const Tensor *h0, const Tensor *cu)
{
    four("q", q);
    need_real("q", q);
    four("k", k, &q);
    four("v", v, &q);
    same_shape("k", k, q.sizes());
    if (v.size(0) != q.size(0) || v.size(1) != q.size(1)) bad_value("v must have q's batch and tokens, got shape " + shape_of(v));
    if (q.size(2) < 1 || v.size(2) < 1 || v.size(2) % q.size(2)) bad_value("the heads of v must be a multiple of those of q");
    if (q.size(3) < 1 || v.size(3) < 1) bad_value("heads must have at least one element");
    gdn_linear_attn_args &a = l.a;
    a.B = (int)q.size(0); a.T = (int)q.size(1); a.H = (int)q.size(2); a.K = (int)q.size(3);
    a.HV = (int)v.size(2); a.V = (int)v.size(3);
    a.dtype = code_of(q);
    l.q = tokens(q); l.k = tokens(k); l.v = tokens(v);
    a.q = l.q.ptr(); a.k = l.k.ptr(); a.v = l.v.ptr();
    a.ldq = l.q.ld; a.ldk = l.k.ld; a.ldv = l.v.ld;
    a.num_seqs = a.B;
    if (cu) {
        l.cu = offsets("cu_seqlens", *cu, q, q.size(0));
        a.cu_seqlens = l.cu.data_ptr<int64_t>();
        a.num_seqs = (int)(l.cu.size(0) - 1);
    }
    if (decay) {
        l.decay = vec("decay", *decay, a.HV, q, false);
        a.decay = l.decay.data_ptr<float>();
    }
    a.scale = scale == Py_None ? 1.f / std::sqrt((float)a.K) : (float)number(scale);
    if (h0) {
        l.h0 = state("initial_state", *h0, q, state_shape(a));
        a.h0 = l.h0.data_ptr<float>();
    }
}

// (q, k, v, decay, scale, initial_state, output_final_state, cu_seqlens, out, final_state, recurrent) -> (o, ht)
PyObject *linear_attn(PyObject *const *p)
{
    const Tensor &q = *tensor("q", p[0]), &k = *tensor("k", p[1]), &v = *tensor("v", p[2]);
    const Tensor *decay = tensor("decay", p[3], true), *h0 = tensor("initial_state", p[5], true), *cu = tensor("cu_seqlens", p[7], true);
    const Tensor *out = tensor("out", p[8], true), *fin = tensor("final_state", p[9], true);
    const bool want = truth(p[6]), recurrent = truth(p[10]);
    if (fin && !want) bad_value("final_state goes with output_final_state");
    cuda("q", q);
    const c10::cuda::CUDAGuard guard(q.device());
    Linear l;
    linear_inputs(l, q, k, v, decay, p[4], h0, cu);
    const Tensor o = output("out", out, v.sizes(), v.scalar_type(), q);
    l.a.o = o.data_ptr();
    Tensor ht;
    if (want) {
        ht = fin ? state("final_state", *fin, q, state_shape(l.a), true) : fresh(state_shape(l.a), at::kFloat, q);
        l.a.ht = ht.data_ptr<float>();
    }
    if (recurrent) checked(gdn_linear_attn_recurrent(&l.a, stream_of(q)), "gdn_linear_attn_recurrent");
    else launch(gdn_linear_attn, gdn_linear_attn_workspace_size, l.a, q, "gdn_linear_attn");
    return tuple_of(o, ht);
}

// (q, k, v, decay, do, scale, initial_state, dht, cu_seqlens) -> (dq, dk, dv, dh0)
PyObject *linear_attn_bwd(PyObject *const *p)
{
    const Tensor &q = *tensor("q", p[0]), &k = *tensor("k", p[1]), &v = *tensor("v", p[2]), &dout = *tensor("do", p[4]);
    const Tensor *decay = tensor("decay", p[3], true), *h0 = tensor("initial_state", p[6], true), *dht = tensor("dht", p[7], true);
    cuda("q", q);
    const c10::cuda::CUDAGuard guard(q.device());
    Linear l;
    linear_inputs(l, q, k, v, decay, p[5], h0, tensor("cu_seqlens", p[8], true));
    four("do", dout, &q);
    same_shape("do", dout, v.sizes());
    const Tokens d = tokens(dout);
    l.a.dout = d.ptr();
    l.a.ld_dout = d.ld;
    Tensor dhtv, dh0;
    if (dht) {
        dhtv = state("dht", *dht, q, state_shape(l.a));
        l.a.dht = dhtv.data_ptr<float>();
    }
    const Tensor dq = fresh(q.sizes(), q.scalar_type(), q), dk = fresh(k.sizes(), q.scalar_type(), q), dv = fresh(v.sizes(), q.scalar_type(), q);
    l.a.dq = dq.data_ptr(); l.a.dk = dk.data_ptr(); l.a.dv = dv.data_ptr();
    if (h0) {
        dh0 = fresh(state_shape(l.a), at::kFloat, q);
        l.a.dh0 = dh0.data_ptr<float>();
    }
    launch(gdn_linear_attn_bwd, gdn_linear_attn_bwd_workspace_size, l.a, q, "gdn_linear_attn_bwd");
    return tuple_of(dq, dk, dv, dh0);
}

struct Window {
    gdn_window_attn_args a{};
    Tokens q, k, v;
    Tensor cu_q, cu_k;
};
// window and sinks as the C entries take them (nothing is longer than 2^31 - 1 tokens)
int count(const char *name, PyObject *o, int64_t least)
{
    const int64_t n = integer(o);
    if (n < least) bad_value(std::string(name) + " must be at least " + std::to_string(least));
    return (int)std::min<int64_t>(n, INT32_MAX);
}
void window_inputs(Window &w, const Tensor &q, const Tensor &k, const Tensor &v, PyObject *window, PyObject *sinks, PyObject *scale, const Tensor *cu,
                   const Tensor *cu_k)
{
    four("q", q);
    need_real("q", q);
    four("k", k, &q);
    four("v", v, &q);
    same_shape("v", v, k.sizes());
    if (k.size(0) != q.size(0) || k.size(3) != q.size(3)) bad_value("k must have q's batch and head size, got shape " + shape_of(k));
    if (q.size(2) < 1 || k.size(2) < 1 || q.size(2) % k.size(2)) bad_value("the heads of q must be a multiple of those of k");
    if (q.size(3) < 1) bad_value("heads must have at least one element");
    if (cu_k && !cu) bad_value("cu_seqlens_k goes with cu_seqlens");
    if (cu && !cu_k && k.size(1) != q.size(1)) bad_value("keys of other lengths than the queries need cu_seqlens_k");
    gdn_window_attn_args &a = w.a;
    a.B = (int)q.size(0); a.Tq = (int)q.size(1); a.Tk = (int)k.size(1); a.H = (int)q.size(2); a.HK = (int)k.size(2); a.D = (int)q.size(3);
    a.dtype = code_of(q);
    a.window = count("window", window, 1);
    a.sinks = count("sinks", sinks, 0);
    a.scale = scale == Py_None ? 1.f / std::sqrt((float)a.D) : (float)number(scale);
    w.q = tokens(q); w.k = tokens(k); w.v = tokens(v);
    a.q = w.q.ptr(); a.k = w.k.ptr(); a.v = w.v.ptr();
    a.ldq = w.q.ld; a.ldk = w.k.ld; a.ldv = w.v.ld;
    a.num_seqs = a.B;
    if (cu) {
        w.cu_q = offsets("cu_seqlens", *cu, q, q.size(0));
        w.cu_k = cu_k ? offsets("cu_seqlens_k", *cu_k, q, q.size(0)) : w.cu_q;
        if (w.cu_k.size(0) != w.cu_q.size(0)) bad_value("cu_seqlens and cu_seqlens_k must have one length");
        a.cu_seqlens_q = w.cu_q.data_ptr<int64_t>();
        a.cu_seqlens_k = w.cu_k.data_ptr<int64_t>();
        a.num_seqs = (int)(w.cu_q.size(0) - 1);
    }
}

// (q, k, v, window, sinks, scale, cu_seqlens, cu_seqlens_k, return_lse, out) -> (o, lse)
PyObject *window_attn(PyObject *const *p)
{
    const Tensor &q = *tensor("q", p[0]), &k = *tensor("k", p[1]), &v = *tensor("v", p[2]);
    cuda("q", q);
    const c10::cuda::CUDAGuard guard(q.device());
    Window w;
    window_inputs(w, q, k, v, p[3], p[4], p[5], tensor("cu_seqlens", p[6], true), tensor("cu_seqlens_k", p[7], true));
    const Tensor o = output("out", tensor("out", p[9], true), q.sizes(), q.scalar_type(), q);
    w.a.o = o.data_ptr();
    Tensor lse;
    if (truth(p[8])) {
        lse = fresh({q.size(0), q.size(2), q.size(1)}, at::kFloat, q);
        w.a.lse = lse.data_ptr<float>();
    }
    launch(gdn_window_attn, gdn_window_attn_workspace_size, w.a, q, "gdn_window_attn");
    return tuple_of(o, lse);
}

// (do, q, k, v, o, lse, window, sinks, scale, cu_seqlens, cu_seqlens_k) -> (dq, dk, dv)
PyObject *window_attn_bwd(PyObject *const *p)
{
    const Tensor &dout = *tensor("do", p[0]), &q = *tensor("q", p[1]), &k = *tensor("k", p[2]), &v = *tensor("v", p[3]), &o = *tensor("o", p[4]),
                 &lse = *tensor("lse", p[5]);
    cuda("q", q);
    const c10::cuda::CUDAGuard guard(q.device());
    Window w;
    window_inputs(w, q, k, v, p[6], p[7], p[8], tensor("cu_seqlens", p[9], true), tensor("cu_seqlens_k", p[10], true));
    four("do", dout, &q);
    four("o", o, &q);
    same_shape("do", dout, q.sizes());
    same_shape("o", o, q.sizes());
    cuda("lse", lse, &q);
    if (lse.scalar_type() != at::kFloat) bad_type("lse must be float32");
    const int64_t stats[] = {q.size(0), q.size(2), q.size(1)};
    same_shape("lse", lse, stats);
    const Tokens d = tokens(dout);
    // o as it lies where the copies can ask for it so, each head's elements together and 16 bytes apart
    bool there = o.size(3) == 1 || o.stride(3) == 1;
    for (int i = 0; i < 3; ++i) there = there && (o.size(i) <= 1 || (o.stride(i) > 0 && o.stride(i) * o.element_size() % 16 == 0));
    const Tensor oc = there ? o : o.contiguous(), lc = lse.contiguous();
    w.a.dout = d.ptr();
    w.a.ld_dout = d.ld;
    w.a.o = oc.data_ptr();
    w.a.o_seq = oc.stride(0); w.a.o_tok = oc.stride(1); w.a.o_head = oc.stride(2);
    w.a.lse = lc.data_ptr<float>();
    const Tensor dq = fresh(q.sizes(), q.scalar_type(), q), dk = fresh(k.sizes(), q.scalar_type(), q), dv = fresh(v.sizes(), q.scalar_type(), q);
    w.a.dq = dq.data_ptr(); w.a.dk = dk.data_ptr(); w.a.dv = dv.data_ptr();
    launch(gdn_window_attn_bwd, gdn_window_attn_bwd_workspace_size, w.a, q, "gdn_window_attn_bwd");
    return tuple_of(dq, dk, dv);
}

// (q, k_cache, v_cache, lengths, window, sinks, scale, out) -> o
PyObject *window_attn_decode(PyObject *const *p)
{
    const Tensor &q = *tensor("q", p[0]), &k = *tensor("k_cache", p[1]), &v = *tensor("v_cache", p[2]), &len = *tensor("lengths", p[3]);
    cuda("q", q);
    const c10::cuda::CUDAGuard guard(q.device());
    four("q", q);
    need_real("q", q);
    four("k_cache", k, &q);
    four("v_cache", v, &q);
    same_shape("v_cache", v, k.sizes());
    if (k.size(0) != q.size(0) || k.size(3) != q.size(3)) bad_value("k_cache must have q's batch and head size, got shape " + shape_of(k));
    if (q.size(2) < 1 || k.size(2) < 1 || q.size(2) % k.size(2)) bad_value("the heads of q must be a multiple of those of k_cache");
    if (q.size(3) < 1) bad_value("heads must have at least one element");
    // a cache is never copied: a call reads a window of it
    for (const auto &c : {std::make_pair("k_cache", &k), std::make_pair("v_cache", &v)})
        if (c.second->size(3) > 1 && c.second->stride(3) != 1) bad_value(std::string(c.first) + " must have consecutive elements in a head");
    cuda("lengths", len, &q);
    if (len.scalar_type() != at::kInt && len.scalar_type() != at::kLong) bad_type("lengths must be int32 or int64");
    if (len.dim() != 1 || len.size(0) != q.size(0)) bad_value("lengths must be [B], got shape " + shape_of(len));
    const Tensor lc = len.contiguous();
    const Tokens qt = tokens(q);
    gdn_window_decode_args a{};
    a.N = (int)q.size(0); a.T = (int)q.size(1); a.S = (int)k.size(1); a.H = (int)q.size(2); a.HK = (int)k.size(2); a.D = (int)q.size(3);
    a.dtype = code_of(q);
    a.window = count("window", p[4], 1);
    a.sinks = count("sinks", p[5], 0);
    a.scale = p[6] == Py_None ? 1.f / std::sqrt((float)a.D) : (float)number(p[6]);
    a.q = qt.ptr(); a.ldq = qt.ld;
    a.k = k.data_ptr(); a.v = v.data_ptr();
    a.k_seq = k.stride(0); a.k_tok = k.stride(1); a.k_head = k.stride(2);
    a.v_seq = v.stride(0); a.v_tok = v.stride(1); a.v_head = v.stride(2);
    a.lengths = lc.data_ptr();
    a.lengths_64 = lc.scalar_type() == at::kLong;
    const Tensor o = output("out", tensor("out", p[7], true), q.sizes(), q.scalar_type(), q);
    a.o = o.data_ptr();
    launch(gdn_window_attn_decode, gdn_window_attn_decode_workspace_size, a, q, "gdn_window_attn_decode");
    return wrap(o);
}

// (device index) -> status code
PyObject *read_status(PyObject *const *p)
{
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)integer(p[0]));
    return PyLong_FromLong(gdn_read_layer_status(c10::cuda::getCurrentCUDAStream().stream()));
}

// (tensor, width) -> (its matrix form, rows, row stride): how inputs are taken
PyObject *row_view(PyObject *const *p)
{
    const Rows r = rows("tensor", *tensor("tensor", p[0]), integer(p[1]));
    return Py_BuildValue("NLL", THPVariable_Wrap(r.t), (long long)r.n, (long long)r.ld);
}

PyObject *set_error(PyObject *const *p)
{
    Py_XDECREF(g_error);
    g_error = p[0];
    Py_INCREF(g_error);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arity(n, N);
        return F(args);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name)
{
    return {name, (PyCFunction)(void (*)(void))entry<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<rms_norm, 7>("rms_norm"),
    method<quantize_rows, 2>("quantize_rows"),
    method<rms_norm_bwd, 5>("rms_norm_bwd"),
    method<linear, 9>("linear"),
    method<linear_bwd, 7>("linear_bwd"),
    method<gated_linear, 6>("gated_linear"),
    method<gated_linear_bwd, 7>("gated_linear_bwd"),
    method<linear_attn, 11>("linear_attn"),
    method<linear_attn_bwd, 9>("linear_attn_bwd"),
    method<window_attn, 10>("window_attn"),
    method<window_attn_bwd, 11>("window_attn_bwd"),
    method<window_attn_decode, 8>("window_attn_decode"),
    method<read_status, 1>("read_status"),
    method<row_view, 2>("row_view"),
    method<set_error, 1>("set_error"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", "decoder-block operators", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__layer() { return PyModule_Create(&module); }
