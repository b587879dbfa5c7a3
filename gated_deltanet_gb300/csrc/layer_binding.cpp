// Python binding of the decoder-block operators (gdn_rms_norm, gdn_linear, gdn_gated_linear and their
// gradients): checks and marshals PyTorch tensors.
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
    method<read_status, 1>("read_status"),
    method<row_view, 2>("row_view"),
    method<set_error, 1>("set_error"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", "decoder-block operators", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__layer() { return PyModule_Create(&module); }
