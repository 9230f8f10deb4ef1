// binding.cpp -- the host side of the serving step's calls (residual norm to
// codes, router top-k, expert layer) between torch tensors and the C ABI of
// include/dg_fp8.h: checks of types and shapes, the outputs, the call.
//
// These calls are made for single tokens too, where a kernel takes 3 to 5 us
// and the same steps in Python took 6 (router) to 12 us (norm, layer), against
// 2 to 3.5 us here. Nothing is computed here, and no device code is built from
// this file.
//
// Each function takes the entry point's address first (the library is loaded
// by _lib.py) and the stream's handle last, returns the outputs, or the status
// where it is not DG_OK.
#include <Python.h>

#include <dlfcn.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "dg_fp8.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int64_t kBlock = 128;

[[noreturn]] void refuse(PyObject *type, const std::string &what)
{
    PyErr_SetString(type, what.c_str());
    throw python_error();
}

[[noreturn]] void bad_value(const std::string &what) { refuse(PyExc_ValueError, what); }
[[noreturn]] void bad_type(const std::string &what) { refuse(PyExc_TypeError, what); }

// Set by tests that call these functions with host tensors and an entry point of their own (this thread's calls).
thread_local bool t_any_device = false;
// The call's entry point is such a callback: code that no loaded file holds.
thread_local bool t_callback = false;

// An address that every entry point refuses as misaligned, before any launch.
void *const kNoAddress = reinterpret_cast<void *>(1);

Tensor tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        bad_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

Tensor optional(PyObject *o, const char *name) { return o == Py_None ? Tensor() : tensor(o, name); }

void *pointer(const Tensor &t, const char *name)
{
    if (t.is_cuda())
        return t.data_ptr();
    if (!t_any_device)
        bad_value(std::string(name) + " must be a device tensor");
    return t_callback ? t.data_ptr() : kNoAddress;  // a host address never reaches the library
}

// DG_DTYPE_F32 or DG_DTYPE_BF16 of a tensor of activations.
int float_type(const Tensor &t, const char *name)
{
    if (t.scalar_type() == ScalarType::Float)
        return DG_DTYPE_F32;
    if (t.scalar_type() != ScalarType::BFloat16)
        bad_type(std::string(name) + " must be float32 or bfloat16");
    return DG_DTYPE_BF16;
}

void need_type(const Tensor &t, const char *name, ScalarType type)
{
    if (t.scalar_type() != type)
        bad_type(std::string(name) + " must be " + c10::toString(type));
}

void need_codes(const Tensor &t, const char *name)
{
    if (t.scalar_type() != ScalarType::Byte && t.scalar_type() != ScalarType::Float8_e4m3fn)
        bad_type(std::string(name) + " must hold e4m3 codes (uint8 or float8_e4m3fn)");
}

// Row stride of a 2-D tensor with contiguous rows (a single row's own stride is free in torch).
int64_t rows(const Tensor &t, const char *name)
{
    if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
        bad_value(std::string(name) + " must be 2-D with contiguous rows");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

void need_shape(const Tensor &t, const char *name, at::IntArrayRef shape)
{
    if (t.sizes() != shape)
        bad_value(std::string("shape mismatch: ") + name);
}

void need_scales(const Tensor &t, const char *name, at::IntArrayRef shape)
{
    need_type(t, name, ScalarType::Float);
    if (t.sizes() != shape)
        bad_value(std::string("scale shape mismatch: ") + name);
}

Tensor make(const Tensor &like, at::IntArrayRef shape, at::IntArrayRef strides, ScalarType type)
{
    return at::empty_strided(shape, strides, like.options().dtype(type));
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return (float)v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}

void *address(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw python_error();
    return p;
}

// The entry point that a call's first argument holds.
template <typename Entry>
Entry entry_point(PyObject *o)
{
    void *const p = address(o);
    if (t_any_device) {
        Dl_info info;
        t_callback = dladdr(p, &info) == 0;
    }
    return reinterpret_cast<Entry>(p);
}

void need_arguments(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want)
        bad_type("takes " + std::to_string(want) + " arguments");
}

// The tensor itself where the caller gave it, else the new one; None where there is none.
PyObject *result(PyObject *given, const Tensor &t)
{
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

template <typename Call>
dg_status without_gil(Call call)
{
    dg_status st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    return st;
}

// rmsnorm_quantize(entry, x, weight, eps, residual, residual_out, normed, y, q, s, stream) -> (q, s, residual_out, y)
PyObject *rmsnorm_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_arguments(n, 11);
    const auto entry = entry_point<decltype(&dg_fp8_rmsnorm_quantize_1x128)>(a[0]);
    const Tensor x = tensor(a[1], "x"), w = tensor(a[2], "weight");
    const float eps = real(a[3]);
    const Tensor r = optional(a[4], "residual");
    Tensor ro = optional(a[5], "residual_out"), y = optional(a[7], "y"), q = optional(a[8], "q"),
           s = optional(a[9], "s");
    const bool normed = truth(a[6]);
    void *stream = address(a[10]);

    const int xt = float_type(x, "x"), wt = float_type(w, "weight");
    const int64_t ldx = rows(x, "x"), M = x.size(0), K = x.size(1), nkb = K / kBlock;
    int rt = 0;
    int64_t ldr = 0, ldro = 0, ldy = 0, ldq = K;
    if (w.dim() != 1 || w.size(0) != K || (w.stride(0) != 1 && K > 1))
        bad_value("weight must be a contiguous [K] tensor");
    if (r.defined()) {
        rt = float_type(r, "residual");
        ldr = rows(r, "residual");
        need_shape(r, "residual", x.sizes());
        ldro = K;
        if (ro.defined()) {
            need_type(ro, "residual_out", r.scalar_type());
            ldro = rows(ro, "residual_out");
            need_shape(ro, "residual_out", x.sizes());
        }
    } else if (ro.defined()) {
        bad_value("residual_out needs a residual");
    }
    if (y.defined()) {
        need_type(y, "y", ScalarType::BFloat16);
        ldy = rows(y, "y");
        need_shape(y, "y", x.sizes());
    }
    if (q.defined()) {
        need_codes(q, "q");
        ldq = rows(q, "q");
        need_shape(q, "q", x.sizes());
    }
    if (s.defined())
        need_scales(s, "s", {M, nkb});
    const void *xp = pointer(x, "x"), *wp = pointer(w, "weight"), *rp = r.defined() ? pointer(r, "residual") : nullptr;
    if (r.defined() && !ro.defined())
        ro = make(x, {M, K}, {K, 1}, r.scalar_type());
    if (normed && !y.defined()) {
        y = make(x, {M, K}, {K, 1}, ScalarType::BFloat16);
        ldy = K;
    }
    if (!q.defined())
        q = make(x, {M, K}, {K, 1}, ScalarType::Byte);
    if (!s.defined())
        s = make(x, {M, nkb}, {1, M}, ScalarType::Float);
    void *rop = ro.defined() ? pointer(ro, "residual_out") : nullptr, *yp = y.defined() ? pointer(y, "y") : nullptr;
    void *qp = pointer(q, "q"), *sp = pointer(s, "s");
    const int64_t s_m = s.stride(0), s_kb = s.stride(1);
    const dg_status st = without_gil([&] {
        return entry(xp, xt, ldx, rp, rt, ldr, rop, ldro, wp, wt, eps, yp, ldy, qp, ldq, (float *)sp, s_m, s_kb, M, K,
                     stream);
    });
    if (st != DG_OK)
        return PyLong_FromLong(st);
    return Py_BuildValue("(NNNN)", result(a[8], q), result(a[9], s), result(a[5], ro), result(a[7], y));
    END_HANDLE_TH_ERRORS
}

void need_slots(const Tensor &t, const char *name, ScalarType type, at::IntArrayRef shape)
{
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        bad_value(std::string(name) + " must be a contiguous " + c10::toString(type) + " [T, top_k] tensor");
}

// gate_topk(entry, logits, top_k, score, renormalize, factor, ids, weights, stream) -> (ids, weights)
PyObject *gate_topk(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_arguments(n, 9);
    const auto entry = entry_point<decltype(&dg_moe_gate_topk)>(a[0]);
    const Tensor logits = tensor(a[1], "logits");
    const int64_t top_k = integer(a[2]);
    const int score = (int)integer(a[3]), renormalize = truth(a[4]);
    const float factor = real(a[5]);
    Tensor ids = optional(a[6], "ids"), weights = optional(a[7], "weights");
    void *stream = address(a[8]);

    const int type = float_type(logits, "logits");
    const int64_t ldl = rows(logits, "logits"), T = logits.size(0), E = logits.size(1);
    if (top_k < 0 || top_k > E)  // before outputs of that size are made
        return PyLong_FromLong(DG_ERR_BAD_SHAPE);
    if (ids.defined())
        need_slots(ids, "ids", ScalarType::Int, {T, top_k});
    if (weights.defined())
        need_slots(weights, "weights", ScalarType::Float, {T, top_k});
    const void *lp = pointer(logits, "logits");
    if (!ids.defined())
        ids = make(logits, {T, top_k}, {top_k, 1}, ScalarType::Int);
    if (!weights.defined())
        weights = make(logits, {T, top_k}, {top_k, 1}, ScalarType::Float);
    int32_t *ip = (int32_t *)pointer(ids, "ids");
    float *wp = (float *)pointer(weights, "weights");
    const dg_status st = without_gil(
        [&] { return entry(lp, type, ldl, score, renormalize, factor, ip, wp, T, E, top_k, stream); });
    if (st != DG_OK)
        return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", result(a[6], ids), result(a[7], weights));
    END_HANDLE_TH_ERRORS
}

// moe_layer(entry, x, sx, w13, s13, w2, s2, topk_ids, topk_weights, workspace, out, stream) -> out
PyObject *moe_layer(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_arguments(n, 12);
    const auto entry = entry_point<decltype(&dg_fp8_moe_layer)>(a[0]);
    const Tensor x = tensor(a[1], "x"), sx = tensor(a[2], "sx"), w13 = tensor(a[3], "w13"), s13 = tensor(a[4], "s13"),
                 w2 = tensor(a[5], "w2"), s2 = tensor(a[6], "s2"), ids = tensor(a[7], "topk_ids"),
                 weights = tensor(a[8], "topk_weights"), ws = optional(a[9], "workspace");
    Tensor out = optional(a[10], "out");
    void *stream = address(a[11]);

    need_codes(x, "x");
    need_codes(w13, "w13");
    need_codes(w2, "w2");
    const int64_t ldx = rows(x, "x"), T = x.size(0), H = x.size(1);
    for (const Tensor *w : {&w13, &w2})
        if (w->dim() != 3 || w->stride(2) != 1)
            bad_value(std::string(w == &w13 ? "w13" : "w2") + " must be 3-D with a contiguous last dimension");
    const int64_t E = w13.size(0), I = w13.size(1) / 2;
    if (w13.size(1) % 2)
        bad_value("w13 must have an even number of rows for each expert");
    need_shape(w13, "w13", {E, 2 * I, H});
    need_shape(w2, "w2", {E, H, I});
    need_scales(sx, "sx", {T, H / kBlock});
    need_scales(s13, "s13", {E, 2 * I / kBlock, H / kBlock});
    need_scales(s2, "s2", {E, H / kBlock, I / kBlock});
    if (ids.dim() != 2)
        bad_value("topk_ids must be [T, top_k]");
    const int64_t top_k = ids.size(1);
    int64_t ldo = H;
    if (out.defined()) {
        need_type(out, "out", ScalarType::BFloat16);
        ldo = rows(out, "out");
        need_shape(out, "out", x.sizes());
    }
    need_slots(ids, "topk_ids", ScalarType::Int, {T, top_k});
    need_slots(weights, "topk_weights", ScalarType::Float, {T, top_k});
    const void *xp = pointer(x, "x"), *w13p = pointer(w13, "w13"), *w2p = pointer(w2, "w2");
    const float *sxp = (const float *)pointer(sx, "sx"), *s13p = (const float *)pointer(s13, "s13"),
                *s2p = (const float *)pointer(s2, "s2");
    const int32_t *ip = (const int32_t *)pointer(ids, "topk_ids");
    const float *wp = (const float *)pointer(weights, "topk_weights");
    void *wsp = nullptr;
    int64_t ws_bytes = 0;
    if (ws.defined() && ws.numel() > 0) {
        if (!ws.is_contiguous())
            bad_value("workspace must be a contiguous device tensor");
        wsp = pointer(ws, "workspace");
        ws_bytes = ws.numel() * ws.element_size();
    }
    if (!out.defined())
        out = make(x, {T, H}, {H, 1}, ScalarType::BFloat16);
    void *op = pointer(out, "out");
    const dg_status st = without_gil([&] {
        return entry(xp, ldx, sxp, sx.stride(0), sx.stride(1), w13p, w13.stride(1), w13.stride(0), s13p, s13.stride(0),
                     s13.stride(1), s13.stride(2), w2p, w2.stride(1), w2.stride(0), s2p, s2.stride(0), s2.stride(1),
                     s2.stride(2), ip, wp, op, ldo, T, top_k, E, H, I, wsp, ws_bytes, stream);
    });
    if (st != DG_OK)
        return PyLong_FromLong(st);
    return result(a[10], out);
    END_HANDLE_TH_ERRORS
}

PyObject *any_device(PyObject *, PyObject *on)
{
    HANDLE_TH_ERRORS
    t_any_device = truth(on);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyCFunction fast()
{
    return (PyCFunction)(void (*)())F;
}

PyMethodDef methods[] = {
    {"rmsnorm_quantize", fast<rmsnorm_quantize>(), METH_FASTCALL, nullptr},
    {"gate_topk", fast<gate_topk>(), METH_FASTCALL, nullptr},
    {"moe_layer", fast<moe_layer>(), METH_FASTCALL, nullptr},
    {"any_device", any_device, METH_O, "Tests only: this thread's calls take host tensors too."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
