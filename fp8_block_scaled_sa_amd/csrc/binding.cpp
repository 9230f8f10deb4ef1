// binding.cpp -- the host side of the serving step's calls (residual norm to
// codes, router top-k, expert layer, the paged cache's write, read and
// attention) between torch tensors and the C ABI of include/dg_fp8.h: checks of
// types and shapes, the outputs, the call.
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

#include <cmath>
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

// A cache from its codes [pages, page_size, heads, head_dim] and scales [pages, page_size, heads].
dg_fp8_cache cache_of(const Tensor &codes, const Tensor &scales, const char *name, const char *scales_name)
{
    need_codes(codes, name);
    if (codes.dim() != 4 || (codes.stride(3) != 1 && codes.size(3) > 1))
        bad_value(std::string(name) + " must be [pages, page_size, heads, head_dim] with a contiguous last dimension");
    need_scales(scales, scales_name, codes.sizes().slice(0, 3));
    return dg_fp8_cache{pointer(codes, name), codes.stride(0), codes.stride(1), codes.stride(2),
                        (float *)pointer(scales, scales_name), scales.stride(0), scales.stride(1), scales.stride(2),
                        codes.size(0), codes.size(1), codes.size(2), codes.size(3)};
}

// [T, heads, D] with contiguous heads.
void need_heads(const Tensor &t, const char *name)
{
    if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1))
        bad_value(std::string(name) + " must be [T, heads, head_dim] with a contiguous last dimension");
}

// A contiguous vector of so many elements.
void need_vector(const Tensor &t, const char *name, ScalarType type, int64_t size)
{
    need_type(t, name, type);
    if (t.dim() != 1 || t.size(0) != size || (t.stride(0) != 1 && size > 1))
        bad_value(std::string(name) + " must be a contiguous vector of " + std::to_string(size) + " elements");
}

// rope_cache_write(entry, k, v, k_cache, k_scales, v_cache, v_scales, slots, positions, freqs, q, interleaved, factor,
//                  q_out, stream) -> q_out
PyObject *rope_cache_write(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_arguments(n, 15);
    const auto entry = entry_point<decltype(&dg_fp8_rope_cache_write)>(a[0]);
    const Tensor k = tensor(a[1], "k"), v = tensor(a[2], "v"), kc = tensor(a[3], "k_cache"), ks = tensor(a[4], "k_scales"),
                 vc = tensor(a[5], "v_cache"), vs = tensor(a[6], "v_scales"), slots = tensor(a[7], "slots"),
                 positions = optional(a[8], "positions"), freqs = optional(a[9], "freqs"), q = optional(a[10], "q");
    const bool interleaved = truth(a[11]);
    const float factor = real(a[12]);
    Tensor qo = optional(a[13], "q_out");
    void *stream = address(a[14]);

    const int type = float_type(k, "k");
    need_heads(k, "k");
    need_type(v, "v", k.scalar_type());
    need_heads(v, "v");
    need_shape(v, "v", k.sizes());
    const int64_t T = k.size(0), heads = k.size(1), D = k.size(2);
    const dg_fp8_cache kcache = cache_of(kc, ks, "k_cache", "k_scales"), vcache = cache_of(vc, vs, "v_cache", "v_scales");
    need_shape(kc, "k_cache", {kc.size(0), kc.size(1), heads, D});
    need_shape(vc, "v_cache", kc.sizes());
    need_vector(slots, "slots", ScalarType::Long, T);
    int64_t rot = 0;
    if (freqs.defined()) {
        if (!positions.defined())
            bad_value("freqs needs positions");
        need_type(freqs, "freqs", ScalarType::Double);
        rot = 2 * freqs.numel();
        need_vector(freqs, "freqs", ScalarType::Double, rot / 2);
        need_vector(positions, "positions", ScalarType::Int, T);
    }
    int64_t q_heads = 0;
    if (q.defined()) {
        need_type(q, "q", k.scalar_type());
        need_heads(q, "q");
        q_heads = q.size(1);
        need_shape(q, "q", {T, q_heads, D});
        if (q_heads == 0)
            bad_value("q must have heads");
        if (qo.defined()) {
            need_type(qo, "q_out", ScalarType::BFloat16);
            need_heads(qo, "q_out");
            need_shape(qo, "q_out", q.sizes());
        }
    } else if (qo.defined()) {
        bad_value("q_out needs q");
    }
    const void *kp = pointer(k, "k"), *vp = pointer(v, "v"), *qp = q.defined() ? pointer(q, "q") : nullptr;
    const int64_t *sp = (const int64_t *)pointer(slots, "slots");
    const int32_t *pp = rot ? (const int32_t *)pointer(positions, "positions") : nullptr;
    const double *fp = rot ? (const double *)pointer(freqs, "freqs") : nullptr;
    if (q.defined() && !qo.defined())
        qo = make(q, {T, q_heads, D}, {q_heads * D, D, 1}, ScalarType::BFloat16);
    void *qop = q.defined() ? pointer(qo, "q_out") : nullptr;
    const int64_t q_t = q.defined() ? q.stride(0) : 0, q_h = q.defined() ? q.stride(1) : 0;
    const int64_t qo_t = q.defined() ? qo.stride(0) : 0, qo_h = q.defined() ? qo.stride(1) : 0;
    const dg_status st = without_gil([&] {
        return entry(qp, q_t, q_h, qop, qo_t, qo_h, q_heads, kp, k.stride(0), k.stride(1), vp, v.stride(0), v.stride(1),
                     type, pp, fp, rot, interleaved, factor, sp, &kcache, &vcache, T, stream);
    });
    if (st != DG_OK)
        return PyLong_FromLong(st);
    return result(a[13], qo);
    END_HANDLE_TH_ERRORS
}

// cache_read(entry, cache, scales, slots, bf16, out, stream) -> out
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_arguments(n, 7);
    const auto entry = entry_point<decltype(&dg_fp8_cache_read)>(a[0]);
    const Tensor codes = tensor(a[1], "cache"), scales = tensor(a[2], "scales"), slots = tensor(a[3], "slots");
    const bool bf16 = truth(a[4]);
    Tensor out = optional(a[5], "out");
    void *stream = address(a[6]);

    const dg_fp8_cache cache = cache_of(codes, scales, "cache", "scales");
    if (slots.dim() != 1)
        bad_value("slots must be a vector");
    const int64_t T = slots.size(0), heads = cache.heads, D = cache.head_dim;
    need_vector(slots, "slots", ScalarType::Long, T);
    if (out.defined()) {
        need_heads(out, "out");
        need_shape(out, "out", {T, heads, D});
    }
    const int64_t *sp = (const int64_t *)pointer(slots, "slots");
    if (!out.defined())
        out = make(codes, {T, heads, D}, {heads * D, D, 1}, bf16 ? ScalarType::BFloat16 : ScalarType::Float);
    const int type = float_type(out, "out");
    void *op = pointer(out, "out");
    const dg_status st =
        without_gil([&] { return entry(&cache, sp, op, type, out.stride(0), out.stride(1), T, stream); });
    if (st != DG_OK)
        return PyLong_FromLong(st);
    return result(a[5], out);
    END_HANDLE_TH_ERRORS
}

// paged_attention(entry, q, k_cache, k_scales, v_cache, v_scales, block_table, kv_lens, q_starts, max_q_len, workspace,
//                 scale, window, out, stream) -> out
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    need_arguments(n, 15);
    const auto entry = entry_point<decltype(&dg_fp8_paged_attention)>(a[0]);
    const Tensor q = tensor(a[1], "q"), kc = tensor(a[2], "k_cache"), ks = tensor(a[3], "k_scales"),
                 vc = tensor(a[4], "v_cache"), vs = tensor(a[5], "v_scales"), table = tensor(a[6], "block_table"),
                 lens = tensor(a[7], "kv_lens"), starts = tensor(a[8], "q_starts");
    const int64_t max_q_len = integer(a[9]);
    const Tensor ws = optional(a[10], "workspace");
    const int64_t window = integer(a[12]);
    Tensor out = optional(a[13], "out");
    void *stream = address(a[14]);

    need_type(q, "q", ScalarType::BFloat16);
    need_heads(q, "q");
    const int64_t T = q.size(0), q_heads = q.size(1), D = q.size(2);
    const float scale = a[11] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : real(a[11]);
    const dg_fp8_cache kcache = cache_of(kc, ks, "k_cache", "k_scales"), vcache = cache_of(vc, vs, "v_cache", "v_scales");
    need_shape(kc, "k_cache", {kc.size(0), kc.size(1), kc.size(2), D});
    need_shape(vc, "v_cache", kc.sizes());
    need_type(table, "block_table", ScalarType::Int);
    if (table.dim() != 2 || (table.stride(1) != 1 && table.size(1) > 1))
        bad_value("block_table must be [B, pages of a sequence] with contiguous rows");
    const int64_t B = table.size(0), width = table.size(1);
    need_vector(lens, "kv_lens", ScalarType::Int, B);
    need_vector(starts, "q_starts", ScalarType::Int, B + 1);
    if (out.defined()) {
        need_type(out, "out", ScalarType::BFloat16);
        need_heads(out, "out");
        need_shape(out, "out", q.sizes());
    }
    const void *qp = pointer(q, "q");
    const int32_t *tp = (const int32_t *)pointer(table, "block_table"), *lp = (const int32_t *)pointer(lens, "kv_lens"),
                  *stp = (const int32_t *)pointer(starts, "q_starts");
    void *wsp = nullptr;
    int64_t ws_bytes = 0;
    if (ws.defined() && ws.numel() > 0) {
        if (!ws.is_contiguous())
            bad_value("workspace must be a contiguous device tensor");
        wsp = pointer(ws, "workspace");
        ws_bytes = ws.numel() * ws.element_size();
    }
    if (!out.defined())
        out = make(q, {T, q_heads, D}, {q_heads * D, D, 1}, ScalarType::BFloat16);
    void *op = pointer(out, "out");
    const int64_t table_stride = B > 1 ? table.stride(0) : width;
    const dg_status st = without_gil([&] {
        return entry(qp, q.stride(0), q.stride(1), q_heads, &kcache, &vcache, tp, table_stride, width, lp, stp, B, T,
                     max_q_len, scale, window, op, out.stride(0), out.stride(1), wsp, ws_bytes, stream);
    });
    if (st != DG_OK)
        return PyLong_FromLong(st);
    return result(a[13], out);
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
    {"rope_cache_write", fast<rope_cache_write>(), METH_FASTCALL, nullptr},
    {"cache_read", fast<cache_read>(), METH_FASTCALL, nullptr},
    {"paged_attention", fast<paged_attention>(), METH_FASTCALL, nullptr},
    {"any_device", any_device, METH_O, "Tests only: this thread's calls take host tensors too."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
