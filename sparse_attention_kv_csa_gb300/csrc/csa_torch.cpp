// The helpers' short way from Python to the entry points of csa_serving.h: one call checks the tensors, allocates the
// outputs and calls the library.  It takes the ordinary case only (contiguous tensors of the right types and shapes on
// the current device, the current stream); for anything else it returns None and the Python helper, whose checks are
// complete, takes over.  Marshalling in Python costs some 8 us of a call whose kernel takes 2.5.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "csa_serving.h"

namespace {

struct Entry {
    decltype(&csa_rms_norm_fwd) norm_fwd;
    decltype(&csa_rms_norm_bwd) norm_bwd;
    decltype(&csa_page_tables) pages;
    decltype(&csa_latent_attention) attention;
    decltype(&csa_layer_norm_fwd) layer_fwd;
    decltype(&csa_layer_norm_bwd) layer_bwd;
    decltype(&csa_append_rows) append;
    decltype(&csa_rotate) rotate;
    decltype(&csa_shared_attention) shared;
} g_entry;

int dtype_code(at::ScalarType t)
{
    return t == at::kBFloat16 ? CSA_DTYPE_BF16 : t == at::kHalf ? CSA_DTYPE_F16 : t == at::kFloat ? CSA_DTYPE_F32
           : t == at::kFloat8_e4m3fn ? CSA_DTYPE_E4M3 : -1;
}

// The current device, if the first argument is a tensor on it (asked in this order: without a GPU there is no current
// device to ask for).
bool device_of(PyObject *o, c10::DeviceIndex *d)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        return false;
    *d = THPVariable_Unpack(o).device().index();
    return *d == c10::cuda::current_device();
}

// An argument that is None or a tensor that the short way takes.
struct Arg {
    const at::Tensor *t = nullptr;
    bool ok = true;
    // strided: rows of any stride whose last dimension is contiguous do too
    Arg(PyObject *o, c10::DeviceIndex device, bool strided = false)
    {
        if (o == Py_None)
            return;
        if (!THPVariable_Check(o)) {
            ok = false;
            return;
        }
        t = &THPVariable_Unpack(o);
        ok = t->is_cuda() && t->device().index() == device && t->layout() == at::kStrided &&
             (t->is_contiguous() || (strided && t->dim() > 0 && (t->size(t->dim() - 1) <= 1 || t->stride(t->dim() - 1) == 1)));
    }
    bool none() const { return ok && !t; }
    bool is(at::ScalarType s, int64_t dim) const { return ok && t && t->scalar_type() == s && t->dim() == dim; }
    int64_t size(int i) const { return t->size(i); }
    // (of a dimension of one element any stride is right: the least that the entry points take)
    int64_t stride(int i, int64_t least) const { return t->size(i) > 1 ? t->stride(i) : std::max(t->stride(i), least); }
    template <typename T = void> T *ptr() const { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }
};

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::DeviceIndex device)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, device));
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

PyObject *own(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

void *stream_of(c10::DeviceIndex device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

bool number(PyObject *o, int64_t *v)
{
    if (!PyLong_CheckExact(o))
        return false;
    *v = PyLong_AsLongLong(o);
    if (*v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}

bool number(PyObject *o, int32_t *v)
{
    int64_t w;
    if (!number(o, &w) || w != (int32_t)w)
        return false;
    *v = (int32_t)w;
    return true;
}

bool number(PyObject *o, double *v)
{
    if (!PyFloat_CheckExact(o))
        return false;
    *v = PyFloat_AS_DOUBLE(o);
    return true;
}

// A status becomes a Python int, which the helper raises; otherwise the tuple of results.
PyObject *status(int rc) { return PyLong_FromLong(rc); }

#define CSA_ORDINARY(cond)     \
    do {                       \
        if (!(cond))           \
            Py_RETURN_NONE;    \
    } while (0)

// (x, weight, eps, residual, bits8, scale_group, slots, out, scales)
PyObject *norm_forward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    c10::DeviceIndex d;
    CSA_ORDINARY(n_args == 9 && device_of(a[0], &d));
    const Arg x(a[0], d), w(a[1], d), res(a[3], d), slots(a[6], d), out(a[7], d), scales(a[8], d);
    double eps;
    int32_t group;
    CSA_ORDINARY(x.ok && !x.none() && x.t->dim() == 2 && number(a[2], &eps) && number(a[5], &group));
    const at::ScalarType type = x.t->scalar_type();
    const int code = dtype_code(type);
    const int64_t n = x.size(0), dim = x.size(1);
    const bool bits8 = a[4] == Py_True;
    CSA_ORDINARY(code >= 0 && code != CSA_DTYPE_E4M3 && dim < (1 << 30) && (group == 0 || (group == 128 && bits8 && dim % 128 == 0)));
    CSA_ORDINARY(w.none() || (w.is(at::kFloat, 1) && w.size(0) == dim));
    CSA_ORDINARY(res.none() || (res.is(type, 2) && res.size(0) == n && res.size(1) == dim));
    CSA_ORDINARY(slots.none() || (slots.is(at::kLong, 1) && slots.size(0) == n && !out.none() && (!bits8 || !scales.none())));
    const at::ScalarType out_type = bits8 ? at::kFloat8_e4m3fn : type;
    const int64_t groups = group ? dim / 128 : 1;
    CSA_ORDINARY(out.none() || (out.is(out_type, 2) && out.size(1) == dim && (!slots.none() || out.size(0) == n)));
    const int64_t rows = out.none() ? n : out.size(0);
    if (!scales.none())
        CSA_ORDINARY(bits8 && ((scales.is(at::kFloat, 2) && scales.size(0) == rows && scales.size(1) == groups) ||
                               (scales.is(at::kFloat, 1) && scales.size(0) == rows && groups == 1)));
    at::Tensor o, s, total, rstd = empty({n}, at::kFloat, d);
    if (out.none())
        o = empty({n, dim}, out_type, d);
    if (bits8 && scales.none())
        s = empty({n, groups}, at::kFloat, d);
    if (!res.none())
        total = empty({n, dim}, type, d);
    const int rc = g_entry.norm_fwd(x.ptr(), dim, res.ptr(), dim, w.ptr<float>(), n, (int32_t)dim, (float)eps, code,
                                    slots.ptr<int64_t>(), rows, out.none() ? o.data_ptr() : out.ptr(), dim,
                                    bits8 ? CSA_DTYPE_E4M3 : code,
                                    !bits8 ? nullptr : scales.none() ? static_cast<float *>(s.data_ptr()) : scales.ptr<float>(),
                                    group, total.defined() ? total.data_ptr() : nullptr, static_cast<float *>(rstd.data_ptr()),
                                    stream_of(d));
    if (rc)
        return status(rc);
    PyObject *r = PyTuple_New(4);
    PyTuple_SET_ITEM(r, 0, out.none() ? wrap(o) : own(a[7]));
    PyTuple_SET_ITEM(r, 1, !bits8 ? own(Py_None) : scales.none() ? wrap(s) : own(a[8]));
    PyTuple_SET_ITEM(r, 2, total.defined() ? wrap(total) : own(Py_None));
    PyTuple_SET_ITEM(r, 3, wrap(rstd));
    return r;
    END_HANDLE_TH_ERRORS
}

// (grad_out, h, weight, rstd, grad_residual)
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    c10::DeviceIndex d;
    CSA_ORDINARY(n_args == 5 && device_of(a[0], &d));
    const Arg g(a[0], d), h(a[1], d), w(a[2], d), rstd(a[3], d), res(a[4], d);
    CSA_ORDINARY(h.ok && !h.none() && h.t->dim() == 2);
    const at::ScalarType type = h.t->scalar_type();
    const int code = dtype_code(type);
    const int64_t n = h.size(0), dim = h.size(1);
    CSA_ORDINARY(code >= 0 && code != CSA_DTYPE_E4M3 && dim < (1 << 30));
    CSA_ORDINARY(g.is(type, 2) && g.size(0) == n && g.size(1) == dim && rstd.is(at::kFloat, 1) && rstd.size(0) == n);
    CSA_ORDINARY(w.none() || (w.is(at::kFloat, 1) && w.size(0) == dim));
    CSA_ORDINARY(res.none() || (res.is(type, 2) && res.size(0) == n && res.size(1) == dim));
    const at::Tensor dx = empty({n, dim}, type, d), dw = empty({dim}, at::kFloat, d);
    const int rc = g_entry.norm_bwd(h.ptr(), dim, g.ptr(), dim, res.ptr(), dim, w.ptr<float>(), rstd.ptr<float>(), n, (int32_t)dim,
                                    code, dx.data_ptr(), static_cast<float *>(dw.data_ptr()), stream_of(d));
    if (rc)
        return status(rc);
    PyObject *r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, wrap(dx));
    PyTuple_SET_ITEM(r, 1, wrap(dw));
    return r;
    END_HANDLE_TH_ERRORS
}

// (before, after, ratio, page_size, free_pages, block_table, capacity, taken, out)
PyObject *page_tables(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    c10::DeviceIndex d;
    CSA_ORDINARY(n_args == 9 && device_of(a[0], &d));
    const Arg before(a[0], d), after(a[1], d), free_pages(a[4], d), table(a[5], d), taken(a[7], d), out(a[8], d);
    int32_t ratio, page;
    int64_t capacity;
    CSA_ORDINARY(number(a[2], &ratio) && number(a[3], &page) && number(a[6], &capacity) && capacity >= 0);
    CSA_ORDINARY(before.is(at::kInt, 1) && after.is(at::kInt, 1) && free_pages.is(at::kInt, 1) && table.is(at::kInt, 2));
    const int64_t n = before.size(0), width = table.size(1), n_free = free_pages.size(0);
    CSA_ORDINARY(after.size(0) == n && table.size(0) == n && n < (1 << 30) && width < (1 << 30) && n_free < (1 << 30));
    CSA_ORDINARY(taken.none() || (taken.is(at::kInt, 1) && taken.size(0) == 1));
    CSA_ORDINARY(out.none() || (out.is(at::kInt, 2) && out.size(0) == n && out.size(1) == width));
    at::Tensor o;
    if (out.none())
        o = empty({n, width}, at::kInt, d);
    const at::Tensor cu = empty({n + 1}, at::kInt, d), slots = empty({capacity}, at::kLong, d), counts = empty({4}, at::kInt, d);
    const int rc = g_entry.pages(before.ptr<int32_t>(), after.ptr<int32_t>(), (int32_t)n, ratio, page, free_pages.ptr<int32_t>(),
                                 (int32_t)n_free, taken.ptr<int32_t>(), table.ptr<int32_t>(), width, (int32_t)width, capacity,
                                 out.none() ? static_cast<int32_t *>(o.data_ptr()) : out.ptr<int32_t>(),
                                 static_cast<int32_t *>(cu.data_ptr()), static_cast<int64_t *>(slots.data_ptr()),
                                 static_cast<int32_t *>(counts.data_ptr()), stream_of(d));
    if (rc)
        return status(rc);
    PyObject *r = PyTuple_New(4);
    PyTuple_SET_ITEM(r, 0, out.none() ? wrap(o) : own(a[8]));
    PyTuple_SET_ITEM(r, 1, wrap(cu));
    PyTuple_SET_ITEM(r, 2, wrap(slots));
    PyTuple_SET_ITEM(r, 3, wrap(counts));
    return r;
    END_HANDLE_TH_ERRORS
}

// (q, cache, block_table, cu_q, seq_lens, ratio, scale, v_dim, row_scales, sink, out); groups: cu_groups and shared_rows, or NULL
PyObject *attend(PyObject *const *a, PyObject *const *groups)
{
    c10::DeviceIndex d;
    CSA_ORDINARY(device_of(a[0], &d));
    const Arg q(a[0], d), cache(a[1], d), table(a[2], d), cu(a[3], d), lens(a[4], d), scales(a[8], d), sink(a[9], d), out(a[10], d);
    int32_t ratio, v_dim = -1;
    double scale;
    CSA_ORDINARY(number(a[5], &ratio) && number(a[6], &scale) && (a[7] == Py_None || (number(a[7], &v_dim) && v_dim > 0)));
    CSA_ORDINARY(q.is(at::kBFloat16, 3) && cache.ok && !cache.none() && cache.t->dim() == 3);
    const bool bits8 = cache.t->scalar_type() == at::kFloat8_e4m3fn;
    const int64_t n = q.size(0), heads = q.size(1), dim = q.size(2), pages = cache.size(0), page = cache.size(1);
    CSA_ORDINARY((bits8 || cache.t->scalar_type() == at::kBFloat16) && cache.size(2) == dim && page >= 1);
    CSA_ORDINARY(heads < (1 << 30) && dim < (1 << 30) && page < (1 << 30));
    CSA_ORDINARY(bits8 ? scales.is(at::kFloat, 2) && scales.size(0) == pages && scales.size(1) == page : scales.none());
    CSA_ORDINARY(cu.is(at::kInt, 1) && cu.size(0) >= 1 && lens.is(at::kInt, 1) && table.is(at::kInt, 2));
    const int64_t n_req = cu.size(0) - 1, width = table.size(1);
    CSA_ORDINARY(lens.size(0) == n_req && table.size(0) == n_req && n_req < (1 << 30) && width < (1 << 30));
    CSA_ORDINARY(sink.none() || (sink.is(at::kFloat, 1) && sink.size(0) == heads));
    const Arg cu_groups(groups ? groups[0] : Py_None, d), shared(groups ? groups[1] : Py_None, d);
    if (groups)
        CSA_ORDINARY(cu_groups.is(at::kInt, 1) && cu_groups.size(0) >= 1 && shared.is(at::kInt, 1) &&
                     shared.size(0) == cu_groups.size(0) - 1 && shared.size(0) < (1 << 30));
    const int64_t v = v_dim < 0 ? dim : v_dim;
    CSA_ORDINARY(out.none() || (out.is(at::kBFloat16, 3) && out.size(0) == n && out.size(1) == heads && out.size(2) == v));
    at::Tensor o;
    if (out.none())
        o = empty({n, heads, v}, at::kBFloat16, d);
    const at::Tensor lse = empty({n, heads}, at::kFloat, d);
    void *const result = out.none() ? o.data_ptr() : out.ptr();
    float *const sums = static_cast<float *>(lse.data_ptr());
    const int kind = bits8 ? CSA_DTYPE_E4M3 : CSA_DTYPE_BF16;
    const int rc =
        groups ? g_entry.shared(q.ptr(), heads * dim, dim, cu.ptr<int32_t>(), (int32_t)n_req, n, (int32_t)heads, (int32_t)dim, (int32_t)v,
                                cache.ptr(), dim, kind, scales.ptr<float>(), pages, (int32_t)page, table.ptr<int32_t>(), width,
                                (int32_t)width, lens.ptr<int32_t>(), cu_groups.ptr<int32_t>(), shared.ptr<int32_t>(),
                                (int32_t)shared.size(0), ratio, (float)scale, sink.ptr<float>(), result, sums, stream_of(d))
               : g_entry.attention(q.ptr(), heads * dim, dim, cu.ptr<int32_t>(), (int32_t)n_req, n, (int32_t)heads, (int32_t)dim,
                                   (int32_t)v, cache.ptr(), dim, kind, scales.ptr<float>(), pages, (int32_t)page, table.ptr<int32_t>(),
                                   width, (int32_t)width, lens.ptr<int32_t>(), ratio, (float)scale, sink.ptr<float>(), result, sums,
                                   stream_of(d));
    if (rc)
        return status(rc);
    PyObject *r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, out.none() ? wrap(o) : own(a[10]));
    PyTuple_SET_ITEM(r, 1, wrap(lse));
    return r;
}

PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    CSA_ORDINARY(n_args == 11);
    return attend(a, nullptr);
    END_HANDLE_TH_ERRORS
}

// (q, cache, block_table, cu_q, seq_lens, cu_groups, shared_rows, ratio, scale, v_dim, row_scales, sink, out)
PyObject *shared_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    CSA_ORDINARY(n_args == 13);
    PyObject *const plain[11] = {a[0], a[1], a[2], a[3], a[4], a[7], a[8], a[9], a[10], a[11], a[12]};
    return attend(plain, a + 5);
    END_HANDLE_TH_ERRORS
}

// (x, weight, bias, eps, residual, out)
PyObject *layer_forward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    c10::DeviceIndex d;
    CSA_ORDINARY(n_args == 6 && device_of(a[0], &d));
    const Arg x(a[0], d), w(a[1], d), b(a[2], d), res(a[4], d), out(a[5], d);
    double eps;
    CSA_ORDINARY(x.ok && !x.none() && x.t->dim() == 2 && number(a[3], &eps));
    const at::ScalarType type = x.t->scalar_type();
    const int code = dtype_code(type);
    const int64_t n = x.size(0), dim = x.size(1);
    CSA_ORDINARY(code >= 0 && code != CSA_DTYPE_E4M3 && dim < (1 << 30));
    CSA_ORDINARY(w.none() || (w.is(at::kFloat, 1) && w.size(0) == dim));
    CSA_ORDINARY(b.none() || (b.is(at::kFloat, 1) && b.size(0) == dim));
    CSA_ORDINARY(res.none() || (res.is(type, 2) && res.size(0) == n && res.size(1) == dim));
    CSA_ORDINARY(out.none() || (out.is(type, 2) && out.size(0) == n && out.size(1) == dim));
    at::Tensor o, total;
    const at::Tensor mean = empty({n}, at::kFloat, d), rstd = empty({n}, at::kFloat, d);
    if (out.none())
        o = empty({n, dim}, type, d);
    if (!res.none())
        total = empty({n, dim}, type, d);
    const int rc = g_entry.layer_fwd(x.ptr(), dim, res.ptr(), dim, w.ptr<float>(), b.ptr<float>(), n, (int32_t)dim, (float)eps, code,
                                     out.none() ? o.data_ptr() : out.ptr(), dim, total.defined() ? total.data_ptr() : nullptr,
                                     static_cast<float *>(mean.data_ptr()), static_cast<float *>(rstd.data_ptr()), stream_of(d));
    if (rc)
        return status(rc);
    PyObject *r = PyTuple_New(4);
    PyTuple_SET_ITEM(r, 0, out.none() ? wrap(o) : own(a[5]));
    PyTuple_SET_ITEM(r, 1, total.defined() ? wrap(total) : own(Py_None));
    PyTuple_SET_ITEM(r, 2, wrap(mean));
    PyTuple_SET_ITEM(r, 3, wrap(rstd));
    return r;
    END_HANDLE_TH_ERRORS
}

// (grad_out, h, weight, mean, rstd, grad_residual)
PyObject *layer_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    c10::DeviceIndex d;
    CSA_ORDINARY(n_args == 6 && device_of(a[0], &d));
    const Arg g(a[0], d), h(a[1], d), w(a[2], d), mean(a[3], d), rstd(a[4], d), res(a[5], d);
    CSA_ORDINARY(h.ok && !h.none() && h.t->dim() == 2);
    const at::ScalarType type = h.t->scalar_type();
    const int code = dtype_code(type);
    const int64_t n = h.size(0), dim = h.size(1);
    CSA_ORDINARY(code >= 0 && code != CSA_DTYPE_E4M3 && dim < (1 << 30));
    CSA_ORDINARY(g.is(type, 2) && g.size(0) == n && g.size(1) == dim && rstd.is(at::kFloat, 1) && rstd.size(0) == n);
    CSA_ORDINARY(mean.is(at::kFloat, 1) && mean.size(0) == n && (w.none() || (w.is(at::kFloat, 1) && w.size(0) == dim)));
    CSA_ORDINARY(res.none() || (res.is(type, 2) && res.size(0) == n && res.size(1) == dim));
    const at::Tensor dx = empty({n, dim}, type, d), dw = empty({dim}, at::kFloat, d), db = empty({dim}, at::kFloat, d);
    const int rc = g_entry.layer_bwd(h.ptr(), dim, g.ptr(), dim, res.ptr(), dim, w.ptr<float>(), mean.ptr<float>(), rstd.ptr<float>(), n,
                                     (int32_t)dim, code, dx.data_ptr(), static_cast<float *>(dw.data_ptr()),
                                     static_cast<float *>(db.data_ptr()), stream_of(d));
    if (rc)
        return status(rc);
    PyObject *r = PyTuple_New(3);
    PyTuple_SET_ITEM(r, 0, wrap(dx));
    PyTuple_SET_ITEM(r, 1, wrap(dw));
    PyTuple_SET_ITEM(r, 2, wrap(db));
    return r;
    END_HANDLE_TH_ERRORS
}

// (rows, positions, rotation, slots, out, scales, rotary, interleaved, queries, query_positions, query_out)
PyObject *append_rows(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    c10::DeviceIndex d;
    CSA_ORDINARY(n_args == 11 && device_of(a[0], &d));
    const Arg rows(a[0], d, true), positions(a[1], d), rotation(a[2], d), slots(a[3], d), out(a[4], d, true), scales(a[5], d),
        rotary(a[6], d, true), q(a[8], d, true), q_positions(a[9], d), q_out(a[10], d, true);
    CSA_ORDINARY(rows.ok && !rows.none() && rows.t->dim() == 2 && (a[7] == Py_True || a[7] == Py_False));
    const at::ScalarType type = rows.t->scalar_type();
    const int code = dtype_code(type);
    const int64_t n = rows.size(0), row_dim = rows.size(1);
    CSA_ORDINARY(code >= 0 && code != CSA_DTYPE_E4M3 && row_dim < (1 << 30));
    CSA_ORDINARY(positions.is(at::kInt, 1) && positions.size(0) == n && slots.is(at::kLong, 1) && slots.size(0) == n);
    CSA_ORDINARY(rotation.is(at::kFloat, 2) && rotation.size(1) < (1 << 30));
    const int64_t rot = rotation.size(1);
    CSA_ORDINARY(rotary.none() || (rotary.is(type, 2) && rotary.size(0) == n && rotary.size(1) == rot));
    const int64_t width = row_dim + (rotary.none() ? 0 : rot);
    CSA_ORDINARY(out.ok && !out.none() && out.t->dim() == 2 && out.size(1) == width);
    const bool bits8 = out.t->scalar_type() == at::kFloat8_e4m3fn;
    CSA_ORDINARY(bits8 ? scales.is(at::kFloat, 1) && scales.size(0) == out.size(0) : out.t->scalar_type() == type && scales.none());
    at::Tensor o;
    int64_t tokens = 0, heads = 1, out_token = 0, out_head = 0;
    const Arg &at = q_positions.none() ? positions : q_positions;
    if (q.none()) {
        CSA_ORDINARY(a[9] == Py_None && a[10] == Py_None);
    } else {
        CSA_ORDINARY(q.is(type, 3) && q.size(2) == rot && q.size(1) > 0 && q.size(1) < (1 << 30));
        tokens = q.size(0);
        heads = q.size(1);
        CSA_ORDINARY(at.is(at::kInt, 1) && at.size(0) == tokens);
        CSA_ORDINARY(q_out.none() || (q_out.is(type, 3) && q_out.size(0) == tokens && q_out.size(1) == heads && q_out.size(2) == rot));
        if (q_out.none())
            o = empty({tokens, heads, rot}, type, d);
        out_token = q_out.none() ? heads * rot : q_out.stride(0, rot);
        out_head = q_out.none() ? rot : q_out.stride(1, rot);
    }
    const int rc = g_entry.append(rows.ptr(), rows.stride(0, row_dim), (int32_t)row_dim, rotary.ptr(), rotary.none() ? 0 : rotary.stride(0, rot),
                                  (int32_t)rot, positions.ptr<int32_t>(), n, code, rotation.ptr<float>(), rotation.size(0), a[7] == Py_True,
                                  slots.ptr<int64_t>(), out.size(0), out.ptr(), out.stride(0, width), bits8 ? CSA_DTYPE_E4M3 : code,
                                  scales.ptr<float>(), q.ptr(), q.none() ? 0 : q.stride(0, rot), q.none() ? 0 : q.stride(1, rot),
                                  q.none() ? nullptr : at.ptr<int32_t>(), tokens, (int32_t)heads, o.defined() ? o.data_ptr() : q_out.ptr(),
                                  out_token, out_head, stream_of(d));
    if (rc)
        return status(rc);
    PyObject *r = PyTuple_New(3);
    PyTuple_SET_ITEM(r, 0, own(a[4]));
    PyTuple_SET_ITEM(r, 1, own(a[5]));
    PyTuple_SET_ITEM(r, 2, o.defined() ? wrap(o) : own(a[10]));
    return r;
    END_HANDLE_TH_ERRORS
}

// (x, positions, rotation, interleaved, inverse, out)
PyObject *rotate(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    c10::DeviceIndex d;
    CSA_ORDINARY(n_args == 6 && device_of(a[0], &d));
    const Arg x(a[0], d, true), positions(a[1], d), rotation(a[2], d), out(a[5], d, true);
    CSA_ORDINARY(x.ok && !x.none() && x.t->dim() == 3 && (a[3] == Py_True || a[3] == Py_False) && (a[4] == Py_True || a[4] == Py_False));
    const at::ScalarType type = x.t->scalar_type();
    const int code = dtype_code(type);
    const int64_t n = x.size(0), heads = x.size(1), rot = x.size(2);
    CSA_ORDINARY(code >= 0 && code != CSA_DTYPE_E4M3 && heads > 0 && heads < (1 << 30) && rot < (1 << 30));
    CSA_ORDINARY(positions.is(at::kInt, 1) && positions.size(0) == n && rotation.is(at::kFloat, 2) && rotation.size(1) == rot);
    CSA_ORDINARY(out.none() || (out.is(type, 3) && out.size(0) == n && out.size(1) == heads && out.size(2) == rot));
    at::Tensor o;
    if (out.none())
        o = empty({n, heads, rot}, type, d);
    const int rc = g_entry.rotate(x.ptr(), x.stride(0, rot), x.stride(1, rot), positions.ptr<int32_t>(), n, (int32_t)heads, (int32_t)rot, code,
                                  rotation.ptr<float>(), rotation.size(0), a[3] == Py_True, a[4] == Py_True,
                                  out.none() ? o.data_ptr() : out.ptr(), out.none() ? heads * rot : out.stride(0, rot),
                                  out.none() ? rot : out.stride(1, rot), stream_of(d));
    if (rc)
        return status(rc);
    return out.none() ? wrap(o) : own(a[5]);
    END_HANDLE_TH_ERRORS
}

// The entry points' addresses in the loaded libcsa, in Entry's order.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    constexpr int kEntries = 9;
    static_assert(sizeof(Entry) == kEntries * sizeof(void *), "");
    void *p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = n_args == kEntries ? PyLong_AsVoidPtr(a[i]) : nullptr;
        if (!p[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "bind takes nine addresses");
            return nullptr;
        }
    }
    g_entry = {reinterpret_cast<decltype(g_entry.norm_fwd)>(p[0]),  reinterpret_cast<decltype(g_entry.norm_bwd)>(p[1]),
               reinterpret_cast<decltype(g_entry.pages)>(p[2]),     reinterpret_cast<decltype(g_entry.attention)>(p[3]),
               reinterpret_cast<decltype(g_entry.layer_fwd)>(p[4]), reinterpret_cast<decltype(g_entry.layer_bwd)>(p[5]),
               reinterpret_cast<decltype(g_entry.append)>(p[6]),    reinterpret_cast<decltype(g_entry.rotate)>(p[7]),
               reinterpret_cast<decltype(g_entry.shared)>(p[8])};
    Py_RETURN_NONE;
}

#define CSA_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CSA_METHOD("bind", bind),
                           CSA_METHOD("rms_norm_forward", norm_forward),
                           CSA_METHOD("rms_norm_backward", norm_backward),
                           CSA_METHOD("page_tables", page_tables),
                           CSA_METHOD("latent_attention", attention),
                           CSA_METHOD("layer_norm_forward", layer_forward),
                           CSA_METHOD("layer_norm_backward", layer_backward),
                           CSA_METHOD("append_rows", append_rows),
                           CSA_METHOD("rotate", rotate),
                           CSA_METHOD("shared_attention", shared_attention),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "csa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_csa_torch() { return PyModule_Create(&g_module); }
