// Python entry of the paged serving operators: argument checks, output and workspace allocation
// on the current stream, and the call of the C ABI (include/infini_attn.h).  A step of a few
// microseconds on the GPU is issued by Python; checks written there cost more than the step.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>

#include "infini_attn.h"

namespace {

PyObject *g_error = nullptr;      // InfiniError(status, message)

using Dims = std::initializer_list<int64_t>;
constexpr auto kI32 = at::kInt, kI64 = at::kLong, kF32 = at::kFloat, kF64 = at::kDouble;

// A Python ValueError on its way out (Python's error is set).
struct Refused {};

[[noreturn]] void refuse(const std::string &what)
{
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Refused{};
}

std::string text(at::IntArrayRef s)
{
    std::ostringstream o;
    o << '(';
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

// The call's device: that of its first tensor, made current for the call.
struct Call {
    int dev;
    std::optional<c10::cuda::CUDAGuard> guard;
    infini_stream_t stream;

    Call(PyObject *o, const char *name)
    {
        const at::Tensor &t = tensor(o, name);
        if (!t.is_cuda()) refuse("the tensors must be on a CUDA device");
        dev = t.get_device();
        if (dev != c10::cuda::current_device()) guard.emplace(static_cast<c10::DeviceIndex>(dev));
        stream = reinterpret_cast<infini_stream_t>(
            c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    }

    void on_device(const at::Tensor &t, const char *name) const
    {
        if (!t.is_cuda() || t.get_device() != dev)
            refuse(std::string(name) + " must be a CUDA tensor on cuda:" + std::to_string(dev));
    }

    // The address of a contiguous tensor of this type and shape; None is null.
    template <typename T = void>
    T *at(PyObject *o, const char *name, at::ScalarType dt, at::IntArrayRef dims) const
    {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o, name);
        on_device(t, name);
        if (t.scalar_type() != dt || !t.sizes().equals(dims) || !t.is_contiguous())
            refuse(std::string(name) + ": expected contiguous " + c10::toString(dt) + " " + text(dims) + ", got " +
                   c10::toString(t.scalar_type()) + " " + text(t.sizes()) +
                   (t.is_contiguous() ? "" : ", not contiguous"));
        return static_cast<T *>(t.data_ptr());
    }

    // A [B, H, L, d] view with contiguous rows: its address, and its element strides (batch, head,
    // token) in `s` unless it is contiguous (null).
    const void *rows(PyObject *o, const char *name, at::ScalarType dt, at::IntArrayRef dims, int64_t (&s)[3],
                     const int64_t *&strides) const
    {
        const at::Tensor &t = tensor(o, name);
        on_device(t, name);
        if (t.scalar_type() != dt || !t.sizes().equals(dims) || (dims[3] > 1 && t.stride(3) != 1))
            refuse(std::string(name) + ": expected " + c10::toString(dt) + " " + text(dims) +
                   " with contiguous rows, got " + c10::toString(t.scalar_type()) + " " + text(t.sizes()) +
                   ", strides " + text(t.strides()));
        strides = nullptr;
        if (!t.is_contiguous()) {
            // a dimension of one entry may carry any stride: name the contiguous one
            s[0] = dims[0] > 1 ? t.stride(0) : dims[1] * dims[2] * dims[3];
            s[1] = dims[1] > 1 ? t.stride(1) : dims[2] * dims[3];
            s[2] = dims[2] > 1 ? t.stride(2) : dims[3];
            strides = s;
        }
        return t.data_ptr();
    }
};

bool wide(const at::Tensor &t)
{
    if (t.scalar_type() == at::kBFloat16) return false;
    if (t.scalar_type() == at::kFloat) return true;
    refuse(std::string("unsupported activation dtype ") + c10::toString(t.scalar_type()));
}

int64_t whole(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

int truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v;
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return static_cast<float>(v);
}

// The C call without the interpreter's lock; a status other than 0 is raised.
template <typename F>
void run(F call)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    if (rc == 0) return;
    PyObject *args = Py_BuildValue("(is)", rc, infini_attn_status_string(rc));
    if (args) {
        PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, args);
        Py_DECREF(args);
    }
    throw Refused{};
}

PyObject *keep(PyObject *given, const at::Tensor &made)
{
    if (given != Py_None) return Py_NewRef(given);
    return THPVariable_Wrap(made);
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F body)
{
    HANDLE_TH_ERRORS
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (backward, q, k, freq, positions, start, interleaved, scale, q_out, k_out) -> (q_out, k_out)
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        const bool back = whole(a[0]) != 0, has_k = a[2] != Py_None;
        const Call c(a[1], "q");
        const at::Tensor &q = THPVariable_Unpack(a[1]);
        if (q.dim() != 4 || (has_k && tensor(a[2], "k").dim() != 4)) refuse("q and k are [B, H, L, d] and [B, Hkv, L, d]");
        const bool f32 = wide(q);
        const at::ScalarType dt = q.scalar_type();
        const int64_t B = q.size(0), H = q.size(1), L = q.size(2), d = q.size(3);
        int64_t sq[3], sk[3], Hkv = 0;
        const int64_t *tq = nullptr, *tk = nullptr;
        const void *kp = nullptr;
        const void *qp = c.rows(a[1], "q", dt, q.sizes(), sq, tq);
        if (has_k) {
            Hkv = THPVariable_Unpack(a[2]).size(1);
            kp = c.rows(a[2], "k", dt, {B, Hkv, L, d}, sk, tk);
        } else if (a[9] != Py_None) {
            refuse("k_out without k");
        }
        const int64_t half = tensor(a[3], "freq").numel();
        const double *freq = c.at<double>(a[3], "freq", kF64, {half});
        const int64_t *pos = c.at<int64_t>(a[4], "positions", kI64, {B, L});
        at::Tensor q_new, k_new;
        void *qo = c.at(a[8], "q_out", dt, {B, H, L, d}), *ko = c.at(a[9], "k_out", dt, {B, Hkv, L, d});
        if (!qo) {
            q_new = at::empty({B, H, L, d}, q.options());
            qo = q_new.data_ptr();
        }
        if (!ko && has_k) {
            k_new = at::empty({B, Hkv, L, d}, q.options());
            ko = k_new.data_ptr();
        }
        const int64_t start = whole(a[5]);
        const int inter = truth(a[6]);
        const float scale = real(a[7]);
        const auto fn = back ? (f32 ? infini_attn_rotary_bwd_f32 : infini_attn_rotary_bwd)
                             : (f32 ? infini_attn_rotary_f32 : infini_attn_rotary);
        run([&] {
            return fn(qp, kp, qo, ko, freq, pos, start, tq, tk, B, H, Hkv, L, d, 2 * half, inter, scale, c.stream);
        });
        PyObject *x = keep(a[8], q_new), *y = has_k ? keep(a[9], k_new) : Py_NewRef(Py_None);
        return Py_BuildValue("(NN)", x, y);
    });
}

// The pool's tensors and sizes, and a page table.
struct Cache {
    void *k, *v;
    float *weights;
    int *table;
    int64_t P, Hkv, page, d, B, max_pages;
    at::ScalarType dt;
    bool f32;

    Cache(const Call &c, PyObject *kp, PyObject *vp, PyObject *w, PyObject *t)
    {
        const at::Tensor &pool = tensor(kp, "k_pages");
        if (pool.dim() != 4) refuse("k_pages and v_pages are [P, Hkv, page, d]");
        dt = pool.scalar_type();
        f32 = wide(pool);
        P = pool.size(0), Hkv = pool.size(1), page = pool.size(2), d = pool.size(3);
        k = c.at(kp, "k_pages", dt, pool.sizes());
        if (vp == Py_None) refuse("v_pages must be a CUDA tensor");
        v = c.at(vp, "v_pages", dt, pool.sizes());
        weights = c.at<float>(w, "weights", kF32, {P, Hkv, page});
        table = pages(c, t, "page_table", B, max_pages);
    }

    static int *pages(const Call &c, PyObject *o, const char *name, int64_t &B, int64_t &n)
    {
        const at::Tensor &t = tensor(o, name);
        if (t.dim() != 2) refuse(std::string(name) + " is [B, pages]");
        B = t.size(0);
        n = t.size(1);
        return c.at<int>(o, name, kI32, t.sizes());
    }
};

// (k, v, k_pages, v_pages, page_table, lens, counts, weights) -> None
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&]() -> PyObject * {
        const Call c(a[2], "k_pages");
        const Cache p(c, a[2], a[3], a[7], a[4]);
        const at::Tensor &k = tensor(a[0], "k");
        if (k.dim() != 4) refuse("k and v are [B, Hkv, T, d]");
        const int64_t T = k.size(2);
        int64_t sk[3], sv[3];
        const int64_t *tk, *tv;
        const void *kr = c.rows(a[0], "k", p.dt, {p.B, p.Hkv, T, p.d}, sk, tk);
        const void *vr = c.rows(a[1], "v", p.dt, {p.B, p.Hkv, T, p.d}, sv, tv);
        const int *lens = c.at<int>(a[5], "lens", kI32, {p.B}), *counts = c.at<int>(a[6], "counts", kI32, {p.B});
        const auto fn = p.f32 ? infini_attn_paged_append_f32 : infini_attn_paged_append;
        run([&] {
            return fn(kr, vr, tk, tv, p.k, p.v, p.weights, p.table, lens, counts, p.B, p.Hkv, T, p.d, p.P, p.page,
                      p.max_pages, c.stream);
        });
        Py_RETURN_NONE;
    });
}

at::Tensor space(int64_t bytes, PyObject *like)
{
    return bytes > 0 ? at::empty({(bytes + 3) / 4}, THPVariable_Unpack(like).options()) : at::Tensor();
}

// (q, k, v, k_pages, v_pages, page_table, lens, beta, M, z, weights, freq, positions, interleaved,
//  scale, out) -> out
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 16, [&]() -> PyObject * {
        const Call c(a[0], "q");
        const Cache p(c, a[3], a[4], a[10], a[5]);
        const at::Tensor &q = THPVariable_Unpack(a[0]);
        if (q.dim() != 3) refuse("q is [B, H, d]");
        const int64_t H = q.size(1);
        const void *qp = c.at(a[0], "q", p.dt, {p.B, H, p.d});
        const void *k = c.at(a[1], "k", p.dt, {p.B, p.Hkv, p.d}), *v = c.at(a[2], "v", p.dt, {p.B, p.Hkv, p.d});
        const int *lens = c.at<int>(a[6], "lens", kI32, {p.B});
        if (!lens) refuse("lens must be a CUDA tensor");
        const float *beta = c.at<float>(a[7], "beta", kF32, {H});
        const float *M = c.at<float>(a[8], "M", kF32, {p.B, p.Hkv, p.d, p.d});
        const float *z = c.at<float>(a[9], "z", kF32, {p.B, p.Hkv, p.d});
        const int64_t half = a[11] == Py_None ? 0 : tensor(a[11], "freq").numel();
        const double *freq = c.at<double>(a[11], "freq", kF64, {half});
        const int64_t *pos = c.at<int64_t>(a[12], "positions", kI64, {p.B});
        if (pos && a[11] == Py_None) refuse("positions without freq");
        const int inter = truth(a[13]);
        const float scale = real(a[14]);
        at::Tensor made;
        void *out = c.at(a[15], "out", p.dt, {p.B, H, p.d});
        if (!out) {
            made = at::empty({p.B, H, p.d}, q.options());
            out = made.data_ptr();
        }
        const int64_t need =
            infini_attn_paged_decode_workspace_bytes(p.B, H, p.Hkv, p.d, p.P, p.page, p.weights != nullptr);
        const at::Tensor ws = space(need, a[6]);
        void *w = need > 0 ? ws.data_ptr() : nullptr;
        const auto fn = p.f32 ? infini_attn_paged_decode_step_f32 : infini_attn_paged_decode_step;
        run([&] {
            return fn(qp, k, v, p.k, p.v, p.table, lens, beta, M, z, p.weights, freq, pos, out, w, need, p.B, H, p.Hkv,
                      p.d, p.P, p.page, p.max_pages, 2 * half, inter, scale, c.stream);
        });
        return keep(a[15], made);
    });
}

// (k_pages, v_pages, weights, page_table, lens, dst_table, budget, recent, M, z, rule, lens_out,
//  kept) -> (lens_out, kept)
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&]() -> PyObject * {
        const Call c(a[0], "k_pages");
        if (a[2] == Py_None) refuse("eviction needs the accumulated weights");
        const Cache p(c, a[0], a[1], a[2], a[3]);
        int64_t Bd, dst_pages;
        const int *dst = Cache::pages(c, a[5], "dst_table", Bd, dst_pages);
        if (Bd != p.B) refuse("dst_table has " + std::to_string(Bd) + " rows, page_table " + std::to_string(p.B));
        const int64_t budget = whole(a[6]), recent = whole(a[7]);
        const int rule = static_cast<int>(whole(a[10]));
        const int *lens = c.at<int>(a[4], "lens", kI32, {p.B});
        if (!lens) refuse("lens must be a CUDA tensor");
        float *M = c.at<float>(a[8], "M", kF32, {p.B, p.Hkv, p.d, p.d});
        float *z = c.at<float>(a[9], "z", kF32, {p.B, p.Hkv, p.d});
        const int64_t rows = budget > 0 ? budget : 0;
        const auto opt = THPVariable_Unpack(a[4]).options();
        at::Tensor lens_new, kept_new;
        int *lens_out = c.at<int>(a[11], "lens_out", kI32, {p.B});
        int *kept = c.at<int>(a[12], "kept", kI32, {p.B, p.Hkv, rows});
        if (!lens_out) {
            lens_new = at::empty({p.B}, opt);
            lens_out = static_cast<int *>(lens_new.data_ptr());
        }
        if (!kept) {
            kept_new = at::empty({p.B, p.Hkv, rows}, opt);
            kept = static_cast<int *>(kept_new.data_ptr());
        }
        const int64_t need =
            infini_attn_paged_evict_workspace_bytes(p.B, p.Hkv, p.d, p.page, p.max_pages, budget, M != nullptr);
        const at::Tensor ws = space(need, a[4]);
        void *w = need > 0 ? ws.data_ptr() : nullptr;
        const auto fn = p.f32 ? infini_attn_paged_evict_f32 : infini_attn_paged_evict;
        run([&] {
            return fn(p.k, p.v, p.weights, p.table, lens, dst, lens_out, kept, M, z, w, need, p.B, p.Hkv, p.d, p.P,
                      p.page, p.max_pages, dst_pages, budget, recent, rule, c.stream);
        });
        PyObject *x = keep(a[11], lens_new), *y = keep(a[12], kept_new);
        return Py_BuildValue("(NN)", x, y);
    });
}

// set_error(cls): the class raised for a status other than 0.
PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_XSETREF(g_error, Py_NewRef(cls));
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&kModule); }
