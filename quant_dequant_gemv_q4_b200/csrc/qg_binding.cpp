// qg_binding.cpp -- the Python side of the operators between the GEMVs: reads sizes, strides and addresses out of
// torch tensors, checks what the C ABI cannot see (types, shapes, devices) and calls include/qg.h.
//
// These operators are short (a few microseconds on the GPU), so what a call does on the host counts: reading the
// tensors' attributes from Python and passing twenty arguments through ctypes took 8.3 us for an append, most of it
// before the launch.  The library stays free of torch: the addresses of its entry points are given to bind().
//
// Each function returns the entry point's status; what is refused here raises ValueError.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <string>

#include "qg.h"

namespace {

using at::Tensor;

struct Entries {
    decltype(&qg_qk_norm_rope) norm_rope;
    decltype(&qg_kv4_append) append;
    decltype(&qg_kv4_read) read;
    decltype(&qg_attn_kv4_workspace) attn_workspace;
    decltype(&qg_attn_kv4) attn;
    decltype(&qg_sample_workspace) sample_workspace;
    decltype(&qg_sample) sample;
} entry;

struct Refused {
    std::string why;
};
struct Raised {};  // a Python error is set

std::string describe(const Tensor &t)
{
    std::string s = std::string(c10::toString(t.scalar_type())) + " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] on " + t.device().str();
}

// The arguments of a call.
struct Args {
    PyObject *const *a;
    const char *what;
    int dev = -1;

    [[noreturn]] void refuse(const std::string &why) const { throw Refused{std::string(what) + ": " + why}; }

    // A tensor, or null for None; it has to be on the current device, where the kernels run.
    const Tensor *maybe(int i, const char *name) const
    {
        PyObject *o = a[i];
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) refuse(std::string(name) + " is a torch tensor");
        const Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != dev)
            refuse("every tensor must be on the current CUDA device (" + std::to_string(dev) + "), " + name + " is " + describe(t));
        if (t.layout() != c10::kStrided) refuse(std::string(name) + " is a dense tensor");
        return &t;
    }
    const Tensor &need(int i, const char *name) const
    {
        const Tensor *t = maybe(i, name);
        if (!t) refuse(std::string(name) + " is a torch tensor");
        return *t;
    }
    int64_t whole(int i) const
    {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) throw Raised{};
        return v;
    }
    int small(int i, const char *name) const
    {
        const int64_t v = whole(i);
        if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
        return (int)v;
    }
    double real(int i) const
    {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) throw Raised{};
        return v;
    }
    // None: torch's current stream
    void *stream(int i, bool *current) const
    {
        void *const now = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        *current = true;
        if (a[i] == Py_None) return now;
        PyObject *o = a[i];
        PyObject *attr = PyLong_Check(o) ? nullptr : PyObject_GetAttrString(o, "cuda_stream");
        if (!PyLong_Check(o) && !attr) throw Raised{};
        void *s = PyLong_AsVoidPtr(attr ? attr : o);
        Py_XDECREF(attr);
        if (!s && PyErr_Occurred()) throw Raised{};
        *current = s == now;
        return s;
    }

    // A [tokens, heads, dims] tensor as a qg_heads.
    qg_heads view(const Tensor &t, const char *name) const
    {
        const auto type = t.scalar_type();
        if ((type != at::kFloat && type != at::kHalf) || t.dim() != 3)
            refuse(std::string(name) + " is fp32 or fp16 [tokens, heads, dims], got " + describe(t));
        return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2), type == at::kFloat ? QG_TYPE_F32 : QG_TYPE_F16};
    }
    // The address of a contiguous vector of n elements, or null.
    template <typename T> T *vec(const Tensor *t, at::ScalarType type, int64_t n, const char *name) const
    {
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->dim() != 1 || t->numel() != n || !t->is_contiguous())
            refuse(std::string(name) + " is a contiguous " + c10::toString(type) + " [" + std::to_string(n) + "], got " + describe(*t));
        return static_cast<T *>(t->data_ptr());
    }
    struct Cache {
        void *p;
        int64_t pages;
        int page, H, D;
    };
    Cache cache(int i, int page_i) const
    {
        const Tensor &t = need(i, "cache");
        const int64_t page = whole(page_i);
        if (t.scalar_type() == at::kByte && t.dim() == 4 && t.is_contiguous() && page >= 16 && page <= INT32_MAX &&
            t.size(2) * 16 == page && t.size(3) % 18 == 0 && t.size(1) <= QG_MAX_HEADS && t.size(3) / 18 <= 256)
            return {t.data_ptr(), t.size(0), (int)page, (int)t.size(1), (int)(t.size(3) / 18)};
        refuse("the cache is contiguous uint8 [pages, heads, page / 16, 18 D] with pages of " + std::to_string(page) + " tokens, got " +
               describe(t));
    }
    struct Rope {
        const int32_t *pos = nullptr;
        const double *freq = nullptr;
        int R = 0;
    };
    Rope rope(int pos_i, int freq_i, int64_t T) const
    {
        Rope r;
        const Tensor *pos = maybe(pos_i, "pos"), *freq = maybe(freq_i, "inv_freq");
        if (!freq) return r;
        if (!pos) refuse("a rotation needs positions");
        if (freq->numel() > 256) refuse("inv_freq has at most 128 elements");
        r.pos = vec<int32_t>(pos, at::kInt, T, "pos");
        r.freq = vec<double>(freq, at::kDouble, freq->numel(), "inv_freq");
        r.R = 2 * (int)freq->numel();
        return r;
    }
};

// The body of a Python function of n arguments; C++ exceptions end here.
template <int N, typename F> PyObject *call(const char *what, PyObject *const *a, Py_ssize_t n, F body)
{
    try {
        if (n != N) throw Refused{std::string(what) + ": wrong number of arguments"};
        Args args{a, what};
        args.dev = c10::cuda::current_device();
        return PyLong_FromLong(body(args));
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.why.c_str());
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (a launch may wait for room in the stream's queue: other Python threads run meanwhile)
template <typename F> int without_gil(F f)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

PyObject *norm_rope(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call<11>("qg_qk_norm_rope", args, n, [](const Args &a) {
        const Tensor *q = a.maybe(0, "q"), *k = a.maybe(1, "k"), *wq = a.maybe(2, "wq"), *wk = a.maybe(3, "wk");
        const Tensor *qo = a.maybe(8, "q_out"), *ko = a.maybe(9, "k_out");
        const Tensor *some = q ? q : k;
        if (!some || some->dim() != 3) a.refuse("q or k, [tokens, heads, dims]");
        const int64_t T = some->size(0), D = some->size(2);
        if (D > 256) a.refuse("heads have 64, 128 or 256 dimensions");
        if (q && (!qo || qo->sizes() != q->sizes())) a.refuse("q_out is as q");
        if (k && (!ko || ko->sizes() != k->sizes() || k->dim() != 3 || k->size(0) != T || k->size(2) != D))
            a.refuse("k and k_out are [" + std::to_string(T) + ", heads, " + std::to_string(D) + "]");
        const int64_t Hq = q ? q->size(1) : 0, Hk = k ? k->size(1) : 0;
        if (Hq > QG_MAX_HEADS || Hk > QG_MAX_HEADS) return (int)QG_ERR_SHAPE;
        qg_heads vq, vk, oq, ok;
        if (q) vq = a.view(*q, "q"), oq = a.view(*qo, "q_out");
        if (k) vk = a.view(*k, "k"), ok = a.view(*ko, "k_out");
        const Args::Rope r = a.rope(5, 6, T);
        const float *pq = a.vec<float>(wq, at::kFloat, D, "wq"), *pk = a.vec<float>(wk, at::kFloat, D, "wk");
        const double eps = a.real(4);
        const int pairing = a.small(7, "pairing");
        bool current;
        void *const st = a.stream(10, &current);
        return without_gil([&] {
            return entry.norm_rope(q ? &vq : nullptr, k ? &vk : nullptr, T, (int)Hq, (int)Hk, (int)D, pq, pk, eps, r.pos, r.freq, r.R,
                                   pairing, q ? &oq : nullptr, k ? &ok : nullptr, st);
        });
    });
}

PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call<11>("qg_kv4_append", args, n, [](const Args &a) {
        const Tensor &k = a.need(0, "k"), &v = a.need(1, "v"), &slot = a.need(7, "slot");
        const Tensor *wk = a.maybe(2, "wk");
        const Args::Cache c = a.cache(8, 9);
        const qg_heads vk = a.view(k, "k"), vv = a.view(v, "v");
        const int64_t T = k.size(0);
        if (k.sizes() != v.sizes() || k.size(1) != c.H || k.size(2) != c.D)
            a.refuse("k and v are [tokens, " + std::to_string(c.H) + ", " + std::to_string(c.D) + "], got " + describe(k) + " and " + describe(v));
        const Args::Rope r = a.rope(4, 5, T);
        const float *pk = a.vec<float>(wk, at::kFloat, c.D, "wk");
        const int64_t *ps = a.vec<int64_t>(&slot, at::kLong, T, "slot");
        const double eps = a.real(3);
        const int pairing = a.small(6, "pairing");
        bool current;
        void *const st = a.stream(10, &current);
        return without_gil([&] {
            return entry.append(&vk, &vv, T, c.H, c.D, pk, eps, r.pos, r.freq, r.R, pairing, ps, c.p, c.pages, c.page, st);
        });
    });
}

PyObject *read(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call<6>("qg_kv4_read", args, n, [](const Args &a) {
        const Tensor &slot = a.need(2, "slot"), &ko = a.need(3, "k_out"), &vo = a.need(4, "v_out");
        const Args::Cache c = a.cache(0, 1);
        const int64_t T = slot.numel();
        const qg_heads vk = a.view(ko, "k_out"), vv = a.view(vo, "v_out");
        if (ko.sizes() != vo.sizes() || ko.size(0) != T || ko.size(1) != c.H || ko.size(2) != c.D)
            a.refuse("k_out and v_out are [" + std::to_string(T) + ", " + std::to_string(c.H) + ", " + std::to_string(c.D) + "]");
        const int64_t *ps = a.vec<int64_t>(&slot, at::kLong, T, "slot");
        bool current;
        void *const st = a.stream(5, &current);
        return without_gil([&] { return entry.read(c.p, c.pages, c.page, c.H, c.D, ps, T, &vk, &vv, st); });
    });
}

// A workspace that the caller gives, or one from torch's allocator (which hands it out again on the same stream only
// after this call's kernels).
struct Workspace {
    Tensor own;
    void *p = nullptr;
    size_t bytes = 0;
    void take(const Args &a, const Tensor *given, size_t need, bool current)
    {
        if (given) {
            if (!given->is_contiguous()) a.refuse("the workspace is contiguous");
            p = given->data_ptr();
            bytes = given->nbytes();
        } else if (need) {
            if (!current) a.refuse("a call on a stream that is not torch's current one needs a workspace");
            own = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)a.dev));
            p = own.data_ptr();
            bytes = need;
        }
    }
};

PyObject *attn(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call<11>("qg_attn_kv4", args, n, [](const Args &a) {
        const Tensor &q = a.need(0, "q"), &start = a.need(1, "q_start"), &table = a.need(5, "table");
        const Tensor &len = a.need(6, "kv_len"), &out = a.need(8, "out");
        const Tensor *given = a.maybe(9, "workspace");
        const Args::Cache c = a.cache(3, 4);
        if (q.scalar_type() != at::kHalf || out.scalar_type() != at::kHalf || q.dim() != 3 || q.sizes() != out.sizes() || q.size(2) != c.D)
            a.refuse("q and out are fp16 [tokens, heads, " + std::to_string(c.D) + "]");
        if (table.scalar_type() != at::kInt || table.dim() != 2 || !table.is_contiguous())
            a.refuse("table is contiguous int32 [sequences, pages]");
        const int64_t T = q.size(0), Hq = q.size(1), nseq = table.size(0), width = table.size(1);
        if (Hq > QG_MAX_HEADS || nseq > INT32_MAX || width > INT32_MAX) return (int)QG_ERR_SHAPE;
        const int max_q = a.small(2, "max_q");
        const qg_heads vq = a.view(q, "q"), vo = a.view(out, "out");
        const int32_t *ps = a.vec<int32_t>(&start, at::kInt, nseq + 1, "q_start"), *pl = a.vec<int32_t>(&len, at::kInt, nseq, "kv_len");
        const float scale = (float)a.real(7);
        bool current;
        void *const st = a.stream(10, &current);
        Workspace ws;
        size_t need = 0;
        if (!given) {
            need = entry.attn_workspace((int)Hq, c.H, c.D, max_q);
            if (!need) return (int)QG_ERR_SHAPE;
        }
        ws.take(a, given, need, current);
        return without_gil([&] {
            return entry.attn(&vq, T, (int)nseq, ps, max_q, (int)Hq, c.H, c.D, c.p, c.pages, c.page,
                              static_cast<const int32_t *>(table.data_ptr()), (int)width, pl, scale, &vo, ws.p, ws.bytes, st);
        });
    });
}

PyObject *sample(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call<9>("qg_sample", args, n, [](const Args &a) {
        const Tensor &x = a.need(0, "logits"), &u = a.need(5, "u"), &token = a.need(6, "token");
        const Tensor *t = a.maybe(1, "temperature"), *k = a.maybe(2, "top_k"), *p = a.maybe(3, "top_p"), *mp = a.maybe(4, "min_p");
        const Tensor *given = a.maybe(7, "workspace");
        if (x.scalar_type() != at::kFloat || x.dim() != 2) a.refuse("logits are fp32 [rows, V], got " + describe(x));
        const int64_t R = x.size(0), V = x.size(1), rs = x.stride(0), es = x.stride(1);
        const float *pt = a.vec<float>(t, at::kFloat, R, "temperature"), *pp = a.vec<float>(p, at::kFloat, R, "top_p");
        const float *pm = a.vec<float>(mp, at::kFloat, R, "min_p"), *pu = a.vec<float>(&u, at::kFloat, R, "u");
        const int32_t *pk = a.vec<int32_t>(k, at::kInt, R, "top_k");
        int32_t *to = a.vec<int32_t>(&token, at::kInt, R, "token");
        bool current;
        void *const st = a.stream(8, &current);
        Workspace ws;
        ws.take(a, given, given ? 0 : entry.sample_workspace(R, V, es), current);
        return without_gil([&] {
            return entry.sample(static_cast<const float *>(x.data_ptr()), R, V, rs, es, pt, pk, pp, pm, pu, to, ws.p, ws.bytes, st);
        });
    });
}

// bind(addresses): of the entry points, in the order of Entries.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    void *p[7];
    if (n != 7) {
        PyErr_SetString(PyExc_ValueError, "bind: seven addresses");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    entry.norm_rope = reinterpret_cast<decltype(entry.norm_rope)>(p[0]);
    entry.append = reinterpret_cast<decltype(entry.append)>(p[1]);
    entry.read = reinterpret_cast<decltype(entry.read)>(p[2]);
    entry.attn_workspace = reinterpret_cast<decltype(entry.attn_workspace)>(p[3]);
    entry.attn = reinterpret_cast<decltype(entry.attn)>(p[4]);
    entry.sample_workspace = reinterpret_cast<decltype(entry.sample_workspace)>(p[5]);
    entry.sample = reinterpret_cast<decltype(entry.sample)>(p[6]);
    Py_RETURN_NONE;
}

template <typename F> PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", fast(norm_rope), METH_FASTCALL, nullptr},
                         {"kv4_append", fast(append), METH_FASTCALL, nullptr},
                         {"kv4_read", fast(read), METH_FASTCALL, nullptr},
                         {"attn_kv4", fast(attn), METH_FASTCALL, nullptr},
                         {"sample", fast(sample), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "qg_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qg_binding()
{
    PyObject *const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", QG_BUILT_FOR) < 0) {  // the torch and the Python of the build
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
