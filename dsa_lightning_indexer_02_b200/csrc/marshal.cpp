// Argument marshalling of the latency-bound entry points: the checks of the Python binding and the C call
// in one step on the tensors' own C++ objects, a microsecond where ctypes takes fifteen.
// Each function takes its operands by position and returns the C entry point's status, or None when any
// operand is not exactly what the call needs (type, shape, contiguity, device); the Python function of
// the same name then checks the operands one by one and raises, or makes the call itself.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dsa.h"

namespace {

using at::Tensor;

struct No {};  // an operand that this route does not take

int current() {
    return c10::cuda::current_device();
}

const Tensor& any(PyObject* o, int dev, at::ScalarType type, int dims) {
    if (!THPVariable_Check(o)) throw No{};
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != dims ||
        t.layout() != at::kStrided)
        throw No{};
    return t;
}
const Tensor& dense(PyObject* o, int dev, at::ScalarType type, int dims) {
    const Tensor& t = any(o, dev, type, dims);
    if (!t.is_contiguous()) throw No{};
    return t;
}
template <typename... Sizes>
void shape(const Tensor& t, Sizes... want) {
    const int64_t w[] = {int64_t(want)...};
    for (int i = 0; i < (int)sizeof...(want); ++i)
        if (w[i] >= 0 && t.size(i) != w[i]) throw No{};
}
template <typename T>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}
int32_t* ints(PyObject* o, int dev, int64_t n) {  // int32 [n] or None
    if (o == Py_None) return nullptr;
    const Tensor& t = dense(o, dev, at::kInt, 1);
    shape(t, n);
    return ptr<int32_t>(t);
}
int64_t whole(PyObject* o) {
    if (!PyLong_CheckExact(o)) throw No{};
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    if (over) throw No{};
    return v;
}
int small(PyObject* o) {
    const int64_t v = whole(o);
    if (v != (int)v) throw No{};
    return (int)v;
}
float real(PyObject* o) {
    if (PyFloat_CheckExact(o)) return (float)PyFloat_AS_DOUBLE(o);
    if (PyLong_CheckExact(o)) return (float)whole(o);
    throw No{};
}
bool flag(PyObject* o) {
    if (o == Py_True) return true;
    if (o == Py_False) return false;
    throw No{};
}
int fit(int64_t n) {
    if (n > INT32_MAX) throw No{};
    return (int)n;
}
// Strides between tokens and heads of a [T, H, D] operand; those of an axis of one entry are free.
void heads(const Tensor& t, int64_t& ts, int64_t& hs) {
    const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
    if (t.stride(2) != 1 && D != 1) throw No{};
    hs = H == 1 ? (D + 7) / 8 * 8 : t.stride(1);
    ts = T == 1 ? H * hs : t.stride(0);
}
dsa_stream_t stream_of(int dev) {
    return reinterpret_cast<dsa_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}

// Runs `body` (which returns a status) with C++ exceptions turned into None.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body) {
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of operands");
        return nullptr;
    }
    int status = -1;
    try {
        status = body();
    } catch (...) {  // an unusual operand (No) or tensor kind (its accessors throw): the caller's own checks decide
        status = -1;
    }
    if (status < 0) Py_RETURN_NONE;
    return PyLong_FromLong(status);
}

// x, out, inv_freq, pos, pos0, rot_offset, interleaved, mscale, inverse
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const int dev = current();
        if (!THPVariable_Check(a[0])) throw No{};
        const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat) throw No{};
        const Tensor& x = any(a[0], dev, type, 3);
        const Tensor& out = any(a[1], dev, type, 3);
        const int64_t T = x.size(0);
        const int H = fit(x.size(1)), D = fit(x.size(2));
        shape(out, T, H, D);
        const Tensor& f = dense(a[2], dev, at::kDouble, 1);
        const int32_t* pos = ints(a[3], dev, T);
        int64_t xt, xh, ot, oh;
        heads(x, xt, xh), heads(out, ot, oh);
        const int R = fit(2 * f.size(0)), off = small(a[5]);
        const int64_t pos0 = whole(a[4]);
        const bool inter = flag(a[6]), inverse = flag(a[8]);
        const float m = real(a[7]);
        const dsa_stream_t s = stream_of(dev);
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = dsa_rope(ptr<void>(x), type == at::kFloat ? DSA_FP32 : DSA_BF16, T, H, D, xt, xh, pos, pos0, ptr<double>(f),
                      off, R, inter ? DSA_ROPE_INTERLEAVED : DSA_ROPE_HALF, m, inverse, ptr<void>(out), ot, oh, s);
        Py_END_ALLOW_THREADS;
        return st;
    });
}

struct Cache {
    const Tensor &k, &v, &ks, &vs, &table;
    int fmt, pages, page, Hkv, D, B, most;
};
Cache cache(PyObject* const* a, int dev) {  // k_pages, v_pages, k_scale, v_scale, page_table
    if (!THPVariable_Check(a[0])) throw No{};
    const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != at::kFloat8_e4m3fn && type != at::kChar) throw No{};
    Cache c{dense(a[0], dev, type, 4), dense(a[1], dev, type, 4), dense(a[2], dev, at::kFloat, 2),
            dense(a[3], dev, at::kFloat, 2), dense(a[4], dev, at::kInt, 2)};
    c.fmt = type == at::kChar ? DSA_KV_INT8 : DSA_KV_E4M3;
    c.pages = fit(c.k.size(0)), c.page = fit(c.k.size(1)), c.Hkv = fit(c.k.size(2)), c.D = fit(c.k.size(3));
    shape(c.v, c.pages, c.page, c.Hkv, c.D), shape(c.ks, c.pages, c.Hkv), shape(c.vs, c.pages, c.Hkv);
    c.B = fit(c.table.size(0)), c.most = fit(c.table.size(1));
    return c;
}

// k_new, v_new, k_pages, v_pages, k_scale, v_scale, page_table, ctx_len, cu_new, inv_freq, rope_pos, rot_offset,
// interleaved, mscale
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const int dev = current();
        const Cache c = cache(a + 2, dev);
        const Tensor& k = any(a[0], dev, at::kBFloat16, 3);
        const Tensor& v = any(a[1], dev, at::kBFloat16, 3);
        const int64_t N = k.size(0);
        shape(k, N, c.Hkv, c.D), shape(v, N, c.Hkv, c.D);
        int64_t kt, kh, vt, vh;
        heads(k, kt, kh), heads(v, vt, vh);
        const int32_t* ctx = ints(a[7], dev, c.B);
        if (!ctx && c.B) throw No{};
        const int32_t* cu = ints(a[8], dev, (int64_t)c.B + 1);
        if (!cu && N != c.B) throw No{};
        const Tensor* f = a[9] == Py_None ? nullptr : &dense(a[9], dev, at::kDouble, 1);
        const int32_t* pos = ints(a[10], dev, N);
        const int off = small(a[11]), R = f ? fit(2 * f->size(0)) : 0;
        const bool inter = flag(a[12]);
        const float m = real(a[13]);
        const dsa_stream_t s = stream_of(dev);
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = dsa_kv_append(ptr<void>(k), ptr<void>(v), kt, kh, vt, vh, N, cu, ctx, pos, f ? ptr<double>(*f) : nullptr, off,
                           R, inter ? DSA_ROPE_INTERLEAVED : DSA_ROPE_HALF, m, c.fmt, ptr<void>(c.k), ptr<void>(c.v),
                           ptr<float>(c.ks), ptr<float>(c.vs), ptr<int32_t>(c.table), c.B, c.pages, c.page, c.most, c.Hkv,
                           c.D, s);
        Py_END_ALLOW_THREADS;
        return st;
    });
}

// q, k_pages, v_pages, k_scale, v_scale, page_table, n_keys, scale, out, seq, idx, lse, ws
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const int dev = current();
        const Cache c = cache(a + 1, dev);
        const Tensor& q = dense(a[0], dev, at::kBFloat16, 3);
        const int T = fit(q.size(0)), Hq = fit(q.size(1));
        shape(q, T, Hq, c.D);
        const int32_t* n_keys = ints(a[6], dev, T);
        if (!n_keys && T) throw No{};
        const float scale = real(a[7]);
        const Tensor& out = dense(a[8], dev, at::kBFloat16, 3);
        shape(out, T, Hq, c.D);
        const int32_t* seq = ints(a[9], dev, T);
        if (!seq && T != c.B) throw No{};
        const Tensor* idx = a[10] == Py_None ? nullptr : &dense(a[10], dev, at::kInt, 2);
        if (idx) shape(*idx, T, -1);
        const Tensor* lse = a[11] == Py_None ? nullptr : &dense(a[11], dev, at::kFloat, 2);
        if (lse) shape(*lse, T, Hq);
        Tensor ws;
        if (a[12] == Py_None) {
            ws = at::empty({(int64_t)dsa_workspace_size(DSA_OP_PAGED_ATTN, 1, T, Hq, 1, 1)}, q.options().dtype(at::kByte));
        } else {
            if (!THPVariable_Check(a[12])) throw No{};
            ws = THPVariable_Unpack(a[12]);
            if (!ws.is_cuda() || ws.get_device() != dev || !ws.is_contiguous()) throw No{};
        }
        const dsa_stream_t s = stream_of(dev);
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = dsa_paged_attn(ptr<void>(q), ptr<void>(c.k), ptr<void>(c.v), ptr<float>(c.ks), ptr<float>(c.vs),
                            ptr<int32_t>(c.table), seq, n_keys, idx ? ptr<int32_t>(*idx) : nullptr, c.fmt, T, c.B, c.pages,
                            c.page, c.most, Hq, c.Hkv, c.D, idx ? fit(idx->size(1)) : 0, scale, ptr<void>(out),
                            lse ? ptr<float>(*lse) : nullptr, ptr<void>(ws), ws.nbytes(), s);
        Py_END_ALLOW_THREADS;
        return st;
    });
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"paged_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attn)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
