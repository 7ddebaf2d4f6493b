// torch_calls.cpp -- the attention and key-value cache calls of the binding, marshalled in C++.
//
// These calls are short on the GPU, and checking and unpacking a dozen tensors in Python
// takes longer than the kernels of a small call (35 us of host time for two head groups of
// 256 tokens through ctypes, 11 through this module).  This module does what the ctypes binding does for the other
// calls: checks shapes, types, strides and devices, allocates results and workspace from torch on
// the current stream, and calls the C ABI, whose entry points binding.py hands over.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tf_ulysses.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct EntryPoints {
    decltype(&tf_ulysses_attention) attention;
    decltype(&tf_ulysses_attention_backward) attention_backward;
    decltype(&tf_ulysses_attention_workspace) attention_workspace;
    decltype(&tf_ulysses_kv_append) kv_append;
    decltype(&tf_ulysses_kv_attend) kv_attend;
    decltype(&tf_ulysses_kv_attend_workspace) kv_attend_workspace;
};
EntryPoints g_abi{};
PyObject* g_check = nullptr;  // raises for a status that is not TF_OK

struct PythonError {};  // an exception is set

[[noreturn]] void refuse(const std::string& message) {
    PyErr_SetString(PyExc_ValueError, message.c_str());
    throw PythonError{};
}

void check(tf_status s) {
    if (s == TF_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "i", int(s));
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call failed");
    throw PythonError{};
}

// The ABI's calls run without the interpreter's lock: they may wait for another thread's.
template <typename F>
void call(F f) {
    PyThreadState* state = PyEval_SaveThread();
    const tf_status s = f();
    PyEval_RestoreThread(state);
    check(s);
}

std::string text(IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}
std::string text(const Tensor& t) {
    return std::string(c10::toString(t.scalar_type())) + " " + text(t.sizes()) + " with strides " + text(t.strides()) + " on " +
           t.device().str();
}

const Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

tf_dtype dtype_code(ScalarType t) {
    switch (t) {
        case ScalarType::Half: return TF_FP16;
        case ScalarType::BFloat16: return TF_BF16;
        case ScalarType::Float:
        case ScalarType::Int: return TF_FP32;
        case ScalarType::Byte:
        case ScalarType::Char:
        case ScalarType::Float8_e4m3fn:
        case ScalarType::Float8_e5m2: return TF_BYTE;
        default: refuse(std::string("unsupported dtype ") + c10::toString(t));
    }
}

// P tensors of a list or tuple.
struct List {
    Tensor t[TF_ULYSSES_MAX_SHARDS];
    int P = 0;
    List(const char* name, PyObject* o, int want = 0) {
        if (!PyList_Check(o) && !PyTuple_Check(o)) refuse(std::string(name) + " must be a list of head groups");
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
        if (n < 1 || n > TF_ULYSSES_MAX_SHARDS || (want && n != want))
            refuse(std::string(name) + " must be a list of " + (want ? std::to_string(want) : "1 to 8") + " head groups, not " +
                   std::to_string(n));
        P = int(n);
        for (int i = 0; i < P; ++i) t[i] = tensor(name, PySequence_Fast_GET_ITEM(o, i));
    }
    // new contiguous tensors
    List(int groups, IntArrayRef shape, const at::TensorOptions& options) : P(groups) {
        for (int i = 0; i < P; ++i) t[i] = at::empty(shape, options);
    }
    PyObject* wrap() const {
        PyObject* list = PyList_New(P);
        if (!list) throw PythonError{};
        for (int i = 0; i < P; ++i) {
            PyObject* o = THPVariable_Wrap(t[i]);
            if (!o) {
                Py_DECREF(list);
                throw PythonError{};
            }
            PyList_SET_ITEM(list, i, o);
        }
        return list;
    }
};

// Pointers and strides of P views of one shape, type and device, whose last stride is 1.
struct Views {
    void* ptr[TF_ULYSSES_MAX_SHARDS] = {};
    tf_strides st{};
    Views(const char* name, const List& l, IntArrayRef shape, ScalarType type, int device) {
        const IntArrayRef s = l.t[0].strides();
        for (int i = 0; i < l.P; ++i) {
            const Tensor& t = l.t[i];
            if (t.sizes() != shape || t.scalar_type() != type || t.strides() != s || !t.is_cuda() || t.get_device() != device)
                refuse(std::string(name) + " must be " + c10::toString(type) + " views of shape " + text(shape) +
                       " with the same strides on the current device cuda:" + std::to_string(device) + ", not " + text(t));
            ptr[i] = t.data_ptr();
        }
        if (s.back() != 1 && shape.back() > 1) refuse("the D dimension must have stride 1");
        if (s.size() == 4)
            st = {s[0], s[1], s[2]};
        else
            st = {0, s[0], s[1]};
    }
};

// Data pointer of a contiguous tensor of this type and shape on the device, or null for None.
void* plain(const char* name, PyObject* o, ScalarType type, IntArrayRef shape, int device) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(name, o);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || !t.is_cuda() || t.get_device() != device)
        refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + text(shape) + " on cuda:" +
               std::to_string(device) + ", not " + text(t));
    return t.data_ptr();
}

struct Lse {
    float* ptr[TF_ULYSSES_MAX_SHARDS] = {};
    Lse(const List& l, IntArrayRef shape, int device) {
        for (int i = 0; i < l.P; ++i) {
            const Tensor& t = l.t[i];
            if (t.scalar_type() != ScalarType::Float || t.sizes() != shape || !t.is_contiguous() || !t.is_cuda() ||
                t.get_device() != device)
                refuse("lse must be contiguous fp32 tensors of shape " + text(shape) + " on cuda:" + std::to_string(device) +
                       ", not " + text(t));
            ptr[i] = static_cast<float*>(t.data_ptr());
        }
    }
};

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}
long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
int small(const char* name, PyObject* o) {
    const long long v = integer(o);
    if (v != int(v)) refuse(std::string(name) + "=" + std::to_string(v) + " is out of range");
    return int(v);
}
int extent(int64_t v) {
    if (v != int(v)) refuse("a dimension of " + std::to_string(v) + " is out of range");
    return int(v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v != 0;
}
void* address(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return p;
}

struct Workspace {
    Tensor t;
    size_t bytes;
    Workspace(size_t n, const at::TensorOptions& like) : bytes(n) {
        if (n) t = at::empty({int64_t(n)}, like.dtype(ScalarType::Byte));
    }
    void* at_() const { return bytes ? t.data_ptr() : nullptr; }
};

// what attention and its gradient share: (q, k, v, scale, softcap, slopes, causal, prefix, q_docs, k_docs, device)
struct Attention {
    List q, k, v;
    tf_attention a{};
    ScalarType type;
    std::vector<int64_t> q_shape, k_shape;
    Views qv, kv, vv;
    Attention(PyObject* const* x, int device)
        : q("q", x[0]), k("k", x[1], q.P), v("v", x[2], q.P), type(q.t[0].scalar_type()), q_shape(shape(q)), k_shape(shape(k)),
          qv("q", q, q_shape, type, device), kv("k", k, k_shape, type, device), vv("v", v, k_shape, type, device) {
        if (k_shape[0] != q_shape[0] || k_shape[3] != q_shape[3])
            refuse("q " + text(IntArrayRef(q_shape)) + " and k " + text(IntArrayRef(k_shape)) + " must agree in batch and D");
        a.P = q.P;
        a.B = extent(q_shape[0]);
        a.Sq = extent(q_shape[1]);
        a.Sk = extent(k_shape[1]);
        a.H = extent(q.P * q_shape[2]);
        a.Hkv = extent(q.P * k_shape[2]);
        a.D = extent(q_shape[3]);
        a.dtype = dtype_code(type);
        a.scale = float(x[3] == Py_None ? 1.0 / std::sqrt(double(a.D)) : number(x[3]));
        a.softcap = float(number(x[4]));
        a.slopes = static_cast<float*>(plain("slopes", x[5], ScalarType::Float, {a.H}, device));
        a.causal = truth(x[6]);
        a.prefix = static_cast<int32_t*>(plain("prefix", x[7], ScalarType::Int, {a.B}, device));
        a.q_docs = static_cast<int32_t*>(plain("q_docs", x[8], ScalarType::Int, {a.B, a.Sq}, device));
        a.k_docs = static_cast<int32_t*>(plain("k_docs", x[9], ScalarType::Int, {a.B, a.Sk}, device));
    }
    static std::vector<int64_t> shape(const List& l) {
        if (l.t[0].dim() != 4) refuse("expected 4-d views [B, tokens, heads, D]");
        return l.t[0].sizes().vec();
    }
    at::TensorOptions options() const { return q.t[0].options(); }
    std::vector<int64_t> rows() const { return {a.B, a.H / a.P, a.Sq}; }
    size_t workspace(bool backward) const {
        size_t n = 0;
        check(g_abi.attention_workspace(&a, backward, &n));
        return n;
    }
};

PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* t = PyTuple_New(2);
    if (!t) throw PythonError{};
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}
PyObject* same(PyObject* o) {
    Py_INCREF(o);
    return o;
}
void count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, not %zd", want, n);
    throw PythonError{};
}

// (q, k, v, scale, softcap, slopes, causal, prefix, q_docs, k_docs, device, stream, out, lse) -> (out, lse)
PyObject* attention(PyObject* const* x, Py_ssize_t n) {
    count(n, 14);
    const int device = small("device", x[10]);
    void* stream = address(x[11]);
    const Attention c(x, device);
    const List out = x[12] == Py_None ? List(c.a.P, c.q_shape, c.options()) : List("out", x[12], c.a.P);
    const List lse = x[13] == Py_None ? List(c.a.P, c.rows(), c.options().dtype(ScalarType::Float)) : List("lse", x[13], c.a.P);
    const Views ov("out", out, c.q_shape, c.type, device);
    const Lse lp(lse, c.rows(), device);
    const Workspace ws(c.workspace(false), c.options());
    const tf_strides st[3] = {c.qv.st, c.kv.st, c.vv.st};
    call([&] {
        return g_abi.attention(&c.a, c.qv.ptr, c.kv.ptr, c.vv.ptr, st, ov.ptr, &ov.st, lp.ptr, ws.at_(), ws.bytes, stream);
    });
    return pair(x[12] == Py_None ? out.wrap() : same(x[12]), x[13] == Py_None ? lse.wrap() : same(x[13]));
}

// (q, k, v, scale, softcap, slopes, causal, prefix, q_docs, k_docs, device, stream, dout, out, lse, dq, dk, dv) -> (dq, dk, dv)
PyObject* attention_backward(PyObject* const* x, Py_ssize_t n) {
    count(n, 18);
    const int device = small("device", x[10]);
    void* stream = address(x[11]);
    const Attention c(x, device);
    const List dout("dout", x[12], c.a.P), out("out", x[13], c.a.P), lse("lse", x[14], c.a.P);
    const Views dv("dout", dout, c.q_shape, c.type, device), ov("out", out, c.q_shape, c.type, device);
    const Lse lp(lse, c.rows(), device);
    auto made = [&](const char* name, PyObject* o, const std::vector<int64_t>& shape) {
        return o == Py_None ? List(c.a.P, shape, c.options()) : List(name, o, c.a.P);
    };
    const List gq = made("dq", x[15], c.q_shape), gk = made("dk", x[16], c.k_shape), gv = made("dv", x[17], c.k_shape);
    const Views gqv("dq", gq, c.q_shape, c.type, device), gkv("dk", gk, c.k_shape, c.type, device),
        gvv("dv", gv, c.k_shape, c.type, device);
    const Workspace ws(c.workspace(true), c.options());
    const tf_strides st[5] = {dv.st, c.qv.st, c.kv.st, c.vv.st, ov.st}, gs[3] = {gqv.st, gkv.st, gvv.st};
    call([&] {
        return g_abi.attention_backward(&c.a, dv.ptr, c.qv.ptr, c.kv.ptr, c.vv.ptr, ov.ptr, lp.ptr, st, gqv.ptr, gkv.ptr, gvv.ptr, gs,
                                        ws.at_(), ws.bytes, stream);
    });
    PyObject* t = PyTuple_New(3);
    if (!t) throw PythonError{};
    PyTuple_SET_ITEM(t, 0, x[15] == Py_None ? gq.wrap() : same(x[15]));
    PyTuple_SET_ITEM(t, 1, x[16] == Py_None ? gk.wrap() : same(x[16]));
    PyTuple_SET_ITEM(t, 2, x[17] == Py_None ? gv.wrap() : same(x[17]));
    return t;
}

// x: k, v, k_scale, v_scale, page_table, lens, starts
struct Cache {
    tf_kv_cache c{};
    Cache(PyObject* const* x, int device) {
        const Tensor& k = tensor("k", x[0]);
        if (k.dim() != 4) refuse("the cache's codes must be [pages, Hkv, page_size, D]");
        const IntArrayRef s = k.sizes();
        const Tensor& table = tensor("page_table", x[4]);
        if (table.dim() != 2 || table.scalar_type() != ScalarType::Int || !table.is_cuda() || table.get_device() != device)
            refuse("page_table must be int32 [N, max_pages] on cuda:" + std::to_string(device));
        const int64_t N = table.size(0), most = table.size(1);
        if (most > 1 && table.stride(1) != 1) refuse("page_table must have unit stride along a row");
        for (int i = 0; i < 7; ++i)
            if (x[i] == Py_None) refuse("a tensor of the cache is None");
        c.k = plain("k", x[0], ScalarType::Float8_e4m3fn, s, device);
        c.v = plain("v", x[1], ScalarType::Float8_e4m3fn, s, device);
        c.k_scale = static_cast<float*>(plain("k_scale", x[2], ScalarType::Float, s.slice(0, 2), device));
        c.v_scale = static_cast<float*>(plain("v_scale", x[3], ScalarType::Float, s.slice(0, 2), device));
        c.num_pages = extent(s[0]);
        c.Hkv = extent(s[1]);
        c.page_size = extent(s[2]);
        c.D = extent(s[3]);
        c.N = extent(N);
        c.max_pages = extent(most);
        c.page_table = static_cast<int32_t*>(table.data_ptr());
        c.table_stride = N > 1 ? table.stride(0) : most;
        c.lens = static_cast<int32_t*>(plain("lens", x[5], ScalarType::Int, {N}, device));
        c.starts = static_cast<int32_t*>(plain("starts", x[6], ScalarType::Int, {N + 1}, device));
    }
};

// (cache's 7, device, stream, k, v, q, q_out, q_weight, k_weight, eps, theta, cos_sin, rope) -> q_out or None
PyObject* kv_append(PyObject* const* x, Py_ssize_t n) {
    count(n, 19);
    const int device = small("device", x[7]);
    void* stream = address(x[8]);
    const Cache c(x, device);
    const List k("k", x[9]), v("v", x[10], k.P);
    const int P = k.P;
    if (k.t[0].dim() != 3) refuse("expected 3-d views [T, heads, D]");
    const int T = extent(k.t[0].size(0));
    const int64_t D = c.c.D;
    const ScalarType type = k.t[0].scalar_type();
    if (c.c.Hkv % P) refuse("the " + std::to_string(P) + " head groups of k do not divide Hkv=" + std::to_string(c.c.Hkv));
    const int64_t shape[3] = {T, c.c.Hkv / P, D};
    const Views kv("k", k, shape, type, device), vv("v", v, shape, type, device);
    tf_norm_rope nr{};
    nr.q_weight = plain("q_weight", x[13], type, {D}, device);
    nr.k_weight = plain("k_weight", x[14], type, {D}, device);
    nr.eps = float(number(x[15]));
    nr.theta = float(number(x[16]));
    int rows = 0;
    if (x[17] != Py_None) {
        const Tensor& table = tensor("cos_sin", x[17]);
        rows = extent(table.dim() ? table.size(0) : 0);
        nr.cos_sin = static_cast<float*>(plain("cos_sin", x[17], ScalarType::Float, {rows, D / 2, 2}, device));
    }
    const tf_rope rope = tf_rope(small("rope", x[18]));
    const tf_dtype code = dtype_code(type);
    if (x[11] == Py_None) {
        const tf_strides st[3] = {kv.st, vv.st, kv.st};
        call([&] {
            return g_abi.kv_append(&c.c, P, T, 0, code, kv.ptr, vv.ptr, nullptr, st, nullptr, nullptr, &nr, rope, rows, stream);
        });
        Py_RETURN_NONE;
    }
    const List q("q", x[11], P);
    if (q.t[0].dim() != 3) refuse("expected 3-d views [T, heads, D]");
    const int64_t q_shape[3] = {T, q.t[0].size(1), D};
    const Views qv("q", q, q_shape, type, device);
    const List out = x[12] == Py_None ? List(P, q_shape, q.t[0].options()) : List("q_out", x[12], P);
    const Views ov("q_out", out, q_shape, type, device);
    const tf_strides st[3] = {kv.st, vv.st, qv.st};
    const int H = extent(P * q_shape[1]);
    call([&] {
        return g_abi.kv_append(&c.c, P, T, H, code, kv.ptr, vv.ptr, qv.ptr, st, ov.ptr, &ov.st, &nr, rope, rows,
                               stream);
    });
    return x[12] == Py_None ? out.wrap() : same(x[12]);
}

// (cache's 7, device, stream, q, out, lse, max_tokens, max_len, scale, softcap, slopes, causal) -> (out, lse)
PyObject* kv_attend(PyObject* const* x, Py_ssize_t n) {
    count(n, 18);
    const int device = small("device", x[7]);
    void* stream = address(x[8]);
    const Cache c(x, device);
    const List q("q", x[9]);
    if (q.t[0].dim() != 3 || q.t[0].size(2) != c.c.D) refuse("q must be views [T, heads, " + std::to_string(c.c.D) + "]");
    const std::vector<int64_t> shape = q.t[0].sizes().vec();
    const ScalarType type = q.t[0].scalar_type();
    const Views qv("q", q, shape, type, device);
    tf_kv_attention a{};
    a.P = q.P;
    a.T = extent(shape[0]);
    a.H = extent(q.P * shape[1]);
    a.dtype = dtype_code(type);
    a.max_tokens = x[12] == Py_None ? a.T : small("max_tokens", x[12]);
    a.max_len = x[13] == Py_None ? extent(int64_t(c.c.max_pages) * c.c.page_size) : small("max_len", x[13]);
    a.scale = float(x[14] == Py_None ? 1.0 / std::sqrt(double(c.c.D)) : number(x[14]));
    a.softcap = float(number(x[15]));
    a.slopes = static_cast<float*>(plain("slopes", x[16], ScalarType::Float, {a.H}, device));
    a.causal = truth(x[17]);
    const int64_t rows[2] = {shape[1], shape[0]};
    const at::TensorOptions options = q.t[0].options();
    const List out = x[10] == Py_None ? List(q.P, shape, options) : List("out", x[10], q.P);
    const List lse = x[11] == Py_None ? List(q.P, rows, options.dtype(ScalarType::Float)) : List("lse", x[11], q.P);
    const Views ov("out", out, shape, type, device);
    const Lse lp(lse, rows, device);
    size_t need = 0;
    check(g_abi.kv_attend_workspace(&c.c, &a, &need));
    const Workspace ws(need, options);
    call([&] { return g_abi.kv_attend(&c.c, &a, qv.ptr, &qv.st, ov.ptr, &ov.st, lp.ptr, ws.at_(), ws.bytes, stream); });
    return pair(x[10] == Py_None ? out.wrap() : same(x[10]), x[11] == Py_None ? lse.wrap() : same(x[11]));
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* x, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(x, n);
    } catch (const PythonError&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(check, six addresses in the order of EntryPoints)
PyObject* bind(PyObject*, PyObject* const* x, Py_ssize_t n) {
    try {
        count(n, 7);
        EntryPoints e;
        void** slots = reinterpret_cast<void**>(&e);
        for (int i = 0; i < 6; ++i) slots[i] = address(x[1 + i]);
        Py_INCREF(x[0]);
        Py_XDECREF(g_check);
        g_check = x[0];
        g_abi = e;
    } catch (const PythonError&) {
        return nullptr;
    }
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef g_methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                           {"attention", fast(entry<attention>), METH_FASTCALL, nullptr},
                           {"attention_backward", fast(entry<attention_backward>), METH_FASTCALL, nullptr},
                           {"kv_append", fast(entry<kv_append>), METH_FASTCALL, nullptr},
                           {"kv_attend", fast(entry<kv_attend>), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
