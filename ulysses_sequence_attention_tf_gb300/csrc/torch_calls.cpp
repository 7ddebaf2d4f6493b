// torch_calls.cpp -- the attention, linear attention, rotation and key-value cache calls of the binding, marshalled in C++.
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
    decltype(&tf_ulysses_kv_plan) kv_plan;
    decltype(&tf_ulysses_rope) rope;
    decltype(&tf_ulysses_rope_frequencies) rope_frequencies;
    decltype(&tf_ulysses_linear_attention) linear_attention;
    decltype(&tf_ulysses_linear_attention_backward) linear_attention_backward;
    decltype(&tf_ulysses_linear_attention_workspace) linear_attention_workspace;
    decltype(&tf_ulysses_linear_attend) linear_attend;
    decltype(&tf_ulysses_linear_attend_workspace) linear_attend_workspace;
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

// New contiguous results of one call.  An allocation takes 1.6 us of host time, as much as two kernels' launches, so small results
// -- up to kSmall bytes altogether -- share one (five of the plan: 12 -> 8 us a call); each of large ones gives its memory back
// by itself.
class Results {
    static constexpr int64_t kSmall = 1 << 20, kAlign = 512;
    at::TensorOptions like;
    Tensor all;
    int64_t room = 0, used = 0, number = 0;
    static int64_t bytes(IntArrayRef shape, ScalarType type) {
        int64_t n = int64_t(c10::elementSize(type));
        for (const int64_t d : shape) n = d > 0 && n > kSmall / d ? kSmall + 1 : n * d;
        return n;
    }
    static int64_t up(int64_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

public:
    explicit Results(const at::TensorOptions& options) : like(options) {}
    // announces what make() is then asked for
    void plan(IntArrayRef shape, ScalarType type, int64_t times = 1) {
        room += times * up(bytes(shape, type));
        number += times;
    }
    Tensor make(IntArrayRef shape, ScalarType type) {
        const int64_t n = up(bytes(shape, type));
        if (number < 2 || room > kSmall || used + n > room) return at::empty(shape, like.dtype(type));
        if (!all.defined()) all = at::empty({room}, like.dtype(ScalarType::Byte));
        Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(used / int64_t(c10::elementSize(type)));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        used += n;
        return t;
    }
};

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
    List(int groups, IntArrayRef shape, ScalarType type, Results& results) : P(groups) {
        for (int i = 0; i < P; ++i) t[i] = results.make(shape, type);
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

// (page_table, lens, new, free, span, device, stream, page_size, rows, lens_out, starts, positions, slots, span_out)
//   -> (lens_out, starts, positions, slots, span_out)
PyObject* kv_plan(PyObject* const* x, Py_ssize_t n) {
    count(n, 14);
    const int device = small("device", x[5]);
    void* stream = address(x[6]);
    const Tensor& table = tensor("page_table", x[0]);
    if (table.dim() != 2 || table.scalar_type() != ScalarType::Int || !table.is_cuda() || table.get_device() != device)
        refuse("page_table must be int32 [N, max_pages] on cuda:" + std::to_string(device));
    const int64_t N = table.size(0), most = table.size(1);
    if (most > 1 && table.stride(1) != 1) refuse("page_table must have unit stride along a row");
    for (int i = 1; i < 5; ++i)
        if (x[i] == Py_None) refuse("lens, new, free and span are required");
    const Tensor& free = tensor("free", x[3]);
    if (free.dim() != 1) refuse("free must be int32 [num_pages]");
    auto ints = [&](const char* name, PyObject* o, int64_t size) { return static_cast<int32_t*>(plain(name, o, ScalarType::Int, {size}, device)); };
    tf_kv_plan p{};
    p.N = extent(N);
    p.max_pages = extent(most);
    p.page_size = small("page_size", x[7]);
    p.num_pages = extent(free.size(0));
    p.T = small("rows", x[8]);
    if (p.T < 0) refuse("rows=" + std::to_string(p.T) + " must be >= 0");
    p.page_table = static_cast<int32_t*>(table.data_ptr());
    p.table_stride = N > 1 ? table.stride(0) : most;
    p.lens = ints("lens", x[1], N);
    p.new_tokens = ints("new", x[2], N);
    p.free_pages = ints("free", x[3], p.num_pages);
    p.free_span = ints("span", x[4], 2);
    const char* names[5] = {"lens_out", "starts", "positions", "slots", "span_out"};
    const int64_t sizes[5] = {N, N + 1, p.T, p.T, 2};
    Results results(table.options());
    for (int i = 0; i < 5; ++i)
        if (x[9 + i] == Py_None) results.plan({sizes[i]}, ScalarType::Int);
    Tensor made[5];
    int32_t* at[5];
    for (int i = 0; i < 5; ++i) {
        if (x[9 + i] == Py_None) {
            made[i] = results.make({sizes[i]}, ScalarType::Int);
            at[i] = static_cast<int32_t*>(made[i].data_ptr());
        } else {
            at[i] = ints(names[i], x[9 + i], sizes[i]);
        }
    }
    p.lens_out = at[0];
    p.starts = at[1];
    p.positions = at[2];
    p.slots = at[3];
    p.span_out = at[4];
    call([&] { return g_abi.kv_plan(&p, stream); });
    PyObject* t = PyTuple_New(5);
    if (!t) throw PythonError{};
    for (int i = 0; i < 5; ++i) {
        PyObject* o = x[9 + i] == Py_None ? THPVariable_Wrap(made[i]) : same(x[9 + i]);
        if (!o) {
            Py_DECREF(t);
            throw PythonError{};
        }
        PyTuple_SET_ITEM(t, i, o);
    }
    return t;
}

// (q, k, device, stream, q_out, k_out, positions, first, frequencies, rotary_dim, theta, magnitude, rope, inverse) -> (q_out, k_out)
PyObject* rope(PyObject* const* x, Py_ssize_t n) {
    count(n, 14);
    const int device = small("device", x[2]);
    void* stream = address(x[3]);
    const List q("q", x[0]);
    const int64_t dims = q.t[0].dim();
    if (dims != 3 && dims != 4) refuse("expected views [B, tokens, heads, D] or [T, heads, D]");
    const ScalarType type = q.t[0].scalar_type();
    const std::vector<int64_t> shape = q.t[0].sizes().vec();
    const Views qv("q", q, shape, type, device);
    tf_rotary r{};
    r.P = q.P;
    r.B = dims == 4 ? extent(shape[0]) : 1;
    r.T = extent(shape[dims - 3]);
    r.H = extent(q.P * shape[dims - 2]);
    r.D = extent(shape[dims - 1]);
    r.dtype = dtype_code(type);
    r.rope = tf_rope(small("rope", x[12]));
    r.inverse = truth(x[13]);
    r.magnitude = float(number(x[11]));
    r.first = small("first", x[7]);
    const std::vector<int64_t> rows(shape.begin(), shape.end() - 2);
    r.positions = static_cast<int32_t*>(plain("positions", x[6], ScalarType::Int, rows, device));
    double made[128];
    if (x[8] == Py_None) {
        r.rotary_dim = x[9] == Py_None ? r.D : small("rotary_dim", x[9]);
        check(g_abi.rope_frequencies(r.rotary_dim, number(x[10]), TF_ROPE_SCALE_NONE, 1.0, 1.0, 0.0, 1.0, made));
        r.frequencies = made;
    } else {
        const Tensor& f = tensor("frequencies", x[8]);
        if (f.dim() != 1 || f.scalar_type() != ScalarType::Double || !f.device().is_cpu() || !f.is_contiguous() || f.size(0) > 128)
            refuse("frequencies must be a contiguous Double tensor [rotary_dim / 2] of up to 128 on the CPU, not " + text(f));
        r.rotary_dim = int(2 * f.size(0));
        if (x[9] != Py_None && small("rotary_dim", x[9]) != r.rotary_dim)
            refuse("rotary_dim does not go with " + std::to_string(f.size(0)) + " frequencies");
        r.frequencies = static_cast<const double*>(f.data_ptr());
    }
    Results results(q.t[0].options());
    if (x[4] == Py_None) results.plan(shape, type, q.P);
    if (x[1] == Py_None) {
        if (x[5] != Py_None) refuse("k_out is given without k");
        const List qo = x[4] == Py_None ? List(q.P, shape, type, results) : List("q_out", x[4], q.P);
        const Views qov("q_out", qo, shape, type, device);
        const tf_strides st[2] = {qv.st, qv.st}, os[2] = {qov.st, qov.st};
        call([&] { return g_abi.rope(&r, qv.ptr, nullptr, st, qov.ptr, nullptr, os, stream); });
        return pair(x[4] == Py_None ? qo.wrap() : same(x[4]), same(Py_None));
    }
    const List k("k", x[1], q.P);
    if (k.t[0].dim() != dims) refuse("q and k must have the same number of dimensions");
    std::vector<int64_t> k_shape = shape;
    k_shape[dims - 2] = k.t[0].size(dims - 2);
    const Views kv("k", k, k_shape, type, device);
    r.Hk = extent(q.P * k_shape[dims - 2]);
    if (x[5] == Py_None) results.plan(k_shape, type, q.P);
    const List qo = x[4] == Py_None ? List(q.P, shape, type, results) : List("q_out", x[4], q.P);
    const List ko = x[5] == Py_None ? List(q.P, k_shape, type, results) : List("k_out", x[5], q.P);
    const Views qov("q_out", qo, shape, type, device);
    const Views kov("k_out", ko, k_shape, type, device);
    const tf_strides st[2] = {qv.st, kv.st}, os[2] = {qov.st, kov.st};
    call([&] { return g_abi.rope(&r, qv.ptr, kv.ptr, st, qov.ptr, kov.ptr, os, stream); });
    return pair(x[4] == Py_None ? qo.wrap() : same(x[4]), x[5] == Py_None ? ko.wrap() : same(x[5]));
}

// what the linear attention calls share: (q, k, v, decay, scale, device)
struct Linear {
    List q, k, v;
    tf_linear a{};
    ScalarType type;
    std::vector<int64_t> shape;
    Views qv, kv, vv;
    Linear(PyObject* const* x, int device, int64_t dims)
        : q("q", x[0]), k("k", x[1], q.P), v("v", x[2], q.P), type(q.t[0].scalar_type()), shape(shape_of(q, dims)),
          qv("q", q, shape, type, device), kv("k", k, shape, type, device), vv("v", v, shape, type, device) {
        a.P = q.P;
        a.B = dims == 4 ? extent(shape[0]) : 1;
        a.S = extent(shape[dims - 3]);
        a.H = extent(q.P * shape[dims - 2]);
        a.D = extent(shape[dims - 1]);
        a.dtype = dtype_code(type);
        if (x[3] == Py_None) refuse("decay is required");
        a.decay = static_cast<float*>(plain("decay", x[3], ScalarType::Float, {a.H}, device));
        a.scale = float(x[4] == Py_None ? 1.0 / std::sqrt(double(a.D)) : number(x[4]));
    }
    static std::vector<int64_t> shape_of(const List& l, int64_t dims) {
        if (l.t[0].dim() != dims) refuse(dims == 4 ? "expected 4-d views [B, tokens, heads, D]" : "expected 3-d views [T, heads, D]");
        return l.t[0].sizes().vec();
    }
    at::TensorOptions options() const { return q.t[0].options(); }
    std::vector<int64_t> states() const { return {a.B, a.H, a.D, a.D}; }
    size_t workspace(bool backward) const {
        size_t n = 0;
        check(g_abi.linear_attention_workspace(&a, backward, &n));
        return n;
    }
};

// A state that may be given (a tensor), asked for (True) or left out (False, None).
struct State {
    Tensor t;
    PyObject* given = nullptr;
    float* at = nullptr;
    State(const char* name, PyObject* o, const Linear& c, int device, Results& results) {
        if (o == Py_None || o == Py_False) return;
        if (o == Py_True) {
            t = results.make(c.states(), ScalarType::Float);
            at = static_cast<float*>(t.data_ptr());
        } else {
            given = o;
            at = static_cast<float*>(plain(name, o, ScalarType::Float, c.states(), device));
        }
    }
    PyObject* wrap() const { return given ? same(given) : at || t.defined() ? THPVariable_Wrap(t) : same(Py_None); }
};

// (q, k, v, decay, scale, state, device, stream, out, final_state) -> (out, final_state)
PyObject* linear_attention(PyObject* const* x, Py_ssize_t n) {
    count(n, 10);
    const int device = small("device", x[6]);
    void* stream = address(x[7]);
    const Linear c(x, device, 4);
    const float* state = static_cast<float*>(plain("state", x[5], ScalarType::Float, c.states(), device));
    Results results(c.options());
    if (x[8] == Py_None) results.plan(c.shape, c.type, c.a.P);
    if (x[9] == Py_True) results.plan(c.states(), ScalarType::Float);
    const List out = x[8] == Py_None ? List(c.a.P, c.shape, c.type, results) : List("out", x[8], c.a.P);
    const Views ov("out", out, c.shape, c.type, device);
    const State last("final_state", x[9], c, device, results);
    const Workspace ws(c.workspace(false), c.options());
    const tf_strides st[3] = {c.qv.st, c.kv.st, c.vv.st};
    call([&] {
        return g_abi.linear_attention(&c.a, c.qv.ptr, c.kv.ptr, c.vv.ptr, st, state, ov.ptr, &ov.st, last.at, ws.at_(), ws.bytes, stream);
    });
    return pair(x[8] == Py_None ? out.wrap() : same(x[8]), last.wrap());
}

// (q, k, v, decay, scale, state, device, stream, dout, dfinal_state, dq, dk, dv, dstate) -> (dq, dk, dv, dstate)
PyObject* linear_attention_backward(PyObject* const* x, Py_ssize_t n) {
    count(n, 14);
    const int device = small("device", x[6]);
    void* stream = address(x[7]);
    const Linear c(x, device, 4);
    const float* state = static_cast<float*>(plain("state", x[5], ScalarType::Float, c.states(), device));
    const List dout("dout", x[8], c.a.P);
    const Views dv("dout", dout, c.shape, c.type, device);
    const float* dfinal = static_cast<float*>(plain("dstate", x[9], ScalarType::Float, c.states(), device));
    const char* names[3] = {"dq", "dk", "dv"};
    PyObject* const asked = x[13] == Py_None && state ? Py_True : x[13];
    Results results(c.options());
    for (int i = 0; i < 3; ++i)
        if (x[10 + i] == Py_None) results.plan(c.shape, c.type, c.a.P);
    if (asked == Py_True) results.plan(c.states(), ScalarType::Float);
    auto made = [&](int i) { return x[10 + i] == Py_None ? List(c.a.P, c.shape, c.type, results) : List(names[i], x[10 + i], c.a.P); };
    const List gq = made(0), gk = made(1), gv = made(2);
    const Views gqv("dq", gq, c.shape, c.type, device), gkv("dk", gk, c.shape, c.type, device), gvv("dv", gv, c.shape, c.type, device);
    const State first("dstate_out", asked, c, device, results);
    const Workspace ws(c.workspace(true), c.options());
    const tf_strides st[4] = {dv.st, c.qv.st, c.kv.st, c.vv.st}, gs[3] = {gqv.st, gkv.st, gvv.st};
    call([&] {
        return g_abi.linear_attention_backward(&c.a, dv.ptr, c.qv.ptr, c.kv.ptr, c.vv.ptr, st, state, dfinal, gqv.ptr, gkv.ptr, gvv.ptr,
                                               gs, first.at, ws.at_(), ws.bytes, stream);
    });
    PyObject* t = PyTuple_New(4);
    if (!t) throw PythonError{};
    PyTuple_SET_ITEM(t, 0, x[10] == Py_None ? gq.wrap() : same(x[10]));
    PyTuple_SET_ITEM(t, 1, x[11] == Py_None ? gk.wrap() : same(x[11]));
    PyTuple_SET_ITEM(t, 2, x[12] == Py_None ? gv.wrap() : same(x[12]));
    PyTuple_SET_ITEM(t, 3, first.wrap());
    return t;
}

// (q, k, v, decay, scale, states, slots, starts, device, stream, out, max_tokens) -> out
PyObject* linear_attend(PyObject* const* x, Py_ssize_t n) {
    count(n, 12);
    const int device = small("device", x[8]);
    void* stream = address(x[9]);
    const Linear c(x, device, 3);
    const Tensor& states = tensor("states", x[5]);
    if (states.dim() != 4) refuse("states must be [slots, H, D, D]");
    const Tensor& slots = tensor("slots", x[6]);
    if (slots.dim() != 1) refuse("slots must be int32 [N]");
    if (x[7] == Py_None) refuse("starts is required");
    tf_linear_pool p{};
    p.states = static_cast<float*>(plain("states", x[5], ScalarType::Float, {states.size(0), c.a.H, c.a.D, c.a.D}, device));
    p.num_slots = extent(states.size(0));
    p.N = extent(slots.size(0));
    p.slots = static_cast<int32_t*>(plain("slots", x[6], ScalarType::Int, {p.N}, device));
    p.starts = static_cast<int32_t*>(plain("starts", x[7], ScalarType::Int, {int64_t(p.N) + 1}, device));
    p.max_tokens = x[11] == Py_None ? c.a.S : small("max_tokens", x[11]);
    Results results(c.options());
    if (x[10] == Py_None) results.plan(c.shape, c.type, c.a.P);
    const List out = x[10] == Py_None ? List(c.a.P, c.shape, c.type, results) : List("out", x[10], c.a.P);
    const Views ov("out", out, c.shape, c.type, device);
    size_t need = 0;
    check(g_abi.linear_attend_workspace(&c.a, &p, &need));
    const Workspace ws(need, c.options());
    const tf_strides st[3] = {c.qv.st, c.kv.st, c.vv.st};
    call([&] {
        return g_abi.linear_attend(&c.a, &p, c.qv.ptr, c.kv.ptr, c.vv.ptr, st, ov.ptr, &ov.st, ws.at_(), ws.bytes, stream);
    });
    return x[10] == Py_None ? out.wrap() : same(x[10]);
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* x, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // results and workspaces are made below autograd, which records none of these calls (2 us of host time a call)
    at::AutoDispatchBelowADInplaceOrView below;
    try {
        return F(x, n);
    } catch (const PythonError&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(check, addresses in the order of EntryPoints)
PyObject* bind(PyObject*, PyObject* const* x, Py_ssize_t n) {
    try {
        constexpr Py_ssize_t kSlots = sizeof(EntryPoints) / sizeof(void*);
        count(n, 1 + kSlots);
        EntryPoints e;
        void** slots = reinterpret_cast<void**>(&e);
        for (Py_ssize_t i = 0; i < kSlots; ++i) slots[i] = address(x[1 + i]);
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
                           {"kv_plan", fast(entry<kv_plan>), METH_FASTCALL, nullptr},
                           {"rope", fast(entry<rope>), METH_FASTCALL, nullptr},
                           {"linear_attention", fast(entry<linear_attention>), METH_FASTCALL, nullptr},
                           {"linear_attention_backward", fast(entry<linear_attention_backward>), METH_FASTCALL, nullptr},
                           {"linear_attend", fast(entry<linear_attend>), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
