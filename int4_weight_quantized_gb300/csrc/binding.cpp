// binding.cpp -- Python entry points of the prompt attention and of the 8-bit
// paged KV cache (the package's functions of the same names document them).
//
// Marshalling only, like the ctypes binding of the other operators: checks of
// the tensors, output allocation from torch's caching allocator, one call of
// the C ABI on the current torch stream.  A decode step calls these once or
// twice per layer, and through ctypes one call took longer than its kernel (21 us
// on the host, 5 of them in the C ABI, against 7 for one sequence of 640 tokens);
// here it takes 5, the C ABI's included (7 with the split kernel's two launches).
//
// Each function returns its outputs, or the library's status as an int where
// that is not W4A8_OK (the package turns it into a W4A8Error).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "w4a8.h"

namespace {

using at::Tensor;

// A check that failed; becomes the Python exception.
struct BadArgument {
    PyObject *type;
    std::string what;
};

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const Tensor &tensor(PyObject *o, const char *name, at::ScalarType dtype) {
    if (!THPVariable_Check(o)) throw BadArgument{PyExc_TypeError, std::string(name) + " must be a CUDA tensor"};
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw BadArgument{PyExc_TypeError, std::string(name) + " must be a CUDA tensor"};
    if (t.scalar_type() != dtype)
        throw BadArgument{PyExc_TypeError, std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type())};
    return t;
}

const Tensor &dense(PyObject *o, const char *name, at::ScalarType dtype, at::IntArrayRef shape) {
    const Tensor &t = tensor(o, name, dtype);
    if (t.sizes() != shape) throw BadArgument{PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes())};
    if (!t.is_contiguous()) throw BadArgument{PyExc_ValueError, std::string(name) + " must be contiguous"};
    return t;
}

int64_t dims(PyObject *o, const char *name, int64_t n, at::ScalarType dtype) {
    const Tensor &t = tensor(o, name, dtype);
    if (t.dim() != n) throw BadArgument{PyExc_ValueError, std::string(name) + " must have " + std::to_string(n) + " dimensions, got " + text(t.sizes())};
    return n;
}

int to_int(int64_t v, const char *name) {
    if (v < 0 || v > 0x7fffffff) throw BadArgument{PyExc_ValueError, std::string(name) + " is out of range"};
    return (int)v;
}

// [tokens][heads][dim] fp16, dense but for the stride between tokens.
struct Rows {
    const uint16_t *p;
    int tokens, heads, dim;
    long long ld;
};

Rows rows(PyObject *o, const char *name, int64_t heads, int64_t dim) {
    dims(o, name, 3, at::kHalf);
    const Tensor &t = THPVariable_Unpack(o);
    if ((heads >= 0 && t.size(1) != heads) || (dim >= 0 && t.size(2) != dim))
        throw BadArgument{PyExc_ValueError, std::string(name) + " must have shape (tokens, " + std::to_string(heads) + ", " + std::to_string(dim) +
                                                "), got " + text(t.sizes())};
    const int64_t h = t.size(1), d = t.size(2);
    if (t.stride(2) != 1 || (h > 1 && t.stride(1) != d)) throw BadArgument{PyExc_ValueError, std::string(name) + "'s heads must be contiguous"};
    return {static_cast<const uint16_t *>(t.data_ptr()), to_int(t.size(0), name), to_int(h, name), to_int(d, name),
            t.size(0) > 1 ? (long long)t.stride(0) : (long long)(h * d)};
}

const int32_t *indices(PyObject *o, const char *name, at::IntArrayRef shape) {
    return static_cast<const int32_t *>(dense(o, name, at::kInt, shape).data_ptr());
}

w4a8_kv8 cache_of(PyObject *o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) throw BadArgument{PyExc_TypeError, "cache must be a KV8Cache"};
    PyObject *kc = PyTuple_GET_ITEM(o, 0);
    dims(kc, "k_codes", 4, at::kChar);
    const auto s = THPVariable_Unpack(kc).sizes();
    const int64_t scales[3] = {s[0], s[1], s[2] / 16};
    w4a8_kv8 c;
    c.k_codes = static_cast<int8_t *>(dense(kc, "k_codes", at::kChar, s).data_ptr());
    c.k_scale = static_cast<float *>(dense(PyTuple_GET_ITEM(o, 1), "k_scale", at::kFloat, scales).data_ptr());
    c.v_codes = static_cast<int8_t *>(dense(PyTuple_GET_ITEM(o, 2), "v_codes", at::kChar, s).data_ptr());
    c.v_scale = static_cast<float *>(dense(PyTuple_GET_ITEM(o, 3), "v_scale", at::kFloat, scales).data_ptr());
    c.pages = to_int(s[0], "pages");
    c.heads = to_int(s[1], "heads");
    c.page_tokens = to_int(s[2], "page_tokens");
    c.dim = to_int(s[3], "dim");
    return c;
}

// `o` where it is given, checked; else a new tensor beside `like`.
Tensor output(PyObject *o, const char *name, at::ScalarType dtype, at::IntArrayRef shape, const Tensor &like) {
    if (o != Py_None) return dense(o, name, dtype, shape);
    return at::empty(shape, like.options().dtype(dtype));
}

// The caller's workspace has to be contiguous: an expanded tensor counts more
// bytes than it has.  Looked at before the other arguments.
void check_workspace(PyObject *o) {
    if (o != Py_None && THPVariable_Check(o) && !THPVariable_Unpack(o).is_contiguous())
        throw BadArgument{PyExc_ValueError, "workspace must be contiguous"};
}

Tensor workspace(PyObject *o, size_t need, const Tensor &like) {
    if (o != Py_None) return tensor(o, "workspace", at::kByte);
    return at::empty({(int64_t)need}, like.options().dtype(at::kByte));
}

cudaStream_t stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

float scale_of(PyObject *o, int dim) {
    if (o == Py_None) return (float)(1.0 / std::sqrt((double)dim));
    const double s = PyFloat_AsDouble(o);
    if (s == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)s;
}

PyObject *result(w4a8_status st, PyObject *(*wrap)(const Tensor &, const Tensor &), const Tensor &a, const Tensor &b) {
    return st == W4A8_OK ? wrap(a, b) : PyLong_FromLong((long)st);
}
PyObject *wrap_one(const Tensor &a, const Tensor &) { return THPVariable_Wrap(a); }
PyObject *wrap_two(const Tensor &a, const Tensor &b) {
    PyObject *t = PyTuple_New(2);
    if (t) {
        PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
        PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    }
    return t;
}
PyObject *wrap_none(const Tensor &, const Tensor &) { Py_RETURN_NONE; }

using Args = PyObject *const *;

// (q, k, v, cu_q, cu_k, causal, scale, out)
PyObject *prompt_attention(Args a) {
    const Rows q = rows(a[0], "q", -1, -1), k = rows(a[1], "k", -1, q.dim), v = rows(a[2], "v", k.heads, q.dim);
    if (k.tokens != v.tokens)
        throw BadArgument{PyExc_ValueError, "k and v must have as many tokens, got " + std::to_string(k.tokens) + " and " + std::to_string(v.tokens)};
    dims(a[3], "cu_q", 1, at::kInt);
    const Tensor &like = THPVariable_Unpack(a[0]);
    const int64_t n = THPVariable_Unpack(a[3]).size(0);
    const int32_t *cu_q = indices(a[3], "cu_q", {n});
    const int32_t *cu_k = a[4] == Py_None ? cu_q : indices(a[4], "cu_k", {n});
    const Tensor out = output(a[7], "out", at::kHalf, {q.tokens, q.heads, q.dim}, like);
    const int causal = PyObject_IsTrue(a[5]);
    if (causal < 0) throw python_error();
    return result(w4a8_prompt_attention(q.p, k.p, v.p, q.ld, k.ld, v.ld, cu_q, cu_k, (int)n - 1, q.tokens, k.tokens, q.heads, k.heads, q.dim,
                                        causal, scale_of(a[6], q.dim), static_cast<uint16_t *>(out.data_ptr()), stream()),
                  wrap_one, out, out);
}

// A table's rows and their length.
struct Table {
    const int32_t *p;
    int rows, pages;
};
Table table_of(PyObject *o) {
    dims(o, "table", 2, at::kInt);
    const auto s = THPVariable_Unpack(o).sizes();
    return {indices(o, "table", s), to_int(s[0], "table"), to_int(s[1], "table")};
}

// (cache, k, v, table, start, cu)
PyObject *kv8_append(Args a) {
    const w4a8_kv8 c = cache_of(a[0]);
    const Rows k = rows(a[1], "k", c.heads, c.dim), v = rows(a[2], "v", c.heads, c.dim);
    if (k.tokens != v.tokens)
        throw BadArgument{PyExc_ValueError, "k and v must have as many tokens, got " + std::to_string(k.tokens) + " and " + std::to_string(v.tokens)};
    const Table t = table_of(a[3]);
    const Tensor none;
    return result(w4a8_kv8_append(&c, k.p, v.p, k.ld, v.ld, t.p, indices(a[4], "start", {t.rows}), indices(a[5], "cu", {t.rows + 1}), t.rows,
                                  t.pages, k.tokens, stream()),
                  wrap_none, none, none);
}

// (cache, table, cu, total, k_out, v_out)
PyObject *kv8_read(Args a) {
    const w4a8_kv8 c = cache_of(a[0]);
    const Table t = table_of(a[1]);
    const int32_t *cu = indices(a[2], "cu", {t.rows + 1});
    const long long total = PyLong_AsLongLong(a[3]);
    if (total == -1 && PyErr_Occurred()) throw python_error();
    const int n = to_int(total, "total");
    const Tensor &like = THPVariable_Unpack(a[1]);
    const int64_t shape[3] = {n, c.heads, c.dim};
    const Tensor k = output(a[4], "k_out", at::kHalf, shape, like), v = output(a[5], "v_out", at::kHalf, shape, like);
    return result(w4a8_kv8_read(&c, t.p, cu, t.rows, t.pages, n, static_cast<uint16_t *>(k.data_ptr()), static_cast<uint16_t *>(v.data_ptr()),
                                stream()),
                  wrap_two, k, v);
}

// (q, cache, table, lens, scale, out, workspace)
PyObject *decode_attention_kv8(Args a) {
    check_workspace(a[6]);
    const w4a8_kv8 c = cache_of(a[1]);
    const Table t = table_of(a[2]);
    dims(a[0], "q", 3, at::kHalf);
    const Tensor &like = THPVariable_Unpack(a[0]);
    const int heads = to_int(like.size(1), "q");
    const int64_t shape[3] = {t.rows, heads, c.dim};
    const Tensor &q = dense(a[0], "q", at::kHalf, shape);
    const int32_t *lens = indices(a[3], "lens", {t.rows});
    const Tensor out = output(a[5], "out", at::kHalf, shape, like);
    const Tensor ws = workspace(a[6], w4a8_decode_attention_kv8_workspace_bytes(t.rows, heads, c.heads, c.dim, c.page_tokens, t.pages), like);
    return result(w4a8_decode_attention_kv8(static_cast<const uint16_t *>(q.data_ptr()), &c, t.p, lens, t.rows, heads, t.pages,
                                            scale_of(a[4], c.dim), static_cast<uint16_t *>(out.data_ptr()), ws.data_ptr(), (size_t)ws.numel(),
                                            stream()),
                  wrap_one, out, out);
}

// (cache, table, lens, ids, count)
PyObject *kv8_free_pages(Args a) {
    const w4a8_kv8 c = cache_of(a[0]);
    const Table t = table_of(a[1]);
    const Tensor &like = THPVariable_Unpack(a[1]);
    const int32_t *lens = indices(a[2], "lens", {t.rows});
    const Tensor ids = output(a[3], "ids", at::kInt, {c.pages}, like), count = output(a[4], "count", at::kInt, {1}, like);
    return result(w4a8_kv8_free_pages(t.p, lens, t.rows, t.pages, c.page_tokens, c.pages, static_cast<int32_t *>(ids.data_ptr()),
                                      static_cast<int32_t *>(count.data_ptr()), stream()),
                  wrap_two, ids, count);
}

// (cache, table, lens, src, dst, fresh)
PyObject *kv8_fork(Args a) {
    const w4a8_kv8 c = cache_of(a[0]);
    const Table t = table_of(a[1]);
    dims(a[3], "src", 1, at::kInt);
    const int64_t n = THPVariable_Unpack(a[3]).size(0);
    const int32_t *lens = indices(a[2], "lens", {t.rows});
    const Tensor none;
    return result(w4a8_kv8_fork(&c, const_cast<int32_t *>(t.p), const_cast<int32_t *>(lens), indices(a[3], "src", {n}), indices(a[4], "dst", {n}),
                                indices(a[5], "fresh", {n}), to_int(n, "src"), t.rows, t.pages, stream()),
                  wrap_none, none, none);
}

// (cache, table, lens, table_out, count, workspace)
PyObject *kv8_compact(Args a) {
    check_workspace(a[5]);
    const w4a8_kv8 c = cache_of(a[0]);
    const Table t = table_of(a[1]);
    const Tensor &like = THPVariable_Unpack(a[1]);
    const int32_t *lens = indices(a[2], "lens", {t.rows});
    const Tensor out = output(a[3], "table_out", at::kInt, {t.rows, t.pages}, like), count = output(a[4], "count", at::kInt, {1}, like);
    const Tensor ws = workspace(a[5], w4a8_kv8_compact_workspace_bytes(c.pages), like);
    return result(w4a8_kv8_compact(&c, t.p, lens, t.rows, t.pages, static_cast<int32_t *>(out.data_ptr()), static_cast<int32_t *>(count.data_ptr()),
                                   ws.data_ptr(), (size_t)ws.numel(), stream()),
                  wrap_two, out, count);
}

// No C++ exception leaves: a check becomes its Python exception, an error of
// torch (out of memory, say) the one that torch makes of it.
template <PyObject *(*F)(Args), int N>
PyObject *entry(PyObject *, Args args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        return F(args);
    } catch (const BadArgument &e) {
        PyErr_SetString(e.type, e.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define W4A8_METHOD(f, n) \
    { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {W4A8_METHOD(prompt_attention, 8),
                         W4A8_METHOD(kv8_append, 6),
                         W4A8_METHOD(kv8_read, 6),
                         W4A8_METHOD(decode_attention_kv8, 7),
                         W4A8_METHOD(kv8_free_pages, 5),
                         W4A8_METHOD(kv8_fork, 6),
                         W4A8_METHOD(kv8_compact, 6),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w4a8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w4a8() { return PyModule_Create(&module); }
