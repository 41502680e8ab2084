// Python entry points of the calls whose kernels take a few microseconds: the
// device tables and the sparse attention.  Marshalling alone: every function
// checks its tensors (type, contiguity, device, shape), takes their addresses and
// the current stream, and returns the status of the C call.  Checked attribute by
// attribute from Python the same costs 4 to 6 us a call, more than most of these
// kernels run.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "pagedkv.h"

namespace {

// Thrown with the Python error set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* format, const char* name, const char* what) {
    PyErr_Format(type, format, name, what);
    throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor%s", name, "");
    return THPVariable_Unpack(o);
}

// What every tensor of a call has to agree with: the current CUDA device.
struct Call {
    int device;
    cudaStream_t stream;

    void* at(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
             bool any_shape = false) const {
        const at::Tensor& t = tensor(o, name);
        if (!t.is_cuda() || !t.is_contiguous() || t.scalar_type() != type)
            refuse(PyExc_TypeError, "%s must be a contiguous CUDA %s tensor", name,
                   c10::toString(type));
        if (t.get_device() != device) {
            char where[96];
            std::snprintf(where, sizeof where, "cuda:%d, but the current device is cuda:%d",
                          int(t.get_device()), device);
            refuse(PyExc_ValueError, "%s is on %s", name, where);
        }
        const at::IntArrayRef have = t.sizes(), want(shape.begin(), shape.size());
        if (!any_shape && have != want) {
            char text[192];
            int n = std::snprintf(text, sizeof text, "(");
            for (const int64_t s : want)
                if (n < int(sizeof text))
                    n += std::snprintf(text + n, sizeof text - n, "%lld, ", (long long)s);
            refuse(PyExc_ValueError, "%s: shape expected %s...)", name, text);
        }
        return t.data_ptr();
    }
    void* at_opt(PyObject* o, const char* name, at::ScalarType type,
                 std::initializer_list<int64_t> shape) const {
        return o == Py_None ? nullptr : at(o, name, type, shape);
    }
};

// The current device and stream (a handle checked by the caller, or None), taken
// once the first tensor is known to be on a GPU.
Call call(PyObject* first, const char* name, PyObject* stream) {
    if (!tensor(first, name).is_cuda())
        refuse(PyExc_TypeError, "%s must be a contiguous CUDA %s", name, "tensor");
    const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream();
    if (stream == Py_None) return Call{int(s.device_index()), s.stream()};
    void* handle = PyLong_AsVoidPtr(stream);
    if (PyErr_Occurred()) throw Refused{};
    return Call{int(s.device_index()), static_cast<cudaStream_t>(handle)};
}

template <typename T>
T structure(PyObject* o, const char* name) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) throw Refused{};
    if (b.len != Py_ssize_t(sizeof(T))) {
        PyBuffer_Release(&b);
        refuse(PyExc_TypeError, "%s: %s", name, "a structure of another size");
    }
    T v;
    std::memcpy(&v, b.buf, sizeof v);
    PyBuffer_Release(&b);
    return v;
}

int32_t int32(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is outside int32%s", name, "");
    return int32_t(v);
}

int32_t rows(const at::Tensor& t, int dim, const char* name) {
    if (t.dim() < 1 || dim >= t.dim() || t.size(dim < 0 ? t.dim() - 1 : dim) > INT32_MAX)
        refuse(PyExc_ValueError, "%s: %s", name, "unexpected shape");
    return int32_t(t.size(dim < 0 ? t.dim() - 1 : dim));
}

at::ScalarType values_of(const pkv_cache_desc& d) {
    if (d.dtype == PKV_F32) return at::kFloat;
    if (d.dtype == PKV_BF16) return at::kBFloat16;
    refuse(PyExc_TypeError, "%s dtype must be float32 or bfloat16%s", "cache", "");
}

PyObject* guarded(PyObject* (*body)(PyObject* const*), PyObject* const* a, Py_ssize_t n,
                  Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
        return nullptr;
    }
    try {
        return body(a);
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// desc, block_table, seq_rows, cached_lens, new_lens, block_tables, context_lens,
// query_start_loc, slot_mapping, positions, free_count_out, stream
PyObject* tables_step(PyObject* const* a) {
    const Call c = call(a[3], "cached_lens", a[11]);
    const int32_t n = rows(tensor(a[3], "cached_lens"), 0, "cached_lens");
    const int32_t tokens = rows(tensor(a[8], "slot_mapping"), 0, "slot_mapping");
    const pkv_device_tables t = structure<pkv_device_tables>(a[0], "tables");
    c.at(a[1], "block_table", at::kInt, {}, true);
    const int32_t width = a[5] == Py_None ? 0 : rows(tensor(a[5], "block_tables"), 1, "block_tables");
    auto* seq_rows = static_cast<int32_t*>(c.at_opt(a[2], "seq_rows", at::kInt, {n}));
    auto* cached = static_cast<int32_t*>(c.at(a[3], "cached_lens", at::kInt, {n}));
    auto* fresh = static_cast<int32_t*>(c.at_opt(a[4], "new_lens", at::kInt, {n}));
    auto* out = static_cast<int32_t*>(c.at_opt(a[5], "block_tables", at::kInt, {n, width}));
    auto* ctx = static_cast<int32_t*>(c.at(a[6], "context_lens", at::kInt, {n}));
    auto* start = static_cast<int32_t*>(c.at(a[7], "query_start_loc", at::kInt, {int64_t(n) + 1}));
    auto* slots = static_cast<int64_t*>(c.at(a[8], "slot_mapping", at::kLong, {tokens}));
    auto* pos = static_cast<int32_t*>(c.at_opt(a[9], "positions", at::kInt, {tokens}));
    auto* count = static_cast<int32_t*>(c.at_opt(a[10], "free_count_out", at::kInt, {1}));
    return PyLong_FromLong(pkv_tables_step(&t, seq_rows, cached, fresh, n, tokens, count, out, width,
                                           ctx, start, slots, pos, c.stream));
}

// desc, block_table, seq_rows, lens, stream
PyObject* tables_release(PyObject* const* a) {
    const Call c = call(a[3], "lens", a[4]);
    const int32_t n = rows(tensor(a[3], "lens"), 0, "lens");
    const pkv_device_tables t = structure<pkv_device_tables>(a[0], "tables");
    c.at(a[1], "block_table", at::kInt, {}, true);
    auto* seq_rows = static_cast<int32_t*>(c.at_opt(a[2], "seq_rows", at::kInt, {n}));
    auto* lens = static_cast<int32_t*>(c.at(a[3], "lens", at::kInt, {n}));
    return PyLong_FromLong(pkv_tables_release(&t, seq_rows, lens, n, c.stream));
}

// The batch of a sparse entry point.
struct Batch {
    int32_t n, width;
    const int32_t *tables, *ctx, *start;
};
Batch batch(const Call& c, PyObject* tables, PyObject* ctx, PyObject* start, int64_t tokens) {
    Batch b;
    b.n = rows(tensor(ctx, "context_lens"), 0, "context_lens");
    b.width = rows(tensor(tables, "block_tables"), 1, "block_tables");
    if (start == Py_None && tokens != b.n)
        refuse(PyExc_ValueError, "query tokens other than one a sequence need %s%s",
               "query_start_loc", "");
    b.tables = static_cast<int32_t*>(c.at(tables, "block_tables", at::kInt, {b.n, b.width}));
    b.ctx = static_cast<int32_t*>(c.at(ctx, "context_lens", at::kInt, {b.n}));
    b.start = static_cast<int32_t*>(
        c.at_opt(start, "query_start_loc", at::kInt, {int64_t(b.n) + 1}));
    return b;
}

// bounds, exps, k_cache, desc, block_tables, context_lens, query_start_loc,
// num_query_tokens or None, stream
PyObject* block_bounds(PyObject* const* a) {
    const Call c = call(a[0], "bounds", a[8]);
    const pkv_cache_desc d = structure<pkv_cache_desc>(a[3], "desc");
    if (a[6] != Py_None && a[7] == Py_None)
        refuse(PyExc_ValueError, "%s is given, so %s has to be", "query_start_loc", "num_query_tokens");
    const int32_t tokens = a[7] == Py_None ? rows(tensor(a[5], "context_lens"), 0, "context_lens")
                                           : int32(a[7], "num_query_tokens");
    const Batch b = batch(c, a[4], a[5], a[6], tokens);
    auto* bounds = static_cast<int8_t*>(
        c.at(a[0], "bounds", at::kChar, {d.num_blocks, d.num_kv_heads, 2, d.head_dim}));
    auto* exps = static_cast<int8_t*>(c.at(a[1], "exps", at::kChar, {d.num_blocks, d.num_kv_heads}));
    const void* k = c.at(a[2], "k_cache", values_of(d),
                         {d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim});
    return PyLong_FromLong(pkv_block_bounds(bounds, exps, k, &d, b.tables, b.width, b.start, b.ctx,
                                            b.n, tokens, c.stream));
}

// selected, q, bounds, exps, desc, block_tables, context_lens, max_context_len,
// num_sink, num_recent, query_start_loc, ws, stream
PyObject* select_blocks(PyObject* const* a) {
    const Call c = call(a[0], "selected", a[12]);
    const pkv_cache_desc d = structure<pkv_cache_desc>(a[4], "desc");
    const int32_t tokens = rows(tensor(a[1], "q"), 0, "q");
    const int32_t top_k = rows(tensor(a[0], "selected"), -1, "selected");
    const Batch b = batch(c, a[5], a[6], a[10], tokens);
    auto* selected = static_cast<int32_t*>(
        c.at(a[0], "selected", at::kInt, {tokens, d.num_kv_heads, top_k}));
    const void* q = c.at(a[1], "q", values_of(d), {tokens, d.num_q_heads, d.head_dim});
    auto* bounds = static_cast<int8_t*>(
        c.at(a[2], "bounds", at::kChar, {d.num_blocks, d.num_kv_heads, 2, d.head_dim}));
    auto* exps = static_cast<int8_t*>(c.at(a[3], "exps", at::kChar, {d.num_blocks, d.num_kv_heads}));
    void* ws = c.at(a[11], "ws", at::kByte, {}, true);
    const size_t bytes = size_t(tensor(a[11], "ws").numel());
    return PyLong_FromLong(pkv_select_blocks(
        selected, q, bounds, exps, &d, b.tables, b.width, b.start, b.ctx, b.n, tokens,
        int32(a[7], "max_context_len"), top_k, int32(a[8], "num_sink"), int32(a[9], "num_recent"),
        ws, bytes, c.stream));
}

// out, q, k_cache, v_cache, desc, block_tables, context_lens, selected,
// query_start_loc, scale or None, stream
PyObject* attention_sparse(PyObject* const* a) {
    const Call c = call(a[0], "out", a[10]);
    const pkv_cache_desc d = structure<pkv_cache_desc>(a[4], "desc");
    const int32_t tokens = rows(tensor(a[1], "q"), 0, "q");
    const int32_t top_k = rows(tensor(a[7], "selected"), -1, "selected");
    const Batch b = batch(c, a[5], a[6], a[8], tokens);
    const at::ScalarType dt = values_of(d);
    void* out = c.at(a[0], "out", dt, {tokens, d.num_q_heads, d.head_dim});
    const void* q = c.at(a[1], "q", dt, {tokens, d.num_q_heads, d.head_dim});
    const void* k = c.at(a[2], "k_cache", dt, {d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim});
    const void* v = c.at(a[3], "v_cache", dt, {d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim});
    auto* selected = static_cast<int32_t*>(
        c.at(a[7], "selected", at::kInt, {tokens, d.num_kv_heads, top_k}));
    double scale = 1.0 / std::sqrt(double(d.head_dim));
    if (a[9] != Py_None) {
        scale = PyFloat_AsDouble(a[9]);
        if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
    }
    return PyLong_FromLong(paged_attention_sparse(out, q, k, v, &d, b.tables, b.width, b.start,
                                                  b.ctx, selected, top_k, b.n, tokens, float(scale),
                                                  c.stream));
}

template <PyObject* (*Body)(PyObject* const*), int Args>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(Body, a, n, Args);
}

template <PyObject* (*Body)(PyObject* const*), int Args>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<Body, Args>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<tables_step, 12>("tables_step"),
                         method<tables_release, 5>("tables_release"),
                         method<block_bounds, 9>("block_bounds"),
                         method<select_blocks, 13>("select_blocks"),
                         method<attention_sparse, 11>("attention_sparse"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hotcalls", nullptr, -1, methods,
                      nullptr,               nullptr,     nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hotcalls() { return PyModule_Create(&module); }
