// pa_bind.cpp -- the tensors' side of pa_kv_append, pa_kv_append_q8 and pa_decode_q8:
// reads the torch tensors, checks that they fit together, and calls the C entry point
// on the current stream of their device.  On single tokens these calls are bound by
// the host: reading a dozen tensors from Python (some fifty attribute lookups) and
// handing thirty arguments through ctypes took 11.8 us a call where the launch itself
// takes 2.
//
// Each function takes its arguments by position and returns the entry point's PA_*
// code; arguments that do not fit raise TypeError or ValueError.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "pa_decode.h"

namespace {

using at::Tensor;

struct Refusal {
    PyObject *type;
    const char *text;
};
// A Python exception is already set.
struct Raised {};

[[noreturn]] void bad_type(const char *text) { throw Refusal{PyExc_TypeError, text}; }
[[noreturn]] void bad_value(const char *text) { throw Refusal{PyExc_ValueError, text}; }

const Tensor &tensor(PyObject *o)
{
    if (!THPVariable_Check(o))
        bad_type("caches, rows, tables, lengths, scales and status must be tensors");
    return THPVariable_Unpack(o);
}

const Tensor *optional(PyObject *o) { return o == Py_None ? nullptr : &tensor(o); }

int to_int(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    if (v < INT32_MIN || v > INT32_MAX)
        bad_value("an integer argument does not fit 32 bits");
    return (int)v;
}

int to_int(int64_t v)
{
    if (v > INT32_MAX)
        bad_value("a dimension does not fit 32 bits");
    return (int)v;
}

template <typename T = void>
T *addr(const Tensor *t)
{
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

// The device all of the tensors (absent ones aside) are on.
template <size_t N>
int device_of(const Tensor *const (&tensors)[N])
{
    int index = -1;
    for (const Tensor *t : tensors) {
        if (!t)
            continue;
        if (!t->is_cuda())
            bad_value("all tensors must be CUDA tensors");
        const int i = t->get_device();
        if (index >= 0 && i != index)
            bad_value("all tensors must be on one device");
        index = i;
    }
    return index;
}

int type_of(const Tensor &t, const char *refusal)
{
    const auto s = t.scalar_type();
    if (s != at::kHalf && s != at::kBFloat16)
        bad_type(refusal);
    return s == at::kBFloat16 ? PA_BF16 : PA_F16;
}

struct Cache {
    int seqs, kv_heads, head_dim, blocks, block_size, max_blocks;
};

Cache cache_of(const Tensor &key_cache, const Tensor &value_cache, const Tensor &tables,
               const Tensor &lens, at::ScalarType type, const Tensor *k_scales, const Tensor *v_scales)
{
    if (key_cache.dim() != 4 || value_cache.sizes() != key_cache.sizes())
        bad_value("cache shapes must be [num_blocks, num_kv_heads, block_size, head_dim]");
    if (key_cache.scalar_type() != type || value_cache.scalar_type() != type)
        bad_type(k_scales ? "key_cache and value_cache must be float8_e4m3fn"
                          : "key_cache and value_cache must be of key's dtype");
    if (tables.scalar_type() != at::kInt || lens.scalar_type() != at::kInt)
        bad_type("block_tables and seq_lens must be int32");
    if (tables.dim() != 2 || lens.dim() != 1 || tables.size(0) != lens.size(0))
        bad_value("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]");
    if (lens.size(0) == 0)
        bad_value("there must be at least one sequence");
    if (!key_cache.is_contiguous() || !value_cache.is_contiguous() || !tables.is_contiguous() ||
        !lens.is_contiguous())
        bad_value("caches, block_tables and seq_lens must be contiguous");
    if (k_scales) {
        if (k_scales->scalar_type() != at::kFloat || v_scales->scalar_type() != at::kFloat)
            bad_type("k_scales and v_scales must be float32");
        for (const Tensor *s : {k_scales, v_scales})
            if (s->dim() != 2 || s->size(0) != key_cache.size(0) || s->size(1) != key_cache.size(1) ||
                !s->is_contiguous())
                bad_value("k_scales and v_scales must be contiguous [num_blocks, num_kv_heads]");
    }
    return {to_int(lens.size(0)),      to_int(key_cache.size(1)), to_int(key_cache.size(3)),
            to_int(key_cache.size(0)), to_int(key_cache.size(2)), to_int(tables.size(1))};
}

// Token rows of t, [tokens, heads, head_dim] or [num_seqs, q_len, heads, head_dim], and
// the elements between them.
struct Rows {
    int64_t n, step;
    int heads;
};

Rows rows_of(const Tensor &t, int heads, int head_dim, at::ScalarType type)
{
    if (t.scalar_type() != type)
        bad_type("key, value, query and query_out must share one dtype: float16 or bfloat16");
    const auto size = t.sizes(), stride = t.strides();
    const int k = (int)size.size();
    if ((k != 3 && k != 4) || size[k - 1] != head_dim || (heads && size[k - 2] != heads))
        bad_value("key, value, query and query_out must be [tokens, heads, head_dim] or "
                  "[num_seqs, q_len, heads, head_dim]");
    if (stride[k - 1] != 1 || (size[k - 2] > 1 && stride[k - 2] != head_dim))
        bad_value("key, value, query and query_out: a token's heads and dims must be contiguous");
    Rows r = {size[0], stride[0], to_int(size[k - 2])};
    if (k == 4) {
        if (size[1] > 1) {
            if (size[0] > 1 && r.step != size[1] * stride[1])
                bad_value("the tokens of all sequences must be evenly spaced");
            r.step = stride[1];
        }
        r.n *= size[1];
    }
    if (r.n <= 1)
        r.step = size[k - 2] * head_dim;
    return r;
}

// Calls f(stream) with the device current.
template <typename F>
int on_device(int index, PyObject *stream, F f)
{
    pa_stream_t handle;
    if (stream == Py_None) {
        handle = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    } else {
        PyObject *const v = PyObject_GetAttrString(stream, "cuda_stream");
        if (!v)
            throw Raised();
        handle = static_cast<pa_stream_t>(PyLong_AsVoidPtr(v));
        Py_DECREF(v);
        if (!handle && PyErr_Occurred())
            throw Raised();
    }
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != index)
        guard.set_index((c10::DeviceIndex)index);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f(handle);
    Py_END_ALLOW_THREADS;
    return rc;
}

// Runs f() -> code; its refusals and any C++ exception become Python exceptions.
template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F f)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, got);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refusal &r) {
        PyErr_SetString(r.type, r.text);
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

int append(PyObject *const *a, bool q8)
{
    if (q8 && (a[6] == Py_None || a[7] == Py_None))
        bad_value("k_scales and v_scales are needed");
    const Tensor &key = tensor(a[0]), &value = tensor(a[1]), &tables = tensor(a[2]), &lens = tensor(a[3]);
    const Tensor &key_cache = tensor(a[4]), &value_cache = tensor(a[5]);
    const Tensor *const k_scales = q8 ? &tensor(a[6]) : nullptr, *const v_scales = q8 ? &tensor(a[7]) : nullptr;
    const Tensor *const cos_sin = optional(a[8]);
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0)
        throw Raised();
    const Tensor *const query = optional(a[10]), *const query_out = optional(a[11]);
    const Tensor *const starts = optional(a[12]), *const status = optional(a[13]);
    const int dtype = type_of(key, "key must be float16 or bfloat16");
    const auto type = key.scalar_type();
    const Tensor *const all[] = {&key,     &value,  &tables, &lens,      &key_cache, &value_cache, k_scales,
                                 v_scales, cos_sin, query,   query_out, starts,     status};
    const int index = device_of(all);
    const Cache c = cache_of(key_cache, value_cache, tables, lens, q8 ? at::kFloat8_e4m3fn : type, k_scales,
                             v_scales);
    const Rows k = rows_of(key, c.kv_heads, c.head_dim, type), v = rows_of(value, c.kv_heads, c.head_dim, type);
    if (v.n != k.n)
        bad_value("key and value must have the same tokens");
    Rows q = {0, 0, 0}, o = {0, 0, 0};
    if (query || query_out) {
        if (!query || !query_out)
            bad_value("query and query_out go together");
        q = rows_of(*query, 0, c.head_dim, type);
        o = rows_of(*query_out, q.heads, c.head_dim, type);
        if (q.n != k.n || o.n != k.n)
            bad_value("key, query and query_out must have the same tokens");
    }
    if (starts) {
        if (starts->scalar_type() != at::kInt || starts->dim() != 1 || starts->size(0) != c.seqs + 1LL ||
            !starts->is_contiguous())
            bad_value("token_starts must be a contiguous int32 [num_seqs + 1]");
    } else if (key.dim() == 4 ? key.size(0) != c.seqs : k.n % c.seqs != 0) {
        bad_value("without token_starts every sequence has the same number of tokens");
    }
    int rotary = 0, positions = 0;
    if (cos_sin) {
        if (cos_sin->scalar_type() != at::kFloat || cos_sin->dim() != 2 || !cos_sin->is_contiguous())
            bad_value("cos_sin must be a contiguous float32 [max_positions, rotary_dim]");
        if (cos_sin->numel() == 0) // (it has no address, which would mean no rotation)
            bad_value("cos_sin must not be empty");
        positions = to_int(cos_sin->size(0));
        rotary = to_int(cos_sin->size(1));
    }
    if (status && (status->scalar_type() != at::kInt || status->numel() < 1))
        bad_value("status must be an int32 tensor");
    const int n = to_int(k.n);
    return on_device(index, a[14], [&](pa_stream_t stream) {
        if (q8)
            return pa_kv_append_q8(addr(&key), addr(&value), k.step, v.step, addr(query), addr(query_out), q.step,
                                   o.step, addr<float>(cos_sin), rotary, positions, interleaved,
                                   addr<int32_t>(&tables), addr<int32_t>(&lens), addr<int32_t>(starts), n, c.seqs,
                                   q.heads, c.kv_heads, c.head_dim, c.blocks, c.block_size, c.max_blocks, dtype,
                                   addr(&key_cache), addr(&value_cache), addr<float>(k_scales),
                                   addr<float>(v_scales), addr<int32_t>(status), stream);
        return pa_kv_append(addr(&key), addr(&value), k.step, v.step, addr(query), addr(query_out), q.step, o.step,
                            addr<float>(cos_sin), rotary, positions, interleaved, addr<int32_t>(&tables),
                            addr<int32_t>(&lens), addr<int32_t>(starts), n, c.seqs, q.heads, c.kv_heads, c.head_dim,
                            c.blocks, c.block_size, c.max_blocks, dtype, addr(&key_cache), addr(&value_cache),
                            addr<int32_t>(status), stream);
    });
}

int decode(PyObject *const *a)
{
    const Tensor &query = tensor(a[0]), &key_cache = tensor(a[1]), &value_cache = tensor(a[2]);
    const Tensor &k_scales = tensor(a[3]), &v_scales = tensor(a[4]), &tables = tensor(a[5]), &lens = tensor(a[6]);
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred())
        throw Raised();
    const int partition = to_int(a[8]);
    const Tensor &out = tensor(a[9]);
    const Tensor *const tmp = optional(a[10]), *const sums = optional(a[11]), *const maxima = optional(a[12]);
    const int hint = to_int(a[13]);
    const Tensor *const status = optional(a[14]);
    const int dtype = type_of(query, "query and out must share one dtype: float16 or bfloat16");
    if (out.scalar_type() != query.scalar_type())
        bad_type("query and out must share one dtype: float16 or bfloat16");
    const Tensor *const all[] = {&query, &key_cache, &value_cache, &k_scales, &v_scales, &tables,
                                 &lens,  &out,       tmp,          sums,      maxima,    status};
    const int index = device_of(all);
    const Cache c = cache_of(key_cache, value_cache, tables, lens, at::kFloat8_e4m3fn, &k_scales, &v_scales);
    const auto size = query.sizes();
    if ((size.size() != 3 && size.size() != 4) || size[0] != c.seqs || size.back() != c.head_dim)
        bad_value("query must be [num_seqs, num_heads, head_dim] or "
                  "[num_seqs, q_len, num_heads, head_dim]");
    const int q_len = size.size() == 3 ? 1 : to_int(size[1]), heads = to_int(size[size.size() - 2]);
    if (out.sizes() != size || !query.is_contiguous() || !out.is_contiguous())
        bad_value("query and out must be contiguous and of one shape");
    int parts = 0;
    if (tmp) {
        const int64_t np = tmp->dim() >= 2 ? tmp->size(-2) : 0, rows = (int64_t)c.seqs * q_len * heads;
        const Tensor *const work[] = {tmp, sums, maxima};
        for (const Tensor *t : work)
            if (!t || t->scalar_type() != at::kFloat || !t->is_contiguous() ||
                t->numel() < rows * np * (t == tmp ? c.head_dim : 1))
                bad_value("tmp_output, exp_sums and max_logits must be what alloc_workspace "
                          "returns for these sizes");
        parts = to_int(np);
    }
    if (status && (status->scalar_type() != at::kInt || status->numel() < 1))
        bad_value("status must be an int32 tensor");
    return on_device(index, a[15], [&](pa_stream_t stream) {
        return pa_decode_q8(addr(&query), addr(&key_cache), addr(&value_cache), addr<float>(&k_scales),
                            addr<float>(&v_scales), addr<int32_t>(&tables), addr<int32_t>(&lens), c.seqs, q_len,
                            heads, c.kv_heads, c.head_dim, c.blocks, c.block_size, c.max_blocks, hint,
                            (float)scale, partition, dtype, addr(&out), addr<float>(tmp), addr<float>(sums),
                            addr<float>(maxima), parts, addr<int32_t>(status), stream);
    });
}

PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 15, [&] { return append(a, false); });
}
PyObject *py_append_q8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 15, [&] { return append(a, true); });
}
PyObject *py_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 16, [&] { return decode(a); });
}

PyMethodDef methods[] = {
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, nullptr},
    {"append_q8", (PyCFunction)(void (*)(void))py_append_q8, METH_FASTCALL, nullptr},
    {"decode_q8", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
