// Python's fast way to the serving step's calls: argument checks, output tensors and the
// current stream, then the C ABI. These calls last a few microseconds on the GPU, and the same
// checks in Python cost as much again (9 to 20 us a call against 2 to 4 here); the GEMMs,
// whose callers bring their own outputs, stay with ctypes.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdio>

#include "w4a16.h"

namespace {

PyObject* g_error = nullptr;   // W4A16Error(status, what)

// A refusal or a failed call, thrown to where the Python error is set.
struct Failure {
    int status;
    char what[224];
};

[[noreturn]] void refuse(const char* what) {
    Failure f{W4A16_ERR_INVALID_ARG, {}};
    std::snprintf(f.what, sizeof f.what, "%s", what);
    throw f;
}

void check(int status, const char* what) {
    if (status == W4A16_OK) return;
    Failure f{status, {}};
    std::snprintf(f.what, sizeof f.what, "%s", what);
    throw f;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) refuse(what);
    return THPVariable_Unpack(o);
}

// Address of a contiguous one-dimensional CUDA tensor of n elements (n < 0: any number).
template <typename T = void>
T* vector(PyObject* o, at::ScalarType type, int64_t n, const char* what) {
    const at::Tensor& t = tensor(o, what);
    if (t.scalar_type() != type || !t.is_cuda() || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous()) refuse(what);
    return static_cast<T*>(t.data_ptr());
}

template <typename T = void>
T* optional_vector(PyObject* o, at::ScalarType type, int64_t n, const char* what) {
    return o == Py_None ? nullptr : vector<T>(o, type, n, what);
}

int integer(PyObject* o, const char* what) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(what);
    }
    if (v < INT32_MIN || v > INT32_MAX) refuse(what);
    return (int)v;
}

// Python's truth of an object: 1 or a numpy bool is as good as True.
bool truth(PyObject* o, const char* what) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        refuse(what);
    }
    return v != 0;
}

int count(int64_t n, const char* what) {
    if (n > INT32_MAX) refuse(what);
    return (int)n;
}

// The current stream: the caller's, or the one asked for (Place makes it current).
w4a16_stream_t stream_of(const at::Tensor& t) {
    return reinterpret_cast<w4a16_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}

int dtype_of(at::ScalarType t, const char* what) {
    if (t == at::kHalf) return W4A16_FP16;
    if (t == at::kBFloat16) return W4A16_BF16;
    if (t == at::kFloat) return W4A16_FP32;
    refuse(what);
}

// The stride of a matrix's rows. That of a single row is never used and may be anything; of more rows the library
// sees the tensor's own: 0 where one row stands for all of them, and one below a row's length is refused there.
int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

struct Cache {
    const at::Tensor& t;
    int pages, heads, dim;
};

Cache cache_of(PyObject* o, int page_size) {
    const char* what = "the cache must be a contiguous uint8 CUDA tensor [pages][kv_heads][page_size / 16][16 * (head_dim + 6)]";
    const at::Tensor& t = tensor(o, what);
    if (t.scalar_type() != at::kByte || !t.is_cuda() || t.dim() != 4 || !t.is_contiguous() || t.size(2) * 16 != page_size ||
        t.size(3) % 16 != 0)
        refuse(what);
    return {t, count(t.size(0), what), count(t.size(1), what), count(t.size(3) / 16 - 6, what)};
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
    return at::empty(size, at::TensorOptions().dtype(type).device(like.device()));
}

// A contiguous tensor over part of another's memory: outputs that come together share one
// allocation (an allocation and its release take 1 us, as long as the kernels of a small call).
at::Tensor part(const at::Tensor& base, int64_t byte, at::IntArrayRef size, at::ScalarType type) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), c10::scalarTypeToTypeMeta(type));
    impl->set_storage_offset(byte / (int64_t)c10::elementSize(type));
    impl->set_sizes_contiguous(size);
    return at::Tensor(std::move(impl));
}

PyObject* tuple(std::initializer_list<at::Tensor> list) {
    PyObject* r = PyTuple_New((Py_ssize_t)list.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : list) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

// (seq_lens, new_lens, free_pages, block_table, page_size, max_tokens, taken, stream)
PyObject* tables(PyObject* const* a) {
    const at::Tensor& seq = tensor(a[0], "seq_lens must be a tensor");
    if (seq.dim() != 1) refuse("seq_lens must be a contiguous int32 CUDA tensor [batch]");
    const int batch = count(seq.size(0), "too many requests");
    const int32_t* seq_at = vector<int32_t>(a[0], at::kInt, batch, "seq_lens must be a contiguous int32 CUDA tensor [batch]");
    const int32_t* new_at = vector<int32_t>(a[1], at::kInt, batch, "new_lens must be a contiguous int32 CUDA tensor [batch]");
    const int32_t* free_at = vector<int32_t>(a[2], at::kInt, -1, "free_pages must be a contiguous int32 CUDA tensor");
    const int n_free = count(THPVariable_Unpack(a[2]).size(0), "too many free pages");
    const at::Tensor& table = tensor(a[3], "block_table must be a tensor");
    if (table.scalar_type() != at::kInt || !table.is_cuda() || table.dim() != 2 || table.size(0) != batch || !table.is_contiguous())
        refuse("block_table must be a contiguous int32 CUDA tensor [batch][pages]");
    const int page_size = integer(a[4], "page_size"), max_tokens = integer(a[5], "max_tokens");
    if (max_tokens < 0) refuse("max_tokens is negative");
    const int32_t* taken = optional_vector<int32_t>(a[6], at::kInt, 1, "taken must be a contiguous int32 CUDA tensor of one element");
    const int64_t at_positions = 8 * (int64_t)max_tokens, at_starts = at_positions + 4 * (int64_t)max_tokens;
    const int64_t at_after = at_starts + 4 * ((int64_t)batch + 1);
    at::Tensor all = empty({at_after + 4}, at::kByte, seq);
    char* const to = static_cast<char*>(all.data_ptr());
    check(w4a16_kv4_tables(seq_at, new_at, batch, free_at, n_free, taken, reinterpret_cast<int32_t*>(to + at_after),
                           table.data_ptr<int32_t>(), count(table.size(1), "too many pages"), page_size,
                           reinterpret_cast<int64_t*>(to), reinterpret_cast<int32_t*>(to + at_positions), max_tokens,
                           reinterpret_cast<int32_t*>(to + at_starts), stream_of(seq)),
          "w4a16_kv4_tables");
    return tuple({part(all, 0, {max_tokens}, at::kLong), part(all, at_positions, {max_tokens}, at::kInt),
                  part(all, at_starts, {(int64_t)batch + 1}, at::kInt), part(all, at_after, {1}, at::kInt)});
}

// (k, v, slots, cache, page_size, stream)
PyObject* append(PyObject* const* a) {
    const char* what = "k and v must be float16 or bfloat16 CUDA tensors [tokens][kv_heads][head_dim], the last dimension contiguous";
    const int page_size = integer(a[4], "page_size");
    const Cache c = cache_of(a[3], page_size);
    const at::Tensor &k = tensor(a[0], what), &v = tensor(a[1], what);
    const int64_t* slots = vector<int64_t>(a[2], at::kLong, -1, "slots must be a contiguous int64 CUDA tensor");
    const int tokens = count(THPVariable_Unpack(a[2]).size(0), "too many slots");
    for (const at::Tensor* t : {&k, &v})
        if (t->scalar_type() != k.scalar_type() || !t->is_cuda() || t->dim() != 3 || t->size(0) != tokens ||
            t->size(1) != c.heads || t->size(2) != c.dim || t->stride(2) != 1)
            refuse(what);
    check(w4a16_kv4_append(k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), slots,
                           c.t.data_ptr<uint8_t>(), c.pages, tokens, c.heads, c.dim, page_size,
                           dtype_of(k.scalar_type(), what), stream_of(k)),
          "w4a16_kv4_append");
    Py_RETURN_NONE;
}

// (cache, slots, page_size, dtype as the C ABI's, stream)
PyObject* read(PyObject* const* a) {
    const int page_size = integer(a[2], "page_size"), dtype = integer(a[3], "dtype");
    const Cache c = cache_of(a[0], page_size);
    const int64_t* slots = vector<int64_t>(a[1], at::kLong, -1, "slots must be a contiguous int64 CUDA tensor");
    const int tokens = count(THPVariable_Unpack(a[1]).size(0), "too many slots");
    const at::ScalarType type = dtype == W4A16_FP16 ? at::kHalf : dtype == W4A16_BF16 ? at::kBFloat16 : at::kFloat;
    at::Tensor all = empty({2, tokens, c.heads, c.dim}, type, c.t);
    const int64_t half = (int64_t)all.nbytes() / 2;
    char* const to = static_cast<char*>(all.data_ptr());
    check(w4a16_kv4_read(c.t.data_ptr<uint8_t>(), c.pages, slots, to, to + half, tokens, c.heads, c.dim, page_size, dtype,
                         stream_of(c.t)),
          "w4a16_kv4_read");
    return tuple({part(all, 0, {tokens, c.heads, c.dim}, type), part(all, half, {tokens, c.heads, c.dim}, type)});
}

// (q, cache, block_table, seq_lens, starts, page_size, max_q, scale, window, out, return_lse, workspace, stream)
PyObject* attention(PyObject* const* a) {
    const char* what = "q must be a float16 or bfloat16 CUDA tensor [tokens][q_heads][head_dim], the last dimension contiguous";
    const int page_size = integer(a[5], "page_size");
    const Cache c = cache_of(a[1], page_size);
    const at::Tensor &q = tensor(a[0], what), &table = tensor(a[2], "block_table must be a tensor");
    if (!q.is_cuda() || q.dim() != 3 || q.size(2) != c.dim || q.stride(2) != 1) refuse(what);
    const int dtype = dtype_of(q.scalar_type(), what);
    const int tokens = count(q.size(0), "too many tokens"), heads = count(q.size(1), "too many heads");
    if (table.scalar_type() != at::kInt || !table.is_cuda() || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
        refuse("block_table must be an int32 CUDA tensor [batch][pages], its rows contiguous");
    const int batch = count(table.size(0), "too many requests"), cols = count(table.size(1), "too many pages");
    const int32_t* seq = vector<int32_t>(a[3], at::kInt, batch, "seq_lens must be a contiguous int32 CUDA tensor [batch]");
    const int32_t* starts = vector<int32_t>(a[4], at::kInt, (int64_t)batch + 1, "starts must be a contiguous int32 CUDA tensor [batch + 1]");
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)c.dim) : PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("scale must be a number");
    }
    at::Tensor out;
    if (a[9] == Py_None) {
        out = empty({tokens, heads, c.dim}, q.scalar_type(), q);
    } else {
        out = tensor(a[9], "out must be a tensor");
        if (out.scalar_type() != q.scalar_type() || !out.is_cuda() || out.sizes() != q.sizes() || out.stride(2) != 1)
            refuse("out must be a CUDA tensor of q's type and shape, the last dimension contiguous");
    }
    at::Tensor lse;
    if (truth(a[10], "return_lse must be true or false")) lse = empty({tokens, heads}, at::kFloat, q);
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[11] != Py_None) {
        const at::Tensor& w = tensor(a[11], "workspace must be a tensor");
        if (!w.is_cuda() || !w.is_contiguous()) refuse("workspace must be a contiguous CUDA tensor");
        ws = w.data_ptr();
        ws_bytes = w.nbytes();
    }
    check(w4a16_kv4_attention(q.data_ptr(), q.stride(0), q.stride(1), c.t.data_ptr<uint8_t>(), c.pages,
                              table.data_ptr<int32_t>(), row_stride(table), cols, seq, starts,
                              out.data_ptr(), out.stride(0), out.stride(1), lse.defined() ? lse.data_ptr<float>() : nullptr,
                              batch, tokens, heads, c.heads, c.dim, page_size, integer(a[6], "max_q"), (float)scale,
                              integer(a[8], "window"), dtype, ws, ws_bytes, stream_of(q)),
          "w4a16_kv4_attention");
    return lse.defined() ? tuple({out, lse}) : THPVariable_Wrap(out);
}

// (logits, u, temperature, top_k, top_p, min_p, stream)
PyObject* sample(PyObject* const* a) {
    const char* what = "logits must be a float16, bfloat16 or float32 CUDA tensor [batch][vocab], its rows contiguous";
    const at::Tensor& x = tensor(a[0], what);
    if (!x.is_cuda() || x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1)) refuse(what);
    const int dtype = dtype_of(x.scalar_type(), what);
    const int batch = count(x.size(0), "too many rows"), vocab = count(x.size(1), "too many tokens");
    const float* u = vector<float>(a[1], at::kFloat, batch, "u must be a contiguous float32 CUDA tensor [batch]");
    const float* temperature = optional_vector<float>(a[2], at::kFloat, batch, "temperature must be a contiguous float32 CUDA tensor [batch]");
    const int32_t* top_k = optional_vector<int32_t>(a[3], at::kInt, batch, "top_k must be a contiguous int32 CUDA tensor [batch]");
    const float* top_p = optional_vector<float>(a[4], at::kFloat, batch, "top_p must be a contiguous float32 CUDA tensor [batch]");
    const float* min_p = optional_vector<float>(a[5], at::kFloat, batch, "min_p must be a contiguous float32 CUDA tensor [batch]");
    at::Tensor all = empty({2, batch}, at::kInt, x);
    int32_t* const to = all.data_ptr<int32_t>();
    check(w4a16_sample(x.data_ptr(), row_stride(x), u, temperature, top_k, top_p, min_p, to,
                       reinterpret_cast<float*>(to + batch), batch, vocab, dtype, stream_of(x)),
          "w4a16_sample");
    return tuple({part(all, 0, {batch}, at::kInt), part(all, 4 * (int64_t)batch, {batch}, at::kFloat)});
}

// Where a call runs: on the device that its tensors share (the library launches on the current device), and on the
// stream asked for, the last argument (a handle or None), as under torch.cuda.stream(): its outputs then come from that stream's
// pool. From another stream's pool, the memory could still be in use by work there, or be handed out again there
// while this call's kernel writes it.
class Place {
public:
    Place(PyObject* const* args, int n) {
        int at = -1;   // no CUDA tensor: the call refuses its arguments
        for (int i = 0; i < n; ++i) {
            // None and numbers by their own types: asking whether they are tensors takes longer
            if (args[i] == Py_None || PyLong_Check(args[i]) || PyFloat_Check(args[i])) continue;
            if (!THPVariable_Check(args[i]) || !THPVariable_Unpack(args[i]).is_cuda()) continue;
            const int d = THPVariable_Unpack(args[i]).device().index();
            if (at >= 0 && d != at) refuse("the tensors are not all on one device");
            at = d;
        }
        if (at < 0) return;
        if (c10::cuda::current_device() != at) device_.set_index((c10::DeviceIndex)at);
        if (args[n - 1] == Py_None) return;
        void* const handle = PyLong_AsVoidPtr(args[n - 1]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            refuse("stream must be a stream's handle");
        }
        stream_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), (c10::DeviceIndex)at));
    }

private:
    c10::cuda::OptionalCUDAGuard device_;
    c10::cuda::OptionalCUDAStreamGuard stream_;
};

// Each call's arguments, a stream's handle or None the last of them.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS   // torch's own exceptions (out of memory, no driver) keep their Python types
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments wanted, %zd given", N, n);
        return nullptr;
    }
    try {
        const Place place(args, N);
        return F(args);
    } catch (const Failure& f) {
        PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", f.status, f.what) : nullptr;
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, f.what);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

#define FAST(f, n) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<f, n>)), METH_FASTCALL
PyMethodDef g_methods[] = {{"kv4_tables", FAST(tables, 8), nullptr},   {"kv4_append", FAST(append, 6), nullptr},
                           {"kv4_read", FAST(read, 5), nullptr},       {"kv4_attention", FAST(attention, 13), nullptr},
                           {"sample", FAST(sample, 7), nullptr},       {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_w4a16_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w4a16_torch(void) { return PyModule_Create(&g_module); }
