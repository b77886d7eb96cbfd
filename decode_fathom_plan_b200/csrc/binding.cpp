// Arguments of the calls on a paged cache, from torch tensors to the C ABI.
//
// A decode step makes several of these calls per layer, and their kernels take
// a few microseconds: reading the tensors' addresses, strides and types in
// Python and converting them with ctypes took 10 to 15 us a call, longer than
// the kernels.  Here a call costs 1 to 2 us before its launches.  The module
// marshals and checks arguments only; every function returns the
// fathom_status of its C call (include/fathom.h), or raises ValueError for a
// tensor that the call would misread.
#include <Python.h>

#include <ATen/core/TensorBase.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <string>

#include "fathom.h"

namespace {

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

const at::Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o)) refuse(std::string(what) + ": a tensor is wanted");
    return THPVariable_Unpack(o);
}

int dtype_code(at::ScalarType t, const char *what)
{
    switch (t) {
    case at::kFloat: return FATHOM_F32;
    case at::kBFloat16: return FATHOM_BF16;
    case at::kHalf: return FATHOM_F16;
    default: refuse(std::string(what) + ": float32, bfloat16 or float16 rows are wanted");
    }
}

// View of a CUDA tensor [tokens][heads][channels].
fathom_rows rows(const at::Tensor &x, const char *what)
{
    if (x.dim() != 3 || !x.is_cuda() || (x.size(2) > 1 && x.stride(2) != 1))
        refuse(std::string(what) + ": a CUDA tensor [tokens][heads][channels] with contiguous channels is wanted");
    if (x.size(0) > INT32_MAX || x.size(1) > INT32_MAX) refuse(std::string(what) + ": too many rows");
    return fathom_rows{x.data_ptr(), x.stride(0), x.stride(1), (int32_t)x.size(1), dtype_code(x.scalar_type(), what)};
}

// Address of a contiguous tensor of the given type and shape on x's device.
void *dense(const at::Tensor &t, const char *what, at::ScalarType type, at::IntArrayRef shape, const at::Tensor &x)
{
    if (t.scalar_type() != type || t.sizes() != shape || t.device() != x.device() || !t.is_contiguous()) {
        std::string want = std::string(what) + ": a contiguous " + c10::toString(type) + " tensor [";
        for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
        refuse(want + "] on " + x.device().str() + " is wanted");
    }
    return t.data_ptr();
}

void same_shape(const at::Tensor &x, const at::Tensor &y, const char *what)
{
    if (x.sizes() != y.sizes() || x.device() != y.device())
        refuse(std::string(what) + ": shape or device differs from that of the rows it belongs to");
}

const void *weight(PyObject *w, const at::Tensor &x, const char *what)
{
    if (w == Py_None) return nullptr;
    const int64_t shape[1] = {x.size(2)};
    return dense(tensor(w, what), what, x.scalar_type(), shape, x);
}

// A ctypes structure by its buffer.
template <typename S>
struct Struct {
    Py_buffer buf{};
    S *p = nullptr;
    explicit Struct(PyObject *o, const char *what)
    {
        if (o == Py_None) return;
        if (PyObject_GetBuffer(o, &buf, PyBUF_WRITABLE) != 0) {
            PyErr_Clear();
            buf.obj = nullptr;
            refuse(std::string(what) + ": a descriptor is wanted");
        }
        if (buf.len != (Py_ssize_t)sizeof(S)) {
            PyBuffer_Release(&buf);
            refuse(std::string(what) + ": another structure is wanted");
        }
        p = static_cast<S *>(buf.buf);
    }
    ~Struct() { if (p) PyBuffer_Release(&buf); }
    Struct(const Struct &) = delete;
    Struct &operator=(const Struct &) = delete;
};

// The turns of a rotation must lie on the rows' device: (descriptor, device index).
struct Rotary : Struct<fathom_rotary> {
    Rotary(PyObject *o, PyObject *device, const at::Tensor &x) : Struct(o, "rotary")
    {
        if (p && PyLong_AsLong(device) != x.get_device()) refuse("rotary: the table lies on another device");
    }
};

// Makes x's device current for the call; the stream as given, or that device's current one.
struct Where {
    std::optional<c10::cuda::CUDAGuard> guard;
    cudaStream_t stream;
    Where(const at::Tensor &x, PyObject *s)
    {
        if (!x.is_cuda()) refuse("rows: a CUDA tensor is wanted");
        if (c10::cuda::current_device() != x.get_device()) guard.emplace(x.device());
        if (s == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(x.get_device()).stream();
            return;
        }
        PyObject *v = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
        stream = v ? static_cast<cudaStream_t>(PyLong_AsVoidPtr(v)) : nullptr;
        Py_XDECREF(v);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            refuse("stream: a stream, its address or None is wanted");
        }
    }
};

int32_t to_int(PyObject *o, const char *what)
{
    const long long v = PyLong_AsLongLong(o);
    if (PyErr_Occurred() || v < INT32_MIN || v > INT32_MAX) {
        PyErr_Clear();
        refuse(std::string(what) + ": an integer of 32 bits is wanted");
    }
    return (int32_t)v;
}

float to_float(PyObject *o, const char *what)
{
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(what) + ": a number is wanted");
    }
    return (float)v;
}

// C++ exceptions end here: as ValueError, or RuntimeError where torch raised.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)f());
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <typename F>
fathom_status without_gil(F f)
{
    PyThreadState *s = PyEval_SaveThread();
    const fathom_status rc = f();
    PyEval_RestoreThread(s);
    return rc;
}

// q, k, pos, q_out, k_out, rotary, rotary device, q_weight, k_weight, eps, stream
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const bool has[2] = {a[0] != Py_None, a[1] != Py_None};
        if ((!has[0] && !has[1]) || has[0] != (a[3] != Py_None) || has[1] != (a[4] != Py_None))
            refuse("q with q_out, k with k_out, or both are wanted");
        const at::Tensor &lead = tensor(a[has[0] ? 0 : 1], "rows");
        fathom_rows in[2], out[2];
        const void *w[2] = {nullptr, nullptr};
        for (int i = 0; i < 2; ++i) {
            if (!has[i]) {
                if (a[7 + i] != Py_None) refuse("a weight of rows that are not given");
                continue;
            }
            const at::Tensor &x = tensor(a[i], i ? "k" : "q"), &y = tensor(a[3 + i], i ? "k_out" : "q_out");
            in[i] = rows(x, i ? "k" : "q");
            same_shape(x, y, i ? "k_out" : "q_out");
            out[i] = rows(y, i ? "k_out" : "q_out");
            if (x.size(0) != lead.size(0) || x.size(2) != lead.size(2) || x.device() != lead.device())
                refuse("q and k differ in tokens, channels or device");
            w[i] = weight(a[7 + i], x, i ? "k_weight" : "q_weight");
        }
        const int64_t shape[1] = {lead.size(0)};
        const void *pos = a[2] == Py_None ? nullptr : dense(tensor(a[2], "pos"), "pos", at::kInt, shape, lead);
        const Rotary rot(a[5], a[6], lead);
        const float eps = to_float(a[9], "eps");
        const Where at(lead, a[10]);
        return without_gil([&] {
            return fathom_qk_norm_rope((int32_t)lead.size(0), (int32_t)lead.size(2), (const int32_t *)pos, rot.p,
                                       w[0], w[1], eps, has[0] ? &in[0] : nullptr, has[0] ? &out[0] : nullptr,
                                       has[1] ? &in[1] : nullptr, has[1] ? &out[1] : nullptr, at.stream);
        });
    });
}

const int32_t *page_table(PyObject *o, int64_t n_seqs, const at::Tensor &x, int32_t *seqs, int32_t *stride)
{
    const at::Tensor &t = tensor(o, "page_table");
    if (t.dim() != 2 || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
        refuse("page_table: int32 [sequences][pages] is wanted");
    const int64_t shape[2] = {n_seqs < 0 ? t.size(0) : n_seqs, t.size(1)};
    *seqs = (int32_t)shape[0];
    *stride = (int32_t)shape[1];
    return (const int32_t *)dense(t, "page_table", at::kInt, shape, x);
}

const fathom_kv_cache *cache_of(const Struct<fathom_kv_cache> &c, const at::Tensor &x)
{
    if (!c.p) refuse("cache: a descriptor is wanted");
    if (x.dim() != 3 || x.size(2) != c.p->head_dim) refuse("rows of another number of channels than the cache's");
    return c.p;
}

// cache, k, v, seq, pos, page_table, rotary, rotary device, k_weight, eps, stream
PyObject *append_kv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const Struct<fathom_kv_cache> desc(a[0], "cache");
        const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        same_shape(k, v, "v");
        const fathom_kv_cache *cache = cache_of(desc, k);
        const fathom_rows kr = rows(k, "k"), vr = rows(v, "v");
        const int64_t shape[1] = {k.size(0)};
        const void *seq = dense(tensor(a[3], "seq"), "seq", at::kInt, shape, k);
        const void *pos = dense(tensor(a[4], "pos"), "pos", at::kInt, shape, k);
        int32_t seqs, stride;
        const int32_t *table = page_table(a[5], -1, k, &seqs, &stride);
        const Rotary rot(a[6], a[7], k);
        const void *w = weight(a[8], k, "k_weight");
        const float eps = to_float(a[9], "eps");
        const Where at(k, a[10]);
        return without_gil([&] {
            return fathom_append_kv(cache, (int32_t)k.size(0), &kr, &vr, (const int32_t *)seq, (const int32_t *)pos,
                                    table, seqs, stride, rot.p, w, eps, at.stream);
        });
    });
}

// What the two attentions take alike.
struct Attention {
    fathom_rows q, out;
    const int32_t *table, *lens;
    int32_t seqs, stride;
    const float *slopes = nullptr;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    Attention(const at::Tensor &x, PyObject *table_, PyObject *lens_, PyObject *out_, PyObject *ws_,
              PyObject *slopes_)
        : q(rows(x, "q")), out(rows(tensor(out_, "out"), "out"))
    {
        same_shape(x, tensor(out_, "out"), "out");
        table = page_table(table_, x.size(0), x, &seqs, &stride);
        const int64_t n[1] = {x.size(0)}, h[1] = {x.size(1)};
        lens = (const int32_t *)dense(tensor(lens_, "seq_lens"), "seq_lens", at::kInt, n, x);
        if (slopes_ != Py_None) slopes = (const float *)dense(tensor(slopes_, "slopes"), "slopes", at::kFloat, h, x);
        if (ws_ == Py_None) return;
        const at::Tensor &w = tensor(ws_, "workspace");
        if (w.device() != x.device() || !w.is_contiguous()) refuse("workspace: contiguous memory of the rows' device is wanted");
        ws = w.data_ptr();
        ws_bytes = w.nbytes();
    }
};

// cache, q, page_table, seq_lens, max_len, out, workspace, softmax_scale, prefix_len, softcap, slopes, stream
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 12, [&] {
        const Struct<fathom_kv_cache> desc(a[0], "cache");
        const at::Tensor &q = tensor(a[1], "q");
        const fathom_kv_cache *cache = cache_of(desc, q);
        const Attention t(q, a[2], a[3], a[5], a[6], a[10]);
        const int32_t max_len = to_int(a[4], "max_len"), prefix = to_int(a[8], "prefix_len");
        const float scale = to_float(a[7], "softmax_scale"), cap = to_float(a[9], "softcap");
        const Where at(q, a[11]);
        return without_gil([&] {
            return fathom_paged_attention(cache, &t.q, t.table, t.stride, t.lens, t.seqs, max_len, prefix, scale, cap,
                                          t.slopes, &t.out, t.ws, t.ws_bytes, at.stream);
        });
    });
}

// cache, q, idx, page_table, seq_lens, out, workspace, softmax_scale, softcap, slopes, stream
PyObject *sparse_attention_paged(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const Struct<fathom_kv_cache> desc(a[0], "cache");
        const at::Tensor &q = tensor(a[1], "q"), &idx = tensor(a[2], "idx");
        const fathom_kv_cache *cache = cache_of(desc, q);
        const Attention t(q, a[3], a[4], a[5], a[6], a[9]);
        if (idx.dim() != 3 || idx.size(2) > INT32_MAX) refuse("idx: int32 [sequences][heads][k] is wanted");
        const int64_t shape[3] = {q.size(0), q.size(1), idx.size(2)};
        const void *ix = dense(idx, "idx", at::kInt, shape, q);
        const float scale = to_float(a[7], "softmax_scale"), cap = to_float(a[8], "softcap");
        const Where at(q, a[10]);
        return without_gil([&] {
            return fathom_sparse_attention_paged(cache, &t.q, (const int32_t *)ix, (int32_t)shape[2], t.table, t.stride,
                                                 t.lens, t.seqs, scale, cap, t.slopes, &t.out, t.ws, t.ws_bytes,
                                                 at.stream);
        });
    });
}

PyMethodDef methods[] = {
    {"qk_norm_rope", (PyCFunction)(void *)qk_norm_rope, METH_FASTCALL, nullptr},
    {"append_kv", (PyCFunction)(void *)append_kv, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void *)paged_attention, METH_FASTCALL, nullptr},
    {"sparse_attention_paged", (PyCFunction)(void *)sparse_attention_paged, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", FATHOM_TORCH_MARK, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
