// The Python side of the calls that are a few microseconds long on the GPU: checks of their tensors, the
// stream, the device, and the C call, in compiled code. Python's own attribute access and ctypes took 6 us
// of the 9 us that a call of one token cost the host; this takes well under one.
//
// Each function has the arguments of the Python function of its name (all of them, in order), raises what
// that documents and returns the C status. It only marshals: the computation is in the CUDA library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <limits>

#include "kda.h"

namespace {

constexpr int64_t kHeadDim = 128;

struct Raised {};  // a Python exception is set

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
        throw Raised();
    }
    return THPVariable_Unpack(o);
}

const at::Tensor &tensor(PyObject *o, const char *name, int64_t dims) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != dims) {
        PyErr_Format(PyExc_ValueError, "%s: expected %d dimensions, got %d", name, (int)dims, (int)t.dim());
        throw Raised();
    }
    return t;
}

const char *dtype_name(at::ScalarType type) {
    return type == at::kBFloat16 ? "torch.bfloat16" : type == at::kFloat ? "torch.float32" : "torch.int32";
}

// Type, shape, order and device of a tensor; -1 in `shape` takes any extent.
const at::Tensor &need(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, at::Device device,
                       bool pages = false) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type) {
        PyObject *const got = PyObject_GetAttrString(o, "dtype");
        if (got) PyErr_Format(PyExc_TypeError, "%s: expected %s, got %S", name, dtype_name(type), got);
        Py_XDECREF(got);
        throw Raised();
    }
    const at::IntArrayRef sizes = t.sizes();
    bool same = sizes.size() == shape.size();
    for (size_t i = 0; same && i < shape.size(); ++i) same = shape.begin()[i] < 0 || sizes[i] == shape.begin()[i];
    if (!same) {
        PyObject *const want = PyTuple_New((Py_ssize_t)shape.size());
        for (size_t i = 0; want && i < shape.size(); ++i)
            PyTuple_SET_ITEM(want, i, shape.begin()[i] < 0 ? PyUnicode_FromString("any") : PyLong_FromLongLong(shape.begin()[i]));
        PyObject *const size = PyObject_GetAttrString(o, "shape"), *const got = size ? PySequence_Tuple(size) : nullptr;
        if (want && got) PyErr_Format(PyExc_ValueError, "%s: expected shape %R, got %R", name, want, got);
        Py_XDECREF(want);
        Py_XDECREF(size);
        Py_XDECREF(got);
        throw Raised();
    }
    if (pages) {  // [pages, heads, page size, 128]: contiguous but for the distance between pages
        const at::IntArrayRef s = t.strides();
        if ((sizes[1] != 1 && s[1] != sizes[2] * kHeadDim) || s[2] != kHeadDim || s[3] != 1) {
            PyErr_Format(PyExc_ValueError, "%s: a page must be contiguous", name);
            throw Raised();
        }
    } else if (!t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s: must be contiguous", name);
        throw Raised();
    }
    if (t.device() != device) {
        PyErr_Format(PyExc_ValueError, "%s: expected device %s, got %s", name, device.str().c_str(), t.device().str().c_str());
        throw Raised();
    }
    return t;
}

template <typename T = void>
T *address(const at::Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

template <typename T = void>
T *optional(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, at::Device device) {
    return o == Py_None ? nullptr : address<T>(need(o, name, type, shape, device));
}

int32_t int_of(int64_t x, const char *name) {
    if (x < std::numeric_limits<int32_t>::min() || x > std::numeric_limits<int32_t>::max()) {
        PyErr_Format(PyExc_ValueError, "%s: %lld does not fit 32 bits", name, (long long)x);
        throw Raised();
    }
    return (int32_t)x;
}

int32_t int_of(PyObject *o, const char *name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised();
    return int_of((int64_t)x, name);
}

float float_of(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)x;
}

struct Workspace {
    void *base = nullptr;
    int64_t bytes = 0;
};

Workspace workspace_of(PyObject *o, at::Device device) {
    if (o == Py_None) return {};
    const at::Tensor &t = tensor(o, "workspace");
    if (t.device() != device || !t.is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "workspace: must be a contiguous tensor on the inputs' device");
        throw Raised();
    }
    return {t.data_ptr(), (int64_t)t.nbytes()};
}

// Runs `call(stream)` on `device` and the given stream (None: the device's current one).
template <typename F>
PyObject *run(at::Device device, PyObject *stream, F call) {
    if (!device.is_cuda()) {  // the kernels would read host memory as device addresses
        PyErr_Format(PyExc_ValueError, "tensors must be on a CUDA device, got %s", device.str().c_str());
        throw Raised();
    }
    kda_stream_t handle;
    if (stream == Py_None) {
        handle = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    } else {
        PyObject *const raw = PyObject_GetAttrString(stream, "cuda_stream");
        handle = raw ? static_cast<kda_stream_t>(PyLong_AsVoidPtr(raw)) : nullptr;
        Py_XDECREF(raw);
        if (PyErr_Occurred()) throw Raised();
    }
    int status;
    {
        const c10::cuda::CUDAGuard guard(device);
        PyThreadState *const state = PyEval_SaveThread();
        status = call(handle);
        PyEval_RestoreThread(state);
    }
    return PyLong_FromLong(status);
}

// 0 for a decay per head [H], 1 for one per row and head.
int32_t decay_rows(PyObject *o, int64_t rows, int64_t heads, at::Device device) {
    const bool per_head = tensor(o, "log_decay").dim() == 1;
    if (per_head) need(o, "log_decay", at::kFloat, {heads}, device);
    else need(o, "log_decay", at::kFloat, {rows, heads}, device);
    return per_head ? 0 : 1;
}

struct Cache {
    const at::Tensor &k, &v, &lens, &table;
    int64_t batch, heads, page_size, pages, width;
    int64_t stride(const at::Tensor &t) const { return pages == 1 ? heads * page_size * kHeadDim : t.stride(0); }  // (any, for one page)
};

Cache cache_of(PyObject *const *a, at::Device device) {
    const at::Tensor &k = need(a[0], "k_cache", at::kBFloat16, {-1, -1, -1, kHeadDim}, device, true);
    const int64_t pages = k.size(0), heads = k.size(1), size = k.size(2);
    const at::Tensor &v = need(a[1], "v_cache", at::kBFloat16, {pages, heads, size, kHeadDim}, device, true);
    const at::Tensor &lens = need(a[3], "seq_lens", at::kInt, {-1}, device);
    const at::Tensor &table = need(a[2], "block_table", at::kInt, {lens.size(0), -1}, device);
    return {k, v, lens, table, lens.size(0), heads, size, pages, table.size(1)};
}

// (q, k, v, log_decay, cu_seqlens, init_state, out, final_state, scale, workspace, stream)
PyObject *linear_prefill(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q", 3);
    const at::Device device = q.device();
    const int64_t T = q.size(0), H = q.size(1);
    need(a[0], "q", at::kBFloat16, {T, H, kHeadDim}, device);
    const at::Tensor &k = need(a[1], "k", at::kBFloat16, {T, H, kHeadDim}, device);
    const at::Tensor &v = need(a[2], "v", at::kBFloat16, {T, H, kHeadDim}, device);
    const at::Tensor &out = need(a[6], "out", at::kBFloat16, {T, H, kHeadDim}, device);
    const int32_t per_token = decay_rows(a[3], T, H, device);
    const at::Tensor &cu = need(a[4], "cu_seqlens", at::kInt, {-1}, device);
    const int64_t N = cu.size(0) - 1;
    const float *const init = optional<float>(a[5], "init_state", at::kFloat, {N, H, kHeadDim, kHeadDim}, device);
    float *const fin = optional<float>(a[7], "final_state", at::kFloat, {N, H, kHeadDim, kHeadDim}, device);
    const Workspace ws = workspace_of(a[9], device);
    const float scale = float_of(a[8]);
    const int32_t n = int_of(N, "cu_seqlens"), t = int_of(T, "q"), h = int_of(H, "q");
    return run(device, a[10], [&](kda_stream_t stream) {
        return kda_linear_prefill(address(q), address(k), address(v), address<float>(THPVariable_Unpack(a[3])), per_token,
                                  address<int32_t>(cu), init, address(out), fin, n, t, h, scale, ws.base, ws.bytes, stream);
    });
}

// (q, k, v, log_decay, slot_idx, state_pool, out, scale, stream)
PyObject *linear_decode(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q", 3);
    const at::Device device = q.device();
    const int64_t R = q.size(0), H = q.size(1);
    need(a[0], "q", at::kBFloat16, {R, H, kHeadDim}, device);
    const at::Tensor &k = need(a[1], "k", at::kBFloat16, {R, H, kHeadDim}, device);
    const at::Tensor &v = need(a[2], "v", at::kBFloat16, {R, H, kHeadDim}, device);
    const at::Tensor &out = need(a[6], "out", at::kBFloat16, {R, H, kHeadDim}, device);
    const int32_t per_row = decay_rows(a[3], R, H, device);
    const at::Tensor &slots = need(a[4], "slot_idx", at::kInt, {R}, device);
    const at::ScalarType type = tensor(a[5], "state_pool", 4).scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) {
        PyErr_SetString(PyExc_TypeError, "state_pool must be float32 or bfloat16");
        throw Raised();
    }
    const at::Tensor &pool = need(a[5], "state_pool", type, {-1, H, kHeadDim, kHeadDim}, device);
    const float scale = float_of(a[7]);
    const int32_t r = int_of(R, "q"), h = int_of(H, "q");
    return run(device, a[8], [&](kda_stream_t stream) {
        return kda_linear_decode(address(q), address(k), address(v), address<float>(THPVariable_Unpack(a[3])), per_row,
                                 address<int32_t>(slots), address(pool), pool.size(0),
                                 type == at::kFloat ? KDA_STATE_F32 : KDA_STATE_BF16, address(out), r, h, scale, stream);
    });
}

// (q, k_cache, v_cache, block_table, seq_lens, out, scale, workspace, lse, weight, stream)
PyObject *attn_decode(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q", 3);
    const at::Device device = q.device();
    const Cache c = cache_of(a + 1, device);
    const int64_t Hq = q.size(1);
    need(a[0], "q", at::kBFloat16, {c.batch, Hq, kHeadDim}, device);
    const at::Tensor &out = need(a[5], "out", at::kBFloat16, {c.batch, Hq, kHeadDim}, device);
    float *const lse = optional<float>(a[8], "lse", at::kFloat, {c.batch, Hq}, device);
    float *const weight = optional<float>(a[9], "weight", at::kFloat, {c.batch, c.heads, c.width * c.page_size}, device);
    const Workspace ws = workspace_of(a[7], device);
    const float scale = float_of(a[6]);
    const int32_t size = int_of(c.page_size, "k_cache"), width = int_of(c.width, "block_table"), batch = int_of(c.batch, "seq_lens"),
                  hq = int_of(Hq, "q"), heads = int_of(c.heads, "k_cache");
    return run(device, a[10], [&](kda_stream_t stream) {
        return kda_attn_decode(address(q), address(c.k), address(c.v), c.stride(c.k), c.stride(c.v), c.pages, size,
                               address<int32_t>(c.table), width, address<int32_t>(c.lens), address(out), lse, weight, batch, hq,
                               heads, scale, ws.base, ws.bytes, stream);
    });
}

// (k_cache, v_cache, block_table, seq_lens, weight, new_lens, kept, budget, sink, recent, dst_table, dst_weight, stream)
PyObject *cache_evict(PyObject *const *a) {
    const at::Device device = tensor(a[0], "k_cache", 4).device();
    const Cache c = cache_of(a, device);
    const int64_t capacity = c.width * c.page_size;
    const int32_t budget = int_of(a[7], "budget"), sink = int_of(a[8], "sink"), recent = int_of(a[9], "recent");
    const at::Tensor &weight = need(a[4], "weight", at::kFloat, {c.batch, c.heads, capacity}, device);
    float *const dst_weight = a[11] == Py_None ? address<float>(weight)
                                               : optional<float>(a[11], "dst_weight", at::kFloat, {c.batch, c.heads, capacity}, device);
    const int32_t *const dst_table = optional<int32_t>(a[10], "dst_table", at::kInt, {c.batch, c.width}, device);
    const at::Tensor &new_lens = need(a[5], "new_lens", at::kInt, {c.batch}, device);
    // (a budget below one, which no tensor's shape can have, is left to the call to refuse)
    const at::Tensor &kept = need(a[6], "kept", at::kInt, {c.batch, c.heads, budget < 0 ? -1 : (int64_t)budget}, device);
    const int32_t size = int_of(c.page_size, "k_cache"), width = int_of(c.width, "block_table"), batch = int_of(c.batch, "seq_lens"),
                  heads = int_of(c.heads, "k_cache");
    return run(device, a[12], [&](kda_stream_t stream) {
        return kda_cache_evict(address(c.k), address(c.v), c.stride(c.k), c.stride(c.v), c.pages, size, address<int32_t>(c.table),
                               dst_table, width, address<int32_t>(c.lens), address<float>(weight), dst_weight,
                               address<int32_t>(new_lens), address<int32_t>(kept), batch, heads, budget, sink, recent, stream);
    });
}

template <PyObject *(*kCall)(PyObject *const *), int kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != kArgs) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    try {
        return kCall(args);
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <PyObject *(*kCall)(PyObject *const *), int kArgs>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<kCall, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<linear_prefill, 11>("linear_prefill"), method<linear_decode, 9>("linear_decode"),
                         method<attn_decode, 11>("attn_decode"), method<cache_evict, 13>("cache_evict"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kda_gb300_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kda_gb300_binding() { return PyModule_Create(&module); }
