// The torch side of the 8-bit cache and the rotary positions (kv8.py): checks of
// tensors, outputs, workspaces and streams in C++.  A single-token step makes a
// handful of these calls a layer, each a few microseconds on the GPU; through
// ctypes the same checks cost more than the kernels do.
//
// Errors: ValueError and TypeError for arguments, the package's TQError for a
// status of libtq.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <unordered_map>

#include "kv8_bind.h"

namespace {

PyObject* g_error = nullptr;  // TQError(fn, status)

struct Fail {};  // the Python error is set

void check(const char* fn, int status) {
    if (status == TQ_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "si", fn, status);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Fail();
}

struct Cache {
    tq_kv8_t c;
    c10::Device device;
    // per stream: calls of one stream follow one another
    std::unordered_map<cudaStream_t, at::Tensor> ws;
    at::Tensor status;  // c.d_status
};

const at::Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Fail();
    return v;
}
int int32(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, ": ", v, " does not fit 32 bits");
    return (int)v;
}

int code_of(at::ScalarType t) {
    return t == at::kFloat ? TQ_F32 : t == at::kBFloat16 ? TQ_BF16 : t == at::kHalf ? TQ_F16 : -1;
}

// [T, heads, d] with contiguous heads: itself, or a copy.
at::Tensor rows(PyObject* o, int64_t heads, int64_t d, const char* name) {
    const at::Tensor& x = tensor(o, name);
    TORCH_CHECK_VALUE(x.dim() == 3 && (heads < 0 || x.size(1) == heads) && x.size(2) == d, name,
                      ": expected [T, ", heads < 0 ? std::string("heads") : std::to_string(heads),
                      ", ", d, "], got ", x.sizes());
    TORCH_CHECK_TYPE(code_of(x.scalar_type()) >= 0, name, ": unsupported dtype ", x.scalar_type(),
                     "; expected float32, bfloat16 or float16");
    TORCH_CHECK_VALUE(x.is_cuda(), name, ": expected a CUDA tensor, got one on ", x.device());
    return x.stride(2) == 1 ? x : x.contiguous();
}

// What is computed here has no derivative for torch to find.
bool backward_grad(const at::Tensor& x) { return x.requires_grad() && c10::GradMode::is_enabled(); }
bool wants_grad(const at::Tensor& x) { return backward_grad(x) || x._fw_grad(0).defined(); }
void no_grad(const at::Tensor& x, const char* name, const char* call) {
    TORCH_CHECK_VALUE(!wants_grad(x), name, ": ", call, " has no gradient; detach() the tensor, or call it under "
                      "torch.no_grad()");
}

// A tensor that a call has written into: a graph that holds its old values is to know.
void written(const at::Tensor& x) {
    if (!x.is_inference()) x.unsafeGetTensorImpl()->bump_version();
}
// An output whose elements share no memory with each other, and with the input's either
// none or that of the same element.
void disjoint(const at::Tensor& out, const at::Tensor& in) {
    TORCH_CHECK_VALUE(at::has_internal_overlap(out) != at::MemOverlap::Yes,
                      "out: expected a tensor whose elements lie apart");
    TORCH_CHECK_VALUE(at::get_overlap_status(out, in) != at::MemOverlapStatus::Partial,
                      "out: overlaps the input in part");
}

// A contiguous [n] index tensor.
template <typename T>
const T* ints(PyObject* o, const char* name, int64_t n, c10::Device device) {
    const at::Tensor& t = tensor(o, name);
    const at::ScalarType want = sizeof(T) == 4 ? at::kInt : at::kLong;
    TORCH_CHECK_VALUE(t.scalar_type() == want && t.dim() == 1 && t.size(0) == n && t.device() == device,
                      name, ": expected [", n, "] ", want, " on ", device, ", got ", t.sizes(), " ",
                      t.scalar_type(), " on ", t.device());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, ": expected a contiguous tensor");
    return (const T*)t.data_ptr();
}

Cache* cache(PyObject* o) {
    Cache* c = (Cache*)PyCapsule_GetPointer(o, "tq.kv8");
    if (!c) throw Fail();
    TORCH_CHECK_VALUE(c->device.is_cuda(), "expected a CUDA tensor, got one on ", c->device);
    return c;
}
const tq_rope_params_t* rope_params(PyObject* o) {
    if (o == Py_None) return nullptr;
    const auto* r = (const tq_rope_params_t*)PyCapsule_GetPointer(o, "tq.rope");
    if (!r) throw Fail();
    return r;
}

struct Ws {
    void* ptr;
    size_t bytes;
    at::Tensor owner;  // until the call is launched
};
Ws workspace(Cache* c, int op, int n, int64_t total, int max_q, int heads_q, cudaStream_t stream) {
    const size_t need = tq_kv8_workspace_bytes(op, &c->c, n, total, max_q, heads_q);
    if (need == (size_t)-1) check("tq_kv8_workspace_bytes", TQ_ERR_UNSUPPORTED);
    const auto fresh = [&] {
        return at::detail::empty_cuda({(int64_t)(need < 256 ? 256 : need)}, at::kByte, c->device,
                                      std::nullopt);
    };
    // in a capture the graph's own memory: graphs that run side by side share nothing
    at::Tensor t;
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
        t = fresh();
    } else {
        at::Tensor& kept = c->ws[stream];
        if (!kept.defined() || (size_t)kept.numel() < need) kept = fresh();
        t = kept;
    }
    return {t.data_ptr(), (size_t)t.numel(), t};
}

void expect_args(Py_ssize_t got, Py_ssize_t want) {
    TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}

// A batch: entries, slots (or null), cumulative counts.
struct Batch {
    int ns;
    const int32_t *slots, *cu;
};
Batch batch(Cache* c, PyObject* slots, PyObject* cu) {
    const at::Tensor& t = tensor(cu, "cu");
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) >= 1, "cu: expected [entries + 1], got ", t.sizes());
    Batch b;
    b.ns = (int)t.size(0) - 1;
    b.slots = slots == Py_None ? nullptr : ints<int32_t>(slots, "slots", b.ns, c->device);
    b.cu = ints<int32_t>(cu, "cu", b.ns + 1, c->device);
    return b;
}

#define TQ_PY_BEGIN HANDLE_TH_ERRORS try {
#define TQ_PY_END                \
    }                            \
    catch (const Fail&) {        \
        return nullptr;          \
    }                            \
    END_HANDLE_TH_ERRORS

// (address of a tq_kv8_t, its status word) -> handle; the struct is copied.
PyObject* py_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 2);
    const at::Tensor& status = tensor(a[1], "status");
    const auto* s = (const tq_kv8_t*)PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) throw Fail();
    if (tq_kv8_workspace_bytes(TQ_KV8_OP_PAGES, s, 0, 0, 0, 0) == (size_t)-1)
        check("tq_kv8_workspace_bytes", TQ_ERR_UNSUPPORTED);
    return PyCapsule_New(new Cache{*s, status.device(), {}, status}, "tq.kv8", [](PyObject* o) {
        delete (Cache*)PyCapsule_GetPointer(o, "tq.kv8");
    });
    TQ_PY_END
}

// (address of a tq_rope_params_t) -> handle; the struct is copied.
PyObject* py_rope_params(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 1);
    const auto* r = (const tq_rope_params_t*)PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) throw Fail();
    return PyCapsule_New(new tq_rope_params_t(*r), "tq.rope", [](PyObject* o) {
        delete (tq_rope_params_t*)PyCapsule_GetPointer(o, "tq.rope");
    });
    TQ_PY_END
}

// (rope, x, pos, out or None, transpose); None where the caller is to differentiate
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 5);
    const tq_rope_params_t* r = rope_params(a[0]);
    const at::Tensor x = rows(a[1], -1, r->d, "x");
    if (a[3] == Py_None && backward_grad(x)) Py_RETURN_NONE;
    no_grad(x, "x", a[3] == Py_None ? "forward mode" : "a rotation into a given tensor");
    const int64_t T = x.size(0), heads = x.size(1);
    const int64_t* pos = ints<int64_t>(a[2], "pos", T, x.device());
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor out;
    if (a[3] == Py_None) {
        out = at::detail::empty_cuda(x.sizes(), x.scalar_type(), x.device(), std::nullopt);
    } else {
        out = tensor(a[3], "out");
        no_grad(out, "out", "a rotation into a given tensor");
        TORCH_CHECK_VALUE(out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type() &&
                              out.device() == x.device() && out.stride(2) == 1,
                          "out: expected x's shape, type and device, contiguous heads");
        disjoint(out, x);
    }
    TORCH_CHECK_VALUE(heads <= INT32_MAX, "x: too many heads");
    check("tq_rope", tq_rope(r, T, (int)heads, x.data_ptr(), x.stride(0), x.stride(1),
                             code_of(x.scalar_type()), pos, out.data_ptr(), out.stride(0),
                             out.stride(1), PyObject_IsTrue(a[4]),
                             c10::cuda::getCurrentCUDAStream(x.device().index()).stream()));
    if (a[3] != Py_None) written(out);
    return THPVariable_Wrap(std::move(out));
    TQ_PY_END
}

// (cache, operation, list, list): 0 reserve, 1 fork, 2 truncate
PyObject* py_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 4);
    static const struct {
        const char *fn, *first, *second;
        int (*call)(const tq_kv8_t*, int, const int32_t*, const int32_t*, void*, size_t, void*);
    } kOps[] = {{"tq_kv8_reserve", "slots", "counts", tq_kv8_reserve},
                {"tq_kv8_fork", "parents", "children", tq_kv8_fork},
                {"tq_kv8_truncate", "slots", "lens", tq_kv8_truncate}};
    Cache* c = cache(a[0]);
    const int64_t which = integer(a[1]);
    TORCH_CHECK_VALUE(which >= 0 && which < 3, "no such operation");
    const auto& op = kOps[which];
    const at::Tensor& first = tensor(a[2], op.first);
    const int64_t entries = first.dim() == 1 ? first.size(0) : -1;
    const int32_t* l0 = ints<int32_t>(a[2], op.first, entries, c->device);
    const int32_t* l1 = ints<int32_t>(a[3], op.second, entries, c->device);
    if (entries > 4096) check(op.fn, TQ_ERR_UNSUPPORTED);
    const c10::cuda::CUDAGuard guard(c->device);
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(c->device.index()).stream();
    const Ws w = workspace(c, TQ_KV8_OP_PAGES, (int)entries, 0, 0, 0, s);
    check(op.fn, op.call(&c->c, (int)entries, l0, l1, w.ptr, w.bytes, s));
    Py_RETURN_NONE;
    TQ_PY_END
}

// (cache)
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 1);
    Cache* c = cache(a[0]);
    const c10::cuda::CUDAGuard guard(c->device);
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(c->device.index()).stream();
    const Ws w = workspace(c, TQ_KV8_OP_PAGES, 0, 0, 0, 0, s);
    check("tq_kv8_compact", tq_kv8_compact(&c->c, w.ptr, w.bytes, s));
    Py_RETURN_NONE;
    TQ_PY_END
}

// Other threads of the interpreter go on meanwhile.
struct NoGil {
    PyThreadState* state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

// (cache): waits for the device -- a call may have run on any stream, in a graph
// too; what it raises it takes off the cache
PyObject* py_status(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 1);
    Cache* c = cache(a[0]);
    const c10::cuda::CUDAGuard guard(c->device);
    TORCH_CHECK(c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None,
                "status() waits for the device, which a graph capture cannot");
    const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream(c->device.index());
    {
        const NoGil no_gil;
        c10::cuda::device_synchronize();
    }
    const int status = tq_device_status(c->c.d_status, s.stream());
    if (status != TQ_OK && status != TQ_ERR_CUDA) {
        const c10::InferenceMode mode;  // (the cache may have been made in one)
        c->status.zero_();
        s.synchronize();  // (the next call may be on another stream)
    }
    check("tq_device_status", status);
    Py_RETURN_NONE;
    TQ_PY_END
}

// (cache, layer, k, v, cu, max_new, slots, rope)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 8);
    Cache* c = cache(a[0]);
    at::Tensor k = rows(a[2], c->c.heads, c->c.d, "k"), v = rows(a[3], c->c.heads, c->c.d, "v");
    TORCH_CHECK_VALUE(k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type() &&
                          k.device() == c->device && v.device() == c->device,
                      "k, v: expected one shape and type, on the cache's device");
    no_grad(k, "k", "append");
    no_grad(v, "v", "append");
    const c10::cuda::CUDAGuard guard(c->device);
    if (k.strides() != v.strides()) {
        k = k.contiguous();
        v = v.contiguous();
    }
    const Batch b = batch(c, a[6], a[4]);
    check("tq_kv8_append",
          tq_kv8_append(&c->c, int32(a[1], "layer"), b.ns, b.slots, b.cu, k.size(0),
                        int32(a[5], "max_new"), k.data_ptr(), v.data_ptr(), code_of(k.scalar_type()),
                        k.stride(0), k.stride(1), rope_params(a[7]),
                        c10::cuda::getCurrentCUDAStream(c->device.index()).stream()));
    Py_RETURN_NONE;
    TQ_PY_END
}

// (cache, layer, begin, cu, total, max_count, slots, dtype)
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 8);
    Cache* c = cache(a[0]);
    const Batch b = batch(c, a[6], a[3]);
    const int32_t* begin = ints<int32_t>(a[2], "begin", b.ns, c->device);
    TORCH_CHECK_TYPE(THPDtype_Check(a[7]), "dtype: expected a torch.dtype");
    const at::ScalarType t = ((THPDtype*)a[7])->scalar_type;
    TORCH_CHECK_TYPE(code_of(t) >= 0, "unsupported dtype ", t, "; expected float32, bfloat16 or float16");
    const int64_t total = integer(a[4]);
    TORCH_CHECK_VALUE(total >= 0, "total: ", total);
    const c10::cuda::CUDAGuard guard(c->device);
    at::Tensor out[2];
    for (at::Tensor& o : out)
        o = at::detail::empty_cuda({total, c->c.heads, c->c.d}, t, c->device, std::nullopt);
    const int max_count = int32(a[5], "max_count");
    if (b.ns == 0 || max_count == 0)  // (no launch)
        for (at::Tensor& o : out) o.zero_();
    check("tq_kv8_read", tq_kv8_read(&c->c, int32(a[1], "layer"), b.ns, b.slots, begin, b.cu, total,
                                     max_count, out[0].data_ptr(), out[1].data_ptr(), code_of(t),
                                     c10::cuda::getCurrentCUDAStream(c->device.index()).stream()));
    PyObject* pair = PyTuple_New(2);
    if (!pair) throw Fail();
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(out[0])));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(out[1])));
    return pair;
    TQ_PY_END
}

// (cache, layer, q, cu, max_q, slots, scale or None, causal, window, out, lse)
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    TQ_PY_BEGIN
    expect_args(n, 11);
    Cache* c = cache(a[0]);
    at::Tensor q = rows(a[2], -1, c->c.d, "q");
    TORCH_CHECK_VALUE(q.device() == c->device, "q: expected a tensor on ", c->device);
    no_grad(q, "q", "attention over the cache");
    const int64_t total = q.size(0), heads_q = q.size(1);
    TORCH_CHECK_VALUE(heads_q <= INT32_MAX, "q: too many heads");
    const c10::cuda::CUDAGuard guard(c->device);
    if ((uintptr_t)q.data_ptr() % 16 || q.stride(0) % 8 || q.stride(1) % 8)
        q = q.clone(at::MemoryFormat::Contiguous);
    at::Tensor out;
    if (a[9] == Py_None) {
        out = at::detail::empty_cuda(q.sizes(), q.scalar_type(), c->device, std::nullopt);
    } else {
        out = tensor(a[9], "out");
        no_grad(out, "out", "attention over the cache");
        TORCH_CHECK_VALUE(out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type() &&
                              out.device() == c->device && out.is_contiguous(),
                          "out: expected q's shape, type and device, contiguous");
        disjoint(out, q);
    }
    float* lse = nullptr;
    at::Tensor l;
    if (a[10] != Py_None) {
        l = tensor(a[10], "lse");
        no_grad(l, "lse", "attention over the cache");
        TORCH_CHECK_VALUE(l.dim() == 2 && l.size(0) == total && l.size(1) == heads_q &&
                              l.scalar_type() == at::kFloat && l.device() == c->device &&
                              l.is_contiguous(),
                          "lse: expected [total, heads_q] float32, contiguous");
        lse = (float*)l.data_ptr();
    }
    const Batch b = batch(c, a[5], a[3]);
    const bool fresh = a[9] == Py_None;
    double scale = 0.0;
    if (a[6] == Py_None) {
        scale = c->c.d == 64 ? 0.125 : 0.08838834764831845;  // 1 / sqrt(d)
    } else {
        scale = PyFloat_AsDouble(a[6]);
        if (scale == -1.0 && PyErr_Occurred()) throw Fail();
    }
    const int max_q = int32(a[4], "max_q");
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(c->device.index()).stream();
    const int layer = int32(a[1], "layer"), causal = PyObject_IsTrue(a[7]), window = int32(a[8], "window");
    // (a call of bad sizes gets no workspace: the entry point names what is wrong)
    Ws w = {nullptr, 0, {}};
    if (max_q >= 0 && heads_q >= 1 && heads_q % c->c.heads == 0)
        w = workspace(c, TQ_KV8_OP_ATTENTION, b.ns, total, max_q, (int)heads_q, s);
    if (fresh && (b.ns == 0 || max_q == 0)) out.zero_();  // (no launch)
    check("tq_kv8_attention",
          tq_kv8_attention_rows(&c->c, layer, b.ns, b.slots, b.cu, total, max_q, (int)heads_q,
                                q.data_ptr(), code_of(q.scalar_type()), q.stride(0), q.stride(1),
                                (float)scale, causal, window, out.data_ptr(), fresh, lse, w.ptr,
                                w.bytes, s));
    if (!fresh) written(out);
    if (lse) written(l);
    return THPVariable_Wrap(std::move(out));
    TQ_PY_END
}

// (TQError)
PyObject* py_init(PyObject*, PyObject* error) {
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    Py_RETURN_NONE;
}

#define TQ_FAST(f) (PyCFunction)(void (*)()) f, METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {{"init", py_init, METH_O, nullptr},
                           {"cache", TQ_FAST(py_cache)},
                           {"rope_params", TQ_FAST(py_rope_params)},
                           {"rope", TQ_FAST(py_rope)},
                           {"pages", TQ_FAST(py_pages)},
                           {"compact", TQ_FAST(py_compact)},
                           {"status", TQ_FAST(py_status)},
                           {"append", TQ_FAST(py_append)},
                           {"read", TQ_FAST(py_read)},
                           {"attention", TQ_FAST(py_attention)},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kv8", nullptr, -1, g_methods};

}  // namespace

// The torch that the module is built for (build.py looks for it in the file).
#define TQ_STR2(x) #x
#define TQ_STR(x) TQ_STR2(x)
static const char kTorch[] = "built for torch " TQ_STR(TQ_TORCH);

PyMODINIT_FUNC PyInit__kv8() {
    PyObject* m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", kTorch) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
