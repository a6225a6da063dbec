// efla_native.cpp -- the binding's short way for calls whose time is the call itself: the per-channel
// recurrence, the state cache and the steps on it.
//
// A token of a few sequences takes 2 to 6 us on the device, and the checks, allocations and argument
// conversions of the Python layer 8 to 12 us.  Here an ordinary call (plain CUDA tensors of the current device,
// on its current stream) is checked and made in 2 to 3 us.  Whatever is not ordinary, wrong arguments included, gives
// None: the Python layer then makes the call, or says what is wrong with it.  A call that the library
// refuses gives its status, an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>

#include <vector>

#include "../../include/efla.h"

namespace {

// The entry points of the library that the Python layer has loaded.
struct Entries {
    decltype(&efla_scan_workspace_bytes) scan_workspace_bytes;
    decltype(&efla_scan_fwd) scan_fwd;
    decltype(&efla_scan_backward_workspace_bytes) scan_backward_workspace_bytes;
    decltype(&efla_scan_backward) scan_backward;
    decltype(&efla_scan_step) scan_step;
    decltype(&efla_scan_step_paged) scan_step_paged;
    decltype(&efla_recurrent_step_paged) recurrent_step_paged;
    decltype(&efla_pages_fork) pages_fork;
    decltype(&efla_pages_copy) pages_copy;
    decltype(&efla_pages_free) pages_free;
    decltype(&efla_pages_compact) pages_compact;
};
constexpr int kEntries = sizeof(Entries) / sizeof(void*);
constexpr const char* kCapsule = "efla_entries";

struct NotOrdinary {};
void need(bool ok) {
    if (!ok) throw NotOrdinary();
}

using Sizes = at::IntArrayRef;

const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_CheckExact(o));
    return THPVariable_Unpack(o);
}
bool plain(const at::Tensor& t, int dev, at::ScalarType type) {
    return t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.scalar_type() == type;
}
// The address of a contiguous tensor of this device, type and shape (None: null).
void* address(PyObject* o, int dev, at::ScalarType type, Sizes shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    need(plain(t, dev, type) && t.sizes() == shape && t.is_contiguous());
    return t.data_ptr();
}
int to_int(PyObject* o) {
    need(PyLong_CheckExact(o));
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    need(!overflow && v >= INT_MIN && v <= INT_MAX);
    return (int)v;
}
int size(int64_t n) {
    need(n <= INT_MAX);
    return (int)n;
}
int element(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kFloat);
    return t == at::kBFloat16 ? EFLA_DTYPE_BF16 : EFLA_DTYPE_F32;
}

// The call's device has to be the current one; its current stream.
struct Place {
    int dev;
    efla_stream_t stream;
    explicit Place(const at::Tensor& t) {
        need(t.is_cuda());
        dev = t.get_device();
        need(c10::cuda::current_device() == dev);
        stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    }
    // (past the dispatcher, which takes longer than the allocation)
    at::Tensor empty(at::ScalarType type, Sizes shape) const {
        return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, dev), std::nullopt));
    }
};

// An output: the caller's, or one made here.  It is a Python object before the call is made, so that nothing can
// fail behind it.
struct Output {
    PyObject* object = nullptr;
    void* p = nullptr;
    Output() = default;
    Output(const Output&) = delete;
    ~Output() { Py_XDECREF(object); }
    void take(PyObject* given, const Place& at, at::ScalarType type, Sizes shape) {
        p = address(given, at.dev, type, shape);
        Py_INCREF(given);
        object = given;
    }
    void make(const Place& at, at::ScalarType type, Sizes shape, bool zeros = false) {
        at::Tensor t = at.empty(type, shape);
        if (zeros) t.zero_();
        p = t.data_ptr();
        object = THPVariable_Wrap(std::move(t));
        need(object);
    }
    void none() {
        Py_INCREF(Py_None);
        object = Py_None;
    }
    PyObject* release() {
        PyObject* o = object;
        object = nullptr;
        return o;
    }
};

struct Cache {
    void* block;
    int n_pages, n_slots;
    Cache(PyObject* block_, PyObject* pages, PyObject* slots, int dev) {
        const at::Tensor& t = tensor(block_);
        n_pages = to_int(pages);
        n_slots = to_int(slots);
        need(plain(t, dev, at::kInt) && t.dim() == 1 && t.is_contiguous() && n_pages > 0 && n_slots > 0 &&
             (size_t)t.numel() * 4 >= (64 + 2 * (size_t)n_slots + 3 * (size_t)n_pages) * 4);
        block = t.data_ptr();
    }
};
// A pool [n_pages, ...] whose pages may lie apart, each contiguous.
struct Pool {
    void* p;
    size_t page, data;
    Pool(PyObject* o, const Cache& cache, int dev) {
        const at::Tensor& t = tensor(o);
        need(t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.dim() >= 2 &&
             t.size(0) == cache.n_pages && t.numel() > 0);
        data = (size_t)(t.numel() / t.size(0)) * t.element_size();
        int64_t want = 1;
        for (int64_t i = t.dim() - 1; i > 0; want *= t.size(i--)) need(t.size(i) == 1 || t.stride(i) == want);
        need(t.size(0) == 1 || t.stride(0) > 0);
        page = t.size(0) == 1 ? data : (size_t)t.stride(0) * t.element_size();
        p = t.data_ptr();
    }
};
const int* list(PyObject* o, int dev, int64_t n) {
    return static_cast<const int*>(address(o, dev, at::kInt, Sizes(&n, 1)));
}

// Offsets of a packed batch: a list of ints, or a CPU int32 tensor.
struct CuSeqlens {
    std::vector<int> copy;
    const int* p = nullptr;
    int n = 0;      // sequences
    explicit CuSeqlens(PyObject* o) {
        if (o == Py_None) return;
        if (PyList_CheckExact(o)) {
            const Py_ssize_t m = PyList_GET_SIZE(o);
            need(m >= 2 && m <= INT_MAX);
            copy.resize(m);
            for (Py_ssize_t i = 0; i < m; ++i) copy[i] = to_int(PyList_GET_ITEM(o, i));
            p = copy.data();
            n = (int)m - 1;
            return;
        }
        const at::Tensor& t = tensor(o);
        need(t.layout() == at::kStrided && t.is_cpu() && t.scalar_type() == at::kInt && t.dim() == 1 && t.is_contiguous() &&
             t.numel() >= 2);
        p = t.const_data_ptr<int>();
        n = size(t.numel() - 1);
    }
};

struct ScanShape {
    int B, H, T, d, gw, dt;
    at::ScalarType type;
    Sizes x, g;
    int64_t state[3];
    ScanShape(const at::Tensor& xt, const at::Tensor& gt, const CuSeqlens& cu) {
        const int lead = cu.p ? 1 : 2;
        need(xt.dim() == lead + 2 && (gt.dim() == xt.dim() || gt.dim() == xt.dim() - 1));
        B = cu.p ? cu.n : size(xt.size(0));
        H = size(xt.size(lead - 1));
        T = size(xt.size(lead));
        d = size(xt.size(lead + 1));
        gw = gt.dim() == xt.dim() ? d : 1;
        type = xt.scalar_type();
        dt = element(type);
        x = xt.sizes();
        g = gw == d && gt.dim() == xt.dim() ? x : x.slice(0, x.size() - 1);
        need(xt.numel() > 0);
        state[0] = B, state[1] = H, state[2] = d;
    }
};

template <typename Call>
PyObject* ordinary(Call call) {
    try {
        return call();
    } catch (...) {      // what went wrong shows again when the Python layer makes the call
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}
// Without the interpreter's lock: a launch may wait for room in the queue.
template <typename Call>
int unlocked(Call call) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call();
    Py_END_ALLOW_THREADS
    return status;
}
const Entries& entries(PyObject* o) {
    const void* p = PyCapsule_GetPointer(o, kCapsule);
    need(p);
    return *static_cast<const Entries*>(p);
}
PyObject* done(int status, Output& o) { return status == EFLA_OK ? o.release() : PyLong_FromLong(status); }

// (entries, x, g, S0, cu_seqlens, o, S_T, workspace, want_state, rule) -> (o, S_T, workspace)
PyObject* scan_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 10);
        const Entries& e = entries(a[0]);
        const at::Tensor& xt = tensor(a[1]);
        const Place at(xt);
        const CuSeqlens cu(a[4]);
        const ScanShape s(xt, tensor(a[2]), cu);
        const void* x = address(a[1], at.dev, s.type, s.x);
        const float* g = static_cast<const float*>(address(a[2], at.dev, at::kFloat, s.g));
        const float* S0 = static_cast<const float*>(address(a[3], at.dev, at::kFloat, s.state));
        const int rule = to_int(a[9]);
        Output o, S_T, ws;
        if (a[5] == Py_None) o.make(at, s.type, s.x);
        else o.take(a[5], at, s.type, s.x);
        need(PyBool_Check(a[8]));
        if (a[6] == Py_None && a[8] == Py_True) S_T.make(at, at::kFloat, s.state);
        else if (a[6] == Py_None) S_T.none();
        else S_T.take(a[6], at, at::kFloat, s.state);
        int64_t bytes;
        if (a[7] == Py_None) {
            bytes = (int64_t)e.scan_workspace_bytes(s.B, s.H, s.T, s.d, s.gw, s.dt, cu.p != nullptr);
            need(bytes > 0);
            ws.make(at, at::kByte, Sizes(&bytes, 1));
        } else {
            bytes = tensor(a[7]).numel();
            ws.take(a[7], at, at::kByte, Sizes(&bytes, 1));
        }
        PyObject* out = PyTuple_New(3);
        need(out);
        const int status = unlocked([&] {
            return e.scan_fwd(x, g, cu.p, S0, o.p, static_cast<float*>(S_T.p), s.B, s.H, s.T, s.d, s.gw, s.dt, rule, ws.p,
                              (size_t)bytes, at.stream);
        });
        if (status != EFLA_OK) {
            Py_DECREF(out);
            return PyLong_FromLong(status);
        }
        PyTuple_SET_ITEM(out, 0, o.release());
        PyTuple_SET_ITEM(out, 1, S_T.release());
        PyTuple_SET_ITEM(out, 2, ws.release());
        return out;
    });
}

// (entries, x, g, dO, S0, dS_T, saved, cu_seqlens, want_dS0, rule) -> (dx, dg, dS0)
PyObject* scan_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 10);
        const Entries& e = entries(a[0]);
        const at::Tensor& xt = tensor(a[1]);
        const Place at(xt);
        const CuSeqlens cu(a[7]);
        const ScanShape s(xt, tensor(a[2]), cu);
        const void *x = address(a[1], at.dev, s.type, s.x), *dO = address(a[3], at.dev, s.type, s.x);
        const float* g = static_cast<const float*>(address(a[2], at.dev, at::kFloat, s.g));
        const float* S0 = static_cast<const float*>(address(a[4], at.dev, at::kFloat, s.state));
        const float* dS_T = static_cast<const float*>(address(a[5], at.dev, at::kFloat, s.state));
        const int rule = to_int(a[9]);
        int64_t saved_bytes = a[6] == Py_None ? 0 : tensor(a[6]).numel();
        const void* saved = address(a[6], at.dev, at::kByte, Sizes(&saved_bytes, 1));
        const int64_t bytes = (int64_t)e.scan_backward_workspace_bytes(s.B, s.H, s.T, s.d, s.gw, s.dt, cu.p != nullptr,
                                                                       saved != nullptr);
        need(bytes > 0);
        Output dx, dg, dS0;
        dx.make(at, at::kFloat, s.x);
        dg.make(at, at::kFloat, s.g);
        need(PyBool_Check(a[8]));
        if (a[8] == Py_True) dS0.make(at, at::kFloat, s.state);
        else dS0.none();
        const at::Tensor ws = at.empty(at::kByte, Sizes(&bytes, 1));
        void* pws = ws.data_ptr();
        PyObject* out = PyTuple_New(3);
        need(out);
        const int status = unlocked([&] {
            return e.scan_backward(x, g, cu.p, S0, dO, dS_T, static_cast<float*>(dx.p), static_cast<float*>(dg.p),
                                   static_cast<float*>(dS0.p), s.B, s.H, s.T, s.d, s.gw, s.dt, rule, saved,
                                   (size_t)saved_bytes, pws, (size_t)bytes, at.stream);
        });
        if (status != EFLA_OK) {
            Py_DECREF(out);
            return PyLong_FromLong(status);
        }
        PyTuple_SET_ITEM(out, 0, dx.release());
        PyTuple_SET_ITEM(out, 1, dg.release());
        PyTuple_SET_ITEM(out, 2, dS0.release());
        return out;
    });
}

struct StepShape {
    int N, H, d, gw, dt;
    at::ScalarType type;
    Sizes x, g;
    StepShape(const at::Tensor& xt, const at::Tensor& gt) {
        need(xt.dim() == 3 && (gt.dim() == 3 || gt.dim() == 2) && xt.numel() > 0);
        x = xt.sizes();
        N = size(x[0]), H = size(x[1]), d = size(x[2]);
        gw = gt.dim() == 3 ? d : 1;
        g = gt.dim() == 3 ? x : x.slice(0, 2);
        type = xt.scalar_type();
        dt = element(type);
    }
};

// (entries, x, g, S, o, rule) -> o
PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 6);
        const Entries& e = entries(a[0]);
        const at::Tensor& xt = tensor(a[1]);
        const Place at(xt);
        const StepShape s(xt, tensor(a[2]));
        const void* x = address(a[1], at.dev, s.type, s.x);
        const float* g = static_cast<const float*>(address(a[2], at.dev, at::kFloat, s.g));
        float* S = static_cast<float*>(address(a[3], at.dev, at::kFloat, s.x));
        const int rule = to_int(a[5]);
        Output o;
        if (a[4] == Py_None) o.make(at, s.type, s.x);
        else o.take(a[4], at, s.type, s.x);
        return done(unlocked([&] { return e.scan_step(x, g, S, o.p, s.N, s.H, s.d, s.gw, s.dt, rule, at.stream); }), o);
    });
}

// (entries, x, g, block, n_pages, n_slots, pool, slots, source, o, rule) -> o
PyObject* scan_step_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 11);
        const Entries& e = entries(a[0]);
        const at::Tensor& xt = tensor(a[1]);
        const Place at(xt);
        const StepShape s(xt, tensor(a[2]));
        const void* x = address(a[1], at.dev, s.type, s.x);
        const float* g = static_cast<const float*>(address(a[2], at.dev, at::kFloat, s.g));
        const Cache cache(a[3], a[4], a[5], at.dev);
        const at::Tensor& pt = tensor(a[6]);
        need(pt.scalar_type() == at::kFloat && pt.dim() == 3 && pt.sizes().slice(1) == s.x.slice(1));
        const Pool pool(a[6], cache, at.dev);
        const int *slots = list(a[7], at.dev, s.N), *source = list(a[8], at.dev, s.N);
        const int rule = to_int(a[10]);
        Output o;
        if (a[9] == Py_None) o.make(at, s.type, s.x, true);
        else o.take(a[9], at, s.type, s.x);
        return done(unlocked([&] {
                        return e.scan_step_paged(x, g, cache.block, cache.n_pages, cache.n_slots, static_cast<float*>(pool.p),
                                                 pool.page, slots, source, o.p, s.N, s.H, s.d, s.gw, s.dt, rule, at.stream);
                    }), o);
    });
}

// (entries, q, k, v, beta, block, n_pages, n_slots, pool, slots, source, g, o, rule) -> o
PyObject* recurrent_step_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 14);
        const Entries& e = entries(a[0]);
        const at::Tensor &kt = tensor(a[2]), &vt = tensor(a[3]);
        const Place at(kt);
        need(kt.dim() == 3 && vt.dim() == 3 && kt.numel() > 0);
        const Sizes ks = kt.sizes();
        const at::ScalarType type = kt.scalar_type();
        const int dt = element(type), N = size(ks[0]), H = size(ks[1]), dk = size(ks[2]), dv = size(vt.size(2));
        const int64_t vs[3] = {N, H, dv};
        const void *q = address(a[1], at.dev, type, ks), *k = address(a[2], at.dev, type, ks);
        const void *v = address(a[3], at.dev, type, vs), *beta = address(a[4], at.dev, type, ks.slice(0, 2));
        const float* g = static_cast<const float*>(address(a[11], at.dev, at::kFloat, ks.slice(0, 2)));
        const Cache cache(a[5], a[6], a[7], at.dev);
        const at::Tensor& pt = tensor(a[8]);
        need(pt.scalar_type() == at::kFloat && pt.dim() == 4 && pt.size(1) == H && pt.size(2) == dk && pt.size(3) == dv);
        const Pool pool(a[8], cache, at.dev);
        const int *slots = list(a[9], at.dev, N), *source = list(a[10], at.dev, N);
        const int rule = to_int(a[13]);
        Output o;
        if (a[12] == Py_None) o.make(at, type, vs, true);
        else o.take(a[12], at, type, vs);
        return done(unlocked([&] {
                        return e.recurrent_step_paged(q, k, v, beta, g, cache.block, cache.n_pages, cache.n_slots,
                                                      static_cast<float*>(pool.p), pool.page, slots, source, o.p, N, H, dk,
                                                      dv, dt, rule, at.stream);
                    }), o);
    });
}

// (entries, block, n_pages, n_slots, pool, source, dest) -> status; a fork's pool may be None
template <bool kFork>
PyObject* pages_pairs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 7);
        const Entries& e = entries(a[0]);
        const at::Tensor& bt = tensor(a[1]);
        const Place at(bt);
        const Cache cache(a[1], a[2], a[3], at.dev);
        const at::Tensor& dest_t = tensor(a[6]);
        const int count = size(dest_t.numel());
        const int *dest = list(a[6], at.dev, count), *source = list(a[5], at.dev, count);
        void* pool = nullptr;
        size_t page = 0, data = 0;
        if (!kFork || a[4] != Py_None) {
            const Pool p(a[4], cache, at.dev);
            pool = p.p, page = p.page, data = p.data;
        }
        return PyLong_FromLong(unlocked([&] {
            return (kFork ? e.pages_fork : e.pages_copy)(cache.block, cache.n_pages, cache.n_slots, pool, page, data, source,
                                                         dest, count, at.stream);
        }));
    });
}

// (entries, block, n_pages, n_slots, slots) -> status
PyObject* pages_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 5);
        const Entries& e = entries(a[0]);
        const Place at(tensor(a[1]));
        const Cache cache(a[1], a[2], a[3], at.dev);
        const int count = size(tensor(a[4]).numel());
        const int* slots = list(a[4], at.dev, count);
        return PyLong_FromLong(
            unlocked([&] { return e.pages_free(cache.block, cache.n_pages, cache.n_slots, slots, count, at.stream); }));
    });
}

// (entries, block, n_pages, n_slots, pool) -> status
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 5);
        const Entries& e = entries(a[0]);
        const Place at(tensor(a[1]));
        const Cache cache(a[1], a[2], a[3], at.dev);
        const Pool pool(a[4], cache, at.dev);
        return PyLong_FromLong(unlocked([&] {
            return e.pages_compact(cache.block, cache.n_pages, cache.n_slots, pool.p, pool.page, pool.data, at.stream);
        }));
    });
}

// (addresses in the order of Entries) -> the capsule that the calls above take
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != kEntries) {
        PyErr_SetString(PyExc_TypeError, "bind takes the address of every entry point");
        return nullptr;
    }
    void** table = static_cast<void**>(PyMem_Malloc(sizeof(Entries)));
    if (!table) return PyErr_NoMemory();
    for (Py_ssize_t i = 0; i < n; ++i) table[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) {
        PyMem_Free(table);
        return nullptr;
    }
    return PyCapsule_New(table, kCapsule, [](PyObject* o) { PyMem_Free(PyCapsule_GetPointer(o, kCapsule)); });
}

#define EFLA_METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {EFLA_METHOD("bind", bind),
                          EFLA_METHOD("scan_fwd", scan_fwd),
                          EFLA_METHOD("scan_backward", scan_backward),
                          EFLA_METHOD("scan_step", scan_step),
                          EFLA_METHOD("scan_step_paged", scan_step_paged),
                          EFLA_METHOD("recurrent_step_paged", recurrent_step_paged),
                          EFLA_METHOD("pages_fork", pages_pairs<true>),
                          EFLA_METHOD("pages_copy", pages_pairs<false>),
                          EFLA_METHOD("pages_free", pages_free),
                          EFLA_METHOD("pages_compact", pages_compact),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_efla_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// EFLA_BUILT_FOR: the torch and the Python that this was built against, given by the build, which looks for the mark to
// see whether it still holds; the Python layer compares the version before it makes a call.
extern "C" __attribute__((used, visibility("default"))) const char efla_native_mark[] = "efla native: " EFLA_BUILT_FOR;

PyMODINIT_FUNC PyInit__efla_native() {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddStringConstant(m, "torch_version", EFLA_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
