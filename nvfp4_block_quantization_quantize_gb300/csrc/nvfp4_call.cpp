// nvfp4_call.cpp -- the binding's short path for the serving operators.
//
// A call on a single token takes a few microseconds on the GPU, less than checking
// its tensors, allocating its outputs and marshalling its arguments takes in
// Python (12 to 20 us a call on the Grace host, about 5 here).  These functions do
// that for a well-formed call -- tensors of the right types and sizes, contiguous,
// on the current device -- and hand it to the C ABI on the current stream.
// For anything else they return None and enqueue nothing, and the Python function
// of the same name, which calls them first, goes through its own checks.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "nvfp4.h"

namespace {

decltype(&nvfp4_rmsnorm) f_rmsnorm = nullptr;
decltype(&nvfp4_mv) f_mv = nullptr;
decltype(&nvfp4_grouped_mm) f_grouped_mm = nullptr;
decltype(&nvfp4_grouped_mm_workspace) f_grouped_ws = nullptr;
decltype(&nvfp4_qk_norm_rope) f_rope = nullptr;
decltype(&nvfp4_cache_write) f_cache_write = nullptr;
decltype(&nvfp4_cache_read) f_cache_read = nullptr;
decltype(&nvfp4_cache_attention) f_attention = nullptr;
decltype(&nvfp4_cache_attention_workspace) f_attention_ws = nullptr;

PyObject* none() { Py_RETURN_NONE; }

// a contiguous CUDA tensor on device dev, or null
const at::Tensor* tensor(PyObject* o, int dev) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.get_device() == dev && t.is_contiguous() ? &t : nullptr;
}

const at::Tensor* tensor(PyObject* o, int dev, at::ScalarType type, int64_t numel) {
    const at::Tensor* t = tensor(o, dev);
    return t && t->scalar_type() == type && t->numel() == numel ? t : nullptr;
}

// the current device if the call's first tensor is on it, else -1 (a host tensor
// makes no CUDA call)
int call_device(PyObject* o) {
    if (!THPVariable_Check(o)) return -1;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.get_device() == c10::cuda::current_device() ? static_cast<int>(t.get_device()) : -1;
}

bool given(PyObject* o) { return o != Py_None; }

void* data(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// nvfp4_dtype of a floating tensor, -1 for another type
int dtype_of(const at::Tensor& t) {
    return t.scalar_type() == at::kFloat ? NVFP4_F32 : t.scalar_type() == at::kBFloat16 ? NVFP4_BF16 : -1;
}

// the position of a string argument in names, -1 for anything else
int choice(PyObject* o, std::initializer_list<const char*> names) {
    if (!PyUnicode_Check(o)) return -1;
    int i = 0;
    for (const char* n : names) {
        if (PyUnicode_CompareWithASCIIString(o, n) == 0) return i;
        ++i;
    }
    return -1;
}

bool number(PyObject* o, float* v) {
    if (!PyFloat_Check(o)) return false;
    *v = static_cast<float>(PyFloat_AS_DOUBLE(o));
    return true;
}

at::Tensor empty(int64_t rows, int64_t cols, at::ScalarType type, int dev) {
    return at::detail::empty_cuda({rows, cols}, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)),
                                  std::nullopt);
}

// Outputs up to this many bytes together share one allocation (an allocation costs
// about 2 us on the Grace host between other work; larger ones are kept apart so that
// one output does not hold the others' memory).
constexpr int64_t kShared = 1 << 20;

// a contiguous tensor of `base`'s storage from byte `at` on, which moves past it (to a multiple of 256)
at::Tensor part(const at::Tensor& base, int64_t* at, int64_t rows, int64_t cols, at::ScalarType type) {
    const int64_t size = static_cast<int64_t>(c10::elementSize(type));
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(*at / size);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({rows, cols});
    *at += (rows * cols * size + 255) / 256 * 256;
    return t;
}

// the global amax of `rows` rows: one value or one per row
bool rows_gamax(PyObject* o, int64_t rows, int dev, int* mode, const at::Tensor** t) {
    *t = nullptr;
    *mode = NVFP4_GAMAX_NONE;
    if (!given(o)) return true;
    *t = tensor(o, dev);
    if (!*t || (*t)->scalar_type() != at::kFloat) return false;
    *mode = (*t)->numel() == 1 ? NVFP4_GAMAX_TENSOR_GIVEN : NVFP4_GAMAX_ROW_GIVEN;
    return (*t)->numel() == 1 || (*t)->numel() == rows;
}

// *t is the given output if there is one; false if it does not fit
bool taken(PyObject* o, int64_t numel, at::ScalarType type, int dev, at::Tensor* t) {
    if (!given(o)) return true;
    const at::Tensor* g = tensor(o, dev, type, numel);
    if (g) *t = *g;
    return g != nullptr;
}

// While one lives this thread does not hold the interpreter's lock.  Allocations and launches may block (a
// full launch queue, freed memory that other streams still use) until something that another Python thread
// does; the arguments are the caller's and stay.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject* wrap(PyObject* o, const at::Tensor& t) {        // a given output is returned itself
    if (given(o)) {
        Py_INCREF(o);
        return o;
    }
    return THPVariable_Wrap(t);
}

// the Python exception torch makes of the C++ one in flight (torch.OutOfMemoryError of an allocation that failed)
PyObject* raised() {
    HANDLE_TH_ERRORS
    throw;
    END_HANDLE_TH_ERRORS
}

template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (...) {
        return raised();
    }
}

// mv(x, codes, scales, x_scales, gamax, scale_bound, out_dtype, out)
PyObject* mv(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        float bound;
        if (n != 8 || !f_mv || !number(v[5], &bound)) return none();
        const int dev = call_device(v[0]);
        if (dev < 0) return none();
        const at::Tensor *x = tensor(v[0], dev), *codes = tensor(v[1], dev), *xs = nullptr, *g;
        if (!x || !codes || x->dim() != 2 || codes->dim() != 2 || codes->scalar_type() != at::kByte) return none();
        const int64_t M = x->size(0), K = x->size(1), N = codes->size(0);
        if (codes->size(1) * 2 != K || K % 16) return none();
        const at::Tensor* scales = tensor(v[2], dev, at::kByte, N * K / 16);
        if (!scales) return none();
        int type = dtype_of(*x), mode;
        if (given(v[3])) {
            if (x->scalar_type() != at::kByte && x->scalar_type() != at::kFloat8_e4m3fn) return none();
            xs = tensor(v[3], dev);
            if (!xs || xs->numel() != M * ((K + 31) / 32) ||
                (xs->scalar_type() != at::kByte && xs->scalar_type() != at::kFloat8_e8m0fnu))
                return none();
            type = NVFP4_X_MXFP8;
        }
        const int odt = choice(v[6], {"f32", "bf16"});
        at::Tensor out;
        const at::ScalarType ot = odt == NVFP4_F32 ? at::kFloat : at::kBFloat16;
        if (type < 0 || odt < 0 || !rows_gamax(v[4], N, dev, &mode, &g) || !taken(v[7], M * N, ot, dev, &out)) return none();
        int rc;
        {
            const Unlocked unlocked;
            if (!out.defined()) out = empty(M, N, ot, dev);
            rc = f_mv(x->data_ptr(), static_cast<const uint8_t*>(data(xs)), type,
                      static_cast<const uint8_t*>(codes->data_ptr()), static_cast<const uint8_t*>(scales->data_ptr()), M, N, K,
                      mode, static_cast<const float*>(data(g)), bound, out.data_ptr(), odt,
                      c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
        }
        return rc == NVFP4_OK ? wrap(v[7], out) : none();
    });
}

// grouped_mm(codes_a, scales_a, offsets, codes_b, scales_b, gamax_a, gamax_b, scale_bound, out_dtype, out)
PyObject* grouped_mm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        float bound;
        if (n != 10 || !f_grouped_mm || !number(v[7], &bound)) return none();
        const int dev = call_device(v[0]);
        if (dev < 0) return none();
        const at::Tensor *ca = tensor(v[0], dev), *cb = tensor(v[3], dev), *ga, *gb = nullptr;
        if (!ca || !cb || ca->dim() != 2 || cb->dim() != 3 || ca->scalar_type() != at::kByte ||
            cb->scalar_type() != at::kByte)
            return none();
        const int64_t T = ca->size(0), K = ca->size(1) * 2, E = cb->size(0), N = cb->size(1);
        if (cb->size(2) * 2 != K || K % 64) return none();
        const at::Tensor* sa = tensor(v[1], dev, at::kByte, T * K / 16);
        const at::Tensor* off = tensor(v[2], dev, at::kLong, E + 1);
        const at::Tensor* sb = tensor(v[4], dev, at::kByte, E * ((N + 127) / 128 * 128) * (K / 16));
        if (!sa || !off || !sb) return none();
        if (given(v[6]) && !(gb = tensor(v[6], dev, at::kFloat, E))) return none();
        int mode;
        const int odt = choice(v[8], {"f32", "bf16"});
        at::Tensor out;
        const at::ScalarType ot = odt == NVFP4_F32 ? at::kFloat : at::kBFloat16;
        if (odt < 0 || !rows_gamax(v[5], T, dev, &mode, &ga) || !taken(v[9], T * N, ot, dev, &out)) return none();
        int rc;
        {
            const Unlocked unlocked;
            if (!out.defined()) out = empty(T, N, ot, dev);
            const int64_t need = f_grouped_ws(E, T, N, K);
            at::Tensor ws;                                // free for the stream's next work once this call is enqueued
            if (need > 0) ws = empty(1, need, at::kByte, dev);
            rc = f_grouped_mm(
                static_cast<const uint8_t*>(ca->data_ptr()), static_cast<const uint8_t*>(sa->data_ptr()),
                static_cast<const int64_t*>(off->data_ptr()), static_cast<const uint8_t*>(cb->data_ptr()),
                static_cast<const uint8_t*>(sb->data_ptr()), E, T, N, K, mode, static_cast<const float*>(data(ga)),
                static_cast<const float*>(data(gb)), bound, out.data_ptr(), odt,
                need > 0 ? static_cast<uint8_t*>(ws.data_ptr()) : nullptr, need,
                c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
        }
        return rc == NVFP4_OK ? wrap(v[9], out) : none();
    });
}

bool put(PyObject* d, const char* key, PyObject* value) {
    if (!value) return false;
    const int rc = PyDict_SetItemString(d, key, value);
    Py_DECREF(value);
    return rc == 0;
}

// rmsnorm(x, weight, hidden, hidden_out, eps, format, want_out, out, codes, scales): no gamax, codes wanted
PyObject* rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        float eps;
        if (n != 10 || !f_rmsnorm || !number(v[4], &eps)) return none();
        const int dev = call_device(v[0]);
        if (dev < 0) return none();
        const at::Tensor *x = tensor(v[0], dev), *w = nullptr, *hidden = nullptr;
        if (!x || x->dim() != 2 || (v[6] != Py_True && v[6] != Py_False)) return none();
        const int64_t M = x->size(0), K = x->size(1);
        const int dt = dtype_of(*x), fmt = choice(v[5], {"nvfp4", "mxfp8"});
        if (dt < 0 || fmt < 0 || K % 16) return none();
        int wdt = dt;
        if (given(v[1])) {
            w = tensor(v[1], dev);
            if (!w || w->numel() != K || (wdt = dtype_of(*w)) < 0) return none();
        }
        at::Tensor hidden_out, out, codes, scales, shared;
        if (given(v[2]) ? !(hidden = tensor(v[2], dev, x->scalar_type(), M * K)) : given(v[3])) return none();
        const bool want_out = given(v[7]) || v[6] == Py_True, mx = fmt == NVFP4_FMT_MXFP8;
        const int64_t cols = mx ? K : K / 2, groups = mx ? (K + 31) / 32 : K / 16;
        const at::ScalarType xt = x->scalar_type();
        if ((hidden && !taken(v[3], M * K, xt, dev, &hidden_out)) || !taken(v[7], M * K, xt, dev, &out) ||
            !taken(v[8], M * cols, at::kByte, dev, &codes) || !taken(v[9], M * groups, at::kByte, dev, &scales))
            return none();
        int rc;
        {
            const Unlocked unlocked;
            const int64_t full = M * K * static_cast<int64_t>(x->element_size());
            const int64_t bytes = (hidden ? full : 0) + (want_out ? full : 0) + M * (cols + groups) + 4 * 256;
            int64_t at = 0;
            if (bytes <= kShared) shared = empty(1, bytes, at::kByte, dev);
            auto make = [&](at::Tensor& t, int64_t n, at::ScalarType type) {
                if (!t.defined()) t = shared.defined() ? part(shared, &at, M, n, type) : empty(M, n, type, dev);
            };
            if (hidden) make(hidden_out, K, xt);
            if (want_out) make(out, K, xt);
            make(codes, cols, at::kByte);
            make(scales, groups, at::kByte);
            rc = f_rmsnorm(x->data_ptr(), data(hidden), M, K, dt, data(w), wdt, eps, hidden ? hidden_out.data_ptr() : nullptr,
                           want_out ? out.data_ptr() : nullptr, fmt, NVFP4_GAMAX_NONE, nullptr, 448.0f,
                           static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr()),
                           c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
        }
        if (rc != NVFP4_OK) return none();
        PyObject* d = PyDict_New();
        if (!d) return nullptr;
        if ((hidden && !put(d, "hidden", wrap(v[3], hidden_out))) || (want_out && !put(d, "out", wrap(v[7], out))) ||
            !put(d, "codes", wrap(v[8], codes)) || !put(d, "scales", wrap(v[9], scales))) {
            Py_DECREF(d);
            return nullptr;
        }
        return d;
    });
}

// ---- a cache of keys and values ----------------------------------------------------------------
// [T, H, D] heads of a floating type, a token's contiguous, tokens whole 16 bytes apart
const at::Tensor* heads(PyObject* o, int dev, int64_t* stride) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || t.dim() != 3 || t.numel() == 0 || dtype_of(t) < 0) return nullptr;
    const int64_t size = static_cast<int64_t>(t.element_size());
    if (t.stride(2) != 1 || t.stride(1) != t.size(2) || t.stride(0) < 0 || t.stride(0) * size % 16 ||
        reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
        return nullptr;
    *stride = t.stride(0);
    return &t;
}

// a cache and the global scales of its keys and values
struct Cache {
    const at::Tensor *t = nullptr, *k_gamax, *v_gamax;
    int k_mode, v_mode;
    int64_t pages, page_size, Hkv, D;

    bool take(PyObject* o, PyObject* kg, PyObject* vg, int dev) {
        t = tensor(o, dev);
        if (!t || t->scalar_type() != at::kByte || t->dim() != 4 || t->numel() == 0 || t->size(3) % 18) return false;
        pages = t->size(0), Hkv = t->size(1), page_size = t->size(2) * 16, D = t->size(3) / 18;
        return rows_gamax(kg, Hkv, dev, &k_mode, &k_gamax) && rows_gamax(vg, Hkv, dev, &v_mode, &v_gamax);
    }
    uint8_t* bytes() const { return static_cast<uint8_t*>(t->data_ptr()); }
    const float* kg() const { return static_cast<const float*>(data(k_gamax)); }
    const float* vg() const { return static_cast<const float*>(data(v_gamax)); }
};

at::Tensor empty3(int64_t a, int64_t b, int64_t c, at::ScalarType type, int dev) {
    return at::detail::empty_cuda({a, b, c}, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

cudaStream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// qk_norm_rope(q, k, positions, phases, q_weight, k_weight, eps, layout, magnitude, q_out, k_out, cache, v, slots, k_gamax,
// v_gamax, scale_bound)
PyObject* qk_norm_rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        float eps, magnitude, bound;
        if (n != 17 || !f_rope || !number(v[6], &eps) || !number(v[8], &magnitude) || !number(v[16], &bound)) return none();
        const int dev = call_device(v[0]);
        if (dev < 0) return none();
        int64_t qs, ks, vs = 0;
        const at::Tensor *q = heads(v[0], dev, &qs), *k = heads(v[1], dev, &ks), *x = nullptr;
        if (!q || !k) return none();
        const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), Hkv = k->size(1);
        const at::ScalarType type = q->scalar_type();
        if (k->size(0) != T || k->size(2) != D || k->scalar_type() != type) return none();
        const at::Tensor *pos = nullptr, *phases = nullptr, *qw = nullptr, *kw = nullptr, *slots = nullptr;
        int64_t rot = 0;
        if (given(v[2]) != given(v[3]) || given(v[4]) != given(v[5]) || given(v[11]) != given(v[12]) || given(v[11]) != given(v[13]))
            return none();
        if (given(v[2])) {
            phases = tensor(v[3], dev);
            if (!phases || phases->scalar_type() != at::kLong || !(pos = tensor(v[2], dev, at::kLong, T))) return none();
            rot = 2 * phases->numel();
        }
        int wdt = dtype_of(*q);
        if (given(v[4])) {
            qw = tensor(v[4], dev);
            if (!qw || qw->numel() != D || (wdt = dtype_of(*qw)) < 0 || !(kw = tensor(v[5], dev, qw->scalar_type(), D))) return none();
        }
        const int layout = choice(v[7], {"half", "interleaved"});
        if (layout < 0) return none();
        Cache c;
        c.k_mode = c.v_mode = NVFP4_GAMAX_NONE, c.k_gamax = c.v_gamax = nullptr, c.pages = 0, c.page_size = 16;
        if (given(v[11])) {
            if (given(v[10]) || !c.take(v[11], v[14], v[15], dev) || c.Hkv != Hkv || c.D != D) return none();
            x = heads(v[12], dev, &vs);
            if (!x || x->sizes() != k->sizes() || x->scalar_type() != type || !(slots = tensor(v[13], dev, at::kLong, T))) return none();
        } else if (given(v[14]) || given(v[15])) {
            return none();
        }
        at::Tensor qo, ko;
        if (!taken(v[9], T * Hq * D, type, dev, &qo) || !taken(v[10], T * Hkv * D, type, dev, &ko)) return none();
        int rc;
        {
            const Unlocked unlocked;
            if (!qo.defined()) qo = empty3(T, Hq, D, type, dev);
            if (!c.t && !ko.defined()) ko = empty3(T, Hkv, D, type, dev);
            rc = f_rope(q->data_ptr(), k->data_ptr(), data(x), T, Hq, Hkv, D, qs, ks, vs, dtype_of(*q), data(qw), data(kw), wdt,
                        eps, static_cast<const int64_t*>(data(pos)), static_cast<const uint64_t*>(data(phases)), rot, layout,
                        magnitude, qo.data_ptr(), c.t ? nullptr : ko.data_ptr(), c.t ? c.bytes() : nullptr, c.pages,
                        c.page_size, static_cast<const int64_t*>(data(slots)), c.k_mode, c.kg(), c.v_mode, c.vg(), bound,
                        stream_of(dev));
        }
        if (rc != NVFP4_OK) return none();
        PyObject* d = PyDict_New();
        if (!d) return nullptr;
        if (!put(d, "q", wrap(v[9], qo)) || (!c.t && !put(d, "k", wrap(v[10], ko)))) {
            Py_DECREF(d);
            return nullptr;
        }
        return d;
    });
}

// cache_write(cache, k, v, slots, k_gamax, v_gamax, scale_bound): True when it is enqueued
PyObject* cache_write(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        float bound;
        if (n != 7 || !f_cache_write || !number(v[6], &bound)) return none();
        const int dev = call_device(v[0]);
        if (dev < 0) return none();
        Cache c;
        int64_t ks, vs;
        const at::Tensor *k = heads(v[1], dev, &ks), *x = heads(v[2], dev, &vs);
        if (!k || !x || !c.take(v[0], v[4], v[5], dev)) return none();
        const int64_t T = k->size(0);
        if (k->size(1) != c.Hkv || k->size(2) != c.D || x->sizes() != k->sizes() || x->scalar_type() != k->scalar_type()) return none();
        const at::Tensor* slots = tensor(v[3], dev, at::kLong, T);
        if (!slots) return none();
        int rc;
        {
            const Unlocked unlocked;
            rc = f_cache_write(k->data_ptr(), x->data_ptr(), T, c.Hkv, c.D, ks, vs, dtype_of(*k), c.bytes(), c.pages, c.page_size,
                               static_cast<const int64_t*>(slots->data_ptr()), c.k_mode, c.kg(), c.v_mode, c.vg(), bound,
                               stream_of(dev));
        }
        if (rc != NVFP4_OK) return none();
        Py_RETURN_TRUE;
    });
}

PyObject* pair(PyObject* a, PyObject* b) {                // takes both references
    PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return t;
}

// cache_read(cache, slots, k_gamax, v_gamax, scale_bound, out_dtype)
PyObject* cache_read(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        float bound;
        if (n != 6 || !f_cache_read || !number(v[4], &bound)) return none();
        const int dev = call_device(v[0]);
        if (dev < 0) return none();
        Cache c;
        const at::Tensor* slots = tensor(v[1], dev);
        const int odt = choice(v[5], {"f32", "bf16"});
        if (!slots || slots->scalar_type() != at::kLong || slots->numel() == 0 || odt < 0 || !c.take(v[0], v[2], v[3], dev)) return none();
        const int64_t T = slots->numel();
        const at::ScalarType ot = odt == NVFP4_F32 ? at::kFloat : at::kBFloat16;
        at::Tensor k, x;
        int rc;
        {
            const Unlocked unlocked;
            k = empty3(T, c.Hkv, c.D, ot, dev);
            x = empty3(T, c.Hkv, c.D, ot, dev);
            rc = f_cache_read(c.bytes(), c.pages, c.page_size, c.Hkv, c.D, static_cast<const int64_t*>(slots->data_ptr()), T,
                              c.k_mode, c.kg(), c.v_mode, c.vg(), bound, k.data_ptr(), x.data_ptr(), odt, stream_of(dev));
        }
        return rc == NVFP4_OK ? pair(THPVariable_Wrap(k), THPVariable_Wrap(x)) : none();
    });
}

// cache_attention(q, cache, pages, lengths, offsets, k_gamax, v_gamax, scale_bound, scale, causal, window, sinks, out_dtype,
// out, want_lse)
PyObject* cache_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        float bound, scale;
        if (n != 15 || !f_attention || !number(v[7], &bound)) return none();
        const int dev = call_device(v[0]);
        if (dev < 0 || !PyBool_Check(v[9]) || !PyLong_Check(v[10]) || !PyBool_Check(v[14])) return none();
        int64_t qs;
        Cache c;
        const at::Tensor *q = heads(v[0], dev, &qs), *pages = tensor(v[2], dev);
        if (!q || !pages || pages->scalar_type() != at::kInt || pages->dim() != 2 || !c.take(v[1], v[5], v[6], dev)) return none();
        const int64_t T = q->size(0), Hq = q->size(1), B = pages->size(0), width = pages->size(1);
        const at::Tensor *lengths = tensor(v[3], dev, at::kLong, B), *offsets = nullptr, *sinks = nullptr;
        if (!lengths || q->size(2) != c.D || B == 0 || width == 0) return none();
        if (given(v[4]) && !(offsets = tensor(v[4], dev, at::kLong, B + 1))) return none();
        if (given(v[11]) && !(sinks = tensor(v[11], dev, at::kFloat, Hq))) return none();
        if (!given(v[8])) scale = static_cast<float>(std::pow(static_cast<double>(c.D), -0.5));
        else if (!number(v[8], &scale)) return none();
        const int64_t window = PyLong_AsLongLong(v[10]);
        if (window == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            return none();
        }
        const int odt = choice(v[12], {"f32", "bf16"});
        at::Tensor out, lse, ws;
        const at::ScalarType ot = odt == NVFP4_F32 ? at::kFloat : at::kBFloat16;
        if (odt < 0 || !taken(v[13], T * Hq * c.D, ot, dev, &out)) return none();
        const bool want_lse = v[14] == Py_True;
        int rc;
        {
            const Unlocked unlocked;
            const int dt = dtype_of(*q);
            if (!out.defined()) out = empty3(T, Hq, c.D, ot, dev);
            if (want_lse) lse = empty(T, Hq, at::kFloat, dev);
            const int64_t need = f_attention_ws(T, Hq, c.Hkv, c.D, B, width, c.page_size, dt, offsets ? 1 : 0);
            if (need > 0) ws = empty(1, need, at::kByte, dev);      // free for the stream's next work once this call is enqueued
            rc = f_attention(q->data_ptr(), T, Hq, qs, dt, c.bytes(), c.pages, c.page_size, c.Hkv, c.D,
                             static_cast<const int32_t*>(pages->data_ptr()), B, width,
                             static_cast<const int64_t*>(lengths->data_ptr()), static_cast<const int64_t*>(data(offsets)),
                             c.k_mode, c.kg(), c.v_mode, c.vg(), bound, scale, v[9] == Py_True, window,
                             static_cast<const float*>(data(sinks)), out.data_ptr(), odt,
                             want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                             need > 0 ? static_cast<uint8_t*>(ws.data_ptr()) : nullptr, need, stream_of(dev));
        }
        if (rc != NVFP4_OK) return none();
        return want_lse ? pair(wrap(v[13], out), THPVariable_Wrap(lse)) : wrap(v[13], out);
    });
}

// bind_cache(qk_norm_rope, cache_write, cache_read, cache_attention, cache_attention_workspace)
PyObject* bind_cache(PyObject*, PyObject* args) {
    unsigned long long a, b, c, d, e;
    if (!PyArg_ParseTuple(args, "KKKKK", &a, &b, &c, &d, &e)) return nullptr;
    f_rope = reinterpret_cast<decltype(f_rope)>(static_cast<uintptr_t>(a));
    f_cache_write = reinterpret_cast<decltype(f_cache_write)>(static_cast<uintptr_t>(b));
    f_cache_read = reinterpret_cast<decltype(f_cache_read)>(static_cast<uintptr_t>(c));
    f_attention = reinterpret_cast<decltype(f_attention)>(static_cast<uintptr_t>(d));
    f_attention_ws = reinterpret_cast<decltype(f_attention_ws)>(static_cast<uintptr_t>(e));
    Py_RETURN_NONE;
}

// bind(rmsnorm, mv, grouped_mm, grouped_mm_workspace): the addresses of the C ABI's functions in the loaded library
PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long a, b, c, d;
    if (!PyArg_ParseTuple(args, "KKKK", &a, &b, &c, &d)) return nullptr;
    f_rmsnorm = reinterpret_cast<decltype(f_rmsnorm)>(static_cast<uintptr_t>(a));
    f_mv = reinterpret_cast<decltype(f_mv)>(static_cast<uintptr_t>(b));
    f_grouped_mm = reinterpret_cast<decltype(f_grouped_mm)>(static_cast<uintptr_t>(c));
    f_grouped_ws = reinterpret_cast<decltype(f_grouped_ws)>(static_cast<uintptr_t>(d));
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"bind_cache", bind_cache, METH_VARARGS, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"cache_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_write)), METH_FASTCALL, nullptr},
    {"cache_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_read)), METH_FASTCALL, nullptr},
    {"cache_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_attention)), METH_FASTCALL, nullptr},
    {"mv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mv)), METH_FASTCALL, nullptr},
    {"grouped_mm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grouped_mm)), METH_FASTCALL, nullptr},
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nvfp4_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// abi: the torch and the interpreter this file was compiled against
PyMODINIT_FUNC PyInit__nvfp4_call(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "abi", NVFP4_CALL_ABI) < 0) Py_CLEAR(m);
    return m;
}
