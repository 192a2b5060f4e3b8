// tensor_args.cc -- the quick way from Python into the dense operators
// (Python module `_tensor_args`).
//
// A serving loop makes several of these calls per layer and token, and one
// call's nine tensors cost about 5 us to check and to hand over from Python.
// Here a tensor is looked at through DLPack's C exchange table, which torch
// offers on its tensor type: no copy, no reference, nothing kept.  Each
// function returns the status of its mono_* call, or None without having
// called it where something is not as the call expects it; the Python side
// then checks argument by argument and says what is wrong.
//
// Measured (host time of a call on a B200 machine): paged_append 8.9 us by the
// checks in Python and ctypes, 3.4 so, most of it the launch; paged_attend, with
// two launches, 12.1 and 6.2.
#define PY_SSIZE_T_CLEAN
#include <ATen/dlpack.h>
#include <Python.h>

#include <initializer_list>
#include <new>

#include "mono.h"

namespace {

PyTypeObject *g_tensor = nullptr;     // torch.Tensor
PyObject *g_current_device = nullptr;  // () -> int
const DLPackExchangeAPI *g_api = nullptr;

struct Entries {
    decltype(&mono_prompt_attend) prompt;
    decltype(&mono_paged_append) append;
    decltype(&mono_paged_attend) attend;
    decltype(&mono_paged_update) update;
    decltype(&mono_paged_compact) compact;
} g_abi;

// what the checks need of a plan
struct PlanInfo {
    const mono_paged_plan_t *plan;
    int64_t Hq, Hkv, d, page, pages, layers, width, ws_bytes;
    int bf16;
};
constexpr char kPlanName[] = "mono.paged_plan";

enum Kind { kData, kInt, kByte };
constexpr int64_t kAny = -1;

// The tensors of one call: all on one CUDA device, contiguous, of the expected type and shape.
struct Call {
    const PlanInfo &p;
    bool ok = true;
    int device = -1;

    // a tensor of `dims` (kAny: whatever it is, returned in *n)
    void *take(PyObject *o, Kind kind, std::initializer_list<int64_t> dims, int64_t *n = nullptr) {
        DLTensor t;
        if (!ok || Py_TYPE(o) != g_tensor || g_api->dltensor_from_py_object_no_sync(o, &t) != 0) return fail();
        const bool type = kind == kInt    ? t.dtype.code == kDLInt && t.dtype.bits == 32
                          : kind == kByte ? t.dtype.code == kDLUInt && t.dtype.bits == 8
                          : p.bf16        ? t.dtype.code == kDLBfloat && t.dtype.bits == 16
                                          : t.dtype.code == kDLFloat && t.dtype.bits == 32;
        if (!type || t.dtype.lanes != 1 || t.device.device_type != kDLCUDA || t.ndim != (int)dims.size()) return fail();
        if (device >= 0 && t.device.device_id != device) return fail();
        device = t.device.device_id;
        int64_t count = 1;
        bool dense = true;
        for (int i = t.ndim - 1; i >= 0; --i) {
            const int64_t want = dims.begin()[i], have = t.shape[i];
            if (want == kAny) *n = have;
            else if (have != want) return fail();
            dense = dense && (have <= 1 || !t.strides || t.strides[i] == count);
            count *= have;
        }
        if (!dense && count > 0) return fail();  // (without elements any strides are contiguous)
        return (char *)t.data + t.byte_offset;
    }
    // an integer inside [0, below)
    int index(PyObject *o, int64_t below) {
        const long v = ok && PyLong_CheckExact(o) ? PyLong_AsLong(o) : -1;
        if (v < 0 || v >= below) fail();
        return (int)v;
    }
    // the stream of the call: an address, or None for torch's current one; the tensors' device must be the current one
    void *stream(PyObject *o) {
        void *s = nullptr;
        if (!ok || device < 0) return fail();
        PyObject *cur = PyObject_CallNoArgs(g_current_device);
        if (!cur) return fail();
        const long now = PyLong_AsLong(cur);
        Py_DECREF(cur);
        if (now != device) return fail();
        if (o == Py_None) {
            if (g_api->current_work_stream(kDLCUDA, device, &s) != 0) return fail();
        } else if (!PyLong_CheckExact(o)) {
            return fail();
        } else {
            s = PyLong_AsVoidPtr(o);
        }
        return PyErr_Occurred() ? fail() : s;
    }
    void *workspace(PyObject *o) {
        int64_t bytes = 0;
        void *at = take(o, kByte, {kAny}, &bytes);
        return bytes >= p.ws_bytes ? at : fail();
    }
    void *pool(PyObject *o) { return take(o, kData, {p.layers, p.pages, p.Hkv, p.page, p.d}); }
    // sizes that the C interface takes as int
    bool fits(std::initializer_list<int64_t> sizes) {
        for (int64_t v : sizes) ok = ok && v >= 0 && v <= INT32_MAX;
        return ok;
    }

  private:
    void *fail() {
        ok = false;
        return nullptr;
    }
};

const PlanInfo *plan_of(PyObject *o) { return (const PlanInfo *)PyCapsule_GetPointer(o, kPlanName); }

PyObject *none() {
    PyErr_Clear();
    Py_RETURN_NONE;
}

template <typename F>
PyObject *status_of(F call) {
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
}

// Every function: (plan, arguments as the Python function's, workspace, stream or None)
PyObject *prompt_attend(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    const PlanInfo *p = n_args == 9 ? plan_of(a[0]) : nullptr;
    if (!p) return none();
    Call c{*p};
    int64_t nq = 0, nk = 0, n1 = 0;
    void *Q = c.take(a[1], kData, {kAny, p->Hq, p->d}, &nq), *K = c.take(a[2], kData, {kAny, p->Hkv, p->d}, &nk),
         *V = c.take(a[3], kData, {nk, p->Hkv, p->d});
    void *cu_q = c.take(a[4], kInt, {kAny}, &n1), *cu_k = c.take(a[5], kInt, {n1});
    void *O = c.take(a[6], kData, {nq, p->Hq * p->d}), *ws = c.workspace(a[7]), *s = c.stream(a[8]);
    if (!c.fits({n1 - 1, nq, nk})) return none();
    return status_of([&] {
        return g_abi.prompt(p->plan, (int)n1 - 1, (int)nq, (int)nk, Q, K, V, (int32_t *)cu_q, (int32_t *)cu_k, O, ws,
                            s);
    });
}

PyObject *paged_append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    const PlanInfo *p = n_args == 11 ? plan_of(a[0]) : nullptr;
    if (!p) return none();
    Call c{*p};
    int64_t n = 0, total = 0;
    const int layer = c.index(a[1], p->layers);
    void *K = c.take(a[2], kData, {kAny, p->Hkv, p->d}, &total), *V = c.take(a[3], kData, {total, p->Hkv, p->d});
    void *lens = c.take(a[6], kInt, {kAny}, &n), *cu = c.take(a[4], kInt, {n + 1}),
         *table = c.take(a[5], kInt, {n, p->width});
    void *Kp = c.pool(a[7]), *Vp = c.pool(a[8]), *ws = c.workspace(a[9]), *s = c.stream(a[10]);
    if (!c.fits({n, total})) return none();
    return status_of([&] {
        return g_abi.append(p->plan, layer, (int)n, (int)total, K, V, (int32_t *)cu, (int32_t *)table, (int32_t *)lens,
                            Kp, Vp, ws, s);
    });
}

PyObject *paged_attend(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    const PlanInfo *p = n_args == 10 ? plan_of(a[0]) : nullptr;
    if (!p) return none();
    Call c{*p};
    int64_t n = 0;
    const int layer = c.index(a[1], p->layers);
    void *lens = c.take(a[4], kInt, {kAny}, &n), *Q = c.take(a[2], kData, {n, p->Hq, p->d}),
         *table = c.take(a[3], kInt, {n, p->width}), *O = c.take(a[5], kData, {n, p->Hq * p->d});
    void *Kp = c.pool(a[6]), *Vp = c.pool(a[7]), *ws = c.workspace(a[8]), *s = c.stream(a[9]);
    if (!c.fits({n})) return none();
    return status_of([&] {
        return g_abi.attend(p->plan, layer, (int)n, Q, (int32_t *)table, (int32_t *)lens, Kp, Vp, O, ws, s);
    });
}

PyObject *paged_update(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    const PlanInfo *p = n_args == 11 ? plan_of(a[0]) : nullptr;
    if (!p) return none();
    Call c{*p};
    int64_t n_in = 0, n_out = 0;
    void *lens = c.take(a[2], kInt, {kAny}, &n_in), *table = c.take(a[1], kInt, {n_in, p->width});
    void *parents = c.take(a[3], kInt, {kAny}, &n_out), *grow = c.take(a[4], kInt, {n_out});
    void *table_out = c.take(a[5], kInt, {n_out, p->width}), *lens_out = c.take(a[6], kInt, {n_out});
    void *Kp = c.pool(a[7]), *Vp = c.pool(a[8]), *ws = c.workspace(a[9]), *s = c.stream(a[10]);
    if (!c.fits({n_in, n_out})) return none();
    return status_of([&] {
        return g_abi.update(p->plan, (int)n_in, (int32_t *)table, (int32_t *)lens, (int)n_out, (int32_t *)parents,
                            (int32_t *)grow, (int32_t *)table_out, (int32_t *)lens_out, Kp, Vp, ws, s);
    });
}

PyObject *paged_compact(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    const PlanInfo *p = n_args == 8 ? plan_of(a[0]) : nullptr;
    if (!p) return none();
    Call c{*p};
    int64_t n = 0;
    void *lens = c.take(a[2], kInt, {kAny}, &n), *table = c.take(a[1], kInt, {n, p->width}),
         *table_out = c.take(a[3], kInt, {n, p->width});
    void *Kp = c.pool(a[4]), *Vp = c.pool(a[5]), *ws = c.workspace(a[6]), *s = c.stream(a[7]);
    if (!c.fits({n})) return none();
    return status_of([&] {
        return g_abi.compact(p->plan, (int)n, (int32_t *)table, (int32_t *)lens, (int32_t *)table_out, Kp, Vp, ws, s);
    });
}

// plan(handle, Hq, Hkv, d, page, pages, layers, width, workspace bytes, bf16): lives as long as the Python plan does
PyObject *plan(PyObject *, PyObject *args) {
    unsigned long long handle;
    long long v[8];
    int bf16;
    if (!PyArg_ParseTuple(args, "KLLLLLLLLp", &handle, v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7, &bf16))
        return nullptr;
    auto *p = new (std::nothrow)
        PlanInfo{(const mono_paged_plan_t *)handle, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], bf16};
    if (!p) return PyErr_NoMemory();  // (an exception must not pass Python's frames)
    PyObject *o = PyCapsule_New(p, kPlanName, [](PyObject *x) { delete plan_of(x); });
    if (!o) delete p;
    return o;
}

// setup(torch.Tensor, its exchange table, current_device, addresses of the five entry points) -> usable
PyObject *setup(PyObject *, PyObject *args) {
    PyObject *tensor, *table, *current;
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "O!OOKKKKK", &PyType_Type, &tensor, &table, &current, f, f + 1, f + 2, f + 3, f + 4))
        return nullptr;
    auto *api = (const DLPackExchangeAPI *)PyCapsule_GetPointer(table, "dlpack_exchange_api");
    if (!api) {  // a table of another kind
        PyErr_Clear();
        Py_RETURN_FALSE;
    }
    if (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync ||
        !api->current_work_stream)
        Py_RETURN_FALSE;
    g_api = api;
    Py_INCREF(tensor);
    g_tensor = (PyTypeObject *)tensor;
    Py_INCREF(current);
    g_current_device = current;
    g_abi = {(decltype(Entries::prompt))f[0], (decltype(Entries::append))f[1], (decltype(Entries::attend))f[2],
             (decltype(Entries::update))f[3], (decltype(Entries::compact))f[4]};
    Py_RETURN_TRUE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, nullptr},
                         {"plan", plan, METH_VARARGS, nullptr},
                         FAST(prompt_attend),
                         FAST(paged_append),
                         FAST(paged_attend),
                         FAST(paged_update),
                         FAST(paged_compact),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) { return PyModule_Create(&module); }
