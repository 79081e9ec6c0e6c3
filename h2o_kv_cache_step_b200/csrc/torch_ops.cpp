// torch_ops.cpp -- the operators next to the step for torch tensors: checks of
// the arguments, outputs, the current stream, and one call of the C ABI each.
//
// Marshalling only, like the ctypes binding of the other entry points, in C++
// because a small call (one token of a draft, a short step's gradients) costs more on
// the host than on the GPU: checking seven tensors, making four and passing fifteen
// arguments takes 15.1 us a call with ctypes and torch from Python and 7.3 here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <array>
#include <string>

#include "../../include/h2o.h"

namespace {

// What the operators need to know of a context.
struct Ops {
    PyObject_HEAD
    h2o_ctx* ctx;
    int64_t B, Hq, Hkv, d, C;
    at::ScalarType dtype;
    c10::DeviceIndex device;
};

using Shape = std::array<int64_t, 4>;

// A Python error is set; unwinds to the entry point.
struct PythonError {};

std::string describe(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: need a tensor", name);
        throw PythonError();
    }
    return THPVariable_Unpack(o);
}

// The address of a tensor that has to be just so.
void* need(const Ops* s, const char* name, PyObject* o, at::ScalarType dtype, at::IntArrayRef shape) {
    const at::Tensor& t = tensor(name, o);
    if (t.scalar_type() != dtype || t.layout() != at::kStrided || t.sizes() != shape || !t.is_cuda() ||
        t.get_device() != s->device || !t.is_contiguous()) {
        const std::string want = describe(shape), got = describe(t.sizes()), on = t.device().str();
        PyErr_Format(PyExc_ValueError, "%s: need a contiguous %s tensor of shape %s on cuda:%d, got %s %s on %s", name,
                     c10::toString(dtype), want.c_str(), (int)s->device, c10::toString(t.scalar_type()), got.c_str(), on.c_str());
        throw PythonError();
    }
    return t.data_ptr();
}

at::Tensor make(const Ops* s, at::ScalarType dtype, at::IntArrayRef shape) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::Device(at::kCUDA, s->device)));
}

void* stream(const Ops* s) { return c10::cuda::getCurrentCUDAStream(s->device).stream(); }

// Python's other threads run during a call of the library, which may wait for the GPU
// (a context's first call of an operator allocates).
class Unlocked {
    PyThreadState* const state_ = PyEval_SaveThread();

public:
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state_); }
};

template <typename F>
int unlocked(F&& call) {
    const Unlocked u;
    return call();
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}

int narrow(const char* name, int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s: out of range", name);
        throw PythonError();
    }
    return (int)v;
}

void count(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return;
    PyErr_Format(PyExc_TypeError, "%zd arguments, need %zd", got, want);
    throw PythonError();
}

// A tuple of tensors, or the status of a call that failed.
template <typename... T>
PyObject* result(int rc, T&&... t) {
    if (rc != H2O_OK) return PyLong_FromLong(rc);
    PyObject* out = PyTuple_New(sizeof...(t));
    if (!out) throw PythonError();
    Py_ssize_t i = 0;
    for (PyObject* o : {THPVariable_Wrap(std::forward<T>(t))...}) PyTuple_SET_ITEM(out, i++, o);
    return out;
}

int64_t tokens(const char* name, PyObject* o, int64_t dims, const char* layout) {
    const at::Tensor& t = tensor(name, o);
    if (t.dim() != dims) {
        PyErr_Format(PyExc_ValueError, "%s: need %s", name, layout);
        throw PythonError();
    }
    return t.size(2);
}

PyObject* tree_attend(const Ops* s, PyObject* const* a, Py_ssize_t n) {
    count(n, 4);
    const int64_t T = tokens("q", a[0], 4, "[B, Hq, T, d]");
    const Shape rows{s->B, s->Hq, T, s->d}, chunk{s->B, s->Hkv, T, s->d};
    const std::array<int64_t, 2> tree{s->B, T};
    const void *q = need(s, "q", a[0], s->dtype, rows), *k = need(s, "k", a[1], s->dtype, chunk);
    const void *v = need(s, "v", a[2], s->dtype, chunk), *parent = need(s, "parent", a[3], at::kInt, tree);
    at::Tensor out = make(s, s->dtype, rows), lse = make(s, at::kFloat, at::IntArrayRef(rows.data(), 3));
    const int t = narrow("q", T);
    const int rc = unlocked([&] {
        return h2o_tree_attend(s->ctx, q, k, v, static_cast<const int32_t*>(parent), out.data_ptr(),
                               static_cast<float*>(lse.data_ptr()), t, stream(s));
    });
    return result(rc, std::move(out), std::move(lse));
}

// (buffer, n): the record and the valid slots it holds.
PyObject* checkpoint(const Ops* s, PyObject* const* a, Py_ssize_t nargs) {
    count(nargs, 3);
    const int64_t T = tokens("q", a[0], 4, "[B, Hq, T, d]");
    const Shape rows{s->B, s->Hq, T, s->d}, chunk{s->B, s->Hkv, T, s->d};
    const void *q = need(s, "q", a[0], s->dtype, rows), *k = need(s, "k", a[1], s->dtype, chunk),
               *v = need(s, "v", a[2], s->dtype, chunk);
    int64_t P = 0, n = 0;
    size_t bytes = 0;
    int rc = h2o_counters(s->ctx, &P, &n);
    if (rc == H2O_OK) rc = h2o_checkpoint_bytes(s->ctx, narrow("q", T), (int)n, &bytes);
    if (rc != H2O_OK) return PyLong_FromLong(rc);
    at::Tensor buf = make(s, at::kByte, {(int64_t)bytes});
    rc = unlocked([&] { return h2o_checkpoint_save(s->ctx, q, k, v, (int)T, buf.data_ptr(), bytes, stream(s)); });
    if (rc != H2O_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("(NL)", THPVariable_Wrap(std::move(buf)), (long long)n);
}

struct Record {
    const void* p;
    size_t bytes;
    int T, n;
};

// buffer, T, n of a record
Record record(const Ops* s, PyObject* const* a) {
    const at::Tensor& t = tensor("checkpoint", a[0]);
    const std::array<int64_t, 1> shape{t.numel()};
    Record r;
    r.p = need(s, "checkpoint", a[0], at::kByte, shape);
    r.bytes = (size_t)t.numel();
    r.T = narrow("T", integer(a[1]));
    r.n = narrow("n", integer(a[2]));
    return r;
}

PyObject* checkpoint_restore(const Ops* s, PyObject* const* a, Py_ssize_t n) {
    count(n, 3);
    const Record r = record(s, a);
    const Shape rows{s->B, s->Hq, r.T, s->d}, chunk{s->B, s->Hkv, r.T, s->d}, cache{s->B, s->Hkv, s->C, s->d};
    at::Tensor q = make(s, s->dtype, rows), k = make(s, s->dtype, chunk), v = make(s, s->dtype, chunk);
    at::Tensor K = make(s, s->dtype, cache), V = make(s, s->dtype, cache);
    const int rc = unlocked([&] {
        return h2o_checkpoint_restore(s->ctx, r.p, r.bytes, r.T, r.n, q.data_ptr(), k.data_ptr(), v.data_ptr(), K.data_ptr(),
                                      V.data_ptr(), stream(s));
    });
    return result(rc, std::move(q), std::move(k), std::move(v), std::move(K), std::move(V));
}

PyObject* checkpoint_backward(const Ops* s, PyObject* const* a, Py_ssize_t n) {
    count(n, 4);
    const Record r = record(s, a);
    const Shape rows{s->B, s->Hq, r.T, s->d}, chunk{s->B, s->Hkv, r.T, s->d}, cache{s->B, s->Hkv, s->C, s->d};
    const void* dout = need(s, "dout", a[3], s->dtype, rows);
    at::Tensor dq = make(s, s->dtype, rows), dK = make(s, s->dtype, cache), dV = make(s, s->dtype, cache);
    at::Tensor dk = make(s, s->dtype, chunk), dv = make(s, s->dtype, chunk);
    const int rc = unlocked([&] {
        return h2o_checkpoint_backward(s->ctx, r.p, r.bytes, r.T, r.n, dout, dq.data_ptr(), dK.data_ptr(), dV.data_ptr(),
                                       dk.data_ptr(), dv.data_ptr(), stream(s));
    });
    return result(rc, std::move(dq), std::move(dK), std::move(dV), std::move(dk), std::move(dv));
}

// token_slots, n, dK, dV, dk, dv, gK_next, gV_next (the last two may be None)
PyObject* carry_grad(const Ops* s, PyObject* const* a, Py_ssize_t nargs) {
    count(nargs, 8);
    const int64_t T = tokens("token_slots", a[0], 3, "[B, Hkv, T]");
    const int n = narrow("n", integer(a[1]));
    const Shape chunk{s->B, s->Hkv, T, s->d}, cache{s->B, s->Hkv, s->C, s->d};
    const void* slots = need(s, "token_slots", a[0], at::kInt, at::IntArrayRef(chunk.data(), 3));
    const void *dK = need(s, "dK", a[2], s->dtype, cache), *dV = need(s, "dV", a[3], s->dtype, cache);
    const void *dk = need(s, "dk", a[4], s->dtype, chunk), *dv = need(s, "dv", a[5], s->dtype, chunk);
    const void* gKn = a[6] == Py_None ? nullptr : need(s, "gK_next", a[6], at::kFloat, cache);
    const void* gVn = a[7] == Py_None ? nullptr : need(s, "gV_next", a[7], at::kFloat, cache);
    at::Tensor gK = make(s, at::kFloat, cache), gV = make(s, at::kFloat, cache);
    at::Tensor gk = make(s, s->dtype, chunk), gv = make(s, s->dtype, chunk);
    const int t = narrow("token_slots", T);
    const int rc = unlocked([&] {
        return h2o_carry_grad(s->ctx, static_cast<const int32_t*>(slots), t, n, dK, dV, dk, dv,
                              static_cast<const float*>(gKn), static_cast<const float*>(gVn),
                              static_cast<float*>(gK.data_ptr()), static_cast<float*>(gV.data_ptr()), gk.data_ptr(),
                              gv.data_ptr(), stream(s));
    });
    return result(rc, std::move(gK), std::move(gV), std::move(gk), std::move(gv));
}

template <PyObject* (*F)(const Ops*, PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(reinterpret_cast<const Ops*>(self), args, n);
    } catch (const PythonError&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(const Ops*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<tree_attend>("tree_attend"), method<checkpoint>("checkpoint"),
                         method<checkpoint_restore>("checkpoint_restore"),
                         method<checkpoint_backward>("checkpoint_backward"), method<carry_grad>("carry_grad"),
                         {nullptr, nullptr, 0, nullptr}};

// Ops(handle, device, B, Hq, Hkv, d, C, bf16)
int init(PyObject* self, PyObject* args, PyObject*) {
    Ops* s = reinterpret_cast<Ops*>(self);
    unsigned long long handle;
    long long device, B, Hq, Hkv, d, C;
    int bf16;
    if (!PyArg_ParseTuple(args, "KLLLLLLp", &handle, &device, &B, &Hq, &Hkv, &d, &C, &bf16)) return -1;
    s->ctx = reinterpret_cast<h2o_ctx*>(static_cast<uintptr_t>(handle));
    s->device = static_cast<c10::DeviceIndex>(device);
    s->B = B;
    s->Hq = Hq;
    s->Hkv = Hkv;
    s->d = d;
    s->C = C;
    s->dtype = bf16 ? at::kBFloat16 : at::kFloat;
    return 0;
}

PyTypeObject ops_type = {PyVarObject_HEAD_INIT(nullptr, 0)};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_ops", "the operators next to the step, for torch tensors", -1, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops() {
    ops_type.tp_name = "h2o_kv_cache_step_b200._torch_ops.Ops";
    ops_type.tp_basicsize = sizeof(Ops);
    ops_type.tp_flags = Py_TPFLAGS_DEFAULT;
    ops_type.tp_new = PyType_GenericNew;
    ops_type.tp_init = init;
    ops_type.tp_methods = methods;
    if (PyType_Ready(&ops_type) < 0) return nullptr;
    PyObject* m = PyModule_Create(&module);
    if (!m) return nullptr;
    // the tensors' layout is that of the torch this was compiled with
    if (PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    Py_INCREF(&ops_type);
    if (PyModule_AddObject(m, "Ops", reinterpret_cast<PyObject*>(&ops_type)) < 0) {
        Py_DECREF(&ops_type);
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
