// kv_torch.cpp — the cache's calls on torch tensors, as one step from Python: a
// decoding step is a handful of kernels of a few microseconds, and making the
// outputs, the descriptors and the call one by one from Python takes longer than
// they run (a step's attention: 13.7 us so and 7.9 us here).
//
// Each function takes the C entry point's address, the addresses that a cache
// and a batch keep, and the tensors. It returns the outputs; or None where
// something is not as it is most of the time (a layout or a type that the
// Python layer refuses, or words differently), without having done anything; or
// the entry point's status where that is not 0. It checks what the Python layer
// checks: nothing else may come between a tensor and its address. Outputs are
// made and the kernels launched without the interpreter's lock: memory that has
// to be freed first, or a full queue, holds up no other thread of Python, whose
// work the device may be waiting for.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "zc.h"

namespace {

uint64_t number(PyObject *o) {
    const uint64_t v = PyLong_AsUnsignedLongLongMask(o);
    if (v == uint64_t(-1) && PyErr_Occurred()) throw python_error();
    return v;
}
template <class T> T address(PyObject *o) { return reinterpret_cast<T>(number(o)); }
double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

// Where a call runs and what its rows are like.
struct Call {
    void *stream;
    int64_t device, tokens, kv_heads, dim;
    const zc_kv_batch *batch;
    int32_t *status;
    // args: batch, status, stream, device, tokens, kv_heads, dim
    explicit Call(PyObject *const *args)
        : stream(address<void *>(args[2])), device(int64_t(number(args[3]))), tokens(int64_t(number(args[4]))), kv_heads(int64_t(number(args[5]))),
          dim(int64_t(number(args[6]))), batch(address<const zc_kv_batch *>(args[0])), status(address<int32_t *>(args[1])) {}
    static constexpr int kArgs = 7;
};

int code_of(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return ZC_BF16;
    case at::kHalf: return ZC_FP16;
    case at::kFloat: return ZC_FP32;
    default: return 0;
    }
}

// A tensor [tokens][heads][dim] on the call's device, heads as given or any (0).
const at::Tensor *rows_of(PyObject *o, const Call &c, int64_t heads, zc_kv_rows &rows) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != 3 || !t.is_cuda() || t.get_device() != c.device || !code_of(t.scalar_type())) return nullptr;
    if (t.size(0) != c.tokens || (heads ? t.size(1) != heads : t.size(1) < 1) || t.size(2) != c.dim || t.stride(2) != 1) return nullptr;
    rows = {t.data_ptr(), t.stride(0), t.stride(1)};
    return &t;
}

at::Tensor made(const Call &c, int64_t heads, at::ScalarType type, zc_kv_rows &rows) {
    at::Tensor t = at::empty({c.tokens, heads, c.dim}, at::TensorOptions(type).device(at::kCUDA, at::DeviceIndex(c.device)));
    rows = {t.data_ptr(), heads * c.dim, c.dim};
    return t;
}

PyObject *both(at::Tensor a, at::Tensor b) {
    PyObject *r = PyTuple_New(2);
    if (!r) throw python_error();
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(a)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(b)));
    return r;
}
PyObject *none() { Py_RETURN_NONE; }
bool wrong(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return n != want;
}

// The interpreter's lock is someone else's while this lives.
class Unlocked {
    PyThreadState *state_ = PyEval_SaveThread();

public:
    Unlocked() = default;
    ~Unlocked() { PyEval_RestoreThread(state_); }
    Unlocked(const Unlocked &) = delete;
    Unlocked &operator=(const Unlocked &) = delete;
};

using Move = int (*)(const void *, const zc_kv_batch *, int, const zc_kv_rows *, const zc_kv_rows *, int32_t *, void *);
using Attend = int (*)(const void *, const zc_kv_batch *, int, uint32_t, const zc_kv_rows *, const zc_kv_rows *, float *, double, uint32_t, uint32_t,
                       void *, uint64_t, int32_t *, void *);

// attend(entry, cache, the call, q, scale, flags, window, workspace, its bytes) -> (out, lse)
PyObject *attend(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong(n, 2 + Call::kArgs + 6)) return nullptr;
    const Call c(args + 2);
    PyObject *const *a = args + 2 + Call::kArgs;
    zc_kv_rows rq, ro;
    const at::Tensor *q = rows_of(a[0], c, 0, rq);
    if (!q || q->scalar_type() == at::kFloat) return none();
    const int64_t heads = q->size(1);
    const at::ScalarType type = q->scalar_type();
    const auto entry = address<Attend>(args[0]);
    const auto cache = address<const void *>(args[1]);
    const double scale = real(a[1]);
    const uint32_t flags = uint32_t(number(a[2])), window = uint32_t(number(a[3]));
    void *const workspace = address<void *>(a[4]);
    const uint64_t bytes = number(a[5]);
    at::Tensor out, lse;
    int st;
    {
        Unlocked unlocked;
        out = made(c, heads, type, ro), lse = at::empty({c.tokens, heads}, out.options().dtype(at::kFloat));
        st = entry(cache, c.batch, code_of(type), uint32_t(heads), &rq, &ro, lse.data_ptr<float>(), scale, flags, window, workspace, bytes, c.status, c.stream);
    }
    return st ? PyLong_FromLong(st) : both(std::move(out), std::move(lse));
    END_HANDLE_TH_ERRORS
}

// read(entry, cache, the call, type code) -> (k, v)
PyObject *read(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong(n, 2 + Call::kArgs + 1)) return nullptr;
    const Call c(args + 2);
    const int code = int(number(args[2 + Call::kArgs]));
    const at::ScalarType type = code == ZC_BF16 ? at::kBFloat16 : code == ZC_FP16 ? at::kHalf : at::kFloat;
    const auto entry = address<Move>(args[0]);
    const auto cache = address<const void *>(args[1]);
    zc_kv_rows rk, rv;
    at::Tensor k, v;
    int st;
    {
        Unlocked unlocked;
        k = made(c, c.kv_heads, type, rk), v = made(c, c.kv_heads, type, rv);
        st = entry(cache, c.batch, code, &rk, &rv, c.status, c.stream);
    }
    return st ? PyLong_FromLong(st) : both(std::move(k), std::move(v));
    END_HANDLE_TH_ERRORS
}

// move(entry, cache, the call, k, v) -> 0
PyObject *move(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong(n, 2 + Call::kArgs + 2)) return nullptr;
    const Call c(args + 2);
    zc_kv_rows rk, rv;
    const at::Tensor *k = rows_of(args[2 + Call::kArgs], c, c.kv_heads, rk), *v = rows_of(args[3 + Call::kArgs], c, c.kv_heads, rv);
    if (!k || !v || k->scalar_type() != v->scalar_type()) return none();
    const int code = code_of(k->scalar_type());
    const auto entry = address<Move>(args[0]);
    const auto cache = address<const void *>(args[1]);
    int st;
    {
        Unlocked unlocked;
        st = entry(cache, c.batch, code, &rk, &rv, c.status, c.stream);
    }
    return PyLong_FromLong(st);
    END_HANDLE_TH_ERRORS
}

// A norm's weights: [dim], contiguous, float32 or of `type`; both of one type. False where they are not.
bool weights(PyObject *o, const Call &c, at::ScalarType type, const void *&to, int &code) {
    to = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) return false;
    const at::Tensor &w = THPVariable_Unpack(o);
    if (w.dim() != 1 || w.size(0) != c.dim || w.stride(0) != 1 || !w.is_cuda() || w.get_device() != c.device) return false;
    if (w.scalar_type() != at::kFloat && w.scalar_type() != type) return false;
    if (code && code != code_of(w.scalar_type())) return false;
    code = code_of(w.scalar_type());
    to = w.data_ptr();
    return true;
}

// rotate(entry, the call, turns, rot_dim, flags, q, k, q's weights, k's weights, eps) -> (q, k)
PyObject *rotate(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong(n, 1 + Call::kArgs + 8)) return nullptr;
    const Call c(args + 1);
    PyObject *const *a = args + 1 + Call::kArgs;
    zc_kv_rotation r{address<const uint64_t *>(a[0]), uint32_t(number(a[1])), uint32_t(number(a[2])), nullptr, nullptr, 0, float(real(a[7]))};
    zc_kv_rows rq, rk, oq, ok;
    const at::Tensor *q = rows_of(a[3], c, 0, rq), *k = rows_of(a[4], c, c.kv_heads, rk);
    if (!q || !k || q->scalar_type() != k->scalar_type()) return none();
    if (!weights(a[5], c, q->scalar_type(), r.d_q_weight, r.weight_dtype) || !weights(a[6], c, q->scalar_type(), r.d_k_weight, r.weight_dtype)) return none();
    using Rotate = int (*)(const zc_kv_batch *, const zc_kv_rotation *, int, uint32_t, uint32_t, uint32_t, const zc_kv_rows *, const zc_kv_rows *,
                           const zc_kv_rows *, const zc_kv_rows *, int32_t *, void *);
    const int64_t heads = q->size(1);
    const at::ScalarType type = q->scalar_type();
    const auto entry = address<Rotate>(args[0]);
    at::Tensor q2, k2;
    int st;
    {
        Unlocked unlocked;
        q2 = made(c, heads, type, oq), k2 = made(c, c.kv_heads, type, ok);
        st = entry(c.batch, &r, code_of(type), uint32_t(c.dim), uint32_t(heads), uint32_t(c.kv_heads), &rq, &rk, &oq, &ok, c.status, c.stream);
    }
    return st ? PyLong_FromLong(st) : both(std::move(q2), std::move(k2));
    END_HANDLE_TH_ERRORS
}

template <class F> PyCFunction entry(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)); }
PyMethodDef methods[] = {{"attend", entry(attend), METH_FASTCALL, nullptr}, {"read", entry(read), METH_FASTCALL, nullptr},
                         {"move", entry(move), METH_FASTCALL, nullptr}, {"rotate", entry(rotate), METH_FASTCALL, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "zc_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit_zc_torch() { return PyModule_Create(&module); }
