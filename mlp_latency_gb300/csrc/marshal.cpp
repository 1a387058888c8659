// marshal.cpp -- the argument checks of mlp_latency_gb300/block.py: tensors in, a call of the C ABI
// (include/mlp_block.h) out.
//
// A call of a few microseconds is bound by the host: a layer norm of one row took 7.2 us from Python through ctypes, of
// which the checks of its six tensors (dtype, shape, device, strides, address: five attributes each) took 4.  Here they
// read the tensor's fields, and it takes 2.1; a layer norm's gradient 4.1 instead of 10.9, a linear's 6.0 instead of 11.7.
// The functions return the library's status; a wrong argument raises ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>

#include "../../include/mlp_block.h"

namespace {

decltype(&mlp_layernorm_forward) norm_forward_fn;
decltype(&mlp_layernorm_backward) norm_backward_fn;
decltype(&mlp_layernorm_workspace_size) norm_workspace_fn;
decltype(&mlp_linear_workspace_size) linear_workspace_fn;
decltype(&mlp_linear_forward) linear_forward_fn;
decltype(&mlp_linear_backward) linear_backward_fn;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

constexpr auto kBf16 = at::ScalarType::BFloat16;
constexpr auto kF32 = at::ScalarType::Float;

bool absent(PyObject *o) { return o == Py_None; }

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (absent(o))
        throw Refused(std::string(name) + " is missing");
    if (!THPVariable_Check(o))
        throw Refused(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

// All tensors of a call are on one device: a kernel runs on one, with addresses that mean something there.
bool elsewhere(const at::Tensor &t, int device) { return !t.is_cuda() || t.get_device() != device; }

[[noreturn]] void refuse(const at::Tensor &t, const char *name, const char *kind, at::ScalarType dtype, at::IntArrayRef shape, int device)
{
    std::ostringstream s;
    s << name << ": expected a " << kind << "CUDA tensor " << c10::toString(dtype) << ' ' << shape;
    if (device >= 0)
        s << " on cuda:" << device;
    s << ", got " << c10::toString(t.scalar_type()) << ' ' << t.sizes() << " on " << t.device();
    throw Refused(s.str());
}

struct Matrix {
    void *p = nullptr;
    int64_t ld = 0;
};

// What the tensors of a call have to be.
struct Tensors {
    int device;

    // A matrix whose rows are contiguous.
    Matrix matrix(PyObject *o, const char *name, int64_t rows, int64_t cols, at::ScalarType dtype) const
    {
        const at::Tensor &t = tensor(o, name);
        if (t.scalar_type() != dtype || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || elsewhere(t, device))
            refuse(t, name, "", dtype, {rows, cols}, device);
        if (t.stride(1) != 1 && cols > 1)
            throw Refused(std::string(name) + ": rows must be contiguous");
        return {t.data_ptr(), rows > 1 ? t.stride(0) : (cols + 7) & ~int64_t{7}};   // (one row: any stride will do)
    }

    Matrix matrix_or_none(PyObject *o, const char *name, int64_t rows, int64_t cols, at::ScalarType dtype) const
    {
        return absent(o) ? Matrix() : matrix(o, name, rows, cols, dtype);
    }

    void *dense(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dtype) const
    {
        const at::Tensor &t = tensor(o, name);
        if (t.scalar_type() != dtype || t.sizes() != shape || elsewhere(t, device) || !t.is_contiguous())
            refuse(t, name, "contiguous ", dtype, shape, device);
        return t.data_ptr();
    }

    void *dense_or_none(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dtype) const
    {
        return absent(o) ? nullptr : dense(o, name, shape, dtype);
    }

    void *workspace(PyObject *o, size_t need) const
    {
        if (absent(o))
            return nullptr;
        const at::Tensor &t = tensor(o, "workspace");
        if (elsewhere(t, device) || !t.is_contiguous() || t.nbytes() < need)
            throw Refused("workspace: expected a contiguous CUDA tensor of at least " + std::to_string(need) + " bytes on cuda:" +
                          std::to_string(device));
        return t.data_ptr();
    }
};

// None: torch's current stream of the device; an address; or an object with one in cuda_stream.
void *stream_of(PyObject *o, int device)
{
    if (absent(o))
        return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    if (PyLong_Check(o))
        return PyLong_AsVoidPtr(o);
    PyObject *s = PyObject_GetAttrString(o, "cuda_stream");
    void *p = s ? PyLong_AsVoidPtr(s) : nullptr;
    Py_XDECREF(s);
    return p;
}

// A layer norm launches on the current device.  (A guard that sets it whether or not it is another one took 0.2 us.)
struct CurrentDevice {
    c10::cuda::OptionalCUDAGuard guard;
    explicit CurrentDevice(int device)
    {
        if (c10::cuda::current_device() != device)
            guard.set_index(static_cast<c10::DeviceIndex>(device));
    }
};

// Runs `call` (which ends in a call of the library) and turns what goes wrong on the way into Python's exceptions.
template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t wanted, F call)
{
    if (got != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, wanted);
        return nullptr;
    }
    try {
        const int status = call();
        return PyErr_Occurred() ? nullptr : PyLong_FromLong(status);
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (A launch waits where the device's queue is full: other threads run meanwhile.)
template <typename F>
int unlocked(F call)
{
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call();
    Py_END_ALLOW_THREADS
    return status;
}

mlp_dtype code(at::ScalarType t) { return t == kBf16 ? MLP_DT_BF16 : MLP_DT_F32; }

const at::Tensor &norm_input(PyObject *o)
{
    const at::Tensor &x = tensor(o, "x");
    if (x.dim() != 2 || (x.scalar_type() != kBf16 && x.scalar_type() != kF32))
        throw Refused("layer norm takes matrices of bfloat16 or float32");
    return x;
}

// The weights' type: that of the first one there is.
at::ScalarType weight_type(std::initializer_list<PyObject *> weights)
{
    for (PyObject *o : weights)
        if (!absent(o)) {
            const at::ScalarType t = tensor(o, "weight").scalar_type();
            if (t != kBf16 && t != kF32)
                throw Refused("layer norm weights are bfloat16 or float32");
            return t;
        }
    return kF32;
}

PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        norm_forward_fn = reinterpret_cast<decltype(norm_forward_fn)>(PyLong_AsVoidPtr(a[0]));
        norm_backward_fn = reinterpret_cast<decltype(norm_backward_fn)>(PyLong_AsVoidPtr(a[1]));
        norm_workspace_fn = reinterpret_cast<decltype(norm_workspace_fn)>(PyLong_AsVoidPtr(a[2]));
        linear_workspace_fn = reinterpret_cast<decltype(linear_workspace_fn)>(PyLong_AsVoidPtr(a[3]));
        linear_forward_fn = reinterpret_cast<decltype(linear_forward_fn)>(PyLong_AsVoidPtr(a[4]));
        linear_backward_fn = reinterpret_cast<decltype(linear_backward_fn)>(PyLong_AsVoidPtr(a[5]));
        return 0;
    });
}

// x, gamma, beta, y, mean, rstd, eps, stream
PyObject *norm_forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const at::Tensor &t = norm_input(a[0]);
        const at::ScalarType dt = t.scalar_type(), wd = weight_type({a[1], a[2]});
        const int64_t R = t.size(0), C = t.size(1);
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix x = on.matrix(a[0], "x", R, C, dt), y = on.matrix(a[3], "y", R, C, dt);
        const void *gamma = on.dense_or_none(a[1], "gamma", {C}, wd), *beta = on.dense_or_none(a[2], "beta", {C}, wd);
        float *mean = static_cast<float *>(on.dense_or_none(a[4], "mean", {R}, kF32));
        float *rstd = static_cast<float *>(on.dense_or_none(a[5], "rstd", {R}, kF32));
        const float eps = static_cast<float>(PyFloat_AsDouble(a[6]));
        void *st = stream_of(a[7], t.get_device());
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] { return norm_forward_fn(R, C, x.p, x.ld, code(dt), gamma, beta, code(wd), eps, y.p, y.ld, mean, rstd, st); });
    });
}

// dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dx_add, workspace, stream
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const at::Tensor &t = norm_input(a[1]);
        const at::ScalarType dt = t.scalar_type(), wd = weight_type({a[2], a[6], a[7]});
        const int64_t R = t.size(0), C = t.size(1);
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix dy = on.matrix(a[0], "dy", R, C, dt), x = on.matrix(a[1], "x", R, C, dt);
        const Matrix add = on.matrix_or_none(a[8], "dx_add", R, C, dt), dx = on.matrix_or_none(a[5], "dx", R, C, dt);
        const void *gamma = on.dense_or_none(a[2], "gamma", {C}, wd);
        const float *mean = static_cast<float *>(on.dense(a[3], "mean", {R}, kF32)), *rstd = static_cast<float *>(on.dense(a[4], "rstd", {R}, kF32));
        void *dgamma = on.dense_or_none(a[6], "dgamma", {C}, wd), *dbeta = on.dense_or_none(a[7], "dbeta", {C}, wd);
        size_t need = 0;
        if (dgamma || dbeta)
            if (const mlp_status s = norm_workspace_fn(R, C, &need))
                return static_cast<int>(s);
        void *ws = on.workspace(a[9], need), *st = stream_of(a[10], t.get_device());
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] {
            return norm_backward_fn(R, C, dy.p, dy.ld, x.p, x.ld, code(dt), gamma, code(wd), mean, rstd, add.p, add.ld, dx.p, dx.ld,
                                    dgamma, dbeta, ws, st);
        });
    });
}

// ---- a Linear's handle and what its arguments have to look like
struct LinearArgs {
    mlp_linear_t h;
    int64_t K, N;
    int experts, device;
    bool nk, act;
    at::ScalarType bias, dw;
    c10::SmallVector<int64_t, 3> weight_shape, bias_shape;
};

constexpr const char *kCapsule = "mlp_linear";

void linear_free(PyObject *c) { delete static_cast<LinearArgs *>(PyCapsule_GetPointer(c, kCapsule)); }

// handle, K, N, experts, layout (1: nk), activation (0: none), bias and dw dtype codes, device -> capsule
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    PyObject *out = nullptr;
    PyObject *ok = guarded(n, 9, [&] {
        int64_t v[9];
        for (int i = 0; i < 9; ++i)
            v[i] = PyLong_AsLongLong(a[i]);
        if (PyErr_Occurred())
            return 0;
        auto type = [](int64_t c) { return c == MLP_DT_BF16 ? kBf16 : kF32; };
        auto *l = new LinearArgs{reinterpret_cast<mlp_linear_t>(v[0]), v[1], v[2], static_cast<int>(v[3]), static_cast<int>(v[8]),
                                 v[4] != 0, v[5] != 0, type(v[6]), type(v[7]), {}, {}};
        if (l->experts) {
            l->weight_shape.push_back(l->experts);
            l->bias_shape.push_back(l->experts);
        }
        l->weight_shape.push_back(l->nk ? l->N : l->K);
        l->weight_shape.push_back(l->nk ? l->K : l->N);
        l->bias_shape.push_back(l->N);
        out = PyCapsule_New(l, kCapsule, linear_free);
        if (!out)
            delete l;
        return 0;
    });
    if (!ok)
        return nullptr;
    Py_DECREF(ok);
    return out;
}

const LinearArgs &args_of(PyObject *o)
{
    const void *p = PyCapsule_GetPointer(o, kCapsule);
    if (!p) {
        PyErr_Clear();
        throw Refused("not a handle of this module");
    }
    return *static_cast<const LinearArgs *>(p);
}

int64_t rows_of(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2)
        throw Refused(std::string(name) + ": expected a matrix");
    return t.size(0);
}

const int32_t *offsets_of(const LinearArgs &l, PyObject *o)
{
    if (l.experts)
        return static_cast<const int32_t *>(Tensors{l.device}.dense(o, "offsets", {l.experts + int64_t{1}}, at::ScalarType::Int));
    if (!absent(o))
        throw Refused("offsets: this handle has no experts");
    return nullptr;
}

// capsule, X, W, Y, bias, residual, Z, offsets, stream
PyObject *linear_forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        if (absent(a[0]))   // closed
            return static_cast<int>(MLP_ERR_INVALID_ARG);
        const LinearArgs &l = args_of(a[0]);
        const int64_t R = rows_of(a[1], "X");
        const Tensors on{l.device};
        const Matrix x = on.matrix(a[1], "X", R, l.K, kBf16), y = on.matrix(a[3], "Y", R, l.N, kBf16);
        const Matrix r = on.matrix_or_none(a[5], "residual", R, l.N, kBf16), z = on.matrix_or_none(a[6], "Z", R, l.N, kBf16);
        const void *w = on.dense(a[2], "W", l.weight_shape, kBf16), *bias = on.dense_or_none(a[4], "bias", l.bias_shape, l.bias);
        const int32_t *off = offsets_of(l, a[7]);
        void *st = stream_of(a[8], l.device);
        if (PyErr_Occurred())
            return 0;
        return unlocked([&] { return linear_forward_fn(l.h, R, x.p, x.ld, w, bias, r.p, r.ld, off, z.p, z.ld, y.p, y.ld, st); });
    });
}

// capsule, dY, X, W, Z, dX, dW, dbias, offsets, workspace, stream
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        if (absent(a[0]))   // closed
            return static_cast<int>(MLP_ERR_INVALID_ARG);
        const LinearArgs &l = args_of(a[0]);
        const int64_t R = rows_of(a[1], "dY");
        const Tensors on{l.device};
        const Matrix dy = on.matrix(a[1], "dY", R, l.N, kBf16);
        const Matrix x = absent(a[6]) ? on.matrix_or_none(a[2], "X", R, l.K, kBf16) : on.matrix(a[2], "X", R, l.K, kBf16);
        const Matrix z = l.act ? on.matrix(a[4], "Z", R, l.N, kBf16) : on.matrix_or_none(a[4], "Z", R, l.N, kBf16);
        const Matrix dx = on.matrix_or_none(a[5], "dX", R, l.K, kBf16);
        const void *w = absent(a[5]) ? on.dense_or_none(a[3], "W", l.weight_shape, kBf16) : on.dense(a[3], "W", l.weight_shape, kBf16);
        void *dw = on.dense_or_none(a[6], "dW", l.weight_shape, l.dw), *db = on.dense_or_none(a[7], "dbias", l.bias_shape, l.bias);
        const int32_t *off = offsets_of(l, a[8]);
        size_t need = 0;
        if (l.act || db)
            if (const mlp_status s = linear_workspace_fn(l.h, R, &need))
                return static_cast<int>(s);
        void *ws = on.workspace(a[9], need), *st = stream_of(a[10], l.device);
        if (PyErr_Occurred())
            return 0;
        return unlocked([&] { return linear_backward_fn(l.h, R, dy.p, dy.ld, x.p, x.ld, w, z.p, z.ld, off, dx.p, dx.ld, dw, db, ws, st); });
    });
}

template <typename F>
PyCFunction fast(F *f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)); }

PyMethodDef kMethods[] = {
    {"bind", fast(bind), METH_FASTCALL, "addresses of the library's functions"},
    {"norm_forward", fast(norm_forward), METH_FASTCALL, nullptr},
    {"norm_backward", fast(norm_backward), METH_FASTCALL, nullptr},
    {"linear", fast(linear), METH_FASTCALL, nullptr},
    {"linear_forward", fast(linear_forward), METH_FASTCALL, nullptr},
    {"linear_backward", fast(linear_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
