// marshal.cpp -- the argument checks of mlp_latency_gb300/block.py, experts.py and clip.py: tensors in, a call of the C ABI
// (include/mlp_block.h, mlp_experts.h, mlp_clip.h) out.
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

#include <algorithm>
#include <sstream>
#include <stdexcept>

#include "../../include/mlp_block.h"
#include "../../include/mlp_clip.h"
#include "../../include/mlp_experts.h"

namespace {

decltype(&mlp_layernorm_forward) norm_forward_fn;
decltype(&mlp_layernorm_backward) norm_backward_fn;
decltype(&mlp_layernorm_workspace_size) norm_workspace_fn;
decltype(&mlp_linear_workspace_size) linear_workspace_fn;
decltype(&mlp_linear_forward) linear_forward_fn;
decltype(&mlp_linear_backward) linear_backward_fn;

decltype(&mlp_route_workspace_size) route_workspace_fn;
decltype(&mlp_route_forward) route_forward_fn;
decltype(&mlp_route_backward) route_backward_fn;
decltype(&mlp_dispatch_forward) dispatch_forward_fn;
decltype(&mlp_dispatch_backward) dispatch_backward_fn;
decltype(&mlp_combine_forward) combine_forward_fn;
decltype(&mlp_combine_backward) combine_backward_fn;
decltype(&mlp_clip_workspace_size) clip_workspace_fn;
decltype(&mlp_gradient_norm) gradient_norm_fn;
decltype(&mlp_clip_gradients) clip_gradients_fn;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

constexpr auto kBf16 = at::ScalarType::BFloat16;
constexpr auto kF32 = at::ScalarType::Float;
constexpr auto kI32 = at::ScalarType::Int;

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
void address(F *&f, PyObject *a) { f = reinterpret_cast<F *>(PyLong_AsVoidPtr(a)); }

PyObject *bind_experts(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        address(route_workspace_fn, a[0]);
        address(route_forward_fn, a[1]);
        address(route_backward_fn, a[2]);
        address(dispatch_forward_fn, a[3]);
        address(dispatch_backward_fn, a[4]);
        address(combine_forward_fn, a[5]);
        address(combine_backward_fn, a[6]);
        return 0;
    });
}

PyObject *bind_clip(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 3, [&] {
        address(clip_workspace_fn, a[0]);
        address(gradient_norm_fn, a[1]);
        address(clip_gradients_fn, a[2]);
        return 0;
    });
}

// The matrix that a call's other tensors go by.
const at::Tensor &matrix_of(PyObject *o, const char *name, const char *op)
{
    const at::Tensor &x = tensor(o, name);
    if (x.dim() != 2 || (x.scalar_type() != kBf16 && x.scalar_type() != kF32))
        throw Refused(std::string(op) + ": " + name + " is a matrix of bfloat16 or float32");
    return x;
}

// int32 [tokens, top]: the choices, or their rows
const at::Tensor &choices_of(PyObject *o, const char *name, int64_t tokens)
{
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2 || t.size(0) != tokens || t.size(1) < 1 || t.size(1) > MLP_MAX_TOP)
        throw Refused(std::string(name) + ": expected int32 [" + std::to_string(tokens) + ", top], top 1 to " + std::to_string(MLP_MAX_TOP));
    return t;
}

// logits, gates, experts, slots, offsets, counts, loss, mask, normalize, workspace, stream
PyObject *route_forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const at::Tensor &t = matrix_of(a[0], "logits", "route");
        const int64_t T = t.size(0), E = t.size(1), k = choices_of(a[2], "experts", T).size(1);
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix l = on.matrix(a[0], "logits", T, E, t.scalar_type());
        float *gates = static_cast<float *>(on.dense(a[1], "gates", {T, k}, kF32));
        auto *chosen = static_cast<int32_t *>(on.dense(a[2], "experts", {T, k}, kI32)), *slots = static_cast<int32_t *>(on.dense(a[3], "slots", {T, k}, kI32));
        auto *offsets = static_cast<int32_t *>(on.dense(a[4], "offsets", {E + 1}, kI32));
        auto *counts = static_cast<int32_t *>(on.dense_or_none(a[5], "counts", {E}, kI32));
        float *loss = static_cast<float *>(on.dense_or_none(a[6], "loss", {1}, kF32));
        auto *mask = static_cast<uint8_t *>(on.dense_or_none(a[7], "mask", {T}, at::ScalarType::Bool));
        const int normalize = PyObject_IsTrue(a[8]);
        size_t need = 0;
        if (const mlp_status s = route_workspace_fn(T, E, &need))
            return static_cast<int>(s);
        void *ws = on.workspace(a[9], need), *st = stream_of(a[10], on.device);
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] {
            return route_forward_fn(T, E, static_cast<int32_t>(k), l.p, l.ld, code(t.scalar_type()), mask, normalize, gates, chosen, slots,
                                    offsets, counts, loss, ws, st);
        });
    });
}

// logits, experts, offsets, dlogits, dgates, dloss, normalize, stream
PyObject *route_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const at::Tensor &t = matrix_of(a[0], "logits", "route");
        const int64_t T = t.size(0), E = t.size(1), k = choices_of(a[1], "experts", T).size(1);
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix l = on.matrix(a[0], "logits", T, E, t.scalar_type()), d = on.matrix(a[3], "dlogits", T, E, t.scalar_type());
        const auto *chosen = static_cast<int32_t *>(on.dense(a[1], "experts", {T, k}, kI32));
        const auto *offsets = static_cast<int32_t *>(on.dense(a[2], "offsets", {E + 1}, kI32));
        const float *dgates = static_cast<float *>(on.dense_or_none(a[4], "dgates", {T, k}, kF32));
        const float *dloss = static_cast<float *>(on.dense_or_none(a[5], "dloss", {1}, kF32));
        const int normalize = PyObject_IsTrue(a[6]);
        void *st = stream_of(a[7], on.device);
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] {
            return route_backward_fn(T, E, static_cast<int32_t>(k), l.p, l.ld, code(t.scalar_type()), normalize, chosen, offsets, dgates,
                                     dloss, d.p, d.ld, st);
        });
    });
}

struct Slots {
    const int32_t *p;
    int64_t tokens, top;
};

Slots slots_of(const Tensors &on, PyObject *o, int64_t tokens)
{
    const int64_t k = choices_of(o, "slots", tokens).size(1);
    return {static_cast<const int32_t *>(on.dense(o, "slots", {tokens, k}, kI32)), tokens, k};
}

// x, slots, y, stream
PyObject *dispatch_forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 4, [&] {
        const at::Tensor &t = matrix_of(a[0], "x", "dispatch");
        const at::ScalarType dt = t.scalar_type();
        const int64_t T = t.size(0), C = t.size(1), R = rows_of(a[2], "y");
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix x = on.matrix(a[0], "x", T, C, dt), y = on.matrix(a[2], "y", R, C, dt);
        const Slots s = slots_of(on, a[1], T);
        void *st = stream_of(a[3], on.device);
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] { return dispatch_forward_fn(T, C, static_cast<int32_t>(s.top), x.p, x.ld, code(dt), s.p, R, y.p, y.ld, st); });
    });
}

// dy, slots, dx, dx_add, stream
PyObject *dispatch_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 5, [&] {
        const at::Tensor &t = matrix_of(a[2], "dx", "dispatch");
        const at::ScalarType dt = t.scalar_type();
        const int64_t T = t.size(0), C = t.size(1), R = rows_of(a[0], "dy");
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix dx = on.matrix(a[2], "dx", T, C, dt), dy = on.matrix(a[0], "dy", R, C, dt);
        const Matrix add = on.matrix_or_none(a[3], "dx_add", T, C, dt);
        const Slots s = slots_of(on, a[1], T);
        void *st = stream_of(a[4], on.device);
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] {
            return dispatch_backward_fn(T, C, static_cast<int32_t>(s.top), dy.p, dy.ld, code(dt), s.p, R, add.p, add.ld, dx.p, dx.ld, st);
        });
    });
}

// z, gates, slots, y, residual, stream
PyObject *combine_forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        const at::Tensor &t = matrix_of(a[3], "y", "combine");
        const at::ScalarType dt = t.scalar_type();
        const int64_t T = t.size(0), C = t.size(1), R = rows_of(a[0], "z");
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix y = on.matrix(a[3], "y", T, C, dt), z = on.matrix(a[0], "z", R, C, dt);
        const Matrix res = on.matrix_or_none(a[4], "residual", T, C, dt);
        const Slots s = slots_of(on, a[2], T);
        const float *gates = static_cast<float *>(on.dense(a[1], "gates", {T, s.top}, kF32));
        void *st = stream_of(a[5], on.device);
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] {
            return combine_forward_fn(T, C, static_cast<int32_t>(s.top), z.p, z.ld, code(dt), gates, s.p, R, res.p, res.ld, y.p, y.ld, st);
        });
    });
}

// dy, z, gates, slots, dz, dgates, stream
PyObject *combine_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        const at::Tensor &t = matrix_of(a[0], "dy", "combine");
        const at::ScalarType dt = t.scalar_type();
        const int64_t T = t.size(0), C = t.size(1);
        const int64_t R = absent(a[1]) ? absent(a[4]) ? 0 : rows_of(a[4], "dz") : rows_of(a[1], "z");
        const Tensors on{static_cast<int>(t.get_device())};
        const Matrix dy = on.matrix(a[0], "dy", T, C, dt);
        const Matrix z = absent(a[5]) ? on.matrix_or_none(a[1], "z", R, C, dt) : on.matrix(a[1], "z", R, C, dt);
        const Matrix dz = on.matrix_or_none(a[4], "dz", R, C, dt);
        const Slots s = slots_of(on, a[3], T);
        const float *gates = static_cast<float *>(absent(a[4]) ? on.dense_or_none(a[2], "gates", {T, s.top}, kF32) : on.dense(a[2], "gates", {T, s.top}, kF32));
        float *dgates = static_cast<float *>(on.dense_or_none(a[5], "dgates", {T, s.top}, kF32));
        void *st = stream_of(a[6], on.device);
        if (PyErr_Occurred())
            return 0;
        const CurrentDevice current(on.device);
        return unlocked([&] {
            return combine_backward_fn(T, C, static_cast<int32_t>(s.top), dy.p, dy.ld, z.p, z.ld, code(dt), gates, s.p, R, dz.p, dz.ld, dgates, st);
        });
    });
}

// A list or tuple of tensors, seen without a copy.
struct Sequence {
    PyObject *o;
    Sequence(PyObject *list, const char *name)
    {
        if (!PyList_Check(list) && !PyTuple_Check(list))
            throw Refused(std::string(name) + ": expected a list or tuple of tensors");
        o = list;
    }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(o); }
    PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(o, i); }
};

// Bytes at an address.
struct Span {
    uintptr_t from, to;
    Span(const void *p, size_t bytes) : from(reinterpret_cast<uintptr_t>(p)), to(from + bytes) {}
    bool meets(const Span &o) const { return from < o.to && o.from < to && from < to && o.from < o.to; }
    void take(const Span &o)
    {
        from = std::min(from, o.from);
        to = std::max(to, o.to);
    }
};

Span data_of(const mlp_tensor &t) { return {t.data, static_cast<size_t>(t.count) * (t.dtype == MLP_DT_BF16 ? 2 : 4)}; }
Span out_of(const mlp_tensor &t) { return {t.out, static_cast<size_t>(t.count) * (t.dtype == MLP_DT_BF16 ? 2 : 4)}; }

// grads, out (None: in place), max_norm (None: the norm only), norm, eps, workspace, stream
PyObject *clip(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        const Sequence grads(a[0], "grads");
        const bool clipped = !absent(a[2]), elsewhere_out = clipped && !absent(a[1]);
        const Tensors on{static_cast<int>(tensor(a[3], "norm").get_device())};
        float *norm = static_cast<float *>(on.dense(a[3], "norm", {1}, kF32));
        c10::SmallVector<mlp_tensor, 64> list(static_cast<size_t>(grads.size()));
        Span all(reinterpret_cast<void *>(UINTPTR_MAX), 0);   // from the first byte of a tensor to the last
        all.to = 0;
        for (Py_ssize_t i = 0; i < grads.size(); ++i) {
            const at::Tensor &t = tensor(grads[i], "grads");
            if ((t.scalar_type() != kBf16 && t.scalar_type() != kF32) || elsewhere(t, on.device) || !t.is_contiguous())
                throw Refused("grads[" + std::to_string(i) + "]: expected a contiguous CUDA tensor of bfloat16 or float32 on cuda:" + std::to_string(on.device));
            list[i] = {t.data_ptr(), t.data_ptr(), t.numel(), code(t.scalar_type())};
            all.take(data_of(list[i]));
        }
        if (elsewhere_out) {
            const Sequence out(a[1], "out");
            if (out.size() != grads.size())
                throw Refused("out: expected as many tensors as gradients");
            for (Py_ssize_t i = 0; i < grads.size(); ++i) {
                const at::Tensor &t = THPVariable_Unpack(grads[i]);
                list[i].out = on.dense(out[i], "out", t.sizes(), t.scalar_type());
                all.take(out_of(list[i]));
            }
        }
        const float max_norm = clipped ? static_cast<float>(PyFloat_AsDouble(a[2])) : 0.0f, eps = static_cast<float>(PyFloat_AsDouble(a[4]));
        size_t need = 0;
        if (const mlp_status s = clip_workspace_fn(grads.size(), &need))
            return static_cast<int>(s);
        void *ws = on.workspace(a[5], need), *st = stream_of(a[6], on.device);
        if (PyErr_Occurred())
            return 0;
        // Nothing that is written may be read by others meanwhile.  (Each tensor is looked at where one of the two lies among them: 2 us for
        // 1000, which take 30 otherwise.)
        const Span used(ws, ws ? need : 0), result(norm, clipped ? sizeof(float) : 0);
        bool bad = result.meets(used);
        if (all.meets(used) || all.meets(result))
            for (const mlp_tensor &t : list)
                for (const Span &s : {data_of(t), out_of(t)})
                    bad = bad || s.meets(used) || s.meets(result);
        if (bad)
            throw Refused("norm and workspace: one overlaps the other or a tensor of the list");
        const CurrentDevice current(on.device);
        return unlocked([&]() -> int {
            const int64_t count = static_cast<int64_t>(list.size());
            return clipped ? clip_gradients_fn(count, list.data(), max_norm, eps, norm, ws, st) : gradient_norm_fn(count, list.data(), norm, ws, st);
        });
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
    {"bind_experts", fast(bind_experts), METH_FASTCALL, "addresses of the library's functions"},
    {"bind_clip", fast(bind_clip), METH_FASTCALL, "addresses of the library's functions"},
    {"route_forward", fast(route_forward), METH_FASTCALL, nullptr},
    {"route_backward", fast(route_backward), METH_FASTCALL, nullptr},
    {"dispatch_forward", fast(dispatch_forward), METH_FASTCALL, nullptr},
    {"dispatch_backward", fast(dispatch_backward), METH_FASTCALL, nullptr},
    {"combine_forward", fast(combine_forward), METH_FASTCALL, nullptr},
    {"combine_backward", fast(combine_backward), METH_FASTCALL, nullptr},
    {"clip", fast(clip), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
