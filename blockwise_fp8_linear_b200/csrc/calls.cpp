// calls.cpp -- the Python calls of the few-token and mixture-of-experts operators in
// compiled form: argument checks, output allocation, the current stream and the C ABI
// call.  A decode step makes several of these calls for each token it gives, and most
// finish on the GPU in less time than Python needs to look at their arguments (one token
// through a 2048 x 2048 linear: 4 us on the GPU, 11 us of checks and calls in Python).
//
// A function here handles the plain case, in which every argument is as it should be, on
// the current device and stream, and returns NotImplemented for all others: the Python
// function of the same name then names the fault, or makes the call on another device or
// stream.  Nothing but the handling of arguments is done here.  The interpreter lock is held
// while arguments are looked at and released for what may wait: the allocation of outputs
// (which may synchronize the device) and the call itself (a full launch queue; a host
// function in the stream, ahead of the launch, may be waiting for the lock).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <initializer_list>

#include "fp8bw.h"

namespace {

// The library's entry points, by address (the library is opened by the package).
struct Abi {
    decltype(&fp8_linear_few_workspace) linear_few_workspace;
    decltype(&fp8_linear_few) linear_few;
    decltype(&fp8_moe_route) moe_route;
    decltype(&fp8_moe_route_bwd) moe_route_bwd;
    decltype(&fp8_moe_plan_rows) moe_plan_rows;
    decltype(&fp8_moe_plan_workspace) moe_plan_workspace;
    decltype(&fp8_moe_plan) moe_plan;
    decltype(&fp8_gemm_grouped) gemm_grouped;
    decltype(&fp8_gemm_grouped_wgrad_acc32) gemm_grouped_wgrad_acc32;
    decltype(&fp8_moe_few_workspace) moe_few_workspace;
    decltype(&fp8_moe_few) moe_few;
} abi;

PyObject *error_class;  // Fp8bwError(status, what)

using Shape = std::initializer_list<int64_t>;

// Thrown for whatever is not the plain case.
struct Other {};

const at::Tensor &tensor(PyObject *o)
{
    if (!THPVariable_CheckExact(o))
        throw Other();
    return THPVariable_Unpack(o);
}

bool given(PyObject *o) { return o != Py_None; }

int64_t integer(PyObject *o)
{
    if (!PyLong_CheckExact(o))
        throw Other();
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Other();
    }
    return v;
}

bool truth(PyObject *o)
{
    if (!PyBool_Check(o))
        throw Other();
    return o == Py_True;
}

// Releases the interpreter lock for a scope.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// An output or workspace: the caller's, or one that make() allocates (without the lock).
struct Out {
    at::Tensor t;
    at::ScalarType type;
    int64_t shape[3];
    int dims;
    void make(c10::DeviceIndex dev)
    {
        // (not through the dispatcher, which takes longer than the allocator)
        if (!t.defined())
            t = at::Tensor(at::detail::empty_cuda(at::IntArrayRef(shape, size_t(dims)), type,
                                                  at::Device(at::kCUDA, dev), std::nullopt));
    }
};

// One call: the current device and stream, which its tensors have to be on.
struct Call {
    c10::DeviceIndex dev = -1;  // asked for at the first tensor that is on a GPU
    explicit Call(PyObject *stream)
    {
        if (given(stream))
            throw Other();
    }
    void check(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape)
    {
        if (!t.is_cuda() || t.layout() != at::kStrided)
            throw Other();
        if (dev < 0)
            dev = c10::cuda::current_device();
        if (t.get_device() != dev || t.scalar_type() != type || t.sizes() != shape ||
            !t.is_contiguous())
            throw Other();
    }
    void *in(PyObject *o, at::ScalarType type, Shape shape)
    {
        const at::Tensor &t = tensor(o);
        check(t, type, shape);
        return t.data_ptr();
    }
    Out out(PyObject *o, at::ScalarType type, Shape shape)
    {
        Out r = {at::Tensor(), type, {}, int(shape.size())};
        std::copy(shape.begin(), shape.end(), r.shape);
        if (given(o)) {
            r.t = tensor(o);
            check(r.t, type, shape);
        }
        return r;
    }
    Out workspace(PyObject *o, int64_t need)
    {
        if (!given(o))
            return out(o, at::kByte, {need});
        const at::Tensor &t = tensor(o);
        if (t.dim() != 1 || t.numel() < need)
            throw Other();
        check(t, at::kByte, t.sizes());
        return {t, at::kByte, {t.numel()}, 1};
    }
    // Without the lock: allocates those that the caller has not given, then f(stream).
    // (An input has been looked at, so the device is known.)
    template <class F> int run(std::initializer_list<Out *> outs, F f) const
    {
        const Unlocked unlocked;
        for (Out *o : outs)
            o->make(dev);
        return f(c10::cuda::getCurrentCUDAStream(dev).stream());
    }
};

void require(bool plain)
{
    if (!plain)
        throw Other();
}

bool whole(int64_t d) { return d > 0 && d % 128 == 0; }

bool choices(int64_t T, int64_t E, int64_t k)
{
    return T > 0 && E > 0 && E <= FP8BW_MAX_EXPERTS && k > 0 && k <= E && k <= FP8BW_MAX_CHOICES;
}

// Sets the Python error of a status; true for FP8BW_OK.
bool done(int status, const char *what)
{
    if (status == FP8BW_OK)
        return true;
    PyObject *e = PyObject_CallFunction(error_class, "is", status, what);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return false;
}

template <class... T> PyObject *tuple(const T &...t)
{
    PyObject *items[] = {THPVariable_Wrap(t)...};
    PyObject *r = PyTuple_New(sizeof...(T));
    for (size_t i = 0; i < sizeof...(T); ++i)
        PyTuple_SET_ITEM(r, Py_ssize_t(i), items[i]);
    return r;
}

// A Python function around f(args): NotImplemented for Other; other C++ exceptions (out of
// memory, most likely) become torch's Python ones.
template <Py_ssize_t N, class F> PyObject *guarded(PyObject *const *args, Py_ssize_t n, F f)
{
    if (n != N)
        Py_RETURN_NOTIMPLEMENTED;
    HANDLE_TH_ERRORS
    try {
        return f(args);
    } catch (const Other &) {
        Py_RETURN_NOTIMPLEMENTED;
    }
    END_HANDLE_TH_ERRORS
}

// (x, qw, sw, out, workspace, stream)
PyObject *linear_few(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<6>(args, n, [](PyObject *const *a) -> PyObject * {
        Call c(a[5]);
        const at::Tensor &x = tensor(a[0]), &qw = tensor(a[1]);
        require(x.dim() == 2 && qw.dim() == 2);
        const int64_t M = x.size(0), K = x.size(1), N = qw.size(0);
        require(M > 0 && M <= FP8BW_FEW_TOKENS && whole(N) && whole(K));
        const void *xp = c.in(a[0], at::kBFloat16, {M, K});
        const void *qp = c.in(a[1], at::kByte, {N, K});
        const void *sp = c.in(a[2], at::kFloat, {N / 128, K / 128});
        Out y = c.out(a[3], at::kBFloat16, {M, N}), ws = {};
        const int64_t need = abi.linear_few_workspace(M, K);
        if (need)
            ws = c.workspace(a[4], need);
        const auto call = [&](void *stream) {
            return abi.linear_few(xp, static_cast<const uint8_t *>(qp), static_cast<const float *>(sp),
                                  y.t.data_ptr(), M, N, K, need ? ws.t.data_ptr() : nullptr, stream);
        };
        const int status = need ? c.run({&y, &ws}, call) : c.run({&y}, call);
        return done(status, "fp8_linear_few") ? THPVariable_Wrap(y.t) : nullptr;
    });
}

// (logits, k, renorm, weights, ids, stream)
PyObject *moe_route(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<6>(args, n, [](PyObject *const *a) -> PyObject * {
        Call c(a[5]);
        const at::Tensor &l = tensor(a[0]);
        const bool bf16 = l.scalar_type() == at::kBFloat16;
        require(l.dim() == 2 && (bf16 || l.scalar_type() == at::kFloat));
        const int64_t T = l.size(0), E = l.size(1), k = integer(a[1]);
        require(choices(T, E, k));
        const void *lp = c.in(a[0], l.scalar_type(), {T, E});
        const bool renorm = truth(a[2]);
        Out w = c.out(a[3], at::kFloat, {T, k}), ids = c.out(a[4], at::kInt, {T, k});
        const int status = c.run({&w, &ids}, [&](void *stream) {
            return abi.moe_route(lp, bf16, T, E, k, renorm, static_cast<float *>(w.t.data_ptr()),
                                 static_cast<int32_t *>(ids.t.data_ptr()), stream);
        });
        return done(status, "fp8_moe_route") ? tuple(w.t, ids.t) : nullptr;
    });
}

// (dweights, weights, ids, logits, renorm, dlogits, stream)
PyObject *moe_route_bwd(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<7>(args, n, [](PyObject *const *a) -> PyObject * {
        Call c(a[6]);
        const at::Tensor &ids = tensor(a[2]), &l = tensor(a[3]);
        const bool bf16 = l.scalar_type() == at::kBFloat16;
        require(l.dim() == 2 && ids.dim() == 2 && (bf16 || l.scalar_type() == at::kFloat));
        const int64_t T = l.size(0), E = l.size(1), k = ids.size(1);
        require(choices(T, E, k));
        const void *dw = c.in(a[0], at::kFloat, {T, k}), *w = c.in(a[1], at::kFloat, {T, k});
        const void *ip = c.in(a[2], at::kInt, {T, k}), *lp = c.in(a[3], l.scalar_type(), {T, E});
        const bool renorm = truth(a[4]);
        Out dl = c.out(a[5], l.scalar_type(), {T, E});
        const int status = c.run({&dl}, [&](void *stream) {
            return abi.moe_route_bwd(static_cast<const float *>(dw), static_cast<const float *>(w),
                                     static_cast<const int32_t *>(ip), lp, bf16, T, E, k, renorm,
                                     dl.t.data_ptr(), stream);
        });
        return done(status, "fp8_moe_route_bwd") ? THPVariable_Wrap(dl.t) : nullptr;
    });
}

// (ids, E, seg, row, src, workspace, stream)
PyObject *moe_plan(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<7>(args, n, [](PyObject *const *a) -> PyObject * {
        Call c(a[6]);
        const at::Tensor &ids = tensor(a[0]);
        require(ids.dim() == 2);
        const int64_t T = ids.size(0), k = ids.size(1), E = integer(a[1]);
        require(choices(T, E, k));
        const int64_t rows = abi.moe_plan_rows(T, E, k);
        require(rows > 0);
        const void *ip = c.in(a[0], at::kInt, {T, k});
        Out seg = c.out(a[2], at::kInt, {E + 1}), row = c.out(a[3], at::kInt, {T, k});
        Out src = c.out(a[4], at::kInt, {rows});
        Out ws = c.workspace(a[5], abi.moe_plan_workspace(T, E, k));
        const int status = c.run({&seg, &row, &src, &ws}, [&](void *stream) {
            return abi.moe_plan(static_cast<const int32_t *>(ip), T, E, k,
                                static_cast<int32_t *>(seg.t.data_ptr()),
                                static_cast<int32_t *>(row.t.data_ptr()),
                                static_cast<int32_t *>(src.t.data_ptr()), ws.t.data_ptr(), stream);
        });
        return done(status, "fp8_moe_plan") ? tuple(seg.t, row.t, src.t) : nullptr;
    });
}

// A grouped GEMM's operands.
struct Grouped {
    const uint8_t *a, *b;
    const float *sa, *sb;
    const int32_t *seg;
    int64_t E, M, N, K;
    Grouped(Call &c, int64_t mode, PyObject *const *p)  // a, sa, b, sb, seg, M, N, K
    {
        M = integer(p[5]);
        N = integer(p[6]);
        K = integer(p[7]);
        require(whole(M) && whole(N) && whole(K));
        const at::Tensor &s = tensor(p[4]);
        require(s.dim() == 1 && s.numel() >= 2 && s.numel() <= FP8BW_MAX_EXPERTS + 1);
        E = s.numel() - 1;
        a = static_cast<const uint8_t *>(c.in(p[0], at::kByte, {M, K}));
        sa = static_cast<const float *>(c.in(p[1], at::kFloat, {K / 128, M}));
        if (mode == FP8BW_WGRAD) {
            b = static_cast<const uint8_t *>(c.in(p[2], at::kByte, {N, K}));
            sb = static_cast<const float *>(c.in(p[3], at::kFloat, {K / 128, N}));
        } else {
            const int64_t r = mode == FP8BW_FPROP ? N : K, q = mode == FP8BW_FPROP ? K : N;
            b = static_cast<const uint8_t *>(c.in(p[2], at::kByte, {E, r, q}));
            sb = static_cast<const float *>(c.in(p[3], at::kFloat, {E, r / 128, q / 128}));
        }
        seg = static_cast<const int32_t *>(c.in(p[4], at::kInt, {E + 1}));
    }
};

// (mode, a, sa, b, sb, seg, M, N, K, out, stream)
PyObject *gemm_grouped(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<11>(args, n, [](PyObject *const *a) -> PyObject * {
        Call c(a[10]);
        const int64_t mode = integer(a[0]);
        require(mode >= FP8BW_FPROP && mode <= FP8BW_WGRAD);
        const Grouped g(c, mode, a + 1);
        Out d = mode == FP8BW_WGRAD ? c.out(a[9], at::kBFloat16, {g.E, g.M, g.N})
                                    : c.out(a[9], at::kBFloat16, {g.M, g.N});
        const int status = c.run({&d}, [&](void *stream) {
            return abi.gemm_grouped(int(mode), g.a, g.sa, g.b, g.sb, g.seg, g.E, d.t.data_ptr(), g.M,
                                    g.N, g.K, stream);
        });
        return done(status, "fp8_gemm_grouped") ? THPVariable_Wrap(d.t) : nullptr;
    });
}

// (a, sa, b, sb, seg, M, N, K, dw32, stream)
PyObject *gemm_grouped_wgrad_acc32(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<10>(args, n, [](PyObject *const *a) -> PyObject * {
        Call c(a[9]);
        const Grouped g(c, FP8BW_WGRAD, a);
        require(given(a[8]));
        void *dw = c.in(a[8], at::kFloat, {g.E, g.M, g.N});
        const int status = c.run({}, [&](void *stream) {
            return abi.gemm_grouped_wgrad_acc32(g.a, g.sa, g.b, g.sb, g.seg, g.E,
                                                static_cast<float *>(dw), g.M, g.N, g.K, stream);
        });
        if (!done(status, "fp8_gemm_grouped_wgrad_acc32"))
            return nullptr;
        Py_INCREF(a[8]);
        return a[8];
    });
}

// (x, w1, s1, w2, s2, ids, weights, out, workspace, stream)
PyObject *moe_few(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<10>(args, n, [](PyObject *const *a) -> PyObject * {
        Call c(a[9]);
        const at::Tensor &x = tensor(a[0]), &w2 = tensor(a[3]), &ids = tensor(a[5]);
        require(x.dim() == 2 && w2.dim() == 3 && ids.dim() == 2);
        const int64_t T = x.size(0), H = x.size(1), E = w2.size(0), I = w2.size(2), k = ids.size(1);
        require(T <= FP8BW_FEW_TOKENS && whole(H) && whole(I) && choices(T, E, k));
        const void *xp = c.in(a[0], at::kBFloat16, {T, H});
        const void *w1p = c.in(a[1], at::kByte, {E, 2 * I, H});
        const void *s1p = c.in(a[2], at::kFloat, {E, 2 * I / 128, H / 128});
        const void *w2p = c.in(a[3], at::kByte, {E, H, I});
        const void *s2p = c.in(a[4], at::kFloat, {E, H / 128, I / 128});
        const void *ip = c.in(a[5], at::kInt, {T, k}), *wp = c.in(a[6], at::kFloat, {T, k});
        const int64_t need = abi.moe_few_workspace(T, k, H, I);
        require(need > 0);
        Out y = c.out(a[7], at::kBFloat16, {T, H}), ws = c.workspace(a[8], need);
        const int status = c.run({&y, &ws}, [&](void *stream) {
            return abi.moe_few(xp, static_cast<const uint8_t *>(w1p), static_cast<const float *>(s1p),
                               static_cast<const uint8_t *>(w2p), static_cast<const float *>(s2p),
                               static_cast<const int32_t *>(ip), static_cast<const float *>(wp),
                               y.t.data_ptr(), T, E, k, H, I, ws.t.data_ptr(), stream);
        });
        return done(status, "fp8_moe_few") ? THPVariable_Wrap(y.t) : nullptr;
    });
}

// open(error_class, address of each entry point): the addresses in the order of Abi.
PyObject *open_library(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    constexpr Py_ssize_t count = sizeof(Abi) / sizeof(void *);
    if (n != count + 1) {
        PyErr_SetString(PyExc_TypeError, "open(error_class, addresses...)");
        return nullptr;
    }
    void *p[count];
    for (Py_ssize_t i = 0; i < count; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i + 1]);
        if (!p[i])
            return PyErr_Occurred() ? nullptr
                                    : (PyErr_SetString(PyExc_ValueError, "null address"), nullptr);
    }
    static_assert(sizeof p == sizeof abi, "one address per entry point");
    memcpy(&abi, p, sizeof abi);
    Py_INCREF(args[0]);
    Py_XDECREF(error_class);
    error_class = args[0];
    Py_RETURN_NONE;
}

#define FP8BW_CALL(name, f) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    FP8BW_CALL("open", open_library),
    FP8BW_CALL("linear_few", linear_few),
    FP8BW_CALL("moe_route", moe_route),
    FP8BW_CALL("moe_route_bwd", moe_route_bwd),
    FP8BW_CALL("moe_plan", moe_plan),
    FP8BW_CALL("gemm_grouped", gemm_grouped),
    FP8BW_CALL("gemm_grouped_wgrad_acc32", gemm_grouped_wgrad_acc32),
    FP8BW_CALL("moe_few", moe_few),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr,
                      nullptr};

} // namespace

PyMODINIT_FUNC PyInit__calls(void)
{
    return PyModule_Create(&module);
}
