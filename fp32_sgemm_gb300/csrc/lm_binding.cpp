// Python side of the language-model operators: reads torch tensors, checks
// them, asks the C ABI (include/sgemm_gb300_lm.h) for the workspace and makes
// the call.  Argument marshalling only.  In C++ because the same checks in
// Python take 13 to 20 us a call, three times what the smallest products take
// on the device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <optional>

#include "../../include/sgemm_gb300_lm.h"
#include "context.h"

namespace {

PyObject *g_check = nullptr;        // _binding._check(status, where)
PyObject *g_stream_ptr = nullptr;   // _binding._stream_ptr(stream, device index)
PyObject *g_out_of_memory = nullptr;   // torch.OutOfMemoryError
PyObject *g_name_ptr = nullptr;

struct Failed {};                   // a Python error is set

[[noreturn]] void fail(PyObject *type, const char *format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw Failed{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

const char *type_name(at::ScalarType t) { return c10::toString(t); }

sgemmDataType_t type_of(const at::Tensor &t, const char *name) {
    switch (t.scalar_type()) {
        case at::kFloat: return SGEMM_TYPE_F32;
        case at::kHalf: return SGEMM_TYPE_F16;
        case at::kBFloat16: return SGEMM_TYPE_BF16;
        default: fail(PyExc_TypeError, "%s must be float32, float16 or bfloat16, got %s", name,
                      type_name(t.scalar_type()));
    }
}

c10::Device device_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return t.device();
}

struct Matrix {
    void *ptr = nullptr;
    int64_t rows = 0, cols = 0, ld = 1, stride = 0;
};

void check_kind(const at::Tensor &t, const char *name, at::ScalarType type, c10::Device dev) {
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
    if (t.device() != dev) fail(PyExc_ValueError, "%s must be on %s", name, dev.str().c_str());
}

// Row pitch of the matrices whose rows are dimension `d` of t.  Rows that are
// the same memory (a broadcast) have none: with one column, too, whose stride
// of 0 must not pass for a pitch of 1, with which the rows would be read beyond
// the tensor.
int64_t pitch(const at::Tensor &t, int d, const char *name) {
    const int64_t rows = t.size(d), cols = t.size(d + 1);
    if (rows <= 1 || cols == 0) return std::max<int64_t>(1, cols);
    if (t.stride(d) < cols) fail(PyExc_ValueError, "%s has overlapping rows", name);
    return t.stride(d);
}

// Row-major matrix of the call's type and device; rows, cols < 0: any.
Matrix matrix(const at::Tensor &t, const char *name, at::ScalarType type, c10::Device dev, int64_t rows = -1,
              int64_t cols = -1) {
    check_kind(t, name, type, dev);
    if (t.dim() != 2) fail(PyExc_ValueError, "%s must be 2-D", name);
    Matrix m;
    m.rows = t.size(0);
    m.cols = t.size(1);
    if ((rows >= 0 && m.rows != rows) || (cols >= 0 && m.cols != cols))
        fail(PyExc_ValueError, "%s has shape (%lld, %lld), expected (%lld, %lld)", name, (long long)m.rows,
             (long long)m.cols, (long long)(rows < 0 ? m.rows : rows), (long long)(cols < 0 ? m.cols : cols));
    if (m.rows > 0 && m.cols > 1 && t.stride(1) != 1)
        fail(PyExc_ValueError, "%s must be row major (stride(1) == 1)", name);
    m.ld = pitch(t, 0, name);
    m.ptr = const_cast<void *>(t.const_data_ptr());
    return m;
}

// Stack of `n` row-major rows x cols matrices.
Matrix stack(const at::Tensor &t, const char *name, at::ScalarType type, c10::Device dev, int64_t n, int64_t rows,
             int64_t cols) {
    check_kind(t, name, type, dev);
    if (t.dim() != 3) fail(PyExc_ValueError, "%s must be 3-D", name);
    if (t.size(0) != n || t.size(1) != rows || t.size(2) != cols)
        fail(PyExc_ValueError, "%s has shape (%lld, %lld, %lld), expected (%lld, %lld, %lld)", name,
             (long long)t.size(0), (long long)t.size(1), (long long)t.size(2), (long long)n, (long long)rows,
             (long long)cols);
    Matrix m;
    m.rows = rows;
    m.cols = cols;
    if (rows > 0 && cols > 1 && t.stride(2) != 1)
        fail(PyExc_ValueError, "%s must be row major (stride(2) == 1)", name);
    m.ld = pitch(t, 1, name);
    m.stride = n > 1 ? t.stride(0) : 0;
    if (n > 1 && rows > 0 && cols > 0 && m.stride < (rows - 1) * m.ld + cols)
        fail(PyExc_ValueError, "%s must hold one matrix per group (no broadcast)", name);
    m.ptr = const_cast<void *>(t.const_data_ptr());
    return m;
}

// Contiguous T x k table beside T tokens (k < 0: any).
template <class T>
T *table(const at::Tensor &t, const char *name, at::ScalarType type, c10::Device dev, int64_t rows, int64_t k) {
    check_kind(t, name, type, dev);
    if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (k >= 0 && t.size(1) != k) || !t.is_contiguous())
        fail(PyExc_ValueError, "%s must be a contiguous matrix with a row for each token%s", name,
             k >= 0 ? " and a column for each of its choices" : "");
    return static_cast<T *>(const_cast<void *>(t.const_data_ptr()));
}

template <class T>
T *vector(PyObject *o, const char *name, at::ScalarType type, c10::Device dev, int64_t n) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be a %s tensor", name, type_name(type));
    if (t.device() != dev || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
        fail(PyExc_ValueError, "%s must be a contiguous vector%s on %s", name, n >= 0 ? " of the call's length" : "",
             dev.str().c_str());
    return static_cast<T *>(const_cast<void *>(t.const_data_ptr()));
}

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(dev));
}

// `out` or a new matrix.
at::Tensor output(PyObject *out, at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
    return out == Py_None ? make(sizes, type, dev) : tensor(out, "out");
}

void check(sgemmStatus_t st, const char *where) {
    if (st == SGEMM_STATUS_SUCCESS) return;
    PyObject *r = PyObject_CallFunction(g_check, "is", int(st), where);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
    throw Failed{};
}

// A call: the settings and the error word of a Handle of this package, the
// stream, and a workspace of its own.  With a stream given, what the call
// allocates belongs to that stream, and what it reads is kept from reuse until
// that stream has passed.
//
// The workspace comes from torch's allocator for this one call: calls on
// different streams or from different threads share none of it, whatever
// handle they go through, and a captured call's stays in its graph's memory.
// (A buffer kept by the handle would have to be one for each stream and each
// capture.  Asking takes some tenths of a microsecond of the host's time; loss of
// 16 rows, 32000 x 1024, 21.1 us with a kept buffer and 21.3.)
struct Call {
    sgemmContext context;           // the handle's, but for the workspace
    sgemmHandle_t handle = nullptr;
    cudaStream_t stream = nullptr;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    c10::DataPtr buffer;

    Call(PyObject *h, PyObject *s, c10::Device dev, std::initializer_list<PyObject *> read) {
        PyObject *p = PyObject_GetAttr(h, g_name_ptr);
        if (p == nullptr) throw Failed{};
        const sgemmContext *given = static_cast<const sgemmContext *>(PyLong_AsVoidPtr(p));
        Py_DECREF(p);
        if (PyErr_Occurred()) throw Failed{};
        if (given != nullptr) {
            context = *given;
            context.ws = nullptr;
            context.ws_bytes = 0;
            handle = &context;
        }
        if (s == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
            return;
        }
        PyObject *v = PyObject_CallFunction(g_stream_ptr, "Oi", s, int(dev.index()));
        if (v == nullptr) throw Failed{};
        stream = v == Py_None ? nullptr : static_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
        Py_DECREF(v);
        if (PyErr_Occurred()) throw Failed{};
        const c10::cuda::CUDAStream on = stream == nullptr ? c10::cuda::getDefaultCUDAStream(dev.index())
                                                           : c10::cuda::getStreamFromExternal(stream, dev.index());
        if (on == c10::cuda::getCurrentCUDAStream(dev.index())) return;
        guard.emplace(on);
        for (PyObject *t : read)
            if (t != Py_None)
                c10::cuda::CUDACachingAllocator::recordStream(THPVariable_Unpack(t).storage().data_ptr(), on);
    }
    Call(const Call &) = delete;
    void workspace(size_t need) {
        if (need == 0) return;
        buffer = c10::cuda::CUDACachingAllocator::get()->allocate(need);
        context.ws = buffer.get();
        context.ws_bytes = need;
    }
};

void expect(Py_ssize_t given, Py_ssize_t want) {
    if (given != want) fail(PyExc_TypeError, "expected %zd arguments, got %zd", want, given);
}

template <class F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (const Failed &) {
        return nullptr;
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

int64_t whole(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        fail(PyExc_TypeError, "%s must be an integer", name);
    }
    return v;
}

bool truth(PyObject *o) {
    const int is = PyObject_IsTrue(o);
    if (is < 0) throw Failed{};
    return is != 0;
}

// Whether the call belongs into torch's graph, by an operand that requires a gradient
// or has a tangent (which goes on where nothing is recorded): then it answers None,
// and _lm.py takes it there (inside, neither counts).
bool recorded(const at::Tensor &a) {
    return (a.requires_grad() && c10::GradMode::is_enabled()) ||
           (c10::AutogradState::get_tls_state().get_fw_grad_mode() && a._fw_grad(0).defined());
}

bool recorded(const at::Tensor &a, const at::Tensor &b) { return recorded(a) || recorded(b); }

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

// (x, w, group_ends, trans_w, out, handle, stream)
PyObject *py_grouped_gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 7);
        const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
        if (a[4] == Py_None && recorded(x, w)) Py_RETURN_NONE;
        const sgemmDataType_t ty = type_of(x, "x");
        const c10::Device dev = device_of(x, "x");
        const at::ScalarType st = x.scalar_type();
        const Matrix mx = matrix(x, "x", st, dev);
        if (w.dim() != 3) fail(PyExc_ValueError, "w must be a 3-D tensor [groups, rows, cols]");
        const bool trans = truth(a[3]);
        const int64_t T = mx.rows, K = mx.cols, G = w.size(0), N = w.size(trans ? 1 : 2);
        const Matrix mw = stack(w, "w", st, dev, G, trans ? N : K, trans ? K : N);
        const int32_t *ends = vector<int32_t>(a[2], "group_ends", at::kInt, dev, G);
        if (a[4] != Py_None) matrix(tensor(a[4], "out"), "out", st, dev, T, N);   // before it is recorded
        Call c(a[5], a[6], dev, {a[0], a[1], a[2], a[4]});
        const at::Tensor out = output(a[4], {T, N}, st, dev);
        const Matrix my = matrix(out, "out", st, dev, T, N);
        const sgemmOperation_t op = trans ? SGEMM_OP_T : SGEMM_OP_N;
        size_t need = 0;
        check(sgemmGroupedWorkspaceSize(c.handle, ty, op, T, N, K, G, mx.ptr, mx.ld, mw.ptr, mw.ld, mw.stride, &need),
              "sgemmGroupedWorkspaceSize");
        c.workspace(need);
        check(sgemmGrouped(c.handle, ty, op, T, N, K, G, mx.ptr, mx.ld, mw.ptr, mw.ld, mw.stride, ends, my.ptr, my.ld,
                           c.stream), "sgemmGrouped");
        return wrap(out);
    });
}

// (x, dy, group_ends, trans_w, out, handle, stream)
PyObject *py_grouped_gemm_weight_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 7);
        const at::Tensor &x = tensor(a[0], "x"), &dy = tensor(a[1], "dy");
        const sgemmDataType_t ty = type_of(x, "x");
        const c10::Device dev = device_of(x, "x");
        const at::ScalarType st = x.scalar_type();
        Matrix l = matrix(x, "x", st, dev), r = matrix(dy, "dy", st, dev);
        if (l.rows != r.rows)
            fail(PyExc_ValueError, "x has %lld rows, dy has %lld", (long long)l.rows, (long long)r.rows);
        if (truth(a[3])) std::swap(l, r);
        const int64_t T = l.rows, M = l.cols, N = r.cols;
        const int32_t *ends = vector<int32_t>(a[2], "group_ends", at::kInt, dev, -1);
        const int64_t G = THPVariable_Unpack(a[2]).size(0);
        if (a[4] != Py_None) stack(tensor(a[4], "out"), "out", st, dev, G, M, N);   // before it is recorded
        Call c(a[5], a[6], dev, {a[0], a[1], a[2], a[4]});
        const at::Tensor out = output(a[4], {G, M, N}, st, dev);
        const Matrix mc = stack(out, "out", st, dev, G, M, N);
        size_t need = 0;
        check(sgemmGroupedWeightGradWorkspaceSize(c.handle, ty, T, M, N, G, l.ptr, l.ld, r.ptr, r.ld, &need),
              "sgemmGroupedWeightGradWorkspaceSize");
        c.workspace(need);
        check(sgemmGroupedWeightGrad(c.handle, ty, T, M, N, G, l.ptr, l.ld, r.ptr, r.ld, ends, mc.ptr, mc.ld,
                                     mc.stride, c.stream), "sgemmGroupedWeightGrad");
        return wrap(out);
    });
}

struct LossOperands {
    sgemmDataType_t ty;
    c10::Device dev;
    at::ScalarType st;
    Matrix x, w;
    const int64_t *target;
    LossOperands(PyObject *px, PyObject *pw, PyObject *pt) : dev(c10::kCPU) {
        const at::Tensor &tx = tensor(px, "x"), &tw = tensor(pw, "w");
        ty = type_of(tx, "x");
        dev = device_of(tx, "x");
        st = tx.scalar_type();
        x = matrix(tx, "x", st, dev);
        w = matrix(tw, "w", st, dev);
        if (x.cols != w.cols)
            fail(PyExc_ValueError, "x has %lld columns, w %lld", (long long)x.cols, (long long)w.cols);
        target = vector<int64_t>(pt, "target", at::kLong, dev, x.rows);
    }
};

// (x, w, target, handle, stream) -> (loss, lse)
PyObject *py_linear_cross_entropy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 5);
        if (recorded(tensor(a[0], "x"), tensor(a[1], "w"))) Py_RETURN_NONE;
        const LossOperands o(a[0], a[1], a[2]);
        const int64_t T = o.x.rows, V = o.w.rows, D = o.x.cols;
        Call c(a[3], a[4], o.dev, {a[0], a[1], a[2]});
        const at::Tensor loss = make({T}, at::kFloat, o.dev), lse = make({T}, at::kFloat, o.dev);
        size_t need = 0;
        check(sgemmCrossEntropyWorkspaceSize(c.handle, o.ty, T, V, D, o.x.ptr, o.x.ld, o.w.ptr, o.w.ld, &need),
              "sgemmCrossEntropyWorkspaceSize");
        c.workspace(need);
        check(sgemmCrossEntropy(c.handle, o.ty, T, V, D, o.x.ptr, o.x.ld, o.w.ptr, o.w.ld, o.target,
                                static_cast<float *>(loss.mutable_data_ptr()),
                                static_cast<float *>(lse.mutable_data_ptr()), c.stream), "sgemmCrossEntropy");
        return Py_BuildValue("NN", wrap(loss), wrap(lse));
    });
}

// (x, w, target, lse, dloss, handle, stream) -> (dx, dw)
PyObject *py_linear_cross_entropy_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 7);
        const LossOperands o(a[0], a[1], a[2]);
        const int64_t T = o.x.rows, V = o.w.rows, D = o.x.cols;
        const float *lse = vector<float>(a[3], "lse", at::kFloat, o.dev, T);
        const float *dloss = vector<float>(a[4], "dloss", at::kFloat, o.dev, T);
        Call c(a[5], a[6], o.dev, {a[0], a[1], a[2], a[3], a[4]});
        const at::Tensor dx = make({T, D}, o.st, o.dev), dw = make({V, D}, o.st, o.dev);
        size_t need = 0;
        check(sgemmCrossEntropyGradWorkspaceSize(c.handle, o.ty, T, V, D, o.x.ptr, o.x.ld, o.w.ptr, o.w.ld, &need),
              "sgemmCrossEntropyGradWorkspaceSize");
        c.workspace(need);
        check(sgemmCrossEntropyGrad(c.handle, o.ty, T, V, D, o.x.ptr, o.x.ld, o.w.ptr, o.w.ld, o.target, lse, dloss,
                                    dx.mutable_data_ptr(), std::max<int64_t>(D, 1), dw.mutable_data_ptr(),
                                    std::max<int64_t>(D, 1), c.stream), "sgemmCrossEntropyGrad");
        return Py_BuildValue("NN", wrap(dx), wrap(dw));
    });
}

// (x, q, scales, zeros, out, handle, stream)
PyObject *py_w4_gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 7);
        const at::Tensor &x = tensor(a[0], "x"), &q = tensor(a[1], "q"), &s = tensor(a[2], "scales");
        if (a[4] == Py_None && recorded(x, s)) Py_RETURN_NONE;
        const sgemmDataType_t ty = type_of(x, "x");
        const c10::Device dev = device_of(x, "x");
        const at::ScalarType st = x.scalar_type();
        const Matrix mx = matrix(x, "x", st, dev);
        const int64_t M = mx.rows, K = mx.cols;
        const Matrix mq = matrix(q, "q", at::kByte, dev, -1, K / 2);
        const int64_t N = mq.rows;
        const Matrix ms = matrix(s, "scales", st, dev, N, -1);
        const int64_t groups = ms.cols;
        if (groups == 0 ? K != 0 : K % groups != 0 || K == 0)
            fail(PyExc_ValueError, "%lld groups do not divide %lld columns", (long long)groups, (long long)K);
        const int64_t group = groups == 0 ? 32 : K / groups;
        Matrix mz;
        mz.ld = 0;
        if (a[3] != Py_None) mz = matrix(tensor(a[3], "zeros"), "zeros", at::kByte, dev, N, groups);
        if (a[4] != Py_None) matrix(tensor(a[4], "out"), "out", st, dev, M, N);   // before it is recorded
        Call c(a[5], a[6], dev, {a[0], a[1], a[2], a[3], a[4]});
        const at::Tensor out = output(a[4], {M, N}, st, dev);
        const Matrix my = matrix(out, "out", st, dev, M, N);
        const int gr = group > 1024 ? 1024 : int(group);       // beyond any that is taken
        size_t need = 0;
        check(sgemmW4WorkspaceSize(c.handle, ty, M, N, K, gr, &need), "sgemmW4WorkspaceSize");
        c.workspace(need);
        check(sgemmW4(c.handle, ty, M, N, K, gr, mx.ptr, mx.ld, static_cast<const uint8_t *>(mq.ptr), mq.ld, ms.ptr,
                      ms.ld, static_cast<const uint8_t *>(mz.ptr), mz.ld, my.ptr, my.ld, c.stream), "sgemmW4");
        return wrap(out);
    });
}

// (logits, k, normalize, handle, stream) -> (weights, experts)
PyObject *py_route_topk(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 5);
        const at::Tensor &l = tensor(a[0], "logits");
        if (recorded(l)) Py_RETURN_NONE;
        const sgemmDataType_t ty = type_of(l, "logits");
        const c10::Device dev = device_of(l, "logits");
        const Matrix ml = matrix(l, "logits", l.scalar_type(), dev);
        const int64_t k = whole(a[1], "k");
        const bool normalize = truth(a[2]);
        if (k < 1 || k > ml.cols)
            fail(PyExc_ValueError, "k is %lld, of %lld experts", (long long)k, (long long)ml.cols);
        Call c(a[3], a[4], dev, {a[0]});
        const at::Tensor weights = make({ml.rows, k}, at::kFloat, dev), experts = make({ml.rows, k}, at::kLong, dev);
        check(sgemmRouteTopK(c.handle, ty, ml.rows, ml.cols, k, normalize, ml.ptr, ml.ld,
                             static_cast<float *>(weights.mutable_data_ptr()),
                             static_cast<int64_t *>(experts.mutable_data_ptr()), c.stream), "sgemmRouteTopK");
        return Py_BuildValue("NN", wrap(weights), wrap(experts));
    });
}

// (logits, experts, dweights, normalize, handle, stream)
PyObject *py_route_topk_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 6);
        const at::Tensor &l = tensor(a[0], "logits"), &e = tensor(a[1], "experts"), &g = tensor(a[2], "dweights");
        const sgemmDataType_t ty = type_of(l, "logits");
        const c10::Device dev = device_of(l, "logits");
        const Matrix ml = matrix(l, "logits", l.scalar_type(), dev);
        const int64_t *experts = table<int64_t>(e, "experts", at::kLong, dev, ml.rows, -1);
        const int64_t k = e.size(1);
        const float *dweights = table<float>(g, "dweights", at::kFloat, dev, ml.rows, k);
        const bool normalize = truth(a[3]);
        if (k < 1 || k > ml.cols)
            fail(PyExc_ValueError, "%lld choices of %lld experts", (long long)k, (long long)ml.cols);
        Call c(a[4], a[5], dev, {a[0], a[1], a[2]});
        const at::Tensor out = make({ml.rows, ml.cols}, l.scalar_type(), dev);
        check(sgemmRouteTopKGrad(c.handle, ty, ml.rows, ml.cols, k, normalize, ml.ptr, ml.ld, experts, dweights,
                                 out.mutable_data_ptr(), ml.cols, c.stream), "sgemmRouteTopKGrad");
        return wrap(out);
    });
}

// (x, experts, num_experts, handle, stream) -> (rows, slots, group_ends)
PyObject *py_expert_dispatch(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 5);
        const at::Tensor &x = tensor(a[0], "x"), &e = tensor(a[1], "experts");
        if (recorded(x)) Py_RETURN_NONE;
        const sgemmDataType_t ty = type_of(x, "x");
        const c10::Device dev = device_of(x, "x");
        const Matrix mx = matrix(x, "x", x.scalar_type(), dev);
        const int64_t *experts = table<int64_t>(e, "experts", at::kLong, dev, mx.rows, -1);
        const int64_t k = e.size(1), G = whole(a[2], "num_experts");
        if (G < 0) fail(PyExc_ValueError, "num_experts is %lld", (long long)G);
        if (G > SGEMM_MAX_GROUPS) check(SGEMM_STATUS_NOT_SUPPORTED, "sgemmExpertDispatch");
        Call c(a[3], a[4], dev, {a[0], a[1]});
        const at::Tensor rows = make({mx.rows * k, mx.cols}, x.scalar_type(), dev);
        const at::Tensor slots = make({mx.rows, k}, at::kInt, dev), ends = make({G}, at::kInt, dev);
        check(sgemmExpertDispatch(c.handle, ty, mx.rows, mx.cols, k, G, mx.ptr, mx.ld, experts, rows.mutable_data_ptr(),
                                  std::max<int64_t>(mx.cols, 1), static_cast<int32_t *>(slots.mutable_data_ptr()),
                                  static_cast<int32_t *>(ends.mutable_data_ptr()), c.stream), "sgemmExpertDispatch");
        return Py_BuildValue("NNN", wrap(rows), wrap(slots), wrap(ends));
    });
}

// `like`: the rows, or dy in their place where they are not wanted.
struct CombineOperands {
    sgemmDataType_t ty;
    c10::Device dev;
    at::ScalarType st;
    Matrix rows;
    const int32_t *slots;
    const float *weights = nullptr;
    int64_t T, k, D;
    CombineOperands(PyObject *pr, PyObject *ps, PyObject *pw, PyObject *like) : dev(c10::kCPU) {
        const char *name = like == pr ? "rows" : "dy";
        const at::Tensor &t = tensor(like, name), &ts = tensor(ps, "slots");
        ty = type_of(t, name);
        dev = device_of(t, name);
        st = t.scalar_type();
        slots = table<int32_t>(ts, "slots", at::kInt, dev, -1, -1);
        T = ts.size(0);
        k = ts.size(1);
        rows = matrix(t, name, st, dev);
        D = rows.cols;
        if (like != pr) rows = Matrix();
        else if (rows.rows != T * k)
            fail(PyExc_ValueError, "rows has %lld rows for %lld slots", (long long)rows.rows, (long long)(T * k));
        if (pw != Py_None) weights = table<float>(tensor(pw, "weights"), "weights", at::kFloat, dev, T, k);
    }
};

// (rows, slots, weights, out, handle, stream)
PyObject *py_expert_combine(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 6);
        if (a[3] == Py_None && (recorded(tensor(a[0], "rows")) || (a[2] != Py_None && recorded(tensor(a[2], "weights")))))
            Py_RETURN_NONE;
        const CombineOperands o(a[0], a[1], a[2], a[0]);
        if (a[3] != Py_None) matrix(tensor(a[3], "out"), "out", o.st, o.dev, o.T, o.D);   // before it is recorded
        Call c(a[4], a[5], o.dev, {a[0], a[1], a[2], a[3]});
        const at::Tensor out = output(a[3], {o.T, o.D}, o.st, o.dev);
        const Matrix my = matrix(out, "out", o.st, o.dev, o.T, o.D);
        check(sgemmExpertCombine(c.handle, o.ty, o.T, o.D, o.k, o.rows.ptr, o.rows.ld, o.slots, o.weights, my.ptr,
                                 my.ld, c.stream), "sgemmExpertCombine");
        return wrap(out);
    });
}

// (dy, rows, slots, weights, need_drows, need_dweights, handle, stream) -> (drows, dweights)
PyObject *py_expert_combine_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 8);
        const at::Tensor &dy = tensor(a[0], "dy");
        const bool need_rows = truth(a[4]), need_weights = truth(a[5]);
        const CombineOperands o(a[1], a[2], a[3], a[1] != Py_None || need_weights ? a[1] : a[0]);
        const Matrix md = matrix(dy, "dy", o.st, o.dev, o.T, o.D);
        Call c(a[6], a[7], o.dev, {a[0], a[1], a[2], a[3]});
        at::Tensor drows, dweights;
        if (need_rows) drows = make({o.T * o.k, o.D}, o.st, o.dev);
        if (need_weights) dweights = make({o.T, o.k}, at::kFloat, o.dev);
        if (need_rows) c.workspace(size_t(o.T) * size_t(o.k) * sizeof(int32_t));
        check(sgemmExpertCombineGradEx(c.handle, o.ty, o.T, o.D, o.k, md.ptr, md.ld, o.rows.ptr,
                                       std::max(o.rows.ld, o.D), o.slots, o.weights,
                                       need_rows ? drows.mutable_data_ptr() : nullptr, std::max<int64_t>(o.D, 1),
                                       need_weights ? static_cast<float *>(dweights.mutable_data_ptr()) : nullptr,
                                       static_cast<int32_t *>(c.buffer.get()), c.stream), "sgemmExpertCombineGradEx");
        return Py_BuildValue("NN", need_rows ? wrap(drows) : Py_NewRef(Py_None),
                             need_weights ? wrap(dweights) : Py_NewRef(Py_None));
    });
}

// (x, handle, stream) -> (q, scales)
PyObject *py_int8_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 3);
        const at::Tensor &x = tensor(a[0], "x");
        if (recorded(x)) Py_RETURN_NONE;
        const sgemmDataType_t ty = type_of(x, "x");
        const c10::Device dev = device_of(x, "x");
        const Matrix mx = matrix(x, "x", x.scalar_type(), dev);
        Call c(a[1], a[2], dev, {a[0]});
        const at::Tensor q = make({mx.rows, mx.cols}, at::kChar, dev), scales = make({mx.rows}, at::kFloat, dev);
        check(sgemmInt8Quantize(c.handle, ty, mx.rows, mx.cols, mx.ptr, mx.ld,
                                static_cast<int8_t *>(q.mutable_data_ptr()), std::max<int64_t>(mx.cols, 1),
                                static_cast<float *>(scales.mutable_data_ptr()), c.stream), "sgemmInt8Quantize");
        return Py_BuildValue("NN", wrap(q), wrap(scales));
    });
}

// (x, w, scales, x_scales, group_ends, dtype, out, handle, stream); group_ends
// None: one matrix.
PyObject *py_int8_gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 9);
        const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &s = tensor(a[2], "scales");
        const bool integers = a[3] != Py_None, grouped = a[4] != Py_None;
        if (a[6] == Py_None &&
            (recorded(x, s) || (integers && recorded(tensor(a[3], "x_scales")))))
            Py_RETURN_NONE;
        const c10::Device dev = device_of(x, "x");
        if (integers && x.scalar_type() != at::kChar)
            fail(PyExc_TypeError, "x must be int8 where x_scales are given, got %s", type_name(x.scalar_type()));
        const sgemmDataType_t from = integers ? SGEMM_TYPE_S8 : type_of(x, "x");
        at::ScalarType st = x.scalar_type();
        if (a[5] != Py_None) {
            if (!THPDtype_Check(a[5])) fail(PyExc_TypeError, "dtype must be a torch.dtype");
            st = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
        } else if (a[6] != Py_None) {
            st = tensor(a[6], "out").scalar_type();
        } else if (integers) {
            fail(PyExc_TypeError, "dtype (or out) must be given with x of integers");
        }
        if (st != at::kFloat && st != at::kHalf && st != at::kBFloat16)
            fail(PyExc_TypeError, "the result must be float32, float16 or bfloat16, not %s", type_name(st));
        const sgemmDataType_t to = st == at::kFloat ? SGEMM_TYPE_F32 : st == at::kHalf ? SGEMM_TYPE_F16 : SGEMM_TYPE_BF16;
        const Matrix mx = matrix(x, "x", x.scalar_type(), dev);
        const int64_t T = mx.rows, K = mx.cols;
        Matrix mw;
        int64_t G = 1, N;
        if (grouped) {
            if (w.dim() != 3) fail(PyExc_ValueError, "w must be a 3-D tensor [groups, channels, columns of x]");
            G = w.size(0);
            N = w.size(1);
            mw = stack(w, "w", at::kChar, dev, G, N, K);
            check_kind(s, "scales", at::kFloat, dev);
            if (s.dim() != 2 || s.size(0) != G || s.size(1) != N || !s.is_contiguous())
                fail(PyExc_ValueError, "scales must be a contiguous matrix with a row for each group and a column for "
                                       "each of w's channels");
        } else {
            mw = matrix(w, "w", at::kChar, dev, -1, K);
            N = mw.rows;
            vector<float>(a[2], "scales", at::kFloat, dev, N);
        }
        const float *scales = static_cast<const float *>(s.const_data_ptr());
        const float *xs = integers ? vector<float>(a[3], "x_scales", at::kFloat, dev, T) : nullptr;
        const int32_t *ends = grouped ? vector<int32_t>(a[4], "group_ends", at::kInt, dev, G) : nullptr;
        if (a[6] != Py_None) matrix(tensor(a[6], "out"), "out", st, dev, T, N);   // before it is recorded
        Call c(a[7], a[8], dev, {a[0], a[1], a[2], a[3], a[4], a[6]});
        const at::Tensor out = output(a[6], {T, N}, st, dev);
        const Matrix my = matrix(out, "out", st, dev, T, N);
        size_t need = 0;
        check(sgemmInt8WorkspaceSize(c.handle, from, to, T, N, K, G, mx.ptr, mx.ld, static_cast<const int8_t *>(mw.ptr),
                                     mw.ld, mw.stride, &need), "sgemmInt8WorkspaceSize");
        c.workspace(need);
        check(sgemmInt8(c.handle, from, to, T, N, K, G, mx.ptr, mx.ld, xs, static_cast<const int8_t *>(mw.ptr), mw.ld,
                        mw.stride, scales, ends, my.ptr, my.ld, c.stream), "sgemmInt8");
        return wrap(out);
    });
}

PyMethodDef methods[] = {
    {"grouped_gemm", reinterpret_cast<PyCFunction>(py_grouped_gemm), METH_FASTCALL, nullptr},
    {"grouped_gemm_weight_grad", reinterpret_cast<PyCFunction>(py_grouped_gemm_weight_grad), METH_FASTCALL, nullptr},
    {"linear_cross_entropy", reinterpret_cast<PyCFunction>(py_linear_cross_entropy), METH_FASTCALL, nullptr},
    {"linear_cross_entropy_grad", reinterpret_cast<PyCFunction>(py_linear_cross_entropy_grad), METH_FASTCALL,
     nullptr},
    {"w4_gemm", reinterpret_cast<PyCFunction>(py_w4_gemm), METH_FASTCALL, nullptr},
    {"route_topk", reinterpret_cast<PyCFunction>(py_route_topk), METH_FASTCALL, nullptr},
    {"route_topk_grad", reinterpret_cast<PyCFunction>(py_route_topk_grad), METH_FASTCALL, nullptr},
    {"expert_dispatch", reinterpret_cast<PyCFunction>(py_expert_dispatch), METH_FASTCALL, nullptr},
    {"expert_combine", reinterpret_cast<PyCFunction>(py_expert_combine), METH_FASTCALL, nullptr},
    {"expert_combine_grad", reinterpret_cast<PyCFunction>(py_expert_combine_grad), METH_FASTCALL, nullptr},
    {"int8_quantize", reinterpret_cast<PyCFunction>(py_int8_quantize), METH_FASTCALL, nullptr},
    {"int8_gemm", reinterpret_cast<PyCFunction>(py_int8_gemm), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm_binding(void) {
    PyObject *b = PyImport_ImportModule("fp32_sgemm_gb300._binding");
    if (b == nullptr) return nullptr;
    g_check = PyObject_GetAttrString(b, "_check");
    g_stream_ptr = PyObject_GetAttrString(b, "_stream_ptr");
    Py_DECREF(b);
    PyObject *t = PyImport_ImportModule("torch");
    if (t == nullptr) return nullptr;
    g_out_of_memory = PyObject_GetAttrString(t, "OutOfMemoryError");
    Py_DECREF(t);
    g_name_ptr = PyUnicode_InternFromString("address");
    if (g_check == nullptr || g_stream_ptr == nullptr || g_out_of_memory == nullptr || g_name_ptr == nullptr)
        return nullptr;
    return PyModule_Create(&module);
}
