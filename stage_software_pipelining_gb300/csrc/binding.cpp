// binding.cpp -- Python's way into libgemm.so's quantised operators
// (include/quant.h) and training operators (include/linear.h): the checks of
// tensor arguments and their marshalling into (pointer, leading dimension) pairs,
// in C++ because at a token a call they are most of a call's time (measured on a Grace host: 14 us of a 20 us
// gemm_fp8 call when written in Python over ctypes).
//
// Every function takes its arguments by position (quant.py and linear.py hold
// the signatures), raises ValueError for a tensor it cannot take, and returns the
// entry point's gemm_status_t.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <stdexcept>
#include <string>

#include "../../include/linear.h"
#include "../../include/quant.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

std::string text(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// The tensor behind a Python argument; null for None where that is allowed.
const Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

const Tensor& matrix(PyObject* o, const char* name) {
    const Tensor& t = *tensor(o, name);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    if (t.dim() != 2) refuse(std::string(name) + " must be 2-D");
    return t;
}

int type_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return QUANT_F32;
        case at::kHalf: return QUANT_F16;
        case at::kBFloat16: return QUANT_BF16;
        default: return -1;
    }
}

int type_of(const Tensor& t, const char* name) {
    const int c = type_code(t.scalar_type());
    if (c < 0) refuse(std::string(name) + " must be fp32, fp16 or bf16");
    return c;
}

int type16_of(const Tensor& t, const char* name) {
    const int c = type_code(t.scalar_type());
    if (c != QUANT_F16 && c != QUANT_BF16) refuse(std::string(name) + " must be fp16 or bf16");
    return c;
}

struct Rows {
    void* p = nullptr;
    int64_t ld = 0;
};

// A rows x cols matrix of `type` whose elements along dimension `inner` are
// adjacent: its address and the distance between its rows.
Rows rows_of(const Tensor& t, const char* name, at::ScalarType type, int64_t rows, int64_t cols, const Tensor& like,
             int inner = 1) {
    if (t.scalar_type() != type)
        refuse(std::string(name) + " must have type " + c10::toString(type) + ", not " +
               c10::toString(t.scalar_type()));
    if (t.device() != like.device()) refuse(std::string(name) + " must be on " + like.device().str());
    if (t.dim() != 2 || t.size(1 - inner) != rows || t.size(inner) != cols)
        refuse(std::string(name) + " must be " + (inner ? text({rows, cols}) : text({cols, rows})) + ", not " +
               text(t.sizes()));
    if (cols > 1 && rows > 0 && t.stride(inner) != 1)
        refuse(std::string(name) + (inner ? " must be row-major (unit column stride)"
                                          : " must be column-major (a transposed view of its rows)"));
    const int64_t ld = t.stride(1 - inner);
    if (rows > 1 && ld < cols) refuse(std::string(name) + "'s rows overlap");
    return {t.data_ptr(), ld};
}

Rows rows_or_none(PyObject* o, const char* name, at::ScalarType type, int64_t rows, int64_t cols,
                  const Tensor& like) {
    const Tensor* t = tensor(o, name, true);
    return t ? rows_of(*t, name, type, rows, cols, like) : Rows{};
}

void* vector_of(const Tensor& t, const char* name, at::ScalarType type, int64_t n, const Tensor& like) {
    if (t.scalar_type() != type)
        refuse(std::string(name) + " must have type " + c10::toString(type) + ", not " +
               c10::toString(t.scalar_type()));
    if (t.device() != like.device()) refuse(std::string(name) + " must be on " + like.device().str());
    if (t.dim() != 1 || t.size(0) != n)
        refuse(std::string(name) + " must have " + std::to_string(n) + " elements, not " + text(t.sizes()));
    if (n > 1 && t.stride(0) != 1) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

// The stream of a call: the given torch.cuda.Stream, or the device's current one.
void* stream_of(PyObject* o, const Tensor& like) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(like.device().index()).stream();
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) {
        PyErr_Clear();
        refuse("stream must be a torch.cuda.Stream");
    }
    void* s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("stream must be a torch.cuda.Stream");
    }
    return s;
}

bool truth_of(PyObject* o, const char* name) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) {
        PyErr_Clear();
        refuse(std::string(name) + " must be true or false");
    }
    return t != 0;
}

int group_of(int64_t K, int64_t groups) {
    const int64_t g = groups > 0 ? K / groups : 32;
    if (groups * g != K || (g != 32 && g != 64 && g != 128))
        refuse("K = " + std::to_string(K) + " and " + std::to_string(groups) +
               " scales a row: the group must be 32, 64 or 128");
    return static_cast<int>(g);
}

// x, weight, residual, eps, residual_out, y, q, scale, stream
int add_rmsnorm_(PyObject* const* a) {
    const Tensor& x = matrix(a[0], "x");
    const int code = type_of(x, "x");
    const at::ScalarType dt = x.scalar_type();
    const int64_t rows = x.size(0), cols = x.size(1);
    const Rows X = rows_of(x, "x", dt, rows, cols, x);
    const void* w = vector_of(*tensor(a[1], "weight"), "weight", dt, cols, x);
    const Rows R = rows_or_none(a[2], "residual", dt, rows, cols, x);
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("eps must be a number");
    }
    const Rows RO = rows_or_none(a[4], "residual_out", dt, rows, cols, x);
    const Rows Y = rows_or_none(a[5], "y", dt, rows, cols, x);
    if ((a[6] == Py_None) != (a[7] == Py_None)) refuse("q and scale go together");
    if (a[4] == Py_None && a[5] == Py_None && a[6] == Py_None)
        refuse("add_rmsnorm needs an output: residual_out, y, or q with scale");
    const Rows Q = rows_or_none(a[6], "q", at::kFloat8_e4m3fn, rows, cols, x);
    const Tensor* scale = tensor(a[7], "scale", true);
    void* s = scale ? vector_of(*scale, "scale", at::kFloat, rows, x) : nullptr;
    if (rows == 0) return GEMM_OK;
    void* stream = stream_of(a[8], x);
    const c10::cuda::CUDAGuard guard(x.device());
    return add_rmsnorm(rows, cols, X.p, X.ld, R.p, R.ld, w, static_cast<float>(eps), code, RO.p, RO.ld, Y.p, Y.ld,
                       Q.p, Q.ld, static_cast<float*>(s), stream);
}

// x, q, scale, stream
int quantize_fp8_(PyObject* const* a) {
    const Tensor& x = matrix(a[0], "x");
    const int code = type_of(x, "x");
    const int64_t rows = x.size(0), cols = x.size(1);
    const Rows X = rows_of(x, "x", x.scalar_type(), rows, cols, x);
    const Rows Q = rows_of(*tensor(a[1], "q"), "q", at::kFloat8_e4m3fn, rows, cols, x);
    void* s = vector_of(*tensor(a[2], "scale"), "scale", at::kFloat, rows, x);
    if (rows == 0) return GEMM_OK;
    void* stream = stream_of(a[3], x);
    const c10::cuda::CUDAGuard guard(x.device());
    return quantize_fp8(rows, cols, X.p, X.ld, code, Q.p, Q.ld, static_cast<float*>(s), stream);
}

// A, B, C, a_scale, b_scale, stream, checked
int gemm_fp8_(PyObject* const* a) {
    const Tensor& A = matrix(a[0], "A");
    const Tensor& B = matrix(a[1], "B");
    const Tensor& C = matrix(a[2], "C");
    const int64_t M = A.size(0), K = A.size(1), N = B.size(1);
    const int code = type16_of(C, "C");
    const Rows RA = rows_of(A, "A", at::kFloat8_e4m3fn, M, K, A);
    const Rows RB = rows_of(B, "B", at::kFloat8_e4m3fn, N, K, A, 0);
    const Rows RC = rows_of(C, "C", C.scalar_type(), M, N, A);
    const float* sa = static_cast<const float*>(vector_of(*tensor(a[3], "a_scale"), "a_scale", at::kFloat, M, A));
    const float* sb = static_cast<const float*>(vector_of(*tensor(a[4], "b_scale"), "b_scale", at::kFloat, N, A));
    void* stream = stream_of(a[5], A);
    const bool checked = truth_of(a[6], "checked");
    const c10::cuda::CUDAGuard guard(A.device());
    if (checked) {
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = gemm_fp8_checked(M, N, K, RA.p, RA.ld, RB.p, RB.ld, RC.p, RC.ld, sa, sb, code, stream);
        Py_END_ALLOW_THREADS
        return st;
    }
    return gemm_fp8(M, N, K, RA.p, RA.ld, RB.p, RB.ld, RC.p, RC.ld, sa, sb, code, stream);
}

// x, W, scales, C, zeros, stream, checked
int gemv_w4_(PyObject* const* a) {
    const Tensor& x = matrix(a[0], "x");
    const Tensor& W = matrix(a[1], "W");
    const Tensor& scales = matrix(a[2], "scales");
    const int64_t M = x.size(0), K = x.size(1), N = W.size(0), groups = scales.size(1);
    const int code = type16_of(x, "x");
    const at::ScalarType dt = x.scalar_type();
    const int group = group_of(K, groups);
    const Rows X = rows_of(x, "x", dt, M, K, x);
    const Rows RW = rows_of(W, "W", at::kByte, N, K / 2, x);
    const Rows S = rows_of(scales, "scales", dt, N, groups, x);
    const Rows C = rows_of(*tensor(a[3], "C"), "C", dt, M, N, x);
    const Rows Z = rows_or_none(a[4], "zeros", at::kByte, N, groups, x);
    void* stream = stream_of(a[5], x);
    const bool checked = truth_of(a[6], "checked");
    const c10::cuda::CUDAGuard guard(x.device());
    if (checked) {
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = gemv_w4_checked(M, N, K, X.p, X.ld, RW.p, RW.ld, S.p, S.ld, Z.p, Z.ld, group, C.p, C.ld, code, stream);
        Py_END_ALLOW_THREADS
        return st;
    }
    return gemv_w4(M, N, K, X.p, X.ld, RW.p, RW.ld, S.p, S.ld, Z.p, Z.ld, group, C.p, C.ld, code, stream);
}

// w, W, scales, zeros, stream
int quantize_w4_(PyObject* const* a) {
    const Tensor& w = matrix(a[0], "w");
    const int code = type_of(w, "w");
    const Tensor& scales = matrix(a[2], "scales");
    const int64_t N = w.size(0), K = w.size(1), groups = scales.size(1);
    const int scode = type16_of(scales, "scales");
    const int group = group_of(K, groups);
    const Rows IN = rows_of(w, "w", w.scalar_type(), N, K, w);
    const Rows RW = rows_of(*tensor(a[1], "W"), "W", at::kByte, N, K / 2, w);
    const Rows S = rows_of(scales, "scales", scales.scalar_type(), N, groups, w);
    const Rows Z = rows_or_none(a[3], "zeros", at::kByte, N, groups, w);
    void* stream = stream_of(a[4], w);
    const c10::cuda::CUDAGuard guard(w.device());
    return quantize_w4(N, K, IN.p, IN.ld, code, group, RW.p, RW.ld, S.p, S.ld, scode, Z.p, Z.ld, stream);
}

// ---------------------------------------------------------------- include/linear.h
int act_of(PyObject* o) {
    const long a = PyLong_AsLong(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("act must be an activation's number");
    }
    return static_cast<int>(a);
}

void* vector_or_none(PyObject* o, const char* name, at::ScalarType type, int64_t n, const Tensor& like) {
    const Tensor* t = tensor(o, name, true);
    return t ? vector_of(*t, name, type, n, like) : nullptr;
}

float number_of(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be a number");
    }
    return static_cast<float>(v);
}

// One of a product's two entry points; the second waits for the stream.
template <class F, class G>
int call(bool checked, F plain, G waiting) {
    if (!checked) return plain();
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = waiting();
    Py_END_ALLOW_THREADS
    return st;
}

// x, W, y, bias, residual, act, pre, stream, checked
int linear_(PyObject* const* a) {
    const Tensor& x = matrix(a[0], "x");
    const Tensor& W = matrix(a[1], "W");
    const int code = type16_of(x, "x");
    const at::ScalarType dt = x.scalar_type();
    const int64_t M = x.size(0), K = x.size(1), N = W.size(0);
    const Rows X = rows_of(x, "x", dt, M, K, x);
    const Rows RW = rows_of(W, "W", dt, N, K, x);
    const Rows Y = rows_of(*tensor(a[2], "y"), "y", dt, M, N, x);
    const void* bias = vector_or_none(a[3], "bias", dt, N, x);
    const Rows R = rows_or_none(a[4], "residual", dt, M, N, x);
    const int act = act_of(a[5]);
    const Rows P = rows_or_none(a[6], "pre", dt, M, N, x);
    void* s = stream_of(a[7], x);
    const bool checked = truth_of(a[8], "checked");
    const c10::cuda::CUDAGuard guard(x.device());
    auto with = [&](auto f) {
        return f(M, N, K, X.p, X.ld, RW.p, RW.ld, bias, R.p, R.ld, act, P.p, P.ld, Y.p, Y.ld, code, s);
    };
    return call(checked, [&] { return with(linear); }, [&] { return with(linear_checked); });
}

// dy, dz, pre, act, dbias, addend, stream
int act_grad_(PyObject* const* a) {
    const Tensor& dy = matrix(a[0], "dy");
    const int code = type16_of(dy, "dy");
    const at::ScalarType dt = dy.scalar_type();
    const int64_t M = dy.size(0), N = dy.size(1);
    const Rows DY = rows_of(dy, "dy", dt, M, N, dy);
    const Rows DZ = rows_or_none(a[1], "dz", dt, M, N, dy);
    const Rows P = rows_or_none(a[2], "pre", dt, M, N, dy);
    const int act = act_of(a[3]);
    if (act != LINEAR_ACT_NONE && a[2] == Py_None) refuse("pre is needed for an activation's derivative");
    float* db = static_cast<float*>(vector_or_none(a[4], "dbias", at::kFloat, N, dy));
    const float* c = static_cast<const float*>(vector_or_none(a[5], "addend", at::kFloat, N, dy));
    if (a[1] == Py_None && a[4] == Py_None) refuse("act_grad needs an output: dz or dbias");
    if (a[4] == Py_None && a[5] != Py_None) refuse("addend is added to dbias, which is not given");
    void* s = stream_of(a[6], dy);
    const c10::cuda::CUDAGuard guard(dy.device());
    return act_grad(M, N, DY.p, DY.ld, P.p, P.ld, act, DZ.p, DZ.ld, db, c, code, s);
}

// dz, W, dx, residual, act, pre, stream, checked
int linear_dx_(PyObject* const* a) {
    const Tensor& dz = matrix(a[0], "dz");
    const Tensor& W = matrix(a[1], "W");
    const int code = type16_of(dz, "dz");
    const at::ScalarType dt = dz.scalar_type();
    const int64_t M = dz.size(0), N = dz.size(1), K = W.size(1);
    const Rows DZ = rows_of(dz, "dz", dt, M, N, dz);
    const Rows RW = rows_of(W, "W", dt, N, K, dz);
    const Rows DX = rows_of(*tensor(a[2], "dx"), "dx", dt, M, K, dz);
    const Rows R = rows_or_none(a[3], "residual", dt, M, K, dz);
    const int act = act_of(a[4]);
    const Rows P = rows_or_none(a[5], "pre", dt, M, K, dz);
    if ((act == LINEAR_ACT_NONE) != (a[5] == Py_None)) refuse("pre and an activation go together");
    void* s = stream_of(a[6], dz);
    const bool checked = truth_of(a[7], "checked");
    const c10::cuda::CUDAGuard guard(dz.device());
    auto with = [&](auto f) {
        return f(M, N, K, DZ.p, DZ.ld, RW.p, RW.ld, R.p, R.ld, act, P.p, P.ld, DX.p, DX.ld, code, s);
    };
    return call(checked, [&] { return with(linear_dx); }, [&] { return with(linear_dx_checked); });
}

// dz, x, dw, addend, stream, checked
int linear_dw_(PyObject* const* a) {
    const Tensor& dz = matrix(a[0], "dz");
    const Tensor& x = matrix(a[1], "x");
    const Tensor& dw = matrix(a[2], "dw");
    const int code = type16_of(dz, "dz"), out = type_of(dw, "dw");
    const at::ScalarType dt = dz.scalar_type(), to = dw.scalar_type();
    if (out != QUANT_F32 && to != dt) refuse("dw must be fp32 or of dz's type");
    const int64_t M = dz.size(0), N = dz.size(1), K = x.size(1);
    const Rows DZ = rows_of(dz, "dz", dt, M, N, dz);
    const Rows X = rows_of(x, "x", dt, M, K, dz);
    const Rows DW = rows_of(dw, "dw", to, N, K, dz);
    const Rows C = rows_or_none(a[3], "addend", to, N, K, dz);
    void* s = stream_of(a[4], dz);
    const bool checked = truth_of(a[5], "checked");
    const c10::cuda::CUDAGuard guard(dz.device());
    auto with = [&](auto f) {
        return f(M, N, K, DZ.p, DZ.ld, X.p, X.ld, C.p, C.ld, DW.p, DW.ld, code, out, s);
    };
    return call(checked, [&] { return with(linear_dw); }, [&] { return with(linear_dw_checked); });
}

// A matrix, or a batch of matrices in a 3-D tensor, whose rows are contiguous.
struct Batch {
    void* p = nullptr;
    int64_t batch = 1, rows = 0, cols = 0, ld = 0, stride = 0;
};
Batch batch_of(const Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    const int d = static_cast<int>(t.dim());
    if (d != 2 && d != 3) refuse(std::string(name) + " must be 2-D or 3-D");
    Batch b;
    b.batch = d == 3 ? t.size(0) : 1;
    b.rows = t.size(d - 2);
    b.cols = t.size(d - 1);
    b.ld = t.stride(d - 2);
    b.stride = d == 3 ? t.stride(0) : 0;
    if (b.cols > 1 && t.numel() > 0 && t.stride(d - 1) != 1) refuse(std::string(name) + " must be row-major (unit column stride)");
    if (b.rows > 1 && b.ld < b.cols) refuse(std::string(name) + "'s rows overlap");
    const int64_t span = b.rows > 0 ? (b.rows - 1) * (b.rows > 1 ? b.ld : 0) + b.cols : 0;
    if (b.batch > 1 && b.stride < span) refuse(std::string(name) + "'s matrices overlap");
    b.p = t.data_ptr();
    return b;
}

// g, out, workspace, steps, a, b, c, eps, scale, stream, checked
int orthogonalize_(PyObject* const* a) {
    const Tensor& g = *tensor(a[0], "g");
    const Tensor& out = *tensor(a[1], "out");
    const Tensor& ws = *tensor(a[2], "workspace");
    const Batch G = batch_of(g, "g"), O = batch_of(out, "out");
    const int code = type_of(g, "g"), to = type16_of(out, "out");
    if (out.device() != g.device()) refuse("out must be on " + g.device().str());
    if (out.sizes() != g.sizes()) refuse("out must be " + text(g.sizes()) + ", not " + text(out.sizes()));
    const long steps = PyLong_AsLong(a[3]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("steps must be a whole number");
    }
    if (steps < 0 || steps > 100) refuse("steps must be 0 to 100");
    const float abc[3] = {number_of(a[4], "a coefficient"), number_of(a[5], "a coefficient"),
                          number_of(a[6], "a coefficient")};
    const float eps = number_of(a[7], "eps"), scale = number_of(a[8], "scale");
    if (ws.device() != g.device()) refuse("workspace must be on " + g.device().str());
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
    void* s = stream_of(a[9], g);
    const bool checked = truth_of(a[10], "checked");
    const c10::cuda::CUDAGuard guard(g.device());
    const size_t bytes = static_cast<size_t>(ws.numel()) * ws.element_size();
    auto with = [&](auto f) {
        return f(G.batch, G.rows, G.cols, G.p, G.ld, G.stride, code, O.p, O.ld, O.stride, to, static_cast<int>(steps),
                 abc, eps, scale, ws.data_ptr(), bytes, s);
    };
    return call(checked, [&] { return with(orthogonalize); }, [&] { return with(orthogonalize_checked); });
}

template <int (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define ENTRY(name, args) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<name##_, args>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(add_rmsnorm, 9), ENTRY(quantize_fp8, 4), ENTRY(gemm_fp8, 7), ENTRY(gemv_w4, 7),
                         ENTRY(quantize_w4, 5), ENTRY(linear, 9), ENTRY(act_grad, 7), ENTRY(linear_dx, 8),
                         ENTRY(linear_dw, 6), ENTRY(orthogonalize, 11), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quant", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__quant() { return PyModule_Create(&module); }
