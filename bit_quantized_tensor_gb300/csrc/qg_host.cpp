// Host side of the small calls for torch tensors: microscaled 4-bit and 8-bit products, the
// norms, and attention over the 8-bit cache.
//
// A small call takes the device 3 to 10 microseconds, and Python's part of it
// (three allocations and a dozen looks at the operands, cold after every
// launch) about as long again: layer_norm of one row took 17 us through the
// ctypes binding, 3 of them in the library.  The functions here do the usual
// call: operands that need no explanation, outputs and workspaces of their own,
// the current stream.  Anything else (an odd operand, a wrong shape, a failed
// launch) returns None, and the ctypes binding takes the call and reports what
// is wrong with it.  The work itself is the library's: these functions call its
// C entry points, whose addresses they are given once.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qgemm.h"

namespace {

struct Entry {
    decltype(&qg_workspace_size) workspace_size;
    decltype(&::fp4_tensor_scale) fp4_tensor_scale;
    decltype(&::fp4_quantize) fp4_quantize;
    decltype(&::fp4_dequantize) fp4_dequantize;
    decltype(&::fp4_gemm) fp4_gemm;
    decltype(&::fp4_linear) fp4_linear;
    decltype(&::fp4_linear_backward) fp4_linear_backward;
    decltype(&::layer_norm) layer_norm;
    decltype(&::layer_norm_fp4) layer_norm_fp4;
    decltype(&::layer_norm_backward) layer_norm_backward;
    decltype(&::s8_quantize) s8_quantize;
    decltype(&::s8_gemm) s8_gemm;
    decltype(&::s8_linear) s8_linear;
    decltype(&::qk_norm_rope) qk_norm_rope;
    decltype(&::qk_norm_rope_backward) qk_norm_rope_backward;
    decltype(&::kv8_append) kv8_append;
    decltype(&::kv8_gather) kv8_gather;
    decltype(&::kv8_attention) kv8_attention;
} lib;

// None: the call is not an ordinary one.
struct NotHere {};
inline void need(bool ok) {
    if (!ok) throw NotHere{};
}

inline const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

// A 2-D matrix on `dev` with unit column stride.
struct Matrix {
    int64_t rows, cols, ld;
    void* p;
};
inline Matrix matrix(const at::Tensor& t, c10::Device dev) {
    need(t.is_cuda() && t.dim() == 2 && t.device() == dev && t.layout() == at::kStrided);
    Matrix m{t.size(0), t.size(1), t.stride(0), t.data_ptr()};
    need(t.stride(1) == 1 && m.rows > 0 && m.cols > 0 && (m.rows == 1 || m.ld >= m.cols));
    if (m.rows == 1) m.ld = m.cols;
    return m;
}

inline int dtype_id(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kHalf || t == at::kFloat);
    return t == at::kBFloat16 ? QG_BF16 : t == at::kHalf ? QG_F16 : QG_F32;
}

inline int format(PyObject* o) {
    need(PyUnicode_Check(o));
    if (PyUnicode_CompareWithASCIIString(o, "nv") == 0) return QG_FP4_NV;
    need(PyUnicode_CompareWithASCIIString(o, "mx") == 0);
    return QG_FP4_MX;
}

// One fp32 on the device, or null for None.
inline const float* scale(PyObject* o, int fmt, c10::Device dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    need(fmt == QG_FP4_NV && t.device() == dev && t.scalar_type() == at::kFloat && t.numel() == 1);
    return static_cast<const float*>(t.data_ptr());
}

inline const void* vec(PyObject* o, int64_t n, at::ScalarType type, c10::Device dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    need(t.device() == dev && t.scalar_type() == type && t.numel() == n && t.is_contiguous());
    return t.data_ptr();
}

inline int64_t codes_ld(int64_t K) { return (K + 31) / 32 * 16; }
inline int64_t scale_cols(int fmt, int64_t K) {
    const int64_t per = fmt == QG_FP4_NV ? 64 : 128;
    return (K + per - 1) / per;
}

struct Packed {
    int64_t rows;
    uint8_t *q, *s;
};
inline Packed packed(PyObject* codes, PyObject* scales, int fmt, int64_t K, c10::Device dev) {
    const at::Tensor &q = tensor(codes), &s = tensor(scales);
    need(q.device() == dev && s.device() == dev && q.scalar_type() == at::kByte && s.scalar_type() == at::kByte);
    need(q.dim() == 2 && q.size(1) == codes_ld(K) && q.is_contiguous() && s.is_contiguous());
    const int64_t rows = q.size(0);
    need(rows > 0 && s.numel() == (rows + 127) / 128 * scale_cols(fmt, K) * 512);
    return {rows, static_cast<uint8_t*>(q.data_ptr()), static_cast<uint8_t*>(s.data_ptr())};
}

inline at::Tensor empty(at::IntArrayRef size, at::ScalarType type, c10::Device dev) {
    return at::Tensor(at::detail::empty_cuda(size, type, dev, std::nullopt));
}
inline at::Tensor workspace(int op, int64_t M, int64_t N, int64_t K, c10::Device dev, size_t* bytes) {
    *bytes = lib.workspace_size(op, M, N, K);
    return empty({static_cast<int64_t>(*bytes)}, at::kByte, dev);
}

inline void* stream(c10::Device dev) {
    need(dev.index() == c10::cuda::current_device());
    return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}

inline PyObject* give(const at::Tensor& t) { return THPVariable_Wrap(t); }
template <class... T>
PyObject* give_all(const T&... t) {
    PyObject* all = PyTuple_New(sizeof...(T));
    Py_ssize_t i = 0;
    ((PyTuple_SET_ITEM(all, i++, t.defined() ? give(t) : (Py_INCREF(Py_None), Py_None))), ...);
    return all;
}

inline void done(int code) { need(code == QG_OK); }

inline float real(PyObject* o) {
    need(PyFloat_Check(o));
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
}
inline int64_t whole(PyObject* o) {
    need(PyLong_Check(o));
    return PyLong_AsLongLong(o);
}

// gamma and beta, of x's type or fp32, alike.
struct Weights {
    const void *gamma, *beta;
    int type;
};
inline Weights weights(PyObject* gamma, PyObject* beta, int64_t D, at::ScalarType x, c10::Device dev) {
    PyObject* any = gamma != Py_None ? gamma : beta;
    if (any == Py_None) return {nullptr, nullptr, dtype_id(x)};
    const at::ScalarType t = tensor(any).scalar_type();
    need(t == x || t == at::kFloat);
    return {vec(gamma, D, t, dev), vec(beta, D, t, dev), dtype_id(t)};
}

// (X, gamma, beta, eps)
PyObject* norm(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev);
    const Weights w = weights(a[1], a[2], x.cols, X.scalar_type(), dev);
    void* s = stream(dev);
    at::Tensor Y = empty({x.rows, x.cols}, X.scalar_type(), dev);
    at::Tensor mean = empty({x.rows}, at::kFloat, dev), rstd = empty({x.rows}, at::kFloat, dev);
    done(lib.layer_norm(dtype_id(X.scalar_type()), x.rows, x.cols, x.p, x.ld, w.gamma, w.beta, w.type, real(a[3]),
                        Y.data_ptr(), x.cols, static_cast<float*>(mean.data_ptr()),
                        static_cast<float*>(rstd.data_ptr()), s));
    return give_all(Y, mean, rstd);
}

// (X, gamma, beta, eps, fmt, scale, want statistics)
PyObject* norm_fp4(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev);
    const Weights w = weights(a[1], a[2], x.cols, X.scalar_type(), dev);
    const int fmt = format(a[4]);
    const float* ts = scale(a[5], fmt, dev);
    void* s = stream(dev);
    at::Tensor q = empty({x.rows, codes_ld(x.cols)}, at::kByte, dev);
    at::Tensor b = empty({(x.rows + 127) / 128, scale_cols(fmt, x.cols), 512}, at::kByte, dev), mean, rstd;
    if (a[6] == Py_True) {
        mean = empty({x.rows}, at::kFloat, dev);
        rstd = empty({x.rows}, at::kFloat, dev);
    }
    done(lib.layer_norm_fp4(fmt, dtype_id(X.scalar_type()), x.rows, x.cols, x.p, x.ld, w.gamma, w.beta, w.type,
                            real(a[3]), ts, static_cast<uint8_t*>(q.data_ptr()), static_cast<uint8_t*>(b.data_ptr()),
                            mean.defined() ? static_cast<float*>(mean.data_ptr()) : nullptr,
                            rstd.defined() ? static_cast<float*>(rstd.data_ptr()) : nullptr, s));
    return give_all(q, b, mean, rstd);
}

// (dY, X, gamma, mean, rstd)
PyObject* norm_backward(PyObject* const* a) {
    const at::Tensor &dY = tensor(a[0]), &X = tensor(a[1]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev), dy = matrix(dY, dev);
    const at::ScalarType type = X.scalar_type();
    need(dY.scalar_type() == type && dy.rows == x.rows && dy.cols == x.cols);
    const Weights w = weights(a[2], Py_None, x.cols, type, dev);
    need(a[3] != Py_None && a[4] != Py_None);
    const void *mean = vec(a[3], x.rows, at::kFloat, dev), *rstd = vec(a[4], x.rows, at::kFloat, dev);
    void* s = stream(dev);
    at::Tensor dX = empty({x.rows, x.cols}, type, dev);
    at::Tensor dg = empty({x.cols}, at::kFloat, dev), db = empty({x.cols}, at::kFloat, dev);
    size_t bytes = 0;
    at::Tensor ws = workspace(QG_OP_LAYER_NORM_BACKWARD, 1, 1, x.cols, dev, &bytes);
    done(lib.layer_norm_backward(dtype_id(type), x.rows, x.cols, dy.p, dy.ld, x.p, x.ld, w.gamma, w.type,
                                 static_cast<const float*>(mean), static_cast<const float*>(rstd), dX.data_ptr(), x.cols,
                                 static_cast<float*>(dg.data_ptr()), static_cast<float*>(db.data_ptr()), ws.data_ptr(),
                                 bytes, s));
    return give_all(dX, dg, db);
}

// (X)
PyObject* tensor_scale(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev);
    void* s = stream(dev);
    at::Tensor out = empty({1}, at::kFloat, dev);
    size_t bytes = 0;
    at::Tensor ws = workspace(QG_OP_FP4_TENSOR_SCALE, 1, 1, 1, dev, &bytes);
    done(lib.fp4_tensor_scale(dtype_id(X.scalar_type()), x.rows, x.cols, x.p, x.ld, static_cast<float*>(out.data_ptr()),
                              ws.data_ptr(), bytes, s));
    return give(out);
}

// (X, fmt, scale)
PyObject* quantize(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev);
    const int fmt = format(a[1]);
    const float* ts = scale(a[2], fmt, dev);
    void* s = stream(dev);
    at::Tensor q = empty({x.rows, codes_ld(x.cols)}, at::kByte, dev);
    at::Tensor b = empty({(x.rows + 127) / 128, scale_cols(fmt, x.cols), 512}, at::kByte, dev);
    done(lib.fp4_quantize(fmt, dtype_id(X.scalar_type()), x.rows, x.cols, x.p, x.ld, ts,
                          static_cast<uint8_t*>(q.data_ptr()), static_cast<uint8_t*>(b.data_ptr()), s));
    return give_all(q, b);
}

// The type of an output: a torch.dtype, or None for `otherwise`.
inline at::ScalarType out_type(PyObject* o, at::ScalarType otherwise) {
    if (o == Py_None) return otherwise;
    need(THPDtype_Check(o));
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// (codes, scales, K, fmt, scale, dtype)
PyObject* dequantize(PyObject* const* a) {
    const c10::Device dev = tensor(a[0]).device();
    const int64_t K = whole(a[2]);
    const int fmt = format(a[3]);
    need(K > 0 && dev.is_cuda());
    const Packed x = packed(a[0], a[1], fmt, K, dev);
    const float* ts = scale(a[4], fmt, dev);
    const at::ScalarType type = out_type(a[5], at::kFloat);
    const int id = dtype_id(type);
    void* s = stream(dev);
    at::Tensor Y = empty({x.rows, K}, type, dev);
    done(lib.fp4_dequantize(fmt, id, x.rows, K, x.q, x.s, ts, Y.data_ptr(), K, s));
    return give(Y);
}

// (Aq, As, Bq, Bs, K, fmt, a_scale, b_scale, bias, dtype)
PyObject* gemm(PyObject* const* a) {
    const c10::Device dev = tensor(a[0]).device();
    const int64_t K = whole(a[4]);
    const int fmt = format(a[5]);
    need(K > 0 && dev.is_cuda());
    const Packed x = packed(a[0], a[1], fmt, K, dev), w = packed(a[2], a[3], fmt, K, dev);
    const float *ta = scale(a[6], fmt, dev), *tb = scale(a[7], fmt, dev);
    const at::ScalarType type = out_type(a[9], at::kBFloat16);
    const int id = dtype_id(type);
    const void* bias = vec(a[8], w.rows, type, dev);
    void* s = stream(dev);
    at::Tensor Y = empty({x.rows, w.rows}, type, dev);
    done(lib.fp4_gemm(fmt, id, x.rows, w.rows, K, x.q, x.s, ta, w.q, w.s, tb, bias, Y.data_ptr(), w.rows, s));
    return give(Y);
}

// (X, Wq, Ws, fmt, x_scale, w_scale, bias)
PyObject* linear(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev);
    const int fmt = format(a[3]);
    const Packed w = packed(a[1], a[2], fmt, x.cols, dev);
    const float *tx = scale(a[4], fmt, dev), *tw = scale(a[5], fmt, dev);
    const at::ScalarType type = X.scalar_type();
    const int id = dtype_id(type);
    const void* bias = vec(a[6], w.rows, type, dev);
    void* s = stream(dev);
    at::Tensor Y = empty({x.rows, w.rows}, type, dev), ws;
    const size_t bytes = lib.workspace_size(QG_OP_FP4_LINEAR, x.rows, w.rows, x.cols);
    if (bytes) ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
    done(lib.fp4_linear(fmt, id, x.rows, w.rows, x.cols, x.p, x.ld, tx, w.q, w.s, tw, bias, Y.data_ptr(), w.rows,
                        bytes ? ws.data_ptr() : nullptr, bytes, s));
    return give(Y);
}

// (dY, X, Wtq, Wts, fmt, dy_scale, x_scale, w_scale)
PyObject* linear_backward(PyObject* const* a) {
    const at::Tensor &dY = tensor(a[0]), &X = tensor(a[1]);
    const c10::Device dev = dY.device();
    const Matrix dy = matrix(dY, dev), x = matrix(X, dev);
    const at::ScalarType type = dY.scalar_type();
    need(X.scalar_type() == type && x.rows == dy.rows);
    const int64_t M = dy.rows, N = dy.cols, K = x.cols;
    const int fmt = format(a[4]), id = dtype_id(type);
    const Packed w = packed(a[2], a[3], fmt, N, dev);
    need(w.rows == K);
    const float *ty = scale(a[5], fmt, dev), *tx = scale(a[6], fmt, dev), *tw = scale(a[7], fmt, dev);
    void* s = stream(dev);
    at::Tensor dX = empty({M, K}, type, dev), dW = empty({N, K}, type, dev), db = empty({N}, at::kFloat, dev);
    size_t bytes = 0;
    at::Tensor ws = workspace(QG_OP_FP4_LINEAR_BACKWARD, M, N, K, dev, &bytes);
    done(lib.fp4_linear_backward(fmt, id, M, N, K, dy.p, dy.ld, ty, x.p, x.ld, tx, w.q, w.s, tw, dX.data_ptr(), K,
                                 dW.data_ptr(), K, static_cast<float*>(db.data_ptr()), ws.data_ptr(), bytes, s));
    return give_all(dX, dW, db);
}

// ------------------------------------------------------------ 8-bit integers

inline int64_t s8_ld(int64_t K) { return (K + 15) / 16 * 16; }

// An operand: codes and a scale for each row.
struct Codes {
    int64_t rows;
    int8_t* q;
    float* s;
};
inline Codes s8_operand(PyObject* codes, PyObject* scales, int64_t K, c10::Device dev) {
    const at::Tensor &q = tensor(codes), &s = tensor(scales);
    need(q.device() == dev && s.device() == dev && q.scalar_type() == at::kChar && s.scalar_type() == at::kFloat);
    need(q.dim() == 2 && q.size(0) > 0 && q.size(1) == s8_ld(K) && q.is_contiguous());
    need(s.numel() == q.size(0) && s.is_contiguous());
    return {q.size(0), static_cast<int8_t*>(q.data_ptr()), static_cast<float*>(s.data_ptr())};
}

// Workspace of M x N x K; none where the call needs none.
inline at::Tensor s8_workspace(int64_t M, int64_t N, int64_t K, c10::Device dev, size_t* bytes, void** p) {
    *bytes = lib.workspace_size(QG_OP_S8_LINEAR, M, N, K);
    at::Tensor ws;
    *p = nullptr;
    if (*bytes) {
        ws = empty({static_cast<int64_t>(*bytes)}, at::kByte, dev);
        *p = ws.data_ptr();
    }
    return ws;
}

// (X)
PyObject* s8_quantize(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev);
    const int id = dtype_id(X.scalar_type());
    void* s = stream(dev);
    at::Tensor q = empty({x.rows, s8_ld(x.cols)}, at::kChar, dev), sc = empty({x.rows}, at::kFloat, dev);
    done(lib.s8_quantize(id, x.rows, x.cols, x.p, x.ld, static_cast<int8_t*>(q.data_ptr()),
                         static_cast<float*>(sc.data_ptr()), s));
    return give_all(q, sc);
}

// (Aq, As, Bq, Bs, K, bias, dtype)
PyObject* s8_gemm(PyObject* const* a) {
    const c10::Device dev = tensor(a[0]).device();
    const int64_t K = whole(a[4]);
    need(K > 0 && dev.is_cuda());
    const Codes x = s8_operand(a[0], a[1], K, dev), w = s8_operand(a[2], a[3], K, dev);
    const at::ScalarType type = out_type(a[6], at::kBFloat16);
    const int id = dtype_id(type);
    const void* bias = vec(a[5], w.rows, type, dev);
    void *s = stream(dev), *wsp = nullptr;
    at::Tensor Y = empty({x.rows, w.rows}, type, dev);
    size_t bytes = 0;
    at::Tensor ws = s8_workspace(x.rows, w.rows, K, dev, &bytes, &wsp);
    done(lib.s8_gemm(id, x.rows, w.rows, K, x.q, x.s, w.q, w.s, bias, Y.data_ptr(), w.rows, wsp, bytes, s));
    return give(Y);
}

// (X, Wq, Ws, bias)
PyObject* s8_linear(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0]);
    const c10::Device dev = X.device();
    const Matrix x = matrix(X, dev);
    const Codes w = s8_operand(a[1], a[2], x.cols, dev);
    const at::ScalarType type = X.scalar_type();
    const int id = dtype_id(type);
    const void* bias = vec(a[3], w.rows, type, dev);
    void *s = stream(dev), *wsp = nullptr;
    at::Tensor Y = empty({x.rows, w.rows}, type, dev);
    size_t bytes = 0;
    at::Tensor ws = s8_workspace(x.rows, w.rows, x.cols, dev, &bytes, &wsp);
    done(lib.s8_linear(id, x.rows, w.rows, x.cols, x.p, x.ld, w.q, w.s, bias, Y.data_ptr(), w.rows, wsp, bytes, s));
    return give(Y);
}

// ------------------------------------------------------------ queries, keys and the cache

// tokens x heads x D on `dev`, heads one after another.
struct Heads {
    int64_t T, H, D, ld;
    void* p;
};
inline Heads heads(PyObject* o, at::ScalarType type, c10::Device dev) {
    const at::Tensor& t = tensor(o);
    need(t.is_cuda() && t.device() == dev && t.scalar_type() == type && t.dim() == 3);
    Heads h{t.size(0), t.size(1), t.size(2), t.stride(0), t.data_ptr()};
    need(h.T > 0 && h.H > 0 && h.D > 0 && t.stride(2) == 1 && t.stride(1) == h.D);
    if (h.T == 1) h.ld = h.H * h.D;
    need(h.ld >= h.H * h.D);
    return h;
}
inline bool same(const Heads& a, const Heads& b) { return a.T == b.T && a.H == b.H && a.D == b.D; }

inline const int32_t* words(PyObject* o, int64_t n, c10::Device dev) {
    return static_cast<const int32_t*>(vec(o, n, at::kInt, dev));
}

struct Table {
    const float* p;
    int64_t rows, R;
};
inline Table rope_table(PyObject* o, c10::Device dev) {
    if (o == Py_None) return {nullptr, 0, 0};
    const at::Tensor& t = tensor(o);
    need(t.device() == dev && t.scalar_type() == at::kFloat && t.dim() == 2 && t.is_contiguous());
    return {static_cast<const float*>(t.data_ptr()), t.size(0), t.size(1)};
}

inline int rope_style(PyObject* o) {
    need(PyUnicode_Check(o));
    if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return QG_ROPE_HALF;
    need(PyUnicode_CompareWithASCIIString(o, "pairs") == 0);
    return QG_ROPE_PAIRS;
}

// (Q, K, gq, gk, positions, table, eps, style)
PyObject* rope(PyObject* const* a) {
    const at::Tensor& Q = tensor(a[0]);
    const c10::Device dev = Q.device();
    const at::ScalarType type = Q.scalar_type();
    const int id = dtype_id(type);
    const Heads q = heads(a[0], type, dev), k = heads(a[1], type, dev);
    need(k.T == q.T && k.D == q.D);
    const Weights w = weights(a[2], a[3], q.D, type, dev);
    const int32_t* pos = words(a[4], q.T, dev);
    const Table t = rope_table(a[5], dev);
    const float eps = real(a[6]);
    const int style = rope_style(a[7]);
    void* s = stream(dev);
    at::Tensor Yq = empty({q.T, q.H, q.D}, type, dev), Yk = empty({k.T, k.H, k.D}, type, dev);
    at::Tensor rq = empty({q.T, q.H}, at::kFloat, dev), rk = empty({k.T, k.H}, at::kFloat, dev);
    done(lib.qk_norm_rope(id, style, q.T, q.H, k.H, q.D, t.R, q.p, q.ld, k.p, k.ld, w.gamma, w.beta, w.type, pos, t.p,
                          t.rows, eps, Yq.data_ptr(), q.H * q.D, Yk.data_ptr(), k.H * k.D,
                          static_cast<float*>(rq.data_ptr()), static_cast<float*>(rk.data_ptr()), s));
    return give_all(Yq, Yk, rq, rk);
}

// (dYq, dYk, Q, K, gq, gk, positions, table, rq, rk, style)
PyObject* rope_backward(PyObject* const* a) {
    const at::Tensor& Q = tensor(a[2]);
    const c10::Device dev = Q.device();
    const at::ScalarType type = Q.scalar_type();
    const int id = dtype_id(type);
    const Heads q = heads(a[2], type, dev), k = heads(a[3], type, dev);
    const Heads dyq = heads(a[0], type, dev), dyk = heads(a[1], type, dev);
    need(k.T == q.T && k.D == q.D && same(dyq, q) && same(dyk, k));
    const Weights w = weights(a[4], a[5], q.D, type, dev);
    const int32_t* pos = words(a[6], q.T, dev);
    const Table t = rope_table(a[7], dev);
    need(a[8] != Py_None && a[9] != Py_None);
    const void *rq = vec(a[8], q.T * q.H, at::kFloat, dev), *rk = vec(a[9], k.T * k.H, at::kFloat, dev);
    const int style = rope_style(a[10]);
    void* s = stream(dev);
    at::Tensor dQ = empty({q.T, q.H, q.D}, type, dev), dK = empty({k.T, k.H, k.D}, type, dev);
    at::Tensor dgq = empty({q.D}, at::kFloat, dev), dgk = empty({q.D}, at::kFloat, dev);
    size_t bytes = 0;
    at::Tensor ws = workspace(QG_OP_QK_NORM_ROPE_BACKWARD, 1, 1, q.D, dev, &bytes);
    done(lib.qk_norm_rope_backward(id, style, q.T, q.H, k.H, q.D, t.R, dyq.p, dyq.ld, dyk.p, dyk.ld, q.p, q.ld, k.p,
                                   k.ld, w.gamma, w.beta, w.type, pos, t.p, t.rows, static_cast<const float*>(rq),
                                   static_cast<const float*>(rk), dQ.data_ptr(), q.H * q.D, dK.data_ptr(), k.H * k.D,
                                   static_cast<float*>(dgq.data_ptr()), static_cast<float*>(dgk.data_ptr()),
                                   ws.data_ptr(), bytes, s));
    return give_all(dQ, dK, dgq, dgk);
}

// A cache (a tuple of four tensors) and its batch.
struct Cache {
    int64_t B, pages, heads, page, D, cols;
    int8_t *kq, *vq;
    float *ks, *vs;
    const int32_t *table, *starts, *lengths;
};
inline Cache cache(PyObject* o, PyObject* table, PyObject* starts, PyObject* lengths, c10::Device dev) {
    need(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4);
    const at::Tensor &kq = tensor(PyTuple_GET_ITEM(o, 0)), &vq = tensor(PyTuple_GET_ITEM(o, 1));
    const at::Tensor& t = tensor(table);
    need(kq.is_cuda() && kq.device() == dev && kq.scalar_type() == at::kChar && kq.dim() == 4 && kq.is_contiguous());
    need(vq.device() == dev && vq.scalar_type() == at::kChar && vq.sizes() == kq.sizes() && vq.is_contiguous());
    need(t.device() == dev && t.scalar_type() == at::kInt && t.dim() == 2 && t.is_contiguous() && t.size(0) > 0);
    Cache c;
    c.pages = kq.size(0), c.heads = kq.size(1), c.page = kq.size(2), c.D = kq.size(3);
    c.B = t.size(0), c.cols = t.size(1);
    need(c.heads > 0);
    auto scales = [&](PyObject* s) {
        const at::Tensor& v = tensor(s);
        need(v.device() == dev && v.scalar_type() == at::kFloat && v.dim() == 2 && v.size(0) == c.pages &&
             v.size(1) == c.heads && v.is_contiguous());
        return static_cast<float*>(v.data_ptr());
    };
    c.kq = static_cast<int8_t*>(kq.data_ptr()), c.vq = static_cast<int8_t*>(vq.data_ptr());
    c.ks = scales(PyTuple_GET_ITEM(o, 2)), c.vs = scales(PyTuple_GET_ITEM(o, 3));
    c.table = static_cast<const int32_t*>(t.data_ptr());
    need(starts != Py_None && lengths != Py_None && tensor(starts).dim() == 1 && tensor(lengths).dim() == 1);
    c.starts = words(starts, c.B + 1, dev), c.lengths = words(lengths, c.B, dev);
    return c;
}

// (K, V, cache, table, starts, lengths)
PyObject* append(PyObject* const* a) {
    const at::Tensor& K = tensor(a[0]);
    const c10::Device dev = K.device();
    const at::ScalarType type = K.scalar_type();
    const int id = dtype_id(type);
    const Heads k = heads(a[0], type, dev), v = heads(a[1], type, dev);
    const Cache c = cache(a[2], a[3], a[4], a[5], dev);
    need(same(k, v) && k.H == c.heads && k.D == c.D);
    done(lib.kv8_append(id, c.B, k.T, c.heads, c.D, k.p, k.ld, v.p, v.ld, c.kq, c.vq, c.ks, c.vs, c.pages, c.page,
                        c.table, c.cols, c.starts, c.lengths, stream(dev)));
    Py_RETURN_TRUE;
}

// (cache, table, starts, lengths, rows, dtype)
PyObject* gather(PyObject* const* a) {
    const c10::Device dev = tensor(a[1]).device();
    const Cache c = cache(a[0], a[1], a[2], a[3], dev);
    const int64_t rows = whole(a[4]);
    const at::ScalarType type = out_type(a[5], at::kBFloat16);
    const int id = dtype_id(type);
    need(rows > 0);
    void* s = stream(dev);
    at::Tensor K = empty({rows, c.heads, c.D}, type, dev), V = empty({rows, c.heads, c.D}, type, dev);
    done(lib.kv8_gather(id, c.B, rows, c.heads, c.D, c.kq, c.vq, c.ks, c.vs, c.pages, c.page, c.table, c.cols, c.starts,
                        c.lengths, K.data_ptr(), c.heads * c.D, V.data_ptr(), c.heads * c.D, s));
    return give_all(K, V);
}

// (Q, cache, table, starts, lengths, scale, causal)
PyObject* attention(PyObject* const* a) {
    const at::Tensor& Q = tensor(a[0]);
    const c10::Device dev = Q.device();
    const at::ScalarType type = Q.scalar_type();
    need(type == at::kHalf || type == at::kBFloat16);
    const Heads q = heads(a[0], type, dev);
    const Cache c = cache(a[1], a[2], a[3], a[4], dev);
    need(q.D == c.D && q.H % c.heads == 0 && PyBool_Check(a[6]));
    const float scale = real(a[5]);
    void* s = stream(dev);
    at::Tensor O = empty({q.T, q.H, q.D}, type, dev);
    size_t bytes = 0;
    at::Tensor ws = workspace(QG_OP_KV8_ATTENTION, q.T, q.H, q.D, dev, &bytes);
    done(lib.kv8_attention(dtype_id(type), c.B, q.T, q.H, c.heads, c.D, q.p, q.ld, c.kq, c.vq, c.ks, c.vs, c.pages,
                           c.page, c.table, c.cols, c.starts, c.lengths, scale, a[6] == Py_True, O.data_ptr(),
                           q.H * q.D, ws.data_ptr(), bytes, s));
    return give(O);
}

// Every function: exactly ARGS positional arguments; None where it is not an
// ordinary call (an exception of torch's, out of memory above all, is raised).
template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        if (n == ARGS) return F(args);
    } catch (const NotHere&) {
    } catch (const std::exception&) {
        // the ctypes binding meets the same condition and reports it
    }
    if (PyErr_Occurred()) PyErr_Clear();
    Py_RETURN_NONE;
}

// (addresses of the entry points, in the order of Entry)
PyObject* bind(PyObject*, PyObject* list) {
    void** to = reinterpret_cast<void**>(&lib);
    constexpr Py_ssize_t N = sizeof(Entry) / sizeof(void*);
    if (!PyList_Check(list) || PyList_GET_SIZE(list) != N) {
        PyErr_Format(PyExc_ValueError, "%zd addresses are needed", N);
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < N; ++i) {
        to[i] = PyLong_AsVoidPtr(PyList_GET_ITEM(list, i));
        if (PyErr_Occurred()) return nullptr;
    }
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, ARGS>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         method<norm, 4>("layer_norm"),
                         method<norm_fp4, 7>("layer_norm_fp4"),
                         method<norm_backward, 5>("layer_norm_backward"),
                         method<tensor_scale, 1>("fp4_tensor_scale"),
                         method<quantize, 3>("fp4_quantize"),
                         method<dequantize, 6>("fp4_dequantize"),
                         method<gemm, 10>("fp4_gemm"),
                         method<linear, 7>("fp4_linear"),
                         method<linear_backward, 8>("fp4_linear_backward"),
                         method<s8_quantize, 1>("s8_quantize"),
                         method<s8_gemm, 7>("s8_gemm"),
                         method<s8_linear, 4>("s8_linear"),
                         method<rope, 8>("qk_norm_rope"),
                         method<rope_backward, 11>("qk_norm_rope_backward"),
                         method<append, 6>("kv8_append"),
                         method<gather, 6>("kv8_gather"),
                         method<attention, 7>("kv8_attention"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qg_host", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__qg_host(void) { return PyModule_Create(&module); }
