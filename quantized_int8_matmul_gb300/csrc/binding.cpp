// Native argument marshalling for the entry points whose calls are often a few
// microseconds of GPU time: checks torch tensors, allocates outputs, passes
// pointers, sizes and the stream to the C ABI (include/qmm.h) -- what the package's
// Python functions do through ctypes, without their interpreter time (a norm of
// one 4096-wide row: 17.7 us a call marshalled in Python, of which the launch is 3).
// A function returns its tensors, or the C ABI's status as an int if that is not
// QMM_OK; malformed tensors raise ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <limits>
#include <optional>
#include <string>

#include "../../include/qmm.h"

namespace {

struct Error : std::exception {   // a Python exception is set
  const char* what() const noexcept override { return "python error"; }
};
[[noreturn]] void fail(const std::string& msg) {
  PyErr_SetString(PyExc_ValueError, msg.c_str());
  throw Error();
}

using at::ScalarType;
using at::Tensor;
using Types = std::initializer_list<ScalarType>;

int qmm_type(ScalarType t) {
  return t == ScalarType::Float ? QMM_F32 : t == ScalarType::BFloat16 ? QMM_BF16 : t == ScalarType::Char ? QMM_S8
         : t == ScalarType::Byte ? QMM_U8 : QMM_S32;
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw Error();
  }
  return THPVariable_Unpack(o);
}

void check_type(const Tensor& t, Types types, const char* name) {
  if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
  for (ScalarType s : types)
    if (t.scalar_type() == s) return;
  fail(std::string(name) + ": dtype " + at::toString(t.scalar_type()) + " is not accepted");
}

// A contiguous CUDA tensor of one of the types (and, where given, of a shape).
const Tensor& need(PyObject* o, Types types, const char* name) {
  const Tensor& t = tensor(o, name);
  check_type(t, types, name);
  if (!t.is_contiguous()) fail(std::string(name) + " must be contiguous");
  return t;
}
// Operands lie on one device.
void check_device(const Tensor& t, const char* name, const Tensor& first) {
  if (t.device() != first.device())
    fail(std::string(name) + " is on " + t.device().str() + ", the first operand on " + first.device().str());
}
const Tensor& need(PyObject* o, Types types, const char* name, at::IntArrayRef shape, const Tensor& first) {
  const Tensor& t = need(o, types, name);
  if (t.sizes() != shape) fail(std::string(name) + " must be " + shape_text(shape));
  check_device(t, name, first);
  return t;
}

// A 2-D CUDA tensor whose rows are contiguous, at any row stride of its width or
// more; ld receives the stride.
const Tensor& need_rows(PyObject* o, Types types, const char* name, int64_t& ld) {
  const Tensor& t = tensor(o, name);
  check_type(t, types, name);
  if (t.dim() != 2) fail(std::string(name) + " must be 2-D");
  ld = t.size(1);
  if (t.is_contiguous()) return t;
  if (t.size(0) > 1) ld = t.stride(0);
  if ((t.size(1) > 1 && t.stride(1) != 1) || ld < t.size(1))
    fail(std::string(name) + ": rows must be contiguous and not overlap");
  return t;
}
const Tensor& need_rows(PyObject* o, Types types, const char* name, int64_t& ld, at::IntArrayRef shape,
                        const Tensor& first) {
  const Tensor& t = need_rows(o, types, name, ld);
  if (t.sizes() != shape) fail(std::string(name) + " must be " + shape_text(shape));
  check_device(t, name, first);
  return t;
}

constexpr ScalarType F32 = ScalarType::Float, BF16 = ScalarType::BFloat16, S8 = ScalarType::Char, U8 = ScalarType::Byte;
#define FLOATS {F32, BF16}

ScalarType float_type(PyObject* o) {
  if (!THPDtype_Check(o)) fail("out_dtype must be a torch dtype");
  const ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  if (t != F32 && t != BF16) fail("out_dtype must be float32 or bfloat16");
  return t;
}

// The stream of a call and what it allocates: the current stream, or one that the
// caller gives. That one is made current for the allocations, so that outputs and
// workspaces come from its own memory: a block goes to the stream that allocated it
// when it is dropped, and to its next user on that stream only behind the kernels of
// this call.
class Call {
 public:
  Call(PyObject* stream, const Tensor& first) : device_(first.device()) {
    if (stream == Py_None) return;
    PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
    if (!h) throw Error();
    given_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Error();
    has_stream_ = true;
  }
  Tensor empty(at::IntArrayRef shape, ScalarType type) const {
    return on_stream([&] { return Tensor(at::detail::empty_cuda(shape, type, device_, std::nullopt)); });
  }
  void fill(Tensor& t, double value) const {
    on_stream([&] { t.fill_(value); });
  }
  // `out` checked, or a new tensor where it is None.
  Tensor output(PyObject* out, at::IntArrayRef shape, ScalarType type, Types types, const char* name,
                const Tensor& first) const {
    return out == Py_None ? empty(shape, type) : need(out, types, name, shape, first);
  }
  // The stream, for a launch; launches go to the current device.
  void* stream() const {
    const int current = c10::cuda::current_device();
    if (current != device_.index())
      fail("the operands are on " + device_.str() + ", the current device is cuda:" + std::to_string(current));
    return has_stream_ ? given_ : c10::cuda::getCurrentCUDAStream(device_.index()).stream();
  }

 private:
  // f() with a given stream as the current one
  template <typename F>
  auto on_stream(F f) const -> decltype(f()) {
    if (!has_stream_) return f();
    const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(given_, device_.index()));
    return f();
  }

  at::Device device_;
  cudaStream_t given_ = nullptr;
  bool has_stream_ = false;
};

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Error();
  return v;
}

int block_size(PyObject* o) {
  const int64_t v = integer(o);
  if (v != 16 && v != 32) fail("block must be 16 or 32");
  return (int)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Error();
  return v != 0;
}

void* ptr(const Tensor& t) { return t.data_ptr(); }

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, a);
  PyTuple_SET_ITEM(r, 1, b);
  return r;
}

// The interpreter lock let go for a call of the C ABI (a launch waits where the
// stream's queue is full), and taken back however the scope is left.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// fn(args...) without the lock. The pointers are arguments, so all of them are taken
// while it is still held: a tensor without storage (inside a transform) raises there.
template <typename... P, typename... A>
qmm_status unlocked(qmm_status (*fn)(P...), A... args) {
  Unlocked u;
  return fn(static_cast<P>(args)...);
}

// x, weight, residual, eps, out, h_out, save_rstd, stream -> (q, scale, h, rstd)
PyObject* rms_norm_s8(PyObject* const* a) {
  int64_t ldx, ldr = 0;
  const Tensor& x = need_rows(a[0], FLOATS, "x", ldx);
  const auto shape = x.sizes();
  const int64_t M = shape[0], H = shape[1];
  const ScalarType t = x.scalar_type();
  const Tensor& w = need(a[1], FLOATS, "weight", {H}, x);
  const bool res = a[2] != Py_None;
  const double eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) throw Error();
  const bool save = truth(a[6]);
  const void *xp = ptr(x), *wp = ptr(w), *rp = res ? ptr(need_rows(a[2], {t}, "residual", ldr, shape, x)) : nullptr;
  const Call call(a[7], x);
  const Tensor q = call.output(a[4], shape, S8, {S8}, "out", x);
  Tensor h = x;
  if (res) {
    h = call.output(a[5], shape, t, {t}, "h_out", x);
  } else if (a[5] != Py_None) {
    fail("h_out without a residual: h is x");
  }
  Tensor scale = call.empty({M}, F32);
  Tensor rstd;
  if (save) rstd = call.empty({M}, F32);
  if (H == 0 && M > 0) {   // nothing is launched: rows of zeros, and the mean of no squares
    call.fill(scale, 1.0);
    if (save) call.fill(rstd, std::numeric_limits<double>::quiet_NaN());
  }
  const qmm_status st =
      unlocked(qmm_rms_norm_s8, xp, qmm_type(t), M, H, ldx, rp, ldr, wp, qmm_type(w.scalar_type()), eps,
               res ? ptr(h) : nullptr, ptr(q), ptr(scale), save ? ptr(rstd) : nullptr, call.stream());
  if (st != QMM_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(4);
  PyTuple_SET_ITEM(r, 0, wrap(q));
  PyTuple_SET_ITEM(r, 1, wrap(scale));
  if (res) {
    PyTuple_SET_ITEM(r, 2, wrap(h));
  } else {
    Py_INCREF(a[0]);
    PyTuple_SET_ITEM(r, 2, a[0]);
  }
  if (save) {
    PyTuple_SET_ITEM(r, 3, wrap(rstd));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 3, Py_None);
  }
  return r;
}

// q, scale, out, out_dtype, stream -> out
PyObject* s8_dequantize_rows(PyObject* const* a) {
  const Tensor& q = need(a[0], {S8}, "q");
  if (q.dim() != 2) fail("q must be 2-D");
  const int64_t M = q.size(0), H = q.size(1);
  const Tensor& scale = need(a[1], {F32}, "scale", {M}, q);
  const void *qp = ptr(q), *sp = ptr(scale);
  const Call call(a[4], q);
  const Tensor y = call.output(a[2], q.sizes(), float_type(a[3]), FLOATS, "out", q);
  const qmm_status st =
      unlocked(qmm_s8_dequantize_rows, qp, sp, M, H, ptr(y), qmm_type(y.scalar_type()), call.stream());
  return st != QMM_OK ? PyLong_FromLong(st) : wrap(y);
}

// dy, h, weight, rstd, dh, out, dweight, stream, workspace -> (dx, dweight)
PyObject* rms_norm_backward(PyObject* const* a) {
  int64_t ldh, lddy, lddh = 0;
  const Tensor& h = need_rows(a[1], FLOATS, "h", ldh);
  const auto shape = h.sizes();
  const int64_t M = shape[0], H = shape[1];
  const ScalarType t = h.scalar_type();
  const Tensor& dy = need_rows(a[0], {t}, "dy", lddy, shape, h);
  const Tensor& w = need(a[2], FLOATS, "weight", {H}, h);
  const Tensor& rstd = need(a[3], {F32}, "rstd", {M}, h);
  const void* dh = a[4] == Py_None ? nullptr : ptr(need_rows(a[4], {t}, "dh", lddh, shape, h));
  const void *dyp = ptr(dy), *hp = ptr(h), *wp = ptr(w), *rp = ptr(rstd);
  const Call call(a[7], h);
  const Tensor dx = call.output(a[5], shape, t, {t}, "out", h);
  const Tensor dw = call.output(a[6], {H}, F32, {F32}, "dweight", h);
  const size_t bytes = qmm_rms_norm_backward_workspace_bytes(M, H);
  Tensor ws;
  size_t have = 0;
  if (THPVariable_Check(a[8])) {
    ws = tensor(a[8], "workspace");
    if (!ws.is_cuda()) fail("workspace must be a CUDA tensor");
    if (!ws.is_contiguous()) fail("workspace must be contiguous");   // an expanded one has fewer bytes than elements
    check_device(ws, "workspace", h);
    have = ws.nbytes();
  } else if (bytes) {
    if (!PyUnicode_Check(a[8]) || PyUnicode_CompareWithASCIIString(a[8], "auto") != 0)
      fail("workspace must be 'auto' or a device tensor");
    ws = call.empty({(int64_t)bytes}, U8);
    have = bytes;
  }
  const qmm_status st =
      unlocked(qmm_rms_norm_backward, dyp, lddy, hp, ldh, dh, lddh, qmm_type(t), M, H, wp, qmm_type(w.scalar_type()),
               rp, ptr(dx), ptr(dw), ws.defined() ? ptr(ws) : nullptr, have, call.stream());
  return st != QMM_OK ? PyLong_FromLong(st) : pair(wrap(dx), wrap(dw));
}

Tensor packed(const Call& call, PyObject* out, int64_t rows, int64_t cols, int block, const char* name,
              const Tensor& first) {
  if (out == Py_None) return call.empty({(int64_t)qmm_fp4_bytes(rows, cols, block)}, U8);
  const Tensor& t = need(out, {U8}, name);
  check_device(t, name, first);
  return t;
}

// x, block, transpose, out, stream -> buffer
PyObject* fp4_quantize(PyObject* const* a) {
  int64_t ld;
  const Tensor& x = need_rows(a[0], FLOATS, "x", ld);
  const int block = block_size(a[1]);
  const int trans = truth(a[2]);
  const int64_t rows = x.size(trans ? 1 : 0), cols = x.size(trans ? 0 : 1);
  const void* xp = ptr(x);
  const Call call(a[4], x);
  const Tensor b = packed(call, a[3], rows, cols, block, "out", x);
  const qmm_status st = unlocked(qmm_fp4_quantize, xp, qmm_type(x.scalar_type()), rows, cols, ld, trans, block, ptr(b),
                                 b.nbytes(), call.stream());
  return st != QMM_OK ? PyLong_FromLong(st) : wrap(b);
}

// x, block, out, out_t, stream -> (buffer, buffer of the transpose)
PyObject* fp4_quantize_both(PyObject* const* a) {
  int64_t ld;
  const Tensor& x = need_rows(a[0], FLOATS, "x", ld);
  const int block = block_size(a[1]);
  const int64_t R = x.size(0), C = x.size(1);
  const void* xp = ptr(x);
  const Call call(a[4], x);
  const Tensor b = packed(call, a[2], R, C, block, "out", x), bt = packed(call, a[3], C, R, block, "out_t", x);
  const qmm_status st = unlocked(qmm_fp4_quantize_both, xp, qmm_type(x.scalar_type()), R, C, ld, block, ptr(b),
                                 b.nbytes(), ptr(bt), bt.nbytes(), call.stream());
  return st != QMM_OK ? PyLong_FromLong(st) : pair(wrap(b), wrap(bt));
}

// buffer, rows, cols, block, out, out_dtype, stream -> out
PyObject* fp4_dequantize(PyObject* const* a) {
  const Tensor& b = need(a[0], {U8}, "m");
  const int64_t rows = integer(a[1]), cols = integer(a[2]);
  const int block = block_size(a[3]);
  const void* bp = ptr(b);
  const Call call(a[6], b);
  const Tensor y = call.output(a[4], {rows, cols}, float_type(a[5]), FLOATS, "out", b);
  const qmm_status st =
      unlocked(qmm_fp4_dequantize, bp, b.nbytes(), rows, cols, block, ptr(y), qmm_type(y.scalar_type()), call.stream());
  return st != QMM_OK ? PyLong_FromLong(st) : wrap(y);
}

// a, M, b, N, K, block, out, out_dtype, stream -> out
PyObject* fp4_matmul(PyObject* const* a) {
  const Tensor &A = need(a[0], {U8}, "a"), &B = need(a[2], {U8}, "b");
  check_device(B, "b", A);
  const int64_t M = integer(a[1]), N = integer(a[3]), K = integer(a[4]);
  const int block = block_size(a[5]);
  const void *ap = ptr(A), *bp = ptr(B);
  const Call call(a[8], A);
  const Tensor y = call.output(a[6], {M, N}, float_type(a[7]), FLOATS, "out", A);
  const qmm_status st = unlocked(qmm_fp4_matmul, ap, A.nbytes(), M, bp, B.nbytes(), N, K, block, ptr(y),
                                 qmm_type(y.scalar_type()), call.stream());
  return st != QMM_OK ? PyLong_FromLong(st) : wrap(y);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Error&) {
    return nullptr;
  } catch (const std::exception& e) {   // an allocation that failed, for instance
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

#define ENTRY(f, n) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {ENTRY(rms_norm_s8, 8),   ENTRY(s8_dequantize_rows, 5), ENTRY(rms_norm_backward, 9),
                         ENTRY(fp4_quantize, 5),  ENTRY(fp4_quantize_both, 5),  ENTRY(fp4_dequantize, 7),
                         ENTRY(fp4_matmul, 9),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Argument marshalling of the C ABI.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
