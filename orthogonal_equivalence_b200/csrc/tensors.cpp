// The 8-bit operators on torch tensors: checks, output allocation and the C
// call (include/poetx.h) of each function of quantized.py, in one step.  At the
// smallest sizes a call is its host side (one token through the norm is 3 us on
// the device), and the same steps in Python and ctypes take 9 to 15 us of it,
// here 4 to 7.  No arithmetic: the C functions' addresses come from the library
// that the package has loaded.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include "poetx.h"

namespace {

// ---------------------------------------------------------------- errors
struct Refused : std::runtime_error {
  PyObject* type;
  Refused(PyObject* t, const std::string& s) : std::runtime_error(s), type(t) {}
};
struct Raised : std::exception {};  // a Python exception is already set

PyObject* g_check = nullptr;  // _check(status, name): raises the package's error
PyObject* g_oom = nullptr;    // torch.OutOfMemoryError

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kChar: return "torch.int8";
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
  }
}

std::string shape_text(at::IntArrayRef s) {
  std::string o = "(";
  for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
  return o + (s.size() == 1 ? ",)" : ")");
}

// ---------------------------------------------------------------- arguments
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    throw Refused(PyExc_TypeError, std::string(name) + ": expected a torch.Tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

void need_contiguous(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous()) throw Refused(PyExc_ValueError, std::string(name) + ": must be contiguous");
}

void need_dtype(const at::Tensor& t, const char* name, at::ScalarType dtype) {
  if (t.scalar_type() != dtype)
    throw Refused(PyExc_ValueError,
                  std::string(name) + ": dtype " + dtype_name(t.scalar_type()) + ", expected " + dtype_name(dtype));
}

// A tensor of this dtype and shape on the device of the call's first one.
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType dtype, at::IntArrayRef shape, at::Device device) {
  const at::Tensor& t = tensor(o, name);
  need_dtype(t, name, dtype);
  if (t.sizes() != shape)
    throw Refused(PyExc_ValueError, std::string(name) + ": shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
  if (t.device() != device)
    throw Refused(PyExc_ValueError, std::string(name) + ": tensor on " + t.device().str() +
                                        ", the other operands are on " + device.str());
  need_contiguous(t, name);
  return t;
}

// The C calls take widths (and a weight's rows) as 32-bit numbers.
void need_int32(int64_t v, const char* name) {
  if (v > INT32_MAX) throw Refused(PyExc_ValueError, std::string(name) + ": " + std::to_string(v) + " rows or columns are too many");
}

void need_rows(const at::Tensor& t, const char* name, const char* form) {
  if (t.dim() != 2 || t.size(1) == 0)
    throw Refused(PyExc_ValueError, std::string(name) + ": shape " + shape_text(t.sizes()) + ", expected " + form);
  need_int32(t.size(1), name);
}

bool ours(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
int32_t code(at::ScalarType t) { return t == at::kBFloat16 ? POETX_BF16 : POETX_FP32; }

// [T][d] in a dtype of the library
const at::Tensor& activation(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  need_contiguous(t, name);
  if (!ours(t.scalar_type()))
    throw Refused(PyExc_ValueError, std::string(name) + ": dtype " + dtype_name(t.scalar_type()) +
                                        ", expected torch.bfloat16 or torch.float32");
  need_rows(t, name, "[T][d] with d >= 1");
  return t;
}

const at::Tensor& codes(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  need_dtype(t, name, at::kChar);
  need_contiguous(t, name);
  need_rows(t, name, "[rows][d] with d >= 1");
  return t;
}

at::ScalarType out_dtype(PyObject* o) {
  if (!THPDtype_Check(o) || !ours(reinterpret_cast<THPDtype*>(o)->scalar_type))
    throw Refused(PyExc_ValueError, "dtype: expected torch.bfloat16 or torch.float32");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

// The checkpoint's codes and exponents
const at::Tensor& checkpoint(PyObject* c, PyObject* e, const at::Tensor** exps) {
  const at::Tensor& t = codes(c, "checkpoint codes");
  *exps = &need(e, "checkpoint exps", at::kByte, {t.size(0), (t.size(1) + 31) / 32}, t.device());
  return t;
}

// ---------------------------------------------------------------- the call
// Where a call runs: the device of its tensors, made current, and its current stream.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  at::Device device;
  void* stream;
  explicit Place(at::Device d) : device(d), stream(nullptr) {
    if (!d.is_cuda())
      throw Refused(PyExc_ValueError, "tensors on " + d.str() + ": the library runs on CUDA devices");
    guard.set_device(d);
    stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::detail::empty_cuda(shape, t, device, c10::nullopt);
  }
};

void check(int status, const char* name) {
  if (status == 0) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", status, name);
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, status);
  throw Raised();
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <typename... Ts>
PyObject* wrap_all(const Ts&... t) {
  PyObject* items[] = {wrap(t)...};
  constexpr Py_ssize_t n = sizeof...(t);
  PyObject* r = PyTuple_New(n);
  bool bad = !r;
  for (Py_ssize_t i = 0; i < n; ++i) bad = bad || !items[i];
  if (bad) {
    for (PyObject* i : items) Py_XDECREF(i);
    Py_XDECREF(r);
    throw Raised();
  }
  for (Py_ssize_t i = 0; i < n; ++i) PyTuple_SET_ITEM(r, i, items[i]);
  return r;
}

// The C functions, by their names in include/poetx.h.
#define POETX_FUNCTIONS(F)                                                                                            \
  F(poetx_quantize_rows) F(poetx_weight_dequantize) F(poetx_rmsnorm_quantize) F(poetx_rmsnorm_backward)               \
  F(poetx_rmsnorm_backward_workspace_bytes) F(poetx_matmul_int8) F(poetx_matmul_int8_workspace_bytes)                 \
  F(poetx_matmul_int8_grad) F(poetx_matmul_int8_grad_workspace_bytes) F(poetx_checkpoint_save)                        \
  F(poetx_checkpoint_load) F(poetx_block_backward) F(poetx_block_backward_workspace_bytes)
struct {
#define F(name) decltype(&::name) name;
  POETX_FUNCTIONS(F)
#undef F
} c;

// bind(addresses, check, oom): the C functions' addresses by name, _check, and
// the exception for a failed allocation.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3 || !PyDict_Check(a[0])) throw Refused(PyExc_TypeError, "bind(addresses, check, oom)");
  auto address = [&](const char* name) -> void* {
    PyObject* v = PyDict_GetItemString(a[0], name);
    void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
    if (!p) throw Refused(PyExc_RuntimeError, std::string(name) + ": no address");
    return p;
  };
#define F(name) c.name = reinterpret_cast<decltype(&::name)>(address(#name));
  POETX_FUNCTIONS(F)
#undef F
  Py_INCREF(a[1]);
  Py_INCREF(a[2]);
  Py_XDECREF(g_check);
  Py_XDECREF(g_oom);
  g_check = a[1];
  g_oom = a[2];
  Py_RETURN_NONE;
}

void count(Py_ssize_t n, Py_ssize_t want, const char* name) {
  if (!g_check) throw Refused(PyExc_RuntimeError, std::string(name) + ": bind() first");
  if (n != want) throw Refused(PyExc_TypeError, std::string(name) + ": wrong number of arguments");
}

PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 2, "quantize_rows");
  const at::Tensor& x = activation(a[0], "x");
  const int64_t T = x.size(0), d = x.size(1);
  at::Tensor colscale;
  if (a[1] != Py_None) colscale = need(a[1], "colscale", at::kFloat, {d}, x.device());
  Place at(x.device());
  at::Tensor q = at.empty({T, d}, at::kChar), s = at.empty({T}, at::kFloat);
  check(c.poetx_quantize_rows(T, static_cast<int32_t>(d), ptr(x), code(x.scalar_type()),
                              static_cast<const float*>(ptr(colscale)), static_cast<int8_t*>(ptr(q)),
                              static_cast<float*>(ptr(s)), at.stream),
        "poetx_quantize_rows");
  return wrap_all(q, s);
}

PyObject* dequantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 3, "dequantize_rows");
  const at::Tensor& q = codes(a[0], "codes");
  const int64_t T = q.size(0), d = q.size(1);
  need_int32(T, "codes");
  const at::Tensor& s = need(a[1], "scale", at::kFloat, {T}, q.device());
  const at::ScalarType t = out_dtype(a[2]);
  Place at(q.device());
  at::Tensor out = at.empty({T, d}, t);
  check(c.poetx_weight_dequantize(static_cast<int32_t>(T), static_cast<int32_t>(d), static_cast<const int8_t*>(ptr(q)),
                                  static_cast<const float*>(ptr(s)), code(t), ptr(out), at.stream),
        "poetx_weight_dequantize");
  return wrap(out);
}

PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 6, "rmsnorm_quantize");
  const at::Tensor& x = activation(a[0], "x");
  const int64_t T = x.size(0), d = x.size(1);
  const at::ScalarType t = x.scalar_type();
  const at::Tensor& gamma = need(a[1], "gamma", at::kFloat, {d}, x.device());
  at::Tensor residual;
  if (a[2] != Py_None) residual = need(a[2], "residual", t, {T, d}, x.device());
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  const bool want_codes = flag(a[4]), want_y = flag(a[5]);
  Place at(x.device());
  at::Tensor h, q, s, y, rstd = at.empty({T}, at::kFloat);
  if (residual.defined()) h = at.empty({T, d}, t);
  if (want_codes) {
    q = at.empty({T, d}, at::kChar);
    s = at.empty({T}, at::kFloat);
  }
  if (want_y) y = at.empty({T, d}, t);
  check(c.poetx_rmsnorm_quantize(T, static_cast<int32_t>(d), ptr(x), ptr(residual),
                                 static_cast<const float*>(ptr(gamma)), static_cast<float>(eps), code(t), ptr(h),
                                 ptr(y), static_cast<int8_t*>(ptr(q)), static_cast<float*>(ptr(s)),
                                 static_cast<float*>(ptr(rstd)), at.stream),
        "poetx_rmsnorm_quantize");
  return wrap_all(q, s, h.defined() ? h : x, rstd, y);
}

PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 6, "rmsnorm_backward");
  const at::Tensor& dy = activation(a[0], "dy");
  const int64_t T = dy.size(0), d = dy.size(1);
  const at::ScalarType t = dy.scalar_type();
  const at::Tensor& h = need(a[1], "h", t, {T, d}, dy.device());
  const at::Tensor& gamma = need(a[2], "gamma", at::kFloat, {d}, dy.device());
  const at::Tensor& rstd = need(a[3], "rstd", at::kFloat, {T}, dy.device());
  at::Tensor dres, dgamma;
  if (a[4] != Py_None) dres = need(a[4], "dres", t, {T, d}, dy.device());
  const bool accumulate = a[5] != Py_None;
  if (accumulate) dgamma = need(a[5], "dgamma", at::kFloat, {d}, dy.device());
  Place at(dy.device());
  if (!accumulate) dgamma = at.empty({d}, at::kFloat);
  at::Tensor dx = at.empty({T, d}, t);
  const size_t nb = c.poetx_rmsnorm_backward_workspace_bytes(T, static_cast<int32_t>(d), code(t));
  at::Tensor ws = at.empty({static_cast<int64_t>(nb)}, at::kByte);
  check(c.poetx_rmsnorm_backward(T, static_cast<int32_t>(d), ptr(dy), ptr(h), static_cast<const float*>(ptr(gamma)),
                                 static_cast<const float*>(ptr(rstd)), ptr(dres), code(t), ptr(dx),
                                 static_cast<float*>(ptr(dgamma)), accumulate ? 1 : 0, ptr(ws), nb, at.stream),
        "poetx_rmsnorm_backward");
  return wrap_all(dx, dgamma);
}

PyObject* matmul_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 5, "matmul_int8");
  const at::Tensor& xq = codes(a[0], "xq");
  const int64_t T = xq.size(0), m = xq.size(1);
  const at::Tensor& first = codes(a[2], "Wq");
  const int64_t N = first.size(0);
  need_int32(N, "Wq");
  const at::Tensor& Wq = need(a[2], "Wq", at::kChar, {N, m}, xq.device());
  const at::Tensor& xs = need(a[1], "xscale", at::kFloat, {T}, xq.device());
  const at::Tensor& ws = need(a[3], "wscale", at::kFloat, {N}, xq.device());
  const at::ScalarType t = out_dtype(a[4]);
  Place at(xq.device());
  at::Tensor out = at.empty({T, N}, t), scratch;
  const int32_t n32 = static_cast<int32_t>(N), m32 = static_cast<int32_t>(m);
  const size_t nb = m % 16 ? c.poetx_matmul_int8_workspace_bytes(T, n32, m32) : 0;
  if (nb) scratch = at.empty({static_cast<int64_t>(nb)}, at::kByte);
  check(c.poetx_matmul_int8(T, n32, m32, static_cast<const int8_t*>(ptr(xq)), static_cast<const float*>(ptr(xs)),
                            static_cast<const int8_t*>(ptr(Wq)), static_cast<const float*>(ptr(ws)), code(t),
                            ptr(out), ptr(scratch), nb, at.stream),
        "poetx_matmul_int8");
  return wrap(out);
}

PyObject* matmul_int8_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 3, "matmul_int8_grad");
  const at::Tensor& dz = activation(a[0], "dz");
  const int64_t T = dz.size(0), N = dz.size(1);
  const at::Tensor& first = codes(a[1], "Wq");
  const int64_t m = first.size(1);
  const at::Tensor& Wq = need(a[1], "Wq", at::kChar, {N, m}, dz.device());
  const at::Tensor& ws = need(a[2], "wscale", at::kFloat, {N}, dz.device());
  const at::ScalarType t = dz.scalar_type();
  Place at(dz.device());
  const int32_t n32 = static_cast<int32_t>(N), m32 = static_cast<int32_t>(m);
  const size_t nb = c.poetx_matmul_int8_grad_workspace_bytes(T, n32, m32);
  at::Tensor dx = at.empty({T, m}, t), scratch = at.empty({static_cast<int64_t>(nb)}, at::kByte);
  check(c.poetx_matmul_int8_grad(T, n32, m32, ptr(dz), static_cast<const int8_t*>(ptr(Wq)),
                                 static_cast<const float*>(ptr(ws)), code(t), ptr(dx), ptr(scratch), nb, at.stream),
        "poetx_matmul_int8_grad");
  return wrap(dx);
}

PyObject* checkpoint_save(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 1, "checkpoint_save");
  const at::Tensor& x = activation(a[0], "x");
  const int64_t T = x.size(0), d = x.size(1);
  Place at(x.device());
  at::Tensor q = at.empty({T, d}, at::kChar), e = at.empty({T, (d + 31) / 32}, at::kByte);
  check(c.poetx_checkpoint_save(T, static_cast<int32_t>(d), ptr(x), code(x.scalar_type()),
                                static_cast<int8_t*>(ptr(q)), static_cast<uint8_t*>(ptr(e)), at.stream),
        "poetx_checkpoint_save");
  return wrap_all(q, e);
}

PyObject* checkpoint_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 3, "checkpoint_load");
  const at::Tensor* e;
  const at::Tensor& q = checkpoint(a[0], a[1], &e);
  const at::ScalarType t = out_dtype(a[2]);
  Place at(q.device());
  at::Tensor out = at.empty({q.size(0), q.size(1)}, t);
  check(c.poetx_checkpoint_load(q.size(0), static_cast<int32_t>(q.size(1)), static_cast<const int8_t*>(ptr(q)),
                                static_cast<const uint8_t*>(ptr(*e)), code(t), ptr(out), at.stream),
        "poetx_checkpoint_load");
  return wrap(out);
}

PyObject* block_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  count(n, 6, "block_backward");
  const at::Tensor* e;
  const at::Tensor& q = checkpoint(a[0], a[1], &e);
  const int64_t T = q.size(0), d = q.size(1);
  const at::Tensor& D = activation(a[2], "D");
  const at::ScalarType t = D.scalar_type();
  need(a[2], "D", t, {T, d}, q.device());
  const at::Tensor& G0 = tensor(a[3], "G");
  if (G0.dim() != 3 || G0.size(0) == 0 || d % G0.size(0))
    throw Refused(PyExc_ValueError, "G: shape " + shape_text(G0.sizes()) + ", expected [d/b][b][b] with d = " + std::to_string(d));
  const int64_t k = G0.size(0), b = d / k;
  const at::Tensor& G = need(a[3], "G", t, {k, b, b}, q.device());
  const bool want_o = flag(a[4]), accumulate = a[5] != Py_None;
  at::Tensor dG, O;
  if (accumulate) dG = need(a[5], "dG", at::kFloat, {k, b, b}, q.device());
  Place at(q.device());
  if (!accumulate) dG = at.empty({k, b, b}, at::kFloat);
  if (want_o) O = at.empty({T, d}, t);
  const int32_t d32 = static_cast<int32_t>(d), b32 = static_cast<int32_t>(b);
  const size_t nb = c.poetx_block_backward_workspace_bytes(T, d32, b32, code(t));
  at::Tensor ws = at.empty({static_cast<int64_t>(nb)}, at::kByte);
  check(c.poetx_block_backward(T, d32, b32, static_cast<const int8_t*>(ptr(q)), static_cast<const uint8_t*>(ptr(*e)),
                               ptr(D), ptr(G), code(t), ptr(O), static_cast<float*>(ptr(dG)), accumulate ? 1 : 0,
                               ptr(ws), nb, at.stream),
        "poetx_block_backward");
  return wrap_all(O, dG);
}

// No C++ exception leaves a function.
template <PyObject* (*Fn)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return Fn(self, a, n);
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_oom ? g_oom : PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(quantize_rows), METHOD(dequantize_rows), METHOD(rmsnorm_quantize),
                         METHOD(rmsnorm_backward), METHOD(matmul_int8), METHOD(matmul_int8_grad),
                         METHOD(checkpoint_save), METHOD(checkpoint_load), METHOD(block_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "Calls of libpoetx on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What this file was compiled against; build.py looks for it in the built file.
extern "C" __attribute__((used, visibility("default"))) const char poetx_tensors_built_for[] = POETX_BUILT_FOR;

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
