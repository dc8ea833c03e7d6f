// Python calls of the microscaled operators, compiled: argument checks, output
// allocation and the library call without the interpreter between them.  Beside
// kernels of a few microseconds the same steps in Python took most of a call
// (norm with its four outputs 17 to 20 us, now 7).
//
// binding.py declares the functions with their keywords and documentation and
// passes the arguments on by position.  Checks raise TypeError or ValueError;
// a refusal by the library raises the binding's MoeqError.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "moeq.h"

namespace {

PyObject* g_error_class = nullptr;  // binding.MoeqError

// Thrown once the Python error is set.
struct Raised {};

template <typename... Args>
[[noreturn]] void raise(PyObject* type, const char* fmt, Args... args) {
  PyErr_Format(type, fmt, args...);
  throw Raised();
}

void check(int status) {
  if (status == MQ_OK) return;
  PyObject* e = PyObject_CallFunction(g_error_class, "is", status, mq_last_error_message());
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  }
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

void on_cuda(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be on a CUDA device", name);
}

long as_long(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

int bits_of(PyObject* o) {
  const long v = as_long(o);
  if (v != 4 && v != 8) raise(PyExc_ValueError, "bits must be 4 or 8, got %ld", v);
  return (int)v;
}

// MQ_DTYPE_* of a plain tensor; -1 for another type.
int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? MQ_DTYPE_BF16
         : t == at::kHalf   ? MQ_DTYPE_F16
         : t == at::kFloat  ? MQ_DTYPE_F32
                            : -1;
}

at::ScalarType scalar_type(long code) {
  return code == MQ_DTYPE_BF16 ? at::kBFloat16 : code == MQ_DTYPE_F16 ? at::kHalf : at::kFloat;
}

void same_device(const at::Tensor& t, const at::Tensor& first, const char* name) {
  if (t.get_device() != first.get_device())
    raise(PyExc_ValueError, "%s must be on cuda:%d", name, (int)first.get_device());
}

// A dense tensor of a given type, dims (< 0: any) and first's device.
const at::Tensor& dense(PyObject* o, at::ScalarType type, int dims, const at::Tensor& first,
                        const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type),
          c10::toString(t.scalar_type()));
  on_cuda(t, name);
  if (dims >= 0 && t.dim() != dims) raise(PyExc_ValueError, "%s must have %d dims", name, dims);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  same_device(t, first, name);
  return t;
}

// Elements between the rows of a tensor whose rows are dense and evenly spaced.
int64_t row_stride(const at::Tensor& t, const char* name) {
  const int64_t cols = t.size(-1);
  if (t.is_contiguous()) return cols;
  if (cols > 1 && t.stride(-1) != 1)
    raise(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
  int64_t stride = cols;
  bool first = true;
  int64_t expect = 0;  // stride that the next dim outwards has to have
  for (int64_t d = t.dim() - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (first) stride = t.stride(d);
    else if (t.stride(d) != expect)
      raise(PyExc_ValueError, "%s: the rows must be evenly spaced", name);
    first = false;
    expect = t.stride(d) * t.size(d);
  }
  return stride;
}

// MX codes and scales, as bytes or E4M3 / E8M0 numbers; `cols` receives the elements of a row.
const at::Tensor& codes(PyObject* q, PyObject* s, int bits, int dims, const char* name,
                        const char* scale_name, int64_t& cols, const uint8_t*& scale) {
  const at::Tensor& t = tensor(q, name);
  const at::Tensor& u = tensor(s, scale_name);
  const bool e4m3 = bits == 8 && t.scalar_type() == at::kFloat8_e4m3fn;
  if (t.scalar_type() != at::kByte && !e4m3)
    raise(PyExc_TypeError, "%s must be torch.uint8, got %s", name, c10::toString(t.scalar_type()));
  if (u.scalar_type() != at::kByte && u.scalar_type() != at::kFloat8_e8m0fnu)
    raise(PyExc_TypeError, "%s must be torch.uint8, got %s", scale_name,
          c10::toString(u.scalar_type()));
  on_cuda(t, name);
  same_device(u, t, scale_name);
  if (!t.is_contiguous() || !u.is_contiguous())
    raise(PyExc_ValueError, "%s and %s must be contiguous", name, scale_name);
  const int64_t n = t.dim();
  if (dims >= 0 ? n != dims : n < 1)
    raise(PyExc_ValueError, "%s must have %s dims", name, dims == 2 ? "2" : dims == 3 ? "3" : "some");
  cols = t.size(-1) * (bits == 4 ? 2 : 1);
  if (cols == 0 || cols % 32)
    raise(PyExc_ValueError, "%s must have rows of a positive multiple of 32 elements", name);
  bool fits = u.dim() == n && u.size(-1) * 32 == cols;
  for (int64_t d = 0; fits && d < n - 1; ++d) fits = u.size(d) == t.size(d);
  if (!fits)
    raise(PyExc_ValueError, "%s must have %s's shape with one scale per 32 elements", scale_name, name);
  scale = static_cast<const uint8_t*>(u.data_ptr());
  return t;
}

// The caller's output, checked, or a new one.
at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& first,
                  const char* name) {
  if (o == Py_None) return at::empty(shape, first.options().dtype(type));
  const at::Tensor& t = dense(o, type, -1, first, name);
  if (t.sizes() != shape) raise(PyExc_ValueError, "%s has the wrong shape", name);
  return t;
}

// Makes the tensors' device current for the rest of a call: the library plans,
// launches and finds its status word on the current device.  (Where it is current
// already, as almost always, one look-up instead of a guard's two.)
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;  // that device's current stream
  explicit OnDevice(const at::Tensor& t) {
    if (c10::cuda::current_device() != t.get_device()) guard.set_device(t.device());
    stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
  }
};

// Shapes of the codes and scales of rows.
void code_shapes(const at::Tensor& x, int bits, c10::SmallVector<int64_t, 5>& q,
                 c10::SmallVector<int64_t, 5>& s) {
  const int64_t cols = x.dim() ? x.size(-1) : 0;
  if (cols == 0 || cols % 32)
    raise(PyExc_ValueError, "rows must have a positive multiple of 32 elements");
  q.assign(x.sizes().begin(), x.sizes().end());
  s = q;
  q.back() = bits == 4 ? cols / 2 : cols;
  s.back() = cols / 32;
}

uint8_t* bytes(const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw Raised();
  return o;
}

PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {  // (undefined: None)
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw Raised();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

template <typename F>
int call(F&& f) {  // without the interpreter's lock: a full launch queue blocks
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

// (x, bits, q, scale)
PyObject* quantize(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const int dt = dtype_code(x.scalar_type());
  if (dt < 0)
    raise(PyExc_TypeError, "x must be bfloat16, float16 or float32, got %s", c10::toString(x.scalar_type()));
  on_cuda(x, "x");
  const OnDevice on(x);
  const int bits = bits_of(a[1]);
  c10::SmallVector<int64_t, 5> qs, ss;
  code_shapes(x, bits, qs, ss);
  const int64_t cols = x.size(-1), stride = row_stride(x, "x");
  const at::Tensor q = output(a[2], qs, at::kByte, x, "q");
  const at::Tensor s = output(a[3], ss, at::kByte, x, "scale");
  check(call([&] {
    return moe_quantize_mx(x.data_ptr(), dt, x.numel() / cols, cols, stride, bits, bytes(q),
                           bytes(s), on.stream);
  }));
  return wrap_all({q, s});
}

// (q, scale, bits, dtype code, out)
PyObject* dequantize(PyObject* const* a) {
  const int bits = bits_of(a[2]);
  int64_t cols;
  const uint8_t* scale;
  const at::Tensor& q = codes(a[0], a[1], bits, -1, "q", "scale", cols, scale);
  const OnDevice on(q);
  const long dt = as_long(a[3]);
  c10::SmallVector<int64_t, 5> shape(q.sizes().begin(), q.sizes().end());
  shape.back() = cols;
  const at::Tensor out = output(a[4], shape, scalar_type(dt), q, "out");
  check(call([&] {
    return moe_dequantize_mx(bytes(q), scale, out.numel() / cols, cols, bits, out.data_ptr(),
                             (int)dt, on.stream);
  }));
  return wrap(out);
}

// (x, weight, eps, residual, bits, want_y, residual_out, y, q, scale)
PyObject* rmsnorm(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const at::ScalarType xt = x.scalar_type();
  if (xt != at::kBFloat16 && xt != at::kHalf)
    raise(PyExc_TypeError, "x must be bfloat16 or float16, got %s", c10::toString(xt));
  on_cuda(x, "x");
  const OnDevice on(x);
  if (x.dim() != 2) raise(PyExc_ValueError, "x must have 2 dims");
  const int64_t T = x.size(0), H = x.size(1);
  const bool wf = THPVariable_Check(a[1]) && THPVariable_Unpack(a[1]).scalar_type() == at::kFloat;
  const at::Tensor& weight = dense(a[1], wf ? at::kFloat : xt, 1, x, "weight");
  if (weight.size(0) != H) raise(PyExc_ValueError, "weight must hold H = %ld values", (long)H);
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  const int bits = bits_of(a[4]);
  c10::SmallVector<int64_t, 5> qs, ss;
  code_shapes(x, bits, qs, ss);
  const int64_t xst = row_stride(x, "x");
  int64_t rst = H;
  const void* rp = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor& r = tensor(a[3], "residual");
    if (r.scalar_type() != xt)
      raise(PyExc_TypeError, "residual must be %s, got %s", c10::toString(xt), c10::toString(r.scalar_type()));
    if (r.sizes() != x.sizes()) raise(PyExc_ValueError, "residual must have x's shape");
    same_device(r, x, "residual");
    rst = row_stride(r, "residual");
    rp = r.data_ptr();
  }
  const int want_y = PyObject_IsTrue(a[5]);
  if (want_y < 0) throw Raised();
  at::Tensor ro, y;
  if (rp || a[6] != Py_None) ro = output(a[6], x.sizes(), xt, x, "residual_out");
  if (want_y || a[7] != Py_None) y = output(a[7], x.sizes(), xt, x, "y");
  const at::Tensor q = output(a[8], qs, at::kByte, x, "q");
  const at::Tensor s = output(a[9], ss, at::kByte, x, "scale");
  if (T > INT32_MAX || H > INT32_MAX) raise(PyExc_ValueError, "x is too large");
  check(call([&] {
    return moe_rmsnorm_mx(x.data_ptr(), rp, weight.data_ptr(), dtype_code(xt), wf, (int)T, (int)H,
                          xst, rst, (float)eps, ro.defined() ? ro.data_ptr() : nullptr,
                          y.defined() ? y.data_ptr() : nullptr, bits, bytes(q), bytes(s), on.stream);
  }));
  return wrap_all({q, s, ro, y});
}

// A workspace of at least `need` bytes: the caller's, or a new one.
at::Tensor workspace(PyObject* o, size_t need, const at::Tensor& first) {
  if (o != Py_None) return dense(o, at::kByte, -1, first, "workspace");
  if (!need) return at::Tensor();
  return at::empty({(int64_t)need}, first.options().dtype(at::kByte));
}

void int_sizes(std::initializer_list<int64_t> sizes) {
  for (int64_t n : sizes)
    if (n > INT32_MAX) raise(PyExc_ValueError, "a size exceeds 32 bits");
}

// (a, a_scale, w, w_scale, expert_offsets, a_bits, out, out dtype code, workspace)
PyObject* product(PyObject* const* v) {
  const int bits = bits_of(v[5]);
  int64_t K, wk;
  const uint8_t *as, *ws;
  const at::Tensor& a = codes(v[0], v[1], bits, 2, "a", "a_scale", K, as);
  const OnDevice on(a);
  const at::Tensor& w = codes(v[2], v[3], 4, -1, "w", "w_scale", wk, ws);
  same_device(w, a, "w");
  if (wk != K) raise(PyExc_ValueError, "a and w must have rows of the same length");
  if (w.dim() != 2 && w.dim() != 3) raise(PyExc_ValueError, "w must have 2 or 3 dims");
  const int64_t R = a.size(0), E = w.dim() == 3 ? w.size(0) : 1, N = w.size(-2);
  const int32_t* offsets = nullptr;
  if (v[4] != Py_None) {
    const at::Tensor& o = dense(v[4], at::kInt, 1, a, "expert_offsets");
    if (o.size(0) != E + 1)
      raise(PyExc_ValueError, "expert_offsets must hold E + 1 = %ld values", (long)(E + 1));
    offsets = static_cast<const int32_t*>(o.data_ptr());
  }
  const long dt = as_long(v[7]);
  int_sizes({K, N, E});
  const at::Tensor out = output(v[6], {R, N}, scalar_type(dt), a, "out");
  const at::Tensor wksp =
      workspace(v[8], v[8] == Py_None ? moe_mx_product_workspace(R, (int)K, (int)N, (int)E) : 0, a);
  check(call([&] {
    return moe_mx_product(bytes(a), as, bits, R, (int)K, (int)N, (int)E, bytes(w), ws, offsets,
                          out.data_ptr(), (int)dt, wksp.defined() ? wksp.data_ptr() : nullptr,
                          wksp.defined() ? (size_t)wksp.numel() : 0, on.stream);
  }));
  return wrap(out);
}

// (a, a_scale, w13, s13, w2, s2, topk_w, topk_ids, a_bits, out, out dtype code, workspace)
PyObject* forward(PyObject* const* v) {
  const int bits = bits_of(v[8]);
  int64_t H, k13, I;
  const uint8_t *as, *s13, *s2;
  const at::Tensor& a = codes(v[0], v[1], bits, 2, "a", "a_scale", H, as);
  const OnDevice on(a);
  const at::Tensor& w13 = codes(v[2], v[3], 4, 3, "w13", "s13", k13, s13);
  const at::Tensor& w2 = codes(v[4], v[5], 4, 3, "w2", "s2", I, s2);
  const int64_t T = a.size(0), E = w13.size(0);
  if (k13 != H || w2.size(1) != H || w13.size(1) != 2 * I || w2.size(0) != E)
    raise(PyExc_ValueError, "w13 must be [E, 2I, H] and w2 [E, H, I]");
  same_device(w13, a, "w13");
  same_device(w2, a, "w2");
  const at::Tensor& tw = dense(v[6], at::kFloat, 2, a, "topk_w");
  const at::Tensor& ids = dense(v[7], at::kInt, 2, a, "topk_ids");
  if (ids.size(0) != T || tw.sizes() != ids.sizes())
    raise(PyExc_ValueError, "topk_w and topk_ids must be [%ld, k]", (long)T);
  const int64_t k = ids.size(1);
  const long dt = as_long(v[10]);
  int_sizes({T, H, I, E, k});
  const at::Tensor out = output(v[9], {T, H}, scalar_type(dt), a, "out");
  const at::Tensor wksp = workspace(
      v[11],
      v[11] == Py_None
          ? std::max<size_t>(16, moe_mx_forward_workspace((int)T, (int)H, (int)I, (int)E, (int)k, bits))
          : 0,
      a);
  check(call([&] {
    return moe_mx_forward(bytes(a), as, bits, (int)T, (int)H, (int)I, (int)E, (int)k, bytes(w13), s13,
                          bytes(w2), s2, static_cast<const float*>(tw.data_ptr()),
                          static_cast<const int32_t*>(ids.data_ptr()), out.data_ptr(), (int)dt,
                          wksp.data_ptr(), (size_t)wksp.numel(), on.stream);
  }));
  return wrap(out);
}

PyObject* set_error_class(PyObject* const* a) {
  Py_XDECREF(g_error_class);
  g_error_class = Py_NewRef(a[0]);
  Py_RETURN_NONE;
}

// No C++ exception leaves a call.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<quantize, 4>("quantize"),   method<dequantize, 5>("dequantize"),
                           method<rmsnorm, 10>("rmsnorm"),    method<product, 9>("product"),
                           method<forward, 12>("forward"),    method<set_error_class, 1>("set_error_class"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mx_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx_binding(void) { return PyModule_Create(&g_module); }
