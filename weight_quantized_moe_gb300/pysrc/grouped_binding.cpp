// Python calls of the 16-bit operators (grouped product, its gradients, adapters),
// compiled as the microscaled ones are: binding.py declares them and passes the
// arguments on by position.
#include "binding_common.h"

namespace {

// The calls have no forward-mode derivative: a tensor with a tangent is refused, as the result
// would have none.
void no_tangent(const at::Tensor& t, const char* name) {
  if (t._fw_grad(0).defined())
    raise(PyExc_ValueError, "%s has a tangent: there is no forward-mode derivative", name);
}

// 16-bit rows [R, C]: their type, and the elements between rows.
struct Rows {
  const at::Tensor& t;
  int dtype;
  int64_t R, C, stride;
};

Rows rows(PyObject* o, const char* name, const at::Tensor* first = nullptr) {
  const at::Tensor& t = tensor(o, name);
  const at::ScalarType type = t.scalar_type();
  if (first ? type != first->scalar_type() : type != at::kBFloat16 && type != at::kHalf)
    raise(PyExc_TypeError, "%s must be %s, got %s", name,
          first ? c10::toString(first->scalar_type()) : "bfloat16 or float16", c10::toString(type));
  on_cuda(t, name);
  no_tangent(t, name);
  if (first) same_device(t, *first, name);
  if (t.dim() != 2) raise(PyExc_ValueError, "%s must have 2 dims", name);
  if (t.size(1) < 1) raise(PyExc_ValueError, "%s must have rows of at least one element", name);
  if (t.size(1) > 1 && t.stride(1) != 1)
    raise(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
  int64_t stride = t.stride(0);
  if (t.size(0) <= 1) stride = (t.size(1) + 7) / 8 * 8;  // (never taken)
  return {t, dtype_code(type), t.size(0), t.size(1), stride};
}

// Weights [E, N, K] or [N, K], stored so or as [E, K, N].
struct Weights {
  const at::Tensor& t;
  int64_t E, N, K, stride, expert;
  bool transposed;
};

Weights weights(PyObject* o, const char* name, const Rows& a) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != a.t.scalar_type())
    raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(a.t.scalar_type()),
          c10::toString(t.scalar_type()));
  on_cuda(t, name);
  no_tangent(t, name);
  same_device(t, a.t, name);
  if (t.dim() != 2 && t.dim() != 3) raise(PyExc_ValueError, "%s must have 2 or 3 dims", name);
  const int64_t E = t.dim() == 3 ? t.size(0) : 1, N = t.size(-2), K = t.size(-1);
  if (E < 1 || N < 1 || K < 1) raise(PyExc_ValueError, "%s must not be empty", name);
  const int64_t sn = t.stride(-2), sk = t.stride(-1);
  const bool by_k = K == 1 || sk == 1, by_n = N == 1 || sn == 1;
  if (!by_k && !by_n)
    raise(PyExc_ValueError, "%s must have contiguous rows, or be a transposed view of such", name);
  const bool fits_k = by_k && (N == 1 || sn % 8 == 0), fits_n = by_n && (K == 1 || sk % 8 == 0);
  const bool transposed = !fits_k && (fits_n || !by_k);
  int64_t stride = transposed ? sk : sn;
  if ((transposed ? K : N) == 1) stride = ((transposed ? N : K) + 7) / 8 * 8;  // (never taken)
  return {t, E, N, K, stride, E > 1 ? t.stride(0) : 8, transposed};
}

const int32_t* expert_offsets(PyObject* o, int64_t E, const at::Tensor& first) {
  if (o == Py_None) {
    if (E != 1) raise(PyExc_ValueError, "expert_offsets may be missing with one expert only");
    return nullptr;
  }
  const at::Tensor& t = dense(o, at::kInt, 1, first, "expert_offsets");
  if (t.size(0) != E + 1)
    raise(PyExc_ValueError, "expert_offsets must hold E + 1 = %ld values", (long)(E + 1));
  return static_cast<const int32_t*>(t.data_ptr());
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v;
}

// (a, w, expert_offsets, out, out dtype code, workspace)
PyObject* product(PyObject* const* v) {
  const Rows a = rows(v[0], "a");
  const OnDevice on(a.t);
  const Weights w = weights(v[1], "w", a);
  if (w.K != a.C) raise(PyExc_ValueError, "a and w must have rows of the same length");
  const int32_t* offsets = expert_offsets(v[2], w.E, a.t);
  const long dt = as_long(v[4]);
  int_sizes({w.K, w.N, w.E});
  const at::Tensor out = output(v[3], {a.R, w.N}, scalar_type(dt), a.t, "out");
  no_tangent(out, "out");
  const int K = (int)w.K, N = (int)w.N, E = (int)w.E;
  const at::Tensor wksp =
      workspace(v[5], v[5] == Py_None ? moe_grouped_product_workspace(a.R, K, N, E) : 0, a.t);
  check(call([&] {
    return moe_grouped_product(a.t.data_ptr(), a.stride, a.dtype, a.R, K, N, E, w.t.data_ptr(),
                               w.stride, w.expert, w.transposed, offsets, out.data_ptr(), (int)dt,
                               ptr(wksp), wksp.defined() ? (size_t)wksp.numel() : 0, on.stream);
  }));
  written({v[3]});
  return wrap(out);
}

// (dy, a, w, expert_offsets, need_a, need_w, da, dw, dw dtype code, workspace)
PyObject* product_grad(PyObject* const* v) {
  const Rows a = rows(v[1], "a");
  const OnDevice on(a.t);
  const Rows dy = rows(v[0], "dy", &a.t);
  const Weights w = weights(v[2], "w", a);
  if (w.K != a.C || w.N != dy.C || dy.R != a.R)
    raise(PyExc_ValueError, "dy must be [R, N], a [R, K] and w [E, N, K]");
  const int32_t* offsets = expert_offsets(v[3], w.E, a.t);
  const long dt = as_long(v[8]);
  int_sizes({w.K, w.N, w.E});
  const int K = (int)w.K, N = (int)w.N, E = (int)w.E;
  at::Tensor da, dw;
  if (truth(v[4]) || v[6] != Py_None) da = output(v[6], {a.R, w.K}, a.t.scalar_type(), a.t, "da");
  if (truth(v[5]) || v[7] != Py_None) {
    if (v[7] != Py_None) {  // the caller's: dense in the order that w is stored in
      const at::Tensor& t = tensor(v[7], "dw");
      if (t.scalar_type() != scalar_type(dt))
        raise(PyExc_TypeError, "dw must be %s, got %s", c10::toString(scalar_type(dt)),
              c10::toString(t.scalar_type()));
      on_cuda(t, "dw");
      same_device(t, a.t, "dw");
      if (t.sizes() != w.t.sizes()) raise(PyExc_ValueError, "dw must have w's shape");
      if (!(w.transposed ? t.transpose(-1, -2) : t).is_contiguous())
        raise(PyExc_ValueError, "dw must be dense in the order that w is stored in");
      dw = t;
    } else {
      c10::SmallVector<int64_t, 3> shape(w.t.sizes().begin(), w.t.sizes().end());
      if (w.transposed) std::swap(shape[shape.size() - 1], shape[shape.size() - 2]);
      dw = at::empty(shape, a.t.options().dtype(scalar_type(dt)));
      if (w.transposed) dw = dw.transpose(-1, -2);
    }
  }
  if (da.defined()) no_tangent(da, "da");
  if (dw.defined()) no_tangent(dw, "dw");
  const at::Tensor wksp =
      workspace(v[9], v[9] == Py_None ? moe_grouped_product_grad_workspace(a.R, K, N, E) : 0, a.t);
  check(call([&] {
    return moe_grouped_product_grad(dy.t.data_ptr(), dy.stride, a.t.data_ptr(), a.stride, a.dtype,
                                    a.R, K, N, E, w.t.data_ptr(), w.stride, w.expert, w.transposed,
                                    offsets, ptr(da), ptr(dw), (int)dt, ptr(wksp),
                                    wksp.defined() ? (size_t)wksp.numel() : 0, on.stream);
  }));
  written({v[6], v[7]});
  return wrap_all({da, dw});
}

// Adapters [L, E, rows, cols], or [L, rows, cols] for one expert.
const at::Tensor& adapters(PyObject* o, const char* name, const Rows& x, int64_t& L, int64_t& E) {
  const at::Tensor& t = dense(o, x.t.scalar_type(), -1, x.t, name);
  no_tangent(t, name);
  if (t.dim() != 3 && t.dim() != 4) raise(PyExc_ValueError, "%s must have 3 or 4 dims", name);
  L = t.size(0);
  E = t.dim() == 4 ? t.size(1) : 1;
  return t;
}

// Rows [R, N] of a given type that may be strided: their stride.
int64_t strided(const at::Tensor& t, at::ScalarType type, int64_t R, int64_t N, const at::Tensor& first,
                const char* name) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  on_cuda(t, name);
  same_device(t, first, name);
  if (t.dim() != 2 || t.size(0) != R || t.size(1) != N)
    raise(PyExc_ValueError, "%s must be [%ld, %ld]", name, (long)R, (long)N);
  if (N > 1 && t.stride(1) != 1)
    raise(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
  return R <= 1 ? N : t.stride(0);
}

// (x, lora_a, lora_b, adapter_ids, base, expert_offsets, scaling, out, out dtype code, workspace)
PyObject* lora(PyObject* const* v) {
  const Rows x = rows(v[0], "x");
  const OnDevice on(x.t);
  int64_t L, E, Lb, Eb;
  const at::Tensor& a = adapters(v[1], "lora_a", x, L, E);
  const at::Tensor& b = adapters(v[2], "lora_b", x, Lb, Eb);
  const int64_t r = a.size(-2), K = x.C, N = b.size(-2), R = x.R;
  if (a.size(-1) != K || b.size(-1) != r || Lb != L || Eb != E || b.dim() != a.dim())
    raise(PyExc_ValueError, "lora_a must be [L, E, r, K] and lora_b [L, E, N, r] (or both without E)");
  const at::Tensor& ids = dense(v[3], at::kInt, 1, x.t, "adapter_ids");
  if (ids.size(0) != R) raise(PyExc_ValueError, "adapter_ids must hold R = %ld values", (long)R);
  const long dt = as_long(v[8]);
  const at::ScalarType type = scalar_type(dt);
  at::Tensor base, out;
  int64_t base_stride = N, out_stride = N;
  if (v[4] != Py_None) {
    base = tensor(v[4], "base");
    no_tangent(base, "base");
    base_stride = strided(base, type, R, N, x.t, "base");
  }
  const int32_t* offsets = expert_offsets(v[5], E, x.t);
  const float* scaling = nullptr;
  if (v[6] != Py_None) {
    const at::Tensor& s = dense(v[6], at::kFloat, 1, x.t, "scaling");
    no_tangent(s, "scaling");
    if (s.size(0) != L) raise(PyExc_ValueError, "scaling must hold L = %ld values", (long)L);
    scaling = static_cast<const float*>(s.data_ptr());
  }
  int_sizes({K, N, r, L, E});
  if (v[7] != Py_None) {
    out = tensor(v[7], "out");
    no_tangent(out, "out");
    out_stride = strided(out, type, R, N, x.t, "out");
  } else {
    out = at::empty({R, N}, x.t.options().dtype(type));
  }
  const at::Tensor wksp = workspace(
      v[9],
      v[9] == Py_None ? moe_lora_product_workspace(R, (int)K, (int)N, (int)r, (int)L, (int)E) : 0, x.t);
  check(call([&] {
    return moe_lora_product(x.t.data_ptr(), x.stride, x.dtype, R, (int)K, (int)N, (int)r, (int)L, (int)E,
                            a.data_ptr(), b.data_ptr(), static_cast<const int32_t*>(ids.data_ptr()), offsets,
                            scaling, ptr(base), base_stride, out.data_ptr(), out_stride, (int)dt, ptr(wksp),
                            wksp.defined() ? (size_t)wksp.numel() : 0, on.stream);
  }));
  written({v[7]});
  return wrap(out);
}

PyMethodDef g_methods[] = {method<product, 6>("product"),
                           method<product_grad, 10>("product_grad"),
                           method<lora, 10>("lora"),
                           method<set_error_class, 1>("set_error_class"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_grouped_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__grouped_binding(void) { return PyModule_Create(&g_module); }
