// The quantised calls of the Python binding, marshalled in C++: outputs are
// allocated through torch, pointers and the current stream go to the C entry
// points of include/normfuse.h. A call from Python takes some 10 microseconds
// less than through ctypes and torch.empty, which is most of what a call for a
// few tokens takes.
//
// A function here answers a call as it is commonly made: tensors on the current
// CUDA device, on the current stream, of the types and layouts that the entry
// point takes. It returns None where anything is otherwise, and the caller in
// __init__.py, which has the checks and their messages, goes its own way. A
// status other than LN_OK comes back as a number. The entry points are those of the
// library that the caller has loaded: bind() takes their addresses.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <type_traits>

#include "../../include/normfuse.h"

namespace {

using at::Tensor;

struct Library {
  decltype(&::mx_matrix_bytes) matrix_bytes;
  decltype(&::mx_norm_fwd) norm_fwd;
  decltype(&::mx_quantize) quantize;
  decltype(&::mx_dequantize) dequantize;
  decltype(&::mx_product) product;
  decltype(&::ln_fwd_from_partials) fwd_from_partials;
} lib;

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? LN_F32 : t == at::kBFloat16 ? LN_BF16 : t == at::kHalf ? LN_F16 : -1;
}
at::ScalarType dtype_of(long code) {
  return code == LN_F32 ? at::kFloat : code == LN_BF16 ? at::kBFloat16 : at::kHalf;
}

// A tensor, or null for None; *ok falls where it is neither.
const Tensor* tensor(PyObject* o, bool* ok) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    *ok = false;
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}
void* ptr(const Tensor* t) { return t == nullptr || t->numel() == 0 ? nullptr : t->data_ptr(); }

// Whether all tensors given are on the current CUDA device.
bool together(std::initializer_list<const Tensor*> list, int* device) {
  *device = -1;
  for (const Tensor* t : list) {
    if (t == nullptr) continue;
    if (!t->is_cuda() || (*device >= 0 && t->get_device() != *device)) return false;
    *device = (int)t->get_device();
  }
  return *device >= 0 && *device == (int)c10::cuda::current_device();
}
bool row_of(const Tensor* t, int64_t n, at::ScalarType type) {   // nullable [n]
  return t == nullptr || (t->numel() == n && t->scalar_type() == type && t->is_contiguous());
}
bool like(const Tensor* t, const Tensor& x) {                    // nullable, contiguous
  return t == nullptr || (t->sizes() == x.sizes() && t->scalar_type() == x.scalar_type() && t->is_contiguous());
}
// Elements from one row of a matrix to the next; -1 where its columns are apart.
int64_t row_stride(const Tensor& t) {
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1)) return -1;
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
// A tuple of tensors (None for those that are not there).
PyObject* tuple_of(std::initializer_list<Tensor> list) {
  PyObject* out = PyTuple_New((Py_ssize_t)list.size());
  if (out == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : list) {
    PyObject* o = wrap(t);
    if (o == nullptr) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

at::ScalarType code_type(long fmt) { return fmt >= MX_MXFP4 ? at::kByte : at::kFloat8_e4m3fn; }
at::ScalarType scale_type(long fmt) {
  return fmt <= MX_FP8_BLOCK ? at::kFloat : fmt == MX_NVFP4 ? at::kFloat8_e4m3fn : at::kFloat8_e8m0fnu;
}
bool sizes(long fmt, int64_t rows, int64_t cols, size_t* codes, size_t* scales) {
  return lib.matrix_bytes((mx_format)fmt, rows, cols, codes, scales) == LN_OK;
}
// Room for a matrix; false where there is no such one.
bool room(long fmt, int64_t rows, int64_t cols, const at::TensorOptions& at_, Tensor* codes, Tensor* scales) {
  size_t c = 0, s = 0;
  if (!sizes(fmt, rows, cols, &c, &s) || rows == 0) return false;
  *codes = at::empty({rows, (int64_t)c / rows}, at_.dtype(code_type(fmt)));
  const int64_t width = fmt == MX_NVFP4 ? 16 : fmt == MX_FP8_BLOCK ? 128 : 32;
  const int64_t blocks = (cols + width - 1) / width;
  if (fmt == MX_FP8_ROW) *scales = at::empty({rows}, at_.dtype(at::kFloat));
  else if (fmt == MX_FP8_BLOCK) *scales = at::empty({rows, blocks}, at_.dtype(at::kFloat));
  else *scales = at::empty({(rows + 127) / 128, (blocks + 3) / 4, 32, 4, 4}, at_.dtype(scale_type(fmt)));
  return true;
}
// The struct of a matrix whose tensors are as they should be.
bool matrix(const Tensor* codes, const Tensor* scales, const Tensor* mul, long fmt, int64_t rows, int64_t cols,
            mx_matrix* m) {
  size_t c = 0, s = 0;
  if (codes == nullptr || scales == nullptr || !sizes(fmt, rows, cols, &c, &s)) return false;
  if (codes->nbytes() != c || scales->nbytes() != s || !codes->is_contiguous() || !scales->is_contiguous()) return false;
  if (fmt != MX_NVFP4) mul = nullptr;
  if (mul != nullptr && (mul->numel() != 1 || mul->scalar_type() != at::kFloat)) return false;
  *m = {ptr(codes), ptr(scales), static_cast<const float*>(ptr(mul)), (mx_format)fmt, rows, cols};
  return true;
}

// Numbers of a call: *ok falls where one is none.
long integer(PyObject* o, bool* ok) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    *ok = false;
  }
  return v;
}
double real(PyObject* o, bool* ok) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    *ok = false;
  }
  return v;
}
bool flag(PyObject* o) { return PyObject_IsTrue(o) == 1; }

// norm_quant(x, gamma, beta, bias, residual, mul, format, mode, zero_centered, eps,
// store_sum, store_y) -> (codes, scales, sum, y, mean, rstd)
PyObject* norm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) return none();
  bool ok = true;
  const Tensor *x = tensor(a[0], &ok), *gamma = tensor(a[1], &ok), *beta = tensor(a[2], &ok), *bias = tensor(a[3], &ok),
               *res = tensor(a[4], &ok), *mul = tensor(a[5], &ok);
  const long fmt = integer(a[6], &ok), mode = integer(a[7], &ok);
  const double eps = real(a[9], &ok);
  const bool zero = flag(a[8]), store_sum = flag(a[10]), store_y = flag(a[11]), rms = mode == LN_RMSNORM;
  int device;
  if (!ok || x == nullptr || gamma == nullptr || !together({x, gamma, beta, bias, res, mul}, &device)) return none();
  const int dt = dtype_code(x->scalar_type());
  if (dt < 0 || x->dim() < 1 || x->numel() == 0 || !x->is_contiguous()) return none();
  const int64_t hidden = x->size(-1), rows = x->numel() / hidden;
  const at::ScalarType type = x->scalar_type();
  if (rms) beta = nullptr;
  if (!row_of(gamma, hidden, type) || !row_of(beta, hidden, type) || !row_of(bias, hidden, type) || !like(res, *x)) return none();
  ln_status st = LN_OK;
  Tensor codes, scales, sum, y, mean, rstd;
  mx_matrix q;
  bool made;
  {
    pybind11::gil_scoped_release away;
    const at::TensorOptions options = x->options().requires_grad(false);
    made = room(fmt, rows, hidden, options, &codes, &scales) && matrix(&codes, &scales, mul, fmt, rows, hidden, &q);
    if (made) {
      if (store_sum) sum = at::empty(x->sizes(), options);
      if (store_y) y = at::empty(x->sizes(), options);
      if (!rms) mean = at::empty({rows}, options.dtype(at::kFloat));
      rstd = at::empty({rows}, options.dtype(at::kFloat));
      st = lib.norm_fwd(x->data_ptr(), ptr(bias), ptr(res), gamma->data_ptr(), ptr(beta), (float)eps, (ln_mode)mode, zero,
                       store_sum ? sum.data_ptr() : nullptr, store_y ? y.data_ptr() : nullptr,
                       rms ? nullptr : mean.data_ptr<float>(), rstd.data_ptr<float>(), &q,
                       c10::cuda::getCurrentCUDAStream(device).stream(), (ln_dtype)dt);
    }
  }
  if (!made) return none();
  if (st != LN_OK) return PyLong_FromLong(st);
  return tuple_of({codes, scales, sum, y, mean, rstd});
  END_HANDLE_TH_ERRORS
}

// quantize(x, format, transpose, mul) -> (codes, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return none();
  bool ok = true;
  const Tensor *x = tensor(a[0], &ok), *mul = tensor(a[3], &ok);
  const long fmt = integer(a[1], &ok);
  const bool transpose = flag(a[2]);
  int device;
  if (!ok || x == nullptr || !together({x, mul}, &device)) return none();
  const int dt = dtype_code(x->scalar_type());
  const int64_t stride = row_stride(*x);
  if (dt < 0 || stride < 0 || x->numel() == 0) return none();
  const int64_t rows = x->size(transpose ? 1 : 0), cols = x->size(transpose ? 0 : 1);
  ln_status st = LN_OK;
  Tensor codes, scales;
  mx_matrix q;
  bool made;
  {
    pybind11::gil_scoped_release away;
    made = room(fmt, rows, cols, x->options().requires_grad(false), &codes, &scales) &&
           matrix(&codes, &scales, mul, fmt, rows, cols, &q);
    if (made)
      st = lib.quantize(x->data_ptr(), stride, transpose, &q, c10::cuda::getCurrentCUDAStream(device).stream(), (ln_dtype)dt);
  }
  if (!made) return none();
  if (st != LN_OK) return PyLong_FromLong(st);
  return tuple_of({codes, scales});
  END_HANDLE_TH_ERRORS
}

// dequantize(codes, scales, mul, format, rows, cols, dtype) -> y
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) return none();
  bool ok = true;
  const Tensor *codes = tensor(a[0], &ok), *scales = tensor(a[1], &ok), *mul = tensor(a[2], &ok);
  const long fmt = integer(a[3], &ok), rows = integer(a[4], &ok), cols = integer(a[5], &ok), dt = integer(a[6], &ok);
  int device;
  mx_matrix q;
  if (!ok || dt < 0 || rows == 0 || codes == nullptr || !together({codes, scales, mul}, &device) ||
      !matrix(codes, scales, mul, fmt, rows, cols, &q))
    return none();
  ln_status st;
  Tensor y;
  {
    pybind11::gil_scoped_release away;
    y = at::empty({rows, cols}, codes->options().requires_grad(false).dtype(dtype_of(dt)));
    st = lib.dequantize(&q, y.data_ptr(), cols, c10::cuda::getCurrentCUDAStream(device).stream(), (ln_dtype)dt);
  }
  if (st != LN_OK) return PyLong_FromLong(st);
  return wrap(y);
  END_HANDLE_TH_ERRORS
}

// product(a_codes, a_scales, a_mul, b_codes, b_scales, b_mul, format, rows, columns,
// depth, alpha, bias, residual, dtype, out, partials) -> (out, psum, psq)
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 16) return none();
  bool ok = true;
  const Tensor* t[6];
  for (int i = 0; i < 6; ++i) t[i] = tensor(a[i], &ok);
  const long fmt = integer(a[6], &ok), M = integer(a[7], &ok), N = integer(a[8], &ok), K = integer(a[9], &ok);
  const double alpha = real(a[10], &ok);
  const Tensor *bias = tensor(a[11], &ok), *res = tensor(a[12], &ok), *given = tensor(a[14], &ok);
  long dt = integer(a[13], &ok);
  const bool partials = flag(a[15]);
  int device;
  mx_matrix left, right;
  if (!ok || M <= 0 || N <= 0 || t[0] == nullptr ||
      !together({t[0], t[1], t[2], t[3], t[4], t[5], bias, res, given}, &device) ||
      !matrix(t[0], t[1], t[2], fmt, M, K, &left) || !matrix(t[3], t[4], t[5], fmt, N, K, &right))
    return none();
  if (given != nullptr) dt = dtype_code(given->scalar_type());
  if (dt < 0) return none();
  const at::ScalarType type = dtype_of(dt);
  const int64_t out_row = given ? row_stride(*given) : N, res_row = res ? row_stride(*res) : N;
  if (out_row < 0 || res_row < 0 || !row_of(bias, N, type)) return none();
  if (res != nullptr && (res->size(0) != M || res->size(1) != N || res->scalar_type() != type)) return none();
  if (given != nullptr && (given->size(0) != M || given->size(1) != N)) return none();
  ln_status st;
  Tensor out, psum, psq;
  {
    pybind11::gil_scoped_release away;
    const at::TensorOptions options = t[0]->options().requires_grad(false);
    out = given ? *given : at::empty({M, N}, options.dtype(type));
    if (partials) {
      psum = at::empty({M, (N + 127) / 128}, options.dtype(at::kFloat));
      psq = at::empty({M, (N + 127) / 128}, options.dtype(at::kFloat));
    }
    st = lib.product(&left, &right, (float)alpha, ptr(bias), ptr(res), res_row, out.data_ptr(), out_row,
                    partials ? psum.data_ptr<float>() : nullptr, partials ? psq.data_ptr<float>() : nullptr,
                    c10::cuda::getCurrentCUDAStream(device).stream(), (ln_dtype)dt);
  }
  if (st != LN_OK) return PyLong_FromLong(st);
  return tuple_of({out, psum, psq});
  END_HANDLE_TH_ERRORS
}

// norm_from_partials(x, psum, psq, tile_cols, kind, gamma, beta, eps, mode,
// zero_centered) -> (y, mean, rstd)
PyObject* norm_from_partials(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) return none();
  bool ok = true;
  const Tensor *x = tensor(a[0], &ok), *psum = tensor(a[1], &ok), *psq = tensor(a[2], &ok), *gamma = tensor(a[5], &ok),
               *beta = tensor(a[6], &ok);
  const long tile = integer(a[3], &ok), kind = integer(a[4], &ok), mode = integer(a[8], &ok);
  const double eps = real(a[7], &ok);
  const bool zero = flag(a[9]), rms = mode == LN_RMSNORM;
  int device;
  if (!ok || x == nullptr || gamma == nullptr || psum == nullptr || psq == nullptr ||
      !together({x, psum, psq, gamma, beta}, &device))
    return none();
  const int dt = dtype_code(x->scalar_type());
  if (dt < 0 || x->dim() < 1 || x->numel() == 0 || psum->dim() < 1) return none();
  if (!x->is_contiguous() || !psum->is_contiguous() || !psq->is_contiguous() || !gamma->is_contiguous() ||
      (beta != nullptr && !beta->is_contiguous()))
    return none();
  const int64_t hidden = x->size(-1), rows = x->numel() / hidden;
  // as the call through ctypes has it, sizes of the partials and parameters are the caller's
  ln_status st;
  Tensor y, mean, rstd;
  {
    pybind11::gil_scoped_release away;
    const at::TensorOptions options = x->options().requires_grad(false);
    y = at::empty(x->sizes(), options);
    if (!rms) mean = at::empty({rows}, options.dtype(at::kFloat));
    rstd = at::empty({rows}, options.dtype(at::kFloat));
    st = lib.fwd_from_partials(x->data_ptr(), static_cast<const float*>(ptr(psum)), static_cast<const float*>(ptr(psq)),
                              psum->size(-1), tile, (ln_partials)kind, gamma->data_ptr(), rms ? nullptr : ptr(beta),
                              (float)eps, (ln_mode)mode, zero, y.data_ptr(), rms ? nullptr : mean.data_ptr<float>(),
                              rstd.data_ptr<float>(), nullptr, c10::cuda::getCurrentCUDAStream(device).stream(), rows,
                              hidden, (ln_dtype)dt);
  }
  if (st != LN_OK) return PyLong_FromLong(st);
  return tuple_of({y, mean, rstd});
  END_HANDLE_TH_ERRORS
}

// bind(mx_matrix_bytes, mx_norm_fwd, mx_quantize, mx_dequantize, mx_product,
// ln_fwd_from_partials): addresses of the library's entry points. Called once, before
// anything else here.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[6];
  if (n != 6) return PyErr_Format(PyExc_TypeError, "bind: six addresses, not %zd", n);
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (at[i] == nullptr) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "bind: no address");
  }
  const auto set = [&](auto& fn, int i) { fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(at[i]); };
  set(lib.matrix_bytes, 0);
  set(lib.norm_fwd, 1);
  set(lib.quantize, 2);
  set(lib.dequantize, 3);
  set(lib.product, 4);
  set(lib.fwd_from_partials, 5);
  Py_RETURN_NONE;
}

#define FAST(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(norm_quant), FAST(quantize), FAST(dequantize), FAST(product), FAST(norm_from_partials),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module_def); }
