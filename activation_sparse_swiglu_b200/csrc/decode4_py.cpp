// The Python entry of the 4-bit operators' calls: argument checks, result
// tensors and the C ABI call of one operator in one native function.  A decode
// step makes a handful of these per layer on data of a few KB, where the same
// steps in Python take longer than the kernels (an attention call 9 us of the
// host's time for 5.6 us of the device's; this way 4).  Weights, caches and
// their lifetimes stay in Python (decode4.py).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <cstdint>

#include <ATen/Functions.h>
#include <ATen/core/grad_mode.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "prox.h"

namespace {

PyObject* prox_error = nullptr;  // the package's ProxError

// A Python exception is set.
struct Raised {};

#define RAISE(type, ...)               \
  do {                                 \
    PyErr_Format(type, __VA_ARGS__);   \
    throw Raised();                    \
  } while (0)

void check(prox_status st) {
  if (st == PROX_OK) return;
  char msg[1024];
  prox_last_error(msg, sizeof(msg));
  PyObject* e = PyObject_CallFunction(prox_error, "is", (int)st, msg);
  if (e) {
    PyErr_SetObject(prox_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

long long number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int integer(PyObject* o) {
  const long long v = number(o);
  if (v != (int)v) RAISE(PyExc_OverflowError, "%lld does not fit 32 bits", v);
  return (int)v;
}
template <typename T>
T* handle(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised();
  return static_cast<T*>(p);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    RAISE(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}
void on(const at::Tensor& t, int index, const char* name) {
  if (t.get_device() != index)
    RAISE(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d", name, (int)t.get_device(), index);
}
int code_of(at::ScalarType t) {
  return t == at::kFloat ? PROX_F32 : t == at::kHalf ? PROX_F16 : t == at::kBFloat16 ? PROX_BF16 : -1;
}
// The calls give no gradients: a tensor whose gradient or tangent they would
// drop is refused.
void no_gradient(const at::Tensor& t, const char* name) {
  if ((t.requires_grad() && at::GradMode::is_enabled()) || t._fw_grad(0).defined())
    RAISE(PyExc_RuntimeError,
          "%s carries a gradient, which this operator does not give: detach it or call under torch.no_grad()", name);
}
// An activation tensor on the device, and its type's code.
const at::Tensor& act(PyObject* o, int index, const char* name, int* code) {
  const at::Tensor& t = tensor(o, name);
  *code = code_of(t.scalar_type());
  if (*code < 0) RAISE(PyExc_TypeError, "%s must be float32, float16 or bfloat16", name);
  on(t, index, name);
  no_gradient(t, name);
  return t;
}
// A contiguous tensor of `numel` integers on the device.
const at::Tensor& ints(PyObject* o, int index, at::ScalarType type, int64_t numel, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    RAISE(PyExc_TypeError, "%s must be a CUDA tensor of %s", name, type == at::kInt ? "int32" : "int64");
  on(t, index, name);
  if (t.numel() != numel || !t.is_contiguous())
    RAISE(PyExc_ValueError, "%s must hold %lld contiguous values", name, (long long)numel);
  return t;
}
// A page table [rows, cols]: its columns and row stride.
const at::Tensor& page_table(PyObject* o, int index, int64_t rows, int64_t* cols, int64_t* stride) {
  if (!THPVariable_Check(o)) RAISE(PyExc_TypeError, "table must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows || (t.size(1) > 1 && t.stride(1) != 1) ||
      (rows > 1 && t.stride(0) < t.size(1)))
    RAISE(PyExc_ValueError, "table must be int32 [%lld, cols] with contiguous rows", (long long)rows);
  tensor(o, "table");
  on(t, index, "table");
  *cols = t.size(1);
  *stride = std::max(t.stride(0), *cols);
  return t;
}

void* stream_of(PyObject* o, int index) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(index).stream();
  return handle<void>(o);
}
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, index));
}

template <typename F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F&& f) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (handle, device, d_in, d_out, x, out or None, stream or None) -> out
PyObject* linear4_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, [&]() -> PyObject* {
    const int index = integer(a[1]);
    const int64_t d_in = number(a[2]), d_out = number(a[3]);
    int code;
    const at::Tensor& x = act(a[4], index, "x", &code);
    const int64_t dim = x.dim();
    if (dim < 1 || dim > 2 || x.size(-1) != d_in || x.stride(-1) != 1)
      RAISE(PyExc_ValueError, "x must be [B, %lld] or [%lld] with contiguous rows", (long long)d_in, (long long)d_in);
    const int64_t B = dim == 2 ? x.size(0) : 1;
    at::Tensor made;
    const at::Tensor* out = &made;
    if (a[5] == Py_None) {
      made = dim == 2 ? empty({B, d_out}, x.scalar_type(), index) : empty({d_out}, x.scalar_type(), index);
    } else {
      out = &tensor(a[5], "out");
      on(*out, index, "out");
      no_gradient(*out, "out");
      if (out->scalar_type() != x.scalar_type() || out->dim() != dim || out->size(-1) != d_out || out->stride(-1) != 1 ||
          (dim == 2 && out->size(0) != B))
        RAISE(PyExc_ValueError, "out must be of x's type, %lld rows of %lld contiguous values", (long long)B,
              (long long)d_out);
    }
    if (B > INT32_MAX) RAISE(PyExc_ValueError, "x has too many rows");
    check(prox_linear4_forward(handle<prox_linear4>(a[0]), x.data_ptr(), dim == 2 ? x.stride(0) : d_in, out->data_ptr(),
                               dim == 2 ? out->stride(0) : d_out, (int)B, code, stream_of(a[6], index)));
    if (a[5] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[5]);
    return a[5];
  });
}

// (handle, device, heads, head_dim, k, v, slots, stream or None)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&]() -> PyObject* {
    const int index = integer(a[1]);
    const int64_t H = number(a[2]), D = number(a[3]);
    int code, v_code;
    const at::Tensor& k = act(a[4], index, "k", &code);
    const at::Tensor& v = act(a[5], index, "v", &v_code);
    if (k.dim() != 3 || k.size(1) != H || k.size(2) != D || v.sizes() != k.sizes() || k.stride(2) != 1 ||
        v.stride(2) != 1)
      RAISE(PyExc_ValueError, "k and v must be [T, %lld, %lld] with contiguous rows", (long long)H, (long long)D);
    if (code != v_code) RAISE(PyExc_TypeError, "k and v must have one type");
    const int64_t T = k.size(0);
    if (T > INT32_MAX) RAISE(PyExc_ValueError, "k has too many rows");
    const at::Tensor& slots = ints(a[6], index, at::kLong, T, "slots");
    check(prox_kv4_append(handle<prox_kv4>(a[0]), k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0),
                          v.stride(1), slots.data_ptr<int64_t>(), (int)T, code, stream_of(a[7], index)));
    Py_RETURN_NONE;
  });
}

// (handle, device, heads, head_dim, slots, dtype, (k, v) or None, stream or None) -> (k, v)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&]() -> PyObject* {
    const int index = integer(a[1]);
    const int64_t H = number(a[2]), D = number(a[3]);
    if (!THPDtype_Check(a[5]) || code_of(reinterpret_cast<THPDtype*>(a[5])->scalar_type) < 0)
      RAISE(PyExc_TypeError, "dtype must be float32, float16 or bfloat16");
    const at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    const int64_t T = tensor(a[4], "slots").numel();
    const at::Tensor& slots = ints(a[4], index, at::kLong, T, "slots");
    if (T > INT32_MAX) RAISE(PyExc_ValueError, "too many slots");
    at::Tensor k, v;
    if (a[6] == Py_None) {
      k = empty({T, H, D}, type, index);
      v = empty({T, H, D}, type, index);
    } else {  // made by the caller for another stream
      k = tensor(PyTuple_GetItem(a[6], 0), "k");
      v = tensor(PyTuple_GetItem(a[6], 1), "v");
    }
    check(prox_kv4_read(handle<prox_kv4>(a[0]), slots.data_ptr<int64_t>(), (int)T, k.data_ptr(), v.data_ptr(),
                        code_of(type), stream_of(a[7], index)));
    PyObject* kv = PyTuple_New(2);
    if (!kv) return nullptr;
    PyTuple_SET_ITEM(kv, 0, THPVariable_Wrap(std::move(k)));
    PyTuple_SET_ITEM(kv, 1, THPVariable_Wrap(std::move(v)));
    return kv;
  });
}

// (handle, device, head_dim, q, table, lens, scale, out or None, lse or None, stream or None) -> out
PyObject* kv4_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> PyObject* {
    const int index = integer(a[1]);
    const int64_t D = number(a[2]);
    int code;
    const at::Tensor& q = act(a[3], index, "q", &code);
    const int64_t dim = q.dim();
    if (dim < 3 || dim > 4 || q.size(-1) != D || q.stride(-1) != 1)
      RAISE(PyExc_ValueError, "q must be [B, Tq, Hq, %lld] or [B, Hq, %lld] with contiguous rows", (long long)D,
            (long long)D);
    const int64_t B = q.size(0), Hq = q.size(-2), Tq = dim == 4 ? q.size(1) : 1;
    int64_t cols, table_stride;
    const at::Tensor& table = page_table(a[4], index, B, &cols, &table_stride);
    const at::Tensor& lens = ints(a[5], index, at::kInt, B, "lens");
    if (std::max({B, Hq, Tq, cols}) > INT32_MAX) RAISE(PyExc_ValueError, "q or table is too large");
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised();
    at::Tensor made;
    const at::Tensor* out = &made;
    if (a[7] == Py_None) {
      made = empty(q.sizes(), q.scalar_type(), index);
    } else {
      out = &tensor(a[7], "out");
      on(*out, index, "out");
      no_gradient(*out, "out");
      if (out->scalar_type() != q.scalar_type() || out->sizes() != q.sizes() || !out->is_contiguous())
        RAISE(PyExc_ValueError, "out must be a contiguous tensor of q's shape and type");
    }
    float* lse = nullptr;
    if (a[8] != Py_None) {
      const at::Tensor& t = tensor(a[8], "lse");
      on(t, index, "lse");
      no_gradient(t, "lse");
      if (t.scalar_type() != at::kFloat || t.numel() != B * Tq * Hq || !t.is_contiguous())
        RAISE(PyExc_ValueError, "lse must hold %lld contiguous float32 values", (long long)(B * Tq * Hq));
      lse = t.data_ptr<float>();
    }
    check(prox_kv4_attend(handle<prox_kv4>(a[0]), q.data_ptr(), q.stride(0), dim == 4 ? q.stride(1) : 0, q.stride(-2),
                          (int)Hq, (int)B, (int)Tq, table.data_ptr<int32_t>(), table_stride, (int)cols,
                          lens.data_ptr<int32_t>(), (float)scale, out->data_ptr(), lse, code, stream_of(a[9], index)));
    if (a[7] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[7]);
    return a[7];
  });
}

// (lens, delta, table, free_pages, free_count, page_size, max_new, commit,
//  (int32 buffer, slots) or None, stream or None)
// -> (lens, count, cu, slots, positions, status)
PyObject* plan_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> PyObject* {
    const at::Tensor& first = tensor(a[0], "lens");
    const int index = (int)first.get_device();
    const int current = (int)c10::cuda::current_device();
    if (index != current)
      RAISE(PyExc_ValueError, "lens is on cuda:%d, not on the current CUDA device cuda:%d", index, current);
    const int64_t B = first.numel();
    const at::Tensor& lens = ints(a[0], index, at::kInt, B, "lens");
    const at::Tensor& delta = ints(a[1], index, at::kInt, B, "delta");
    int64_t cols, table_stride;
    const at::Tensor& table = page_table(a[2], index, B, &cols, &table_stride);
    const int64_t cap = tensor(a[3], "free_pages").numel();
    const at::Tensor& pages = ints(a[3], index, at::kInt, cap, "free_pages");
    const at::Tensor& count = ints(a[4], index, at::kInt, 1, "free_count");
    const int page = integer(a[5]), room = integer(a[6]);
    if (room < 0) RAISE(PyExc_ValueError, "max_new=%d must be >= 0", room);
    if (std::max({B, cols, cap}) > INT32_MAX) RAISE(PyExc_ValueError, "lens, table or free_pages is too large");
    const int commit = PyObject_IsTrue(a[7]);
    if (commit < 0) throw Raised();
    const int64_t sizes[5] = {room, B, B + 1, 1, 1};
    at::Tensor buf, slots;
    if (a[8] == Py_None) {
      buf = empty({2 * B + 3 + room}, at::kInt, index);
      slots = empty({room}, at::kLong, index);
    } else {  // made by the caller for another stream
      buf = tensor(PyTuple_GetItem(a[8], 0), "buffer");
      slots = tensor(PyTuple_GetItem(a[8], 1), "slots");
    }
    at::Tensor part[5];  // positions, lens, cu, count, status
    {
      at::AutoDispatchBelowADInplaceOrView plain;  // (integers: no gradients to follow)
      int64_t from = 0;
      for (int i = 0; i < 5; ++i) {
        part[i] = buf.as_strided({sizes[i]}, {1}, from);
        from += sizes[i];
      }
    }
    if (commit) part[1] = lens, part[3] = count;
    check(prox_plan_pages(lens.data_ptr<int32_t>(), delta.data_ptr<int32_t>(), (int)B, page, table.data_ptr<int32_t>(),
                          table_stride, (int)cols, pages.data_ptr<int32_t>(), (int)cap, count.data_ptr<int32_t>(),
                          part[1].data_ptr<int32_t>(), part[3].data_ptr<int32_t>(), part[2].data_ptr<int32_t>(),
                          slots.data_ptr<int64_t>(), part[0].data_ptr<int32_t>(), room, part[4].data_ptr<int32_t>(),
                          stream_of(a[9], index)));
    PyObject* all = PyTuple_New(6);
    if (!all) return nullptr;
    PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(std::move(part[1])));
    PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(std::move(part[3])));
    PyTuple_SET_ITEM(all, 2, THPVariable_Wrap(std::move(part[2])));
    PyTuple_SET_ITEM(all, 3, THPVariable_Wrap(std::move(slots)));
    PyTuple_SET_ITEM(all, 4, THPVariable_Wrap(std::move(part[0])));
    PyTuple_SET_ITEM(all, 5, THPVariable_Wrap(std::move(part[4])));
    return all;
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(linear4_forward), FAST(kv4_append), FAST(kv4_read), FAST(kv4_attend), FAST(plan_pages),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode4", "Calls of the 4-bit operators (see decode4.py).", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode4(void) {
  PyObject* m = PyModule_Create(&module);
  if (!m) return nullptr;
  // what this module's C++ interface is that of (see build.py); checked before any call
  if (PyModule_AddStringConstant(m, "built_for", PROX_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  // _lib.py loads libprox.so and defines the error before this module is imported
  PyObject* lib = PyImport_ImportModule("activation_sparse_swiglu_b200._lib");
  prox_error = lib ? PyObject_GetAttrString(lib, "ProxError") : nullptr;
  Py_XDECREF(lib);
  if (!prox_error) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
