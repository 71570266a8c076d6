// The tensor-level calls of mxfp4.py: argument checks, output allocation and
// marshalling to the C ABI (include/mhr_mxfp4.h), nothing else.
//
// They are compiled because a 4-bit product of one token takes 6 us on the GPU,
// and the same steps as Python statements on tensors took 9 us on the Grace host
// (a torch.empty alone 1.5 to 5 us) before the 4 us of the C call.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "mhr_mxfp4.h"

namespace {

// The C ABI's entry points, as the package has loaded them, and its classes.
decltype(&gemm_mxfp4_quantize) g_quantize;
decltype(&gemm_mxfp4) g_product;
decltype(&gemm_mxfp4_quantized) g_quantized;
decltype(&gemm_mxfp4_moe) g_moe;
PyObject* g_matrix;  // MxFp4Matrix
PyObject* g_error;   // GemmError

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* format, const char* name = "") {
  PyErr_Format(type, format, name);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

int dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return MHR_F32;
    case at::kBFloat16: return MHR_BF16;
    case at::kHalf: return MHR_F16;
    default: raise(PyExc_TypeError, "%s must be float32, bfloat16 or float16", name);
  }
}

// A row-major matrix: sizes and row pitch.
struct Plain {
  int64_t rows, cols, ld;
};
Plain plain(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) raise(PyExc_ValueError, "%s must be 2-D", name);
  const int64_t rows = t.size(0), cols = t.size(1);
  if (rows > 0 && cols > 1 && t.stride(1) != 1)
    raise(PyExc_ValueError, "%s must be row-major (last dimension contiguous)", name);
  const int64_t ld = rows > 1 && t.stride(0) > cols ? t.stride(0) : cols;
  // (rows that repeat or overlap have no pitch)
  if (rows > 1 && cols > 0 && t.stride(0) < cols)
    raise(PyExc_ValueError, "%s must be row-major (rows overlap)", name);
  return {rows, cols, ld};
}

int64_t blocks(int64_t cols) { return (cols + 31) / 32; }
int64_t scale_bytes(int64_t rows, int64_t cols) {
  return (rows + 127) / 128 * ((cols + 127) / 128) * 512;
}

struct Packed {
  at::Tensor data, scales;
  int64_t rows, cols, ld;
  const uint8_t* d() const { return static_cast<const uint8_t*>(data.data_ptr()); }
  const uint8_t* s() const { return static_cast<const uint8_t*>(scales.data_ptr()); }
};
bool is_packed(PyObject* o) { return PyObject_TypeCheck(o, (PyTypeObject*)g_matrix); }
Packed packed(PyObject* o, const char* name) {
  if (!is_packed(o)) raise(PyExc_TypeError, "%s must be an MxFp4Matrix", name);
  Packed q{tensor(PyTuple_GET_ITEM(o, 0), name), tensor(PyTuple_GET_ITEM(o, 1), name),
           PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2)), PyLong_AsLongLong(PyTuple_GET_ITEM(o, 3)), 0};
  if (PyErr_Occurred()) throw Raised{};
  if (q.data.scalar_type() != at::kByte || q.scales.scalar_type() != at::kByte)
    raise(PyExc_TypeError, "%s: data and scales must be uint8", name);
  const Plain p = plain(q.data, name);
  if (q.rows < 0 || q.cols < 0 || p.rows != q.rows || p.cols < blocks(q.cols) * 16)
    raise(PyExc_ValueError, "%s: data must be rows x 16 * ceil(cols / 32) bytes", name);
  if (!q.scales.is_contiguous() || q.scales.numel() < scale_bytes(q.rows, q.cols))
    raise(PyExc_ValueError,
          "%s: scales must be contiguous, mxfp4_scale_bytes(rows, cols) bytes", name);
  q.ld = p.ld;
  return q;
}

// The one CUDA device of all tensors.
int device_of(std::initializer_list<const at::Tensor*> tensors) {
  const at::Device d = (*tensors.begin())->device();
  if (!d.is_cuda()) raise(PyExc_ValueError, "%soperands must be CUDA tensors");
  for (const at::Tensor* t : tensors)
    if (t->device() != d) raise(PyExc_ValueError, "%soperands must be on one device");
  return d.index();
}

at::Tensor empty(std::initializer_list<int64_t> sizes, at::ScalarType type, int device) {
  return at::detail::empty_cuda(at::IntArrayRef(sizes.begin(), sizes.size()), type,
                                at::Device(at::kCUDA, static_cast<at::DeviceIndex>(device)),
                                std::nullopt);
}

// The raw stream of a call: the caller's handle, or the current torch stream.
void* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (PyErr_Occurred()) throw Raised{};
  return reinterpret_cast<void*>(v);
}

// Runs the C call without the interpreter's lock; a status other than MHR_OK
// becomes GemmError(status, where).
template <typename Call>
void run(const char* where, int device, const Call& call) {
  int rc;
  {
    const c10::cuda::CUDAGuard guard(static_cast<at::DeviceIndex>(device));
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
  }
  if (rc == MHR_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", rc, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

void count(Py_ssize_t have, Py_ssize_t want) {
  if (have != want) raise(PyExc_TypeError, "%swrong number of arguments");
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// quantize(x, axis, values, stream) -> MxFp4Matrix [, values]
PyObject* quantize(PyObject* const* a, Py_ssize_t n) {
  count(n, 4);
  const at::Tensor& x = tensor(a[0], "x");
  const int type = dtype_of(x, "x");
  const long axis = PyLong_AsLong(a[1]);
  if (axis == -1 && PyErr_Occurred()) throw Raised{};
  if (axis != 0 && axis != 1) raise(PyExc_ValueError, "%saxis must be 0 or 1");
  const int with_values = PyObject_IsTrue(a[2]);
  if (with_values < 0) throw Raised{};
  const Plain p = plain(x, "x");
  const int device = device_of({&x});
  void* stream = stream_of(a[3], device);
  const int64_t rows = axis ? p.rows : p.cols, cols = axis ? p.cols : p.rows;
  const int64_t ldd = blocks(cols) * 16;
  // Codes and scales in one allocation: 0.4 us less than two (of 4.3 a call on the
  // Grace host).
  at::Tensor data = empty({rows * ldd + scale_bytes(rows, cols)}, at::kByte, device);
  at::Tensor scales = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(data.storage()),
                                                               data.key_set(), data.dtype());
  scales.unsafeGetTensorImpl()->set_storage_offset(rows * ldd);
  scales.unsafeGetTensorImpl()->set_sizes_contiguous({scale_bytes(rows, cols)});
  data.unsafeGetTensorImpl()->set_sizes_contiguous({rows, ldd});
  at::Tensor values;
  if (with_values) values = empty({p.rows, p.cols}, x.scalar_type(), device);
  run("gemm_mxfp4_quantize", device, [&] {
    return g_quantize(type, x.data_ptr(), p.rows, p.cols, p.ld, axis ? 0 : 1,
                      static_cast<uint8_t*>(data.data_ptr()), ldd,
                      static_cast<uint8_t*>(scales.data_ptr()),
                      with_values ? values.data_ptr() : nullptr, p.cols, stream);
  });
  PyObject* q = PyObject_CallFunction(g_matrix, "NNLL", THPVariable_Wrap(data),
                                      THPVariable_Wrap(scales), static_cast<long long>(rows),
                                      static_cast<long long>(cols));
  if (!q || !with_values) return q;
  return Py_BuildValue("NN", q, THPVariable_Wrap(values));
}

// matmul(a, b, out or None, out_dtype as a number of mhr_dtype, stream) -> C
PyObject* matmul(PyObject* const* v, Py_ssize_t n) {
  count(n, 5);
  const bool is4 = is_packed(v[0]);
  Packed qa;
  at::Tensor xa;
  int a_type = 0;
  int64_t M, K, lda;
  if (is4) {
    qa = packed(v[0], "a");
    M = qa.rows;
    K = qa.cols;
    lda = qa.ld;
  } else {
    xa = tensor(v[0], "a");
    a_type = dtype_of(xa, "a");
    const Plain p = plain(xa, "a");
    M = p.rows;
    K = p.cols;
    lda = p.ld;
  }
  const Packed b = packed(v[1], "b");
  if (b.cols != K) raise(PyExc_ValueError, "%sinner dimensions of a and b differ");
  const int device = is4 ? device_of({&b.data, &b.scales, &qa.data, &qa.scales})
                         : device_of({&b.data, &b.scales, &xa});
  at::Tensor out;
  if (v[2] == Py_None) {
    const long type = PyLong_AsLong(v[3]);
    if (type < MHR_F32 || type > MHR_F16) {
      PyErr_Clear();
      raise(PyExc_TypeError, "%sout_dtype must be float32, bfloat16 or float16");
    }
    out = empty({M, b.rows},
                type == MHR_F32 ? at::kFloat : type == MHR_BF16 ? at::kBFloat16 : at::kHalf, device);
  } else {
    out = tensor(v[2], "out");
    device_of({&b.data, &out});
  }
  const int c_type = dtype_of(out, "out");
  const Plain c = plain(out, "out");
  if (c.rows != M || c.cols != b.rows) raise(PyExc_TypeError, "%sout must be of shape (M, N)");
  void* stream = stream_of(v[4], device);
  if (is4)
    run("gemm_mxfp4", device, [&] {
      return g_product(c_type, qa.d(), qa.s(), b.d(), b.s(), out.data_ptr(), M, b.rows, K, lda,
                       b.ld, c.ld, stream);
    });
  else
    run("gemm_mxfp4_quantized", device, [&] {
      return g_quantized(a_type, xa.data_ptr(), c_type, b.d(), b.s(), out.data_ptr(), M, b.rows, K,
                         lda, b.ld, c.ld, stream);
    });
  return THPVariable_Wrap(out);
}

// moe(x, router, up, down, top, out or None, stream) -> y, experts, weights
PyObject* moe(PyObject* const* v, Py_ssize_t n) {
  count(n, 7);
  const at::Tensor &x = tensor(v[0], "x"), &router = tensor(v[1], "router");
  if (x.scalar_type() != at::kBFloat16 || router.scalar_type() != at::kBFloat16)
    raise(PyExc_TypeError, "%sx and router must be bfloat16");
  const Plain px = plain(x, "x"), pr = plain(router, "router");
  const Packed up = packed(v[2], "up"), down = packed(v[3], "down");
  const int64_t T = px.rows, H = px.cols, E = pr.rows, I = down.cols;
  if (pr.cols != H || up.cols != H || up.rows != 2 * E * I || down.rows != E * H)
    raise(PyExc_ValueError,
          "%ssizes differ: x is T x H, router E x H, up 2 E I x H, down E H x I");
  const long long top = PyLong_AsLongLong(v[4]);
  if (PyErr_Occurred()) throw Raised{};
  if (top < 1 || top > E) raise(PyExc_ValueError, "%stop must be 1 to the number of experts");
  const int device =
      device_of({&x, &router, &up.data, &up.scales, &down.data, &down.scales});
  at::Tensor out;
  if (v[5] == Py_None) {
    out = empty({T, H}, at::kBFloat16, device);
  } else {
    out = tensor(v[5], "out");
    device_of({&x, &out});
  }
  const Plain py = plain(out, "out");
  if (out.scalar_type() != at::kBFloat16 || py.rows != T || py.cols != H)
    raise(PyExc_TypeError, "%sout must be bfloat16 of x's shape");
  at::Tensor experts = empty({T, top}, at::kInt, device);
  at::Tensor weights = empty({T, top}, at::kFloat, device);
  void* stream = stream_of(v[6], device);
  run("gemm_mxfp4_moe", device, [&] {
    return g_moe(static_cast<const uint16_t*>(x.data_ptr()), px.ld,
                 static_cast<const uint16_t*>(router.data_ptr()), pr.ld, up.d(), up.s(), up.ld,
                 down.d(), down.s(), down.ld, static_cast<uint16_t*>(out.data_ptr()), py.ld,
                 static_cast<int32_t*>(experts.data_ptr()),
                 static_cast<float*>(weights.data_ptr()), T, E, top, H, I, stream);
  });
  return Py_BuildValue("NNN", THPVariable_Wrap(out), THPVariable_Wrap(experts),
                       THPVariable_Wrap(weights));
}

// init(addresses of the four entry points, MxFp4Matrix, GemmError)
PyObject* init(PyObject* const* a, Py_ssize_t n) {
  count(n, 6);
  void* p[4];
  for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) throw Raised{};
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[0]);
  g_product = reinterpret_cast<decltype(g_product)>(p[1]);
  g_quantized = reinterpret_cast<decltype(g_quantized)>(p[2]);
  g_moe = reinterpret_cast<decltype(g_moe)>(p[3]);
  Py_INCREF(a[4]);
  Py_INCREF(a[5]);
  g_matrix = a[4];
  g_error = a[5];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<init>("init"), method<quantize>("quantize"),
                           method<matmul>("matmul"), method<moe>("moe"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_binding(void) {
  return PyModule_Create(&g_module);
}
