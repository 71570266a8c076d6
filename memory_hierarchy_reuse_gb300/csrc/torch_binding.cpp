// The tensor-level calls of mxfp4.py and routed.py: argument checks, output
// allocation and marshalling to the C ABI (include/mhr_mxfp4.h, mhr_routed.h),
// nothing else.
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
#include "mhr_routed.h"

namespace {

// The C ABI's entry points, as the package has loaded them, and its classes.
decltype(&gemm_mxfp4_quantize) g_quantize;
decltype(&gemm_mxfp4) g_product;
decltype(&gemm_mxfp4_quantized) g_quantized;
decltype(&gemm_mxfp4_moe) g_moe;
decltype(&gemm_routed_choose) g_choose;
decltype(&gemm_routed_choose_grad) g_choose_grad;
decltype(&gemm_routed_sort) g_sort;
decltype(&gemm_routed_product_scratch) g_product_scratch;
decltype(&gemm_routed_weight_grad_scratch) g_weight_grad_scratch;
decltype(&gemm_routed_product) g_routed_product;
decltype(&gemm_routed_weight_grad) g_weight_grad;
decltype(&gemm_routed_adapters_scratch) g_adapters_scratch;
decltype(&gemm_routed_adapters) g_adapters;
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

// ------------------------------------------------------ by an index per row (routed.py)

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

// A contiguous tensor of one type.
const at::Tensor& array(PyObject* o, at::ScalarType type, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, type == at::kInt ? "%s must be int32" : "%s must be float32", name);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}

// score and group_score as numbers of the C enums, -1 for another name
void score_ok(int64_t score) {
  if (score < 0) raise(PyExc_ValueError, "%sscore must be 'softmax' or 'sigmoid'");
}

// choose(logits, top, score, bias or None, groups, group_top, group_score, renormalize, scale,
//        stream) -> experts, weights
PyObject* choose(PyObject* const* v, Py_ssize_t n) {
  count(n, 10);
  const at::Tensor& logits = tensor(v[0], "logits");
  const int type = dtype_of(logits, "logits");
  const Plain p = plain(logits, "logits");
  const int64_t top = integer(v[1]), score = integer(v[2]);
  score_ok(score);
  int device = device_of({&logits});
  const float* bias = nullptr;
  if (v[3] != Py_None) {
    const at::Tensor& b = array(v[3], at::kFloat, "bias");
    if (b.dim() != 1 || b.size(0) != p.cols) raise(PyExc_ValueError, "%sbias must be of E values");
    device = device_of({&logits, &b});
    bias = static_cast<const float*>(b.data_ptr());
  }
  const int64_t groups = integer(v[4]), group_top = integer(v[5]), group_score = integer(v[6]);
  if (groups < 1 || p.cols % groups || group_top < 1 || group_top > groups)
    raise(PyExc_ValueError, "%sgroups must divide the experts, group_top be 1 to groups");
  if (group_score < 0) raise(PyExc_ValueError, "%sgroup_score must be 'max' or 'top2'");
  if (top < 1 || top > group_top * (p.cols / groups))
    raise(PyExc_ValueError, "%stop must be 1 to the number of experts in group_top groups");
  const bool renormalize = truth(v[7]);
  const float scale = number(v[8]);
  void* stream = stream_of(v[9], device);
  at::Tensor experts = empty({p.rows, top}, at::kInt, device);
  at::Tensor weights = empty({p.rows, top}, at::kFloat, device);
  run("gemm_routed_choose", device, [&] {
    return g_choose(type, logits.data_ptr(), p.rows, p.cols, p.ld, static_cast<int>(score), bias,
                    groups, group_top, static_cast<int>(group_score), top, renormalize, scale,
                    static_cast<int32_t*>(experts.data_ptr()),
                    static_cast<float*>(weights.data_ptr()), stream);
  });
  return Py_BuildValue("NN", THPVariable_Wrap(experts), THPVariable_Wrap(weights));
}

// choose_grad(logits, experts, grad_weights, score, renormalize, scale, out or None, stream)
PyObject* choose_grad(PyObject* const* v, Py_ssize_t n) {
  count(n, 8);
  const at::Tensor& logits = tensor(v[0], "logits");
  const int type = dtype_of(logits, "logits");
  const Plain p = plain(logits, "logits");
  const at::Tensor& experts = array(v[1], at::kInt, "experts");
  const at::Tensor& grad = array(v[2], at::kFloat, "grad_weights");
  if (experts.dim() != 2 || experts.size(0) != p.rows || grad.sizes() != experts.sizes())
    raise(PyExc_ValueError, "%sexperts and grad_weights must be T x top");
  const int64_t top = experts.size(1), score = integer(v[3]);
  score_ok(score);
  const bool renormalize = truth(v[4]);
  const float scale = number(v[5]);
  const int device = device_of({&logits, &experts, &grad});
  at::Tensor out;
  if (v[6] == Py_None) {
    out = empty({p.rows, p.cols}, logits.scalar_type(), device);
  } else {
    out = tensor(v[6], "out");
    device_of({&logits, &out});
  }
  const Plain po = plain(out, "out");
  if (out.scalar_type() != logits.scalar_type() || po.rows != p.rows || po.cols != p.cols)
    raise(PyExc_TypeError, "%sout must be of the logits' type and shape");
  void* stream = stream_of(v[7], device);
  run("gemm_routed_choose_grad", device, [&] {
    return g_choose_grad(type, logits.data_ptr(), p.ld,
                         static_cast<const int32_t*>(experts.data_ptr()),
                         static_cast<const float*>(grad.data_ptr()), p.rows, p.cols, top,
                         static_cast<int>(score), renormalize, scale, out.data_ptr(), po.ld,
                         stream);
  });
  return THPVariable_Wrap(out);
}

// sort(experts, count, stream) -> offsets, order
PyObject* sort(PyObject* const* v, Py_ssize_t n) {
  count(n, 3);
  const at::Tensor& experts = array(v[0], at::kInt, "experts");
  const int64_t E = integer(v[1]);
  if (E < 1) raise(PyExc_ValueError, "%scount must be at least 1");
  const int device = device_of({&experts});
  void* stream = stream_of(v[2], device);
  at::Tensor offsets = empty({E + 1}, at::kInt, device);
  at::Tensor order = empty({experts.numel()}, at::kInt, device);
  run("gemm_routed_sort", device, [&] {
    return g_sort(static_cast<const int32_t*>(experts.data_ptr()), experts.numel(), E,
                  static_cast<int32_t*>(offsets.data_ptr()),
                  static_cast<int32_t*>(order.data_ptr()), stream);
  });
  return Py_BuildValue("NN", THPVariable_Wrap(offsets), THPVariable_Wrap(order));
}

// An int32 index per sorted position, or none; *rows is their number once one says it.
const int32_t* index_of(PyObject* o, const char* name, int device, int64_t* rows) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = array(o, at::kInt, name);
  if (t.device() != at::Device(at::kCUDA, static_cast<at::DeviceIndex>(device)))
    raise(PyExc_ValueError, "%soperands must be on one device");
  if (*rows >= 0 && t.numel() != *rows)
    raise(PyExc_ValueError, "%s: as many entries as sorted rows", name);
  *rows = t.numel();
  return static_cast<const int32_t*>(t.data_ptr());
}

// Matrices of one shape: the sizes and strides of a 3-D tensor.
struct Parts {
  int64_t parts, rows, cols, ld, stride;
};
Parts parts(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) raise(PyExc_ValueError, "%s must be 3-D", name);
  Parts p{t.size(0), t.size(1), t.size(2), 0, 0};
  const bool some = p.parts > 0 && p.rows > 0 && p.cols > 0;
  if (some && p.cols > 1 && t.stride(2) != 1)
    raise(PyExc_ValueError, "%s must be row-major (last dimension contiguous)", name);
  p.ld = some && p.rows > 1 ? t.stride(1) : p.cols;
  p.stride = some && p.parts > 1 ? t.stride(0) : p.rows * p.ld;
  if (some && (p.ld < p.cols || p.stride < (p.rows - 1) * p.ld + p.cols))
    raise(PyExc_ValueError, "%s must be row-major (rows or parts overlap)", name);
  return p;
}

// 16-bit operands of one type.
int half_type(const at::Tensor& x, const at::Tensor& w, const char* names) {
  const at::ScalarType t = x.scalar_type();
  if ((t != at::kBFloat16 && t != at::kHalf) || w.scalar_type() != t)
    raise(PyExc_TypeError, "%s must both be bfloat16, or both float16", names);
  return t == at::kBFloat16 ? MHR_BF16 : MHR_F16;
}
at::ScalarType type_number(PyObject* o, at::ScalarType same) {
  if (o == Py_None) return same;
  const long type = PyLong_AsLong(o);
  if (type < MHR_F32 || type > MHR_F16) {
    PyErr_Clear();
    raise(PyExc_TypeError, "%sout_dtype must be float32, bfloat16 or float16");
  }
  return type == MHR_F32 ? at::kFloat : type == MHR_BF16 ? at::kBFloat16 : at::kHalf;
}

// Where both are given, out is of that type.
void out_type_ok(PyObject* out, PyObject* type) {
  if (out != Py_None && type != Py_None &&
      tensor(out, "out").scalar_type() != type_number(type, at::kFloat))
    raise(PyExc_TypeError, "%sout must be of out_dtype");
}

// Scratch of a call on `stream`, of that stream's own memory: what another stream gave
// back to the allocator may still have that stream's work ahead of it.
at::Tensor scratch_for(int64_t bytes, int device, void* stream) {
  if (stream == static_cast<void*>(c10::cuda::getCurrentCUDAStream(device).stream()))
    return empty({bytes}, at::kByte, device);
  c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(
      static_cast<cudaStream_t>(stream), static_cast<c10::DeviceIndex>(device)));
  return empty({bytes}, at::kByte, device);
}

// experts(x, w, offsets, gather, scatter, top, transposed, out or None, out_dtype or None,
//         stream) -> out
PyObject* experts(PyObject* const* v, Py_ssize_t n) {
  count(n, 10);
  const at::Tensor &x = tensor(v[0], "x"), &w = tensor(v[1], "w");
  const int type = half_type(x, w, "x and w");
  const Plain px = plain(x, "x");
  const Parts pw = parts(w, "w");
  out_type_ok(v[7], v[8]);
  const at::Tensor& offsets = array(v[2], at::kInt, "offsets");
  const int device = device_of({&x, &w, &offsets});
  int64_t rows = -1;
  const int32_t* gather = index_of(v[3], "gather", device, &rows);
  const int32_t* scatter = index_of(v[4], "scatter", device, &rows);
  if (rows < 0) rows = px.rows;
  const int64_t top = integer(v[5]);
  if (top < 1) raise(PyExc_ValueError, "%stop must be at least 1");
  const bool transposed = truth(v[6]);
  const int64_t K = transposed ? pw.cols : pw.rows, N = transposed ? pw.rows : pw.cols;
  if (px.cols != K) raise(PyExc_ValueError, "%sinner dimensions of x and w differ");
  if (offsets.dim() != 1 || offsets.numel() != pw.parts + 1)
    raise(PyExc_ValueError, "%soffsets must be of experts + 1 values");
  if (!gather && px.rows != rows) raise(PyExc_ValueError, "%sx must have as many rows as scatter");
  at::Tensor out;
  if (v[7] == Py_None) {
    out = empty({rows, N}, type_number(v[8], x.scalar_type()), device);
  } else {
    out = tensor(v[7], "out");
    device_of({&x, &out});
  }
  const int out_type = dtype_of(out, "out");
  const Plain po = plain(out, "out");
  if (po.cols != N || (!scatter && po.rows != rows))
    raise(PyExc_TypeError, "%sout must be of shape (rows, N)");
  void* stream = stream_of(v[9], device);
  const int64_t bytes = g_product_scratch(x.data_ptr(), px.rows, px.ld, gather != nullptr,
                                          w.data_ptr(), pw.ld, pw.stride, transposed, pw.parts,
                                          rows, K, N);
  const int64_t need = bytes > 0 ? bytes : 0;  // (the call says what -1 is about)
  at::Tensor scratch;
  if (need) scratch = scratch_for(need, device, stream);
  run("gemm_routed_product", device, [&] {
    return g_routed_product(type, x.data_ptr(), px.rows, px.ld, gather, top, w.data_ptr(), pw.ld,
                            pw.stride, transposed, static_cast<const int32_t*>(offsets.data_ptr()),
                            pw.parts, out_type, out.data_ptr(), po.rows, po.ld, scatter, rows, K,
                            N, need ? scratch.data_ptr() : nullptr, need, stream);
  });
  return THPVariable_Wrap(out);
}

// experts_grad(x, grad, offsets, gather, scatter, top, out or None, out_dtype or None, stream)
//     -> out
PyObject* experts_grad(PyObject* const* v, Py_ssize_t n) {
  count(n, 9);
  const at::Tensor &x = tensor(v[0], "x"), &grad = tensor(v[1], "grad");
  const int type = half_type(x, grad, "x and grad");
  const Plain px = plain(x, "x"), pg = plain(grad, "grad");
  out_type_ok(v[6], v[7]);
  const at::Tensor& offsets = array(v[2], at::kInt, "offsets");
  const int device = device_of({&x, &grad, &offsets});
  int64_t rows = -1;
  const int32_t* gather = index_of(v[3], "gather", device, &rows);
  const int32_t* scatter = index_of(v[4], "scatter", device, &rows);
  if (rows < 0) rows = px.rows;
  const int64_t top = integer(v[5]);
  if (top < 1) raise(PyExc_ValueError, "%stop must be at least 1");
  if ((!gather && px.rows != rows) || (!scatter && pg.rows != rows))
    raise(PyExc_ValueError, "%sx and grad must have as many rows as there are sorted ones");
  const int64_t E = offsets.numel() - 1;
  if (offsets.dim() != 1 || E < 1)
    raise(PyExc_ValueError, "%soffsets must be of experts + 1 values");
  at::Tensor out;
  if (v[6] == Py_None) {
    out = empty({E, px.cols, pg.cols}, type_number(v[7], x.scalar_type()), device);
  } else {
    out = tensor(v[6], "out");
    device_of({&x, &out});
  }
  const int out_type = dtype_of(out, "out");
  const Parts po = parts(out, "out");
  if (po.parts != E || po.rows != px.cols || po.cols != pg.cols)
    raise(PyExc_TypeError, "%sout must be of shape (experts, K, N)");
  void* stream = stream_of(v[8], device);
  const int64_t bytes =
      g_weight_grad_scratch(x.data_ptr(), px.rows, px.ld, gather != nullptr, grad.data_ptr(),
                            pg.rows, pg.ld, scatter != nullptr, rows, px.cols, pg.cols);
  const int64_t need = bytes > 0 ? bytes : 0;
  at::Tensor scratch;
  if (need) scratch = scratch_for(need, device, stream);
  run("gemm_routed_weight_grad", device, [&] {
    return g_weight_grad(type, x.data_ptr(), px.rows, px.ld, gather, top, grad.data_ptr(), pg.rows,
                         pg.ld, scatter, static_cast<const int32_t*>(offsets.data_ptr()), E,
                         out_type, out.data_ptr(), po.ld, po.stride, rows, px.cols, pg.cols,
                         need ? scratch.data_ptr() : nullptr, need, stream);
  });
  return THPVariable_Wrap(out);
}

// adapters(y, x, down, up, which, scales or None, out or None, stream) -> out
PyObject* adapters(PyObject* const* v, Py_ssize_t n) {
  count(n, 8);
  const at::Tensor &y = tensor(v[0], "y"), &x = tensor(v[1], "x");
  const at::Tensor &down = tensor(v[2], "down"), &up = tensor(v[3], "up");
  const int out_type = dtype_of(y, "y");
  const int type = half_type(x, down, "x and the adapters");
  half_type(x, up, "x and the adapters");
  const Plain py = plain(y, "y"), px = plain(x, "x");
  const Parts pd = parts(down, "down"), pu = parts(up, "up");
  if (px.rows != py.rows || pd.cols != px.cols || pu.cols != py.cols || pu.parts != pd.parts ||
      pu.rows != pd.rows)
    raise(PyExc_ValueError,
          "%ssizes differ: y is T x N, x T x K, down adapters x rank x K, up adapters x rank x N");
  const at::Tensor& which = array(v[4], at::kInt, "which");
  if (which.dim() != 1 || which.numel() != py.rows)
    raise(PyExc_ValueError, "%swhich must be of T values");
  const int device = device_of({&y, &x, &down, &up, &which});
  const float* scales = nullptr;
  if (v[5] != Py_None) {
    const at::Tensor& s = array(v[5], at::kFloat, "scales");
    if (s.dim() != 1 || s.numel() != pd.parts)
      raise(PyExc_ValueError, "%sscales must be of one value an adapter");
    device_of({&y, &s});
    scales = static_cast<const float*>(s.data_ptr());
  }
  at::Tensor out;
  if (v[6] == Py_None) {
    out = empty({py.rows, py.cols}, y.scalar_type(), device);
  } else {
    out = tensor(v[6], "out");
    device_of({&y, &out});
  }
  const Plain po = plain(out, "out");
  if (out.scalar_type() != y.scalar_type() || po.rows != py.rows || po.cols != py.cols)
    raise(PyExc_TypeError, "%sout must be of y's type and shape");
  void* stream = stream_of(v[7], device);
  const int64_t bytes =
      g_adapters_scratch(type, x.data_ptr(), px.ld, down.data_ptr(), pd.ld, pd.stride,
                         up.data_ptr(), pu.ld, pu.stride, pd.parts, pd.rows, out_type, py.rows,
                         px.cols, py.cols);
  const int64_t need = bytes > 0 ? bytes : 0;  // (the call says what -1 is about)
  at::Tensor scratch;
  if (need) scratch = scratch_for(need, device, stream);
  run("gemm_routed_adapters", device, [&] {
    return g_adapters(type, x.data_ptr(), px.ld, down.data_ptr(), pd.ld, pd.stride, up.data_ptr(),
                      pu.ld, pu.stride, static_cast<const int32_t*>(which.data_ptr()), scales,
                      pd.parts, pd.rows, out_type, y.data_ptr(), py.ld, out.data_ptr(), po.ld,
                      py.rows, px.cols, py.cols, need ? scratch.data_ptr() : nullptr, need, stream);
  });
  return THPVariable_Wrap(out);
}

// init_routed(addresses of the entry points)
PyObject* init_routed(PyObject* const* a, Py_ssize_t n) {
  count(n, 9);
  void* p[9];
  for (int i = 0; i < 9; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) throw Raised{};
  g_choose = reinterpret_cast<decltype(g_choose)>(p[0]);
  g_choose_grad = reinterpret_cast<decltype(g_choose_grad)>(p[1]);
  g_sort = reinterpret_cast<decltype(g_sort)>(p[2]);
  g_product_scratch = reinterpret_cast<decltype(g_product_scratch)>(p[3]);
  g_routed_product = reinterpret_cast<decltype(g_routed_product)>(p[4]);
  g_weight_grad_scratch = reinterpret_cast<decltype(g_weight_grad_scratch)>(p[5]);
  g_weight_grad = reinterpret_cast<decltype(g_weight_grad)>(p[6]);
  g_adapters_scratch = reinterpret_cast<decltype(g_adapters_scratch)>(p[7]);
  g_adapters = reinterpret_cast<decltype(g_adapters)>(p[8]);
  Py_RETURN_NONE;
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
                           method<init_routed>("init_routed"), method<choose>("choose"),
                           method<choose_grad>("choose_grad"), method<sort>("sort"),
                           method<experts>("experts"), method<experts_grad>("experts_grad"),
                           method<adapters>("adapters"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_binding(void) {
  return PyModule_Create(&g_module);
}
