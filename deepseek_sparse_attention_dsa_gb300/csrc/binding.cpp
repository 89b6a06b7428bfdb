// binding.cpp -- torch tensors to the C calls of the 8-bit rows and projections
// (dsa_rmsnorm, dsa_quantize_rows, dsa_quantize_weight, dsa_project_fp8), and to
// those between projections and caches (dsa_rotate, dsa_append_latents,
// dsa_append_kv, dsa_prefix_attend).
//
// A norm of one token takes 3 us on the GPU.  Reading its tensors' shapes,
// types and strides and making its outputs took 15 us in Python; here they take
// a few, and nothing else is done: every number goes into the call's shape
// structure, and a status other than DSA_OK goes to the binding's check.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "dsa.h"

namespace {

PyObject *g_check = nullptr;   // dsa._check(status, what, handle): raises

enum Kind { kValues, kCodes, kScales, kPositions };

// DSA_BF16 / DSA_FP32 for values, 0 for the others; -1: not of this kind.
int type_of(at::ScalarType t, Kind kind) {
  switch (kind) {
    case kValues: return t == at::kBFloat16 ? DSA_BF16 : t == at::kFloat ? DSA_FP32 : -1;
    case kPositions: return t == at::kInt ? 0 : -1;
    case kCodes: return t == at::kByte || t == at::kFloat8_e4m3fn ? 0 : -1;
    default: return t == at::kFloat ? 0 : -1;
  }
}

// Where a call's tensors have to be, and the call itself.
struct Call {
  dsa_ctx_t *ctx;
  dsa_plan_t *plan;
  int device;   // -1: a host-only context, whose tensors are the host's
  dsa_stream_t stream;
  bool other;   // a stream was given: it may not be the current one

  // (handle, device, plan, stream): the first four arguments of every function
  bool take(PyObject *const *args) {
    ctx = static_cast<dsa_ctx_t *>(PyLong_AsVoidPtr(args[0]));
    device = static_cast<int>(PyLong_AsLong(args[1]));
    plan = args[2] == Py_None ? nullptr : static_cast<dsa_plan_t *>(PyLong_AsVoidPtr(args[2]));
    other = args[3] != Py_None;
    if (other) stream = static_cast<dsa_stream_t>(PyLong_AsVoidPtr(args[3]));
    else stream = device < 0 ? nullptr : reinterpret_cast<dsa_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
    return !PyErr_Occurred();
  }
  // A new tensor of the call's stream: memory that the current stream has freed
  // but may still be working on is not written from another.
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    c10::cuda::OptionalCUDAStreamGuard guard;
    if (other && device >= 0)
      guard.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream), device));
    return at::empty(shape, at::TensorOptions().dtype(type).device(device < 0 ? at::Device(at::kCPU)
                                                                             : at::Device(at::kCUDA, device)));
  }
  // Checks the outcome; NULL with an exception, or `result`.
  PyObject *done(dsa_status st, const char *what, PyObject *result) const {
    if (st == DSA_OK) return result;
    Py_XDECREF(result);
    PyObject *r = PyObject_CallFunction(g_check, "isN", static_cast<int>(st), what, PyLong_FromVoidPtr(ctx));
    if (r) {   // (the check raises)
      Py_DECREF(r);
      PyErr_SetString(PyExc_RuntimeError, what);
    }
    return nullptr;
  }
};

bool is_none(PyObject *o) { return o == Py_None; }

bool tensor(PyObject *o, const char *name) {
  if (THPVariable_Check(o)) return true;
  PyErr_Format(PyExc_TypeError, "%s must be a torch tensor", name);
  return false;
}

struct View {
  void *p = nullptr;
  int type = 0;
  int64_t stride[2] = {0, 0};   // of the dimensions before the last
};

// o: a tensor of this kind and shape on the call's device, adjacent in its last dimension.
bool view(const Call &call, PyObject *o, const char *name, Kind kind, at::IntArrayRef shape, View *v) {
  if (!tensor(o, name)) return false;
  const at::Tensor &t = THPVariable_Unpack(o);
  v->type = type_of(t.scalar_type(), kind);
  if (v->type < 0) {
    PyErr_Format(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()),
                 kind == kValues ? "bfloat16 or float32" : kind == kCodes ? "uint8 or float8_e4m3fn"
                 : kind == kPositions ? "int32" : "float32");
    return false;
  }
  if (call.device < 0 ? !t.is_cpu() : !t.is_cuda() || t.get_device() != call.device) {
    PyErr_Format(PyExc_ValueError, "%s is on %s, expected %s %d", name, t.device().str().c_str(),
                 call.device < 0 ? "cpu" : "cuda", call.device);
    return false;
  }
  const at::IntArrayRef have = t.sizes(), strides = t.strides();
  if (have != shape) {
    PyErr_Format(PyExc_ValueError, "%s has the wrong shape (%d dimensions, last %lld)", name, static_cast<int>(have.size()),
                 static_cast<long long>(have.empty() ? 0 : have.back()));
    return false;
  }
  if (shape.back() > 1 && strides.back() != 1) {
    PyErr_Format(PyExc_ValueError, "%s must have adjacent values in its last dimension", name);
    return false;
  }
  if (t.is_neg() || t._is_zerotensor()) {   // (their memory does not hold their values)
    PyErr_Format(PyExc_ValueError, "%s is a view that negates its memory, or has none", name);
    return false;
  }
  for (size_t i = 0; i + 1 < shape.size(); ++i) v->stride[i] = strides[i];
  v->p = t.data_ptr();
  return true;
}

// The tensor given as an output, or a new one for None; `kept` holds it.
bool output(const Call &call, PyObject *o, const char *name, Kind kind, at::IntArrayRef shape, at::ScalarType type, View *v,
            PyObject **kept) {
  if (!is_none(o)) {
    if (!view(call, o, name, kind, shape, v)) return false;
    *kept = Py_NewRef(o);
    return true;
  }
  at::Tensor t = call.make(shape, type);
  v->p = t.data_ptr();
  v->type = type_of(type, kind);
  int64_t n = 1;
  for (size_t i = shape.size() - 1; i > 0; --i) v->stride[i - 1] = n *= shape[i];
  *kept = THPVariable_Wrap(std::move(t));
  return *kept != nullptr;
}

// References held until the call is made, dropped on an error.
struct Kept {
  PyObject *o[4] = {nullptr, nullptr, nullptr, nullptr};
  ~Kept() {
    for (PyObject *p : o) Py_XDECREF(p);
  }
  PyObject *take(int i) {
    PyObject *p = o[i];
    o[i] = nullptr;
    return p;
  }
};

int64_t groups(int64_t n) { return (n + 127) / 128; }

// One value, or a tuple of up to three, of what `kept` holds.
PyObject *result(Kept &kept, std::initializer_list<int> which) {
  if (which.size() == 1) return kept.take(*which.begin());
  PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(which.size()));
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (int w : which) PyTuple_SET_ITEM(t, i++, kept.take(w));
  return t;
}

bool wants(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// rmsnorm(handle, device, plan, stream, x, weight, eps, residual, residual_out,
//   out, out_dtype, codes, scales, quantize): with quantize (codes, scales[,
//   residual_out]) and out only where it is given, else out or (out, residual_out)
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 14) || !call.take(a) || !tensor(a[4], "x")) return nullptr;
  const at::Tensor &x = THPVariable_Unpack(a[4]);
  if (x.dim() != 2) {
    PyErr_SetString(PyExc_ValueError, "x must be (rows, width)");
    return nullptr;
  }
  const at::IntArrayRef shape = x.sizes();
  const int64_t width = shape[1];
  const bool quantize = PyObject_IsTrue(a[13]) == 1, with_residual = !is_none(a[7]);
  View vx, vw, vr, vro, vo, vc, vs;
  Kept kept;
  if (!view(call, a[4], "x", kValues, shape, &vx)) return nullptr;
  if (!is_none(a[5]) && !view(call, a[5], "weight", kValues, {width}, &vw)) return nullptr;
  if (with_residual) {
    if (!view(call, a[7], "residual", kValues, shape, &vr) ||
        !output(call, a[8], "residual_out", kValues, shape, vr.type == DSA_BF16 ? at::kBFloat16 : at::kFloat, &vro, &kept.o[0]))
      return nullptr;
    if (vro.type != vr.type) {
      PyErr_SetString(PyExc_TypeError, "residual_out must have the residual's dtype");
      return nullptr;
    }
  } else if (!is_none(a[8])) {
    PyErr_SetString(PyExc_ValueError, "residual_out needs a residual");
    return nullptr;
  }
  if (!quantize || !is_none(a[9])) {
    at::ScalarType type = at::kBFloat16;
    if (is_none(a[9])) {
      if (!THPDtype_Check(a[10]) || type_of(type = reinterpret_cast<THPDtype *>(a[10])->scalar_type, kValues) < 0) {
        PyErr_SetString(PyExc_TypeError, "out_dtype must be bfloat16 or float32");
        return nullptr;
      }
    }
    if (!output(call, a[9], "out", kValues, shape, type, &vo, &kept.o[1])) return nullptr;
  }
  if (quantize && (!output(call, a[11], "codes", kCodes, shape, at::kByte, &vc, &kept.o[2]) ||
                   !output(call, a[12], "scales", kScales, {shape[0], groups(width)}, at::kFloat, &vs, &kept.o[3])))
    return nullptr;
  const double eps = PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred()) return nullptr;
  dsa_norm_t s{};
  s.rows = shape[0];
  s.width = width > INT32_MAX ? INT32_MAX : static_cast<int32_t>(width);   // (refused there)
  s.x_type = vx.type, s.weight_type = vw.type, s.residual_type = vr.type, s.out_type = vo.type;
  s.eps = static_cast<float>(eps);
  s.x_stride = vx.stride[0], s.residual_stride = vr.stride[0], s.residual_out_stride = vro.stride[0];
  s.out_stride = vo.stride[0], s.codes_stride = vc.stride[0], s.scales_stride = vs.stride[0];
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_rmsnorm(call.ctx, call.plan, &s, vx.p, vw.p, vr.p, vro.p, vo.p, vc.p, static_cast<float *>(vs.p), call.stream);
  Py_END_ALLOW_THREADS
  PyObject *r = quantize ? (with_residual ? result(kept, {2, 3, 0}) : result(kept, {2, 3}))
                         : (with_residual ? result(kept, {1, 0}) : result(kept, {1}));
  return call.done(st, "dsa_rmsnorm", r);
  END_HANDLE_TH_ERRORS
}

// quantize_rows(handle, device, plan, stream, x, codes, scales) -> (codes, scales)
PyObject *quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 7) || !call.take(a) || !tensor(a[4], "x")) return nullptr;
  const at::Tensor &x = THPVariable_Unpack(a[4]);
  if (x.dim() != 2) {
    PyErr_SetString(PyExc_ValueError, "x must be (rows, width)");
    return nullptr;
  }
  const at::IntArrayRef shape = x.sizes();
  View vx, vc, vs;
  Kept kept;
  if (!view(call, a[4], "x", kValues, shape, &vx) ||
      !output(call, a[5], "codes", kCodes, shape, at::kByte, &vc, &kept.o[0]) ||
      !output(call, a[6], "scales", kScales, {shape[0], groups(shape[1])}, at::kFloat, &vs, &kept.o[1]))
    return nullptr;
  if (shape[1] > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "x has too wide rows");
    return nullptr;
  }
  dsa_rows_t s{};
  s.rows = shape[0], s.width = static_cast<int32_t>(shape[1]), s.x_type = vx.type;
  s.x_stride = vx.stride[0], s.codes_stride = vc.stride[0], s.scales_stride = vs.stride[0];
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_quantize_rows(call.ctx, call.plan, &s, vx.p, vc.p, static_cast<float *>(vs.p), call.stream);
  Py_END_ALLOW_THREADS
  return call.done(st, "dsa_quantize_rows", result(kept, {0, 1}));
  END_HANDLE_TH_ERRORS
}

bool fits(int64_t batch, int64_t n, int64_t k) {
  if (batch <= INT32_MAX && n <= INT32_MAX && k <= INT32_MAX) return true;
  PyErr_SetString(PyExc_ValueError, "a dimension has too many elements");
  return false;
}

// quantize_weight(handle, device, plan, stream, w, codes, scales) -> (codes, scales)
PyObject *quantize_weight(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 7) || !call.take(a) || !tensor(a[4], "w")) return nullptr;
  const at::Tensor &w = THPVariable_Unpack(a[4]);
  const at::IntArrayRef shape = w.sizes();
  if (shape.size() != 2 && shape.size() != 3) {
    PyErr_SetString(PyExc_ValueError, "w must be (n, k) or (batch, n, k)");
    return nullptr;
  }
  const bool many = shape.size() == 3;
  const int64_t rows = shape[many], k = shape[many + 1], batch = many ? shape[0] : 1;
  const int64_t s3[3] = {batch, groups(rows), groups(k)};
  const at::IntArrayRef s_shape(s3 + (many ? 0 : 1), many ? 3 : 2);
  View vw, vc, vs;
  Kept kept;
  if (!fits(batch, rows, k) || !view(call, a[4], "w", kValues, shape, &vw) ||
      !output(call, a[5], "codes", kCodes, shape, at::kByte, &vc, &kept.o[0]) ||
      !output(call, a[6], "scales", kScales, s_shape, at::kFloat, &vs, &kept.o[1]))
    return nullptr;
  dsa_weight_t s{};
  s.batch = static_cast<int32_t>(batch), s.n = static_cast<int32_t>(rows), s.k = static_cast<int32_t>(k);
  s.w_type = vw.type;
  s.w_stride = vw.stride[many], s.codes_stride = vc.stride[many], s.scales_stride = vs.stride[many];
  if (many) s.w_batch = vw.stride[0], s.codes_batch = vc.stride[0], s.scales_batch = vs.stride[0];
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_quantize_weight(call.ctx, &s, vw.p, vc.p, static_cast<float *>(vs.p), call.stream);
  Py_END_ALLOW_THREADS
  return call.done(st, "dsa_quantize_weight", result(kept, {0, 1}));
  END_HANDLE_TH_ERRORS
}

// project_fp8(handle, device, plan, stream, a, a_scale, w, w_scale, out,
//   out_dtype, query) -> out; with query whether it would run on the tensor cores
PyObject *project_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 11) || !call.take(a) || !tensor(a[4], "a") || !tensor(a[6], "w")) return nullptr;
  const at::IntArrayRef sa = THPVariable_Unpack(a[4]).sizes(), sw = THPVariable_Unpack(a[6]).sizes();
  const bool many = sw.size() == 3;
  if ((sw.size() != 2 && !many) || sa.size() != sw.size()) {
    PyErr_SetString(PyExc_ValueError, "a (rows, k) goes with w (n, k), a (rows, batch, k) with w (batch, n, k)");
    return nullptr;
  }
  const int64_t rows = sa[0], batch = many ? sw[0] : 1, cols = sw[many], k = sw[many + 1];
  const int64_t a3[3] = {rows, batch, k}, as3[3] = {rows, batch, groups(k)}, a2[2] = {rows, k}, as2[2] = {rows, groups(k)};
  const int64_t ws3[3] = {batch, groups(cols), groups(k)}, o3[3] = {rows, batch, cols}, o2[2] = {rows, cols};
  View va, vas, vw, vws, vo;
  Kept kept;
  at::ScalarType type = at::kBFloat16;
  if (is_none(a[8]) &&
      (!THPDtype_Check(a[9]) || type_of(type = reinterpret_cast<THPDtype *>(a[9])->scalar_type, kValues) < 0)) {
    PyErr_SetString(PyExc_TypeError, "out_dtype must be bfloat16 or float32");
    return nullptr;
  }
  auto of = [&](const int64_t *three, const int64_t *two) { return many ? at::IntArrayRef(three, 3) : at::IntArrayRef(two, 2); };
  if (!fits(batch, cols, k) || !view(call, a[4], "a", kCodes, of(a3, a2), &va) ||
      !view(call, a[5], "a_scale", kScales, of(as3, as2), &vas) || !view(call, a[6], "w", kCodes, sw, &vw) ||
      !view(call, a[7], "w_scale", kScales, of(ws3, ws3 + 1), &vws) ||
      !output(call, a[8], "out", kValues, of(o3, o2), type, &vo, &kept.o[0]))
    return nullptr;
  dsa_project_t s{};
  s.rows = rows, s.batch = static_cast<int32_t>(batch), s.n = static_cast<int32_t>(cols), s.k = static_cast<int32_t>(k);
  s.out_type = vo.type;
  s.a_stride = va.stride[0], s.a_scale_stride = vas.stride[0], s.out_stride = vo.stride[0];
  s.w_stride = vw.stride[many], s.w_scale_stride = vws.stride[many];
  if (many) {
    s.a_batch = va.stride[1], s.a_scale_batch = vas.stride[1], s.out_batch = vo.stride[1];
    s.w_batch = vw.stride[0], s.w_scale_batch = vws.stride[0];
  }
  if (PyObject_IsTrue(a[10]) == 1) return PyBool_FromLong(dsa_project_on_tensor_cores(&s, va.p, vw.p));
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_project_fp8(call.ctx, call.plan, &s, va.p, static_cast<const float *>(vas.p), vw.p,
                       static_cast<const float *>(vws.p), vo.p, call.stream);
  Py_END_ALLOW_THREADS
  return call.done(st, "dsa_project_fp8", result(kept, {0}));
  END_HANDLE_TH_ERRORS
}

int64_t integer(PyObject *o) { return PyLong_AsLongLong(o); }
// (out of an int's range: refused by the call)
int32_t small(PyObject *o) { return static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(integer(o), -1), INT32_MAX)); }
template <typename T>
T *handle(PyObject *o) { return is_none(o) ? nullptr : static_cast<T *>(PyLong_AsVoidPtr(o)); }

// A cache: contiguous, of this type (bf16, or packed bytes) and at least this many bytes.
bool cache(const Call &call, PyObject *o, const char *name, bool packed, int64_t bytes, void **p) {
  if (!tensor(o, name)) return false;
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.scalar_type() != (packed ? at::kByte : at::kBFloat16)) {
    PyErr_Format(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()), packed ? "uint8" : "bfloat16");
    return false;
  }
  if (call.device < 0 ? !t.is_cpu() : !t.is_cuda() || t.get_device() != call.device) {
    PyErr_Format(PyExc_ValueError, "%s is on %s, expected %s %d", name, t.device().str().c_str(),
                 call.device < 0 ? "cpu" : "cuda", call.device);
    return false;
  }
  if (!t.is_contiguous() || t.is_neg() || t._is_zerotensor()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return false;
  }
  if (static_cast<int64_t>(t.nbytes()) < bytes) {
    PyErr_Format(PyExc_ValueError, "%s has %lld bytes, the plan's pages take %lld", name, static_cast<long long>(t.nbytes()),
                 static_cast<long long>(bytes));
    return false;
  }
  *p = t.data_ptr();
  return true;
}

// rotary(handle, device, plan, stream, table, x, positions, offset, layout, inverse, out) -> out
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 11) || !call.take(a) || !tensor(a[5], "x")) return nullptr;
  const at::Tensor &x = THPVariable_Unpack(a[5]);
  if (x.dim() != 2 && x.dim() != 3) {
    PyErr_SetString(PyExc_ValueError, "x must be (rows, heads, width) or (rows, width)");
    return nullptr;
  }
  const at::IntArrayRef shape = x.sizes();
  const bool many = shape.size() == 3;
  View vx, vp, vo;
  Kept kept;
  if (!view(call, a[5], "x", kValues, shape, &vx) ||
      (!is_none(a[6]) && !view(call, a[6], "positions", kPositions, {shape[0]}, &vp)) ||
      !output(call, a[10], "out", kValues, shape, x.scalar_type(), &vo, &kept.o[0]))
    return nullptr;
  if (vo.type != vx.type) {
    PyErr_SetString(PyExc_TypeError, "out must have x's dtype");
    return nullptr;
  }
  if ((many && shape[1] > INT32_MAX) || shape.back() > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "a dimension has too many elements");
    return nullptr;
  }
  dsa_rotate_t s{};
  s.rows = shape[0], s.heads = many ? static_cast<int32_t>(shape[1]) : 1, s.width = static_cast<int32_t>(shape.back());
  s.offset = small(a[7]), s.layout = small(a[8]), s.inverse = PyObject_IsTrue(a[9]) == 1, s.type = vx.type;
  s.x_stride = vx.stride[0], s.out_stride = vo.stride[0];
  if (many) s.x_head = vx.stride[1], s.out_head = vo.stride[1];
  const dsa_rotary_t *table = handle<dsa_rotary_t>(a[4]);
  if (PyErr_Occurred()) return nullptr;
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_rotate(call.ctx, call.plan, table, &s, vx.p, static_cast<const int32_t *>(vp.p), vo.p, call.stream);
  Py_END_ALLOW_THREADS
  return call.done(st, "dsa_rotate", result(kept, {0}));
  END_HANDLE_TH_ERRORS
}

// The index keys of an append: (keys, index_dim, index_cache, packed, bytes) at a[0 .. 4].
bool append_keys(const Call &call, PyObject *const *a, int64_t rows, dsa_append_t *s, void **keys, void **index_cache) {
  *keys = *index_cache = nullptr;
  if (is_none(a[0]) && is_none(a[2])) return true;
  View v;
  if (!view(call, a[0], "keys", kValues, {rows, integer(a[1])}, &v) ||
      !cache(call, a[2], "index_cache", PyObject_IsTrue(a[3]) == 1, integer(a[4]), index_cache))
    return false;
  *keys = v.p, s->key_type = v.type, s->keys_stride = v.stride[0];
  return true;
}

// append_latents(handle, device, plan, stream, table, rows, c, kv_lora_rank, k_pe, rope_dim, latent_cache, packed,
//   bytes, keys, index_dim, index_cache, packed, bytes, layout, key_layout, key_offset)
PyObject *append_latents(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 21) || !call.take(a)) return nullptr;
  const int64_t rows = integer(a[5]);
  dsa_append_t s{};
  void *keys, *index_cache, *latent_cache = nullptr;
  View vc, vk;
  if (!is_none(a[6]) || !is_none(a[8]) || !is_none(a[10])) {
    const int64_t rope = integer(a[9]);
    if (!view(call, a[6], "c", kValues, {rows, integer(a[7])}, &vc) ||
        !((rope == 0 && is_none(a[8])) || view(call, a[8], "k_pe", kValues, {rows, rope}, &vk)) ||
        !cache(call, a[10], "latent_cache", PyObject_IsTrue(a[11]) == 1, integer(a[12]), &latent_cache))
      return nullptr;
    s.c_type = vc.type, s.k_pe_type = vk.type, s.c_stride = vc.stride[0], s.k_pe_stride = vk.stride[0];
  }
  if (!append_keys(call, a + 13, rows, &s, &keys, &index_cache)) return nullptr;
  s.layout = small(a[18]), s.key_layout = small(a[19]), s.key_offset = small(a[20]);
  const dsa_rotary_t *table = handle<dsa_rotary_t>(a[4]);
  if (PyErr_Occurred()) return nullptr;
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_append_latents(call.ctx, call.plan, table, &s, vc.p, vk.p, latent_cache, keys, index_cache, call.stream);
  Py_END_ALLOW_THREADS
  return call.done(st, "dsa_append_latents", Py_NewRef(Py_None));
  END_HANDLE_TH_ERRORS
}

// append_kv(handle, device, plan, stream, table, rows, kv_heads, head_dim, k, v, kv_cache, bytes,
//   keys, index_dim, index_cache, packed, bytes, layout, kv_offset, key_layout, key_offset)
PyObject *append_kv(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 21) || !call.take(a)) return nullptr;
  const int64_t rows = integer(a[5]);
  dsa_append_t s{};
  dsa_msa_shape_t msa{};
  msa.kv_heads = small(a[6]), msa.head_dim = small(a[7]);
  void *keys, *index_cache, *kv_cache;
  View vk, vv;
  const int64_t shape[3] = {rows, msa.kv_heads, msa.head_dim};
  if (!view(call, a[8], "k", kValues, shape, &vk) || !view(call, a[9], "v", kValues, shape, &vv) ||
      !cache(call, a[10], "kv_cache", false, integer(a[11]), &kv_cache) ||
      !append_keys(call, a + 12, rows, &s, &keys, &index_cache))
    return nullptr;
  if (vk.type != vv.type) {
    PyErr_SetString(PyExc_TypeError, "k and v must have the same dtype");
    return nullptr;
  }
  s.kv_type = vk.type, s.k_stride = vk.stride[0], s.k_head = vk.stride[1], s.v_stride = vv.stride[0], s.v_head = vv.stride[1];
  s.layout = small(a[17]), s.kv_offset = small(a[18]), s.key_layout = small(a[19]), s.key_offset = small(a[20]);
  const dsa_rotary_t *table = handle<dsa_rotary_t>(a[4]);
  if (PyErr_Occurred()) return nullptr;
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_append_kv(call.ctx, call.plan, table, &msa, &s, vk.p, vv.p, kv_cache, keys, index_cache, call.stream);
  Py_END_ALLOW_THREADS
  return call.done(st, "dsa_append_kv", Py_NewRef(Py_None));
  END_HANDLE_TH_ERRORS
}

// prefix_attend(handle, device, None, stream, prefix plan, rows, q_heads, head_dim, q, kv_cache, bytes, sm_scale, out) -> out
PyObject *prefix_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call call;
  if (!wants(n, 13) || !call.take(a)) return nullptr;
  const int64_t shape[3] = {integer(a[5]), integer(a[6]), integer(a[7])};
  const dsa_prefix_plan_t *pp = handle<dsa_prefix_plan_t>(a[4]);
  const int64_t bytes = integer(a[10]);
  const double scale = PyFloat_AsDouble(a[11]);
  if (PyErr_Occurred()) return nullptr;
  void *kv_cache;
  View vq, vo;
  Kept kept;
  if (!view(call, a[8], "q", kValues, shape, &vq) || !cache(call, a[9], "kv_cache", false, bytes, &kv_cache) ||
      !output(call, a[12], "out", kValues, shape, at::kBFloat16, &vo, &kept.o[0]))
    return nullptr;
  if (vq.type != DSA_BF16 || vo.type != DSA_BF16) {
    PyErr_SetString(PyExc_TypeError, "q and out must be bfloat16");
    return nullptr;
  }
  const bool dense = THPVariable_Unpack(a[8]).is_contiguous() && (is_none(a[12]) || THPVariable_Unpack(a[12]).is_contiguous());
  if (!dense) {
    PyErr_SetString(PyExc_ValueError, "q and out must be contiguous");
    return nullptr;
  }
  dsa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsa_prefix_attend(call.ctx, pp, vq.p, kv_cache, static_cast<float>(scale), vo.p, call.stream);
  Py_END_ALLOW_THREADS
  return call.done(st, "dsa_prefix_attend", result(kept, {0}));
  END_HANDLE_TH_ERRORS
}

PyObject *set_check(PyObject *, PyObject *f) {
  Py_INCREF(f);
  Py_XSETREF(g_check, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rmsnorm)), METH_FASTCALL, nullptr},
    {"quantize_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(quantize_rows)), METH_FASTCALL, nullptr},
    {"quantize_weight", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(quantize_weight)), METH_FASTCALL, nullptr},
    {"project_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(project_fp8)), METH_FASTCALL, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rotary)), METH_FASTCALL, nullptr},
    {"append_latents", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(append_latents)), METH_FASTCALL, nullptr},
    {"append_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(append_kv)), METH_FASTCALL, nullptr},
    {"prefix_attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(prefix_attend)), METH_FASTCALL, nullptr},
    {"set_check", set_check, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dsa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dsa_binding() { return PyModule_Create(&module); }
