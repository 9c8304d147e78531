// Calls of the operators around the layer from Python without its overhead:
// the checks, allocations and the C call of binding.py's functions for the
// ordinary case, tensors on the current device and its current stream. A call
// that is anything else, or wrong, returns None and binding.py makes it (or
// explains what is wrong). A call that the library refuses returns its code.
//
// A selection of one token costs 5 us on the host this way, through ctypes and
// three torch calls 12; the kernel takes 3.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/rawint4_moe.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int64_t kGroup = 32;  // columns under one scale of a checkpoint

int type_of(ScalarType t) {
  if (t == ScalarType::Float) return RAWINT4_TYPE_F32;
  if (t == ScalarType::BFloat16) return RAWINT4_TYPE_BF16;
  if (t == ScalarType::Half) return RAWINT4_TYPE_F16;
  return -1;
}

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// What a call works on: the current device, if the first tensor lies there.
struct Here {
  c10::DeviceIndex device = -1;
  bool at(const Tensor& t) {
    if (!t.is_cuda()) return false;
    if (device < 0) {
      device = t.get_device();
      return device == c10::cuda::current_device();
    }
    return t.get_device() == device;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
  Tensor empty(at::IntArrayRef size, ScalarType type) const {
    return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, device), std::nullopt);
  }
};

// [rows, width] of fp32, bf16 or fp16 with dense rows; fills the pitch.
bool rows_ok(Here& here, const Tensor* t, int64_t* pitch) {
  if (!t || t->dim() != 2 || type_of(t->scalar_type()) < 0 || !here.at(*t)) return false;
  const int64_t rows = t->size(0), width = t->size(1);
  if (rows > INT32_MAX || width > INT32_MAX || (width > 1 && t->stride(1) != 1)) return false;
  *pitch = rows <= 1 ? width : t->stride(0);
  return *pitch >= width;
}

bool dense(Here& here, const Tensor* t, ScalarType type, at::IntArrayRef size) {
  return t && t->scalar_type() == type && here.at(*t) && t->sizes() == size && t->is_contiguous();
}

// None, or a dense [width] vector.
bool vector_ok(Here& here, PyObject* o, int64_t width, const Tensor** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const Tensor* t = tensor(o);
  if (!t || type_of(t->scalar_type()) < 0 || !dense(here, t, t->scalar_type(), {width})) return false;
  *out = t;
  return true;
}

template <class T = void>
T* data(const Tensor* t) {
  return t && t->numel() ? static_cast<T*>(t->data_ptr()) : nullptr;
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// A new tuple of the tensors; undefined ones become None.
PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// The interpreter's lock is let go while results are allocated and the library
// is called: both may wait (for memory, for room in the stream's queue of
// launches), and other threads run on meanwhile. No Python object is touched.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

PyObject* refused(int code) { return PyLong_FromLong(code); }

// The selection's configuration (a ctypes structure), for scores of a type.
bool select_cfg(PyObject* o, ScalarType type, rawint4_moe_select_cfg* cfg) {
  Py_buffer view;
  if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    return false;
  }
  const bool ok = view.len == (Py_ssize_t)sizeof(*cfg);
  if (ok) std::memcpy(cfg, view.buf, sizeof(*cfg));
  PyBuffer_Release(&view);
  cfg->type = type_of(type);
  return ok;
}

// router_select(scores, cfg, bias, counts)
PyObject* router_select(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Here here;
  int64_t pitch = 0;
  rawint4_moe_select_cfg cfg;
  const Tensor* scores = n == 4 ? tensor(args[0]) : nullptr;
  if (!rows_ok(here, scores, &pitch) || !select_cfg(args[1], scores->scalar_type(), &cfg) ||
      scores->size(1) != cfg.experts || cfg.top_k < 1)
    Py_RETURN_NONE;
  const Tensor *bias = nullptr, *counts = nullptr;
  if (args[2] != Py_None && !dense(here, bias = tensor(args[2]), ScalarType::Float, {cfg.experts})) Py_RETURN_NONE;
  if (args[3] != Py_None && !dense(here, counts = tensor(args[3]), ScalarType::Int, {cfg.experts})) Py_RETURN_NONE;
  const int64_t q = scores->size(0);
  Tensor ids, w;
  int rc;
  {
    const Unlocked unlocked;
    ids = here.empty({q, cfg.top_k}, ScalarType::Long);
    w = here.empty({q, cfg.top_k}, ScalarType::Float);
    rc = rawint4_moe_router_select(&cfg, data(scores), pitch, (int32_t)q, data<const float>(bias), data<int64_t>(&ids),
                                   data<float>(&w), data<int32_t>(counts), here.stream());
  }
  return rc == RAWINT4_OK ? tuple_of({ids, w}) : refused(rc);
  END_HANDLE_TH_ERRORS
}

// router_select_bwd(scores, cfg, ids, grad_route)
PyObject* router_select_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Here here;
  int64_t pitch = 0;
  rawint4_moe_select_cfg cfg;
  const Tensor* scores = n == 4 ? tensor(args[0]) : nullptr;
  if (!rows_ok(here, scores, &pitch) || !select_cfg(args[1], scores->scalar_type(), &cfg) ||
      scores->size(1) != cfg.experts)
    Py_RETURN_NONE;
  const int64_t q = scores->size(0);
  const Tensor *ids = tensor(args[2]), *grad = tensor(args[3]);
  if (!dense(here, ids, ScalarType::Long, {q, cfg.top_k}) || !dense(here, grad, ScalarType::Float, {q, cfg.top_k}))
    Py_RETURN_NONE;
  Tensor out;
  int rc;
  {
    const Unlocked unlocked;
    out = here.empty({q, cfg.experts}, scores->scalar_type());
    rc = rawint4_moe_router_select_bwd(&cfg, data(scores), pitch, (int32_t)q, data<const int64_t>(ids),
                                       data<const float>(grad), data(&out), here.stream());
  }
  return rc == RAWINT4_OK ? wrap(out) : refused(rc);
  END_HANDLE_TH_ERRORS
}

// ckpt8_save(x, format) -> (codes, scales)
PyObject* ckpt8_save(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Here here;
  int64_t pitch = 0;
  const Tensor* x = n == 2 ? tensor(args[0]) : nullptr;
  if (!rows_ok(here, x, &pitch)) Py_RETURN_NONE;
  const int64_t rows = x->size(0), width = x->size(1);
  const int32_t format = (int32_t)PyLong_AsLong(args[1]);
  Tensor codes, scales;
  int rc;
  {
    const Unlocked unlocked;
    codes = here.empty({rows, width}, ScalarType::Byte);
    scales = here.empty({rows, (width + kGroup - 1) / kGroup}, ScalarType::Byte);
    rc = rawint4_ckpt8_save(format, type_of(x->scalar_type()), data(x), pitch, rows, (int32_t)width,
                            data<uint8_t>(&codes), data<uint8_t>(&scales), here.stream());
  }
  return rc == RAWINT4_OK ? tuple_of({codes, scales}) : refused(rc);
  END_HANDLE_TH_ERRORS
}

bool ckpt_ok(Here& here, const Tensor* codes, const Tensor* scales) {
  return codes && codes->dim() == 2 && codes->size(0) <= INT32_MAX && codes->size(1) <= INT32_MAX &&
         dense(here, codes, ScalarType::Byte, codes->sizes()) &&
         dense(here, scales, ScalarType::Byte, {codes->size(0), (codes->size(1) + kGroup - 1) / kGroup});
}

// ckpt8_load(codes, scales, format, dtype)
PyObject* ckpt8_load(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Here here;
  const Tensor *codes = n == 4 ? tensor(args[0]) : nullptr, *scales = n == 4 ? tensor(args[1]) : nullptr;
  if (!ckpt_ok(here, codes, scales) || !THPDtype_Check(args[3])) Py_RETURN_NONE;
  const ScalarType type = reinterpret_cast<THPDtype*>(args[3])->scalar_type;
  if (type_of(type) < 0) Py_RETURN_NONE;
  const int64_t rows = codes->size(0), width = codes->size(1);
  const int32_t format = (int32_t)PyLong_AsLong(args[2]);
  Tensor out;
  int rc;
  {
    const Unlocked unlocked;
    out = here.empty({rows, width}, type);
    rc = rawint4_ckpt8_load(format, data<const uint8_t>(codes), data<const uint8_t>(scales), rows, (int32_t)width,
                            type_of(type), data(&out), here.stream());
  }
  return rc == RAWINT4_OK ? wrap(out) : refused(rc);
  END_HANDLE_TH_ERRORS
}

// The input of a norm: a tensor, or (x None) a checkpoint's codes, scales and format.
struct NormInput {
  const Tensor *x = nullptr, *codes = nullptr;
  rawint4_ckpt8 ckpt{};
  int64_t rows = 0, width = 0, pitch = 0;
  bool take(Here& here, PyObject* const* args) {
    if (args[0] != Py_None) {
      x = tensor(args[0]);
      if (!rows_ok(here, x, &pitch)) return false;
      rows = x->size(0);
      width = x->size(1);
      return true;
    }
    codes = tensor(args[1]);
    const Tensor* scales = tensor(args[2]);
    if (!ckpt_ok(here, codes, scales) || PyLong_AsLong(args[3]) < 0) return false;
    rows = codes->size(0);
    width = codes->size(1);
    ckpt = {data<const uint8_t>(codes), data<const uint8_t>(scales), (int32_t)PyLong_AsLong(args[3])};
    return true;
  }
  const rawint4_ckpt8* held() const { return codes ? &ckpt : nullptr; }
};

// norm_fwd(x, codes, scales, format, weight, bias, kind, eps, dtype, save) -> (y, mean, rstd, codes, scales);
// dtype None: that of x; save: a format, or -1
PyObject* norm_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Here here;
  NormInput in;
  if (n != 10 || !in.take(here, args)) Py_RETURN_NONE;
  const Tensor *weight, *bias;
  if (!vector_ok(here, args[4], in.width, &weight) || !vector_ok(here, args[5], in.width, &bias) ||
      (weight && bias && weight->scalar_type() != bias->scalar_type()))
    Py_RETURN_NONE;
  const long kind = PyLong_AsLong(args[6]), save = PyLong_AsLong(args[9]);
  const double eps = PyFloat_AsDouble(args[7]);
  if (PyErr_Occurred()) return nullptr;
  ScalarType type = in.x ? in.x->scalar_type() : ScalarType::BFloat16;
  if (args[8] != Py_None) {
    if (!THPDtype_Check(args[8])) Py_RETURN_NONE;
    const ScalarType asked = reinterpret_cast<THPDtype*>(args[8])->scalar_type;
    if (type_of(asked) < 0 || (in.x && asked != type)) Py_RETURN_NONE;
    type = asked;
  }
  if (save >= 0 && !in.x) Py_RETURN_NONE;
  const ScalarType wtype = weight ? weight->scalar_type() : bias ? bias->scalar_type() : type;
  const rawint4_norm_cfg cfg = {(int32_t)in.rows, (int32_t)in.width, (int32_t)kind, type_of(type), type_of(wtype), (float)eps};
  Tensor y, mean, rstd, codes, scales;
  int rc;
  {
    const Unlocked unlocked;
    y = here.empty({in.rows, in.width}, type);
    rstd = here.empty({in.rows}, ScalarType::Float);
    if (kind == RAWINT4_NORM_LAYER) mean = here.empty({in.rows}, ScalarType::Float);
    if (save >= 0) {
      codes = here.empty({in.rows, in.width}, ScalarType::Byte);
      scales = here.empty({in.rows, (in.width + kGroup - 1) / kGroup}, ScalarType::Byte);
    }
    rc = rawint4_norm_fwd(&cfg, data(in.x), in.pitch, in.held(), data(weight), data(bias), data(&y),
                          mean.defined() ? data<float>(&mean) : nullptr, data<float>(&rstd),
                          save >= 0 ? (int32_t)save : 0, save >= 0 ? data<uint8_t>(&codes) : nullptr,
                          save >= 0 ? data<uint8_t>(&scales) : nullptr, here.stream());
  }
  return rc == RAWINT4_OK ? tuple_of({y, mean, rstd, codes, scales}) : refused(rc);
  END_HANDLE_TH_ERRORS
}

// norm_bwd(x, codes, scales, format, grad_y, rstd, weight, mean, kind, bias_grad, grad_weight, grad_bias,
//          accumulate) -> (grad_x, grad_weight, grad_bias)
PyObject* norm_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Here here;
  NormInput in;
  if (n != 13 || !in.take(here, args)) Py_RETURN_NONE;
  int64_t pitch = 0;
  const Tensor *gy = tensor(args[4]), *rstd = tensor(args[5]), *mean = nullptr, *weight, *gw_in, *gb_in;
  if (!rows_ok(here, gy, &pitch) || gy->size(0) != in.rows || gy->size(1) != in.width ||
      (in.x && gy->scalar_type() != in.x->scalar_type()) || !dense(here, rstd, ScalarType::Float, {in.rows}))
    Py_RETURN_NONE;
  const long kind = PyLong_AsLong(args[8]);
  const int bias_grad = PyObject_IsTrue(args[9]), accumulate = PyObject_IsTrue(args[12]);
  if (PyErr_Occurred()) return nullptr;
  if (kind == RAWINT4_NORM_LAYER ? !dense(here, mean = tensor(args[7]), ScalarType::Float, {in.rows}) : args[7] != Py_None)
    Py_RETURN_NONE;
  if (!vector_ok(here, args[6], in.width, &weight) || !vector_ok(here, args[10], in.width, &gw_in) ||
      !vector_ok(here, args[11], in.width, &gb_in) || (gw_in && !weight) ||
      (accumulate && ((weight && !gw_in) || (bias_grad && !gb_in))))
    Py_RETURN_NONE;
  const ScalarType type = gy->scalar_type();
  const ScalarType wtype = weight ? weight->scalar_type() : gb_in ? gb_in->scalar_type() : type;
  if ((gw_in && gw_in->scalar_type() != wtype) || (gb_in && gb_in->scalar_type() != wtype)) Py_RETURN_NONE;
  const rawint4_norm_cfg cfg = {(int32_t)in.rows, (int32_t)in.width, (int32_t)kind, type_of(type), type_of(wtype), 1.0f};
  size_t bytes = 0;
  int rc = rawint4_norm_bwd_workspace_size(&cfg, &bytes);
  if (rc != RAWINT4_OK) return refused(rc);
  Tensor gx, gw, gb;
  {
    const Unlocked unlocked;
    Tensor ws;
    gx = here.empty({in.rows, in.width}, type);
    if (gw_in) gw = *gw_in;
    else if (weight) gw = here.empty({in.width}, wtype);
    if (gb_in) gb = *gb_in;
    else if (bias_grad) gb = here.empty({in.width}, wtype);
    if (gw.defined() || gb.defined()) ws = here.empty({(int64_t)bytes}, ScalarType::Byte);
    else bytes = 0;
    rc = rawint4_norm_bwd(&cfg, data(in.x), in.pitch, in.held(), data(gy), pitch, data(weight),
                          mean ? data<const float>(mean) : nullptr, data<const float>(rstd), data(&gx),
                          gw.defined() ? data(&gw) : nullptr, gb.defined() ? data(&gb) : nullptr, accumulate,
                          ws.defined() ? data(&ws) : nullptr, bytes, here.stream());
  }
  return rc == RAWINT4_OK ? tuple_of({gx, gw, gb}) : refused(rc);
  END_HANDLE_TH_ERRORS
}

#define R4_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {R4_METHOD(router_select), R4_METHOD(router_select_bwd), R4_METHOD(ckpt8_save),
                         R4_METHOD(ckpt8_load),    R4_METHOD(norm_fwd),          R4_METHOD(norm_bwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module_def); }
