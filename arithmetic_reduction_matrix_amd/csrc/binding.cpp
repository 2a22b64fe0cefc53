// The layer entry points of include/armx.h for PyTorch tensors: a CPython module
// (arithmetic_reduction_matrix_amd._binding) that checks tensors, allocates
// results on the inputs' device, and calls the C ABI on the device's current
// stream.  The kernels of these calls take a few microseconds on small inputs;
// with the checks and allocations in Python the call took longer than they did
// (us per call on MI355X, Python / this: norm of 1 x 4096 with the residual and
// 1 / rms 11.0 / 6.3, product 1 x 4096 x 4096 8.5 / 4.7, backward 515 x 2056
// 15.6 / 9.5).
//
// Every function takes positional arguments (layer.py and training.py give them names,
// defaults and documentation) and returns a tuple of tensors, or the library's status as an
// int when it is not ARMX_OK.  Wrong types raise TypeError, anything else that the
// tensors get wrong ValueError; exceptions of PyTorch (out of memory) pass through.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>

#include <cstdint>

#include "armx.h"

namespace {

using at::ScalarType;
using at::Tensor;

int type_code(ScalarType t) {
  return t == at::kHalf ? ARMX_F16 : t == at::kBFloat16 ? ARMX_BF16 : t == at::kFloat ? ARMX_F32 : -1;
}

// One call's context: its name in messages, and the shape, type and device that
// its operands must have.
struct Call {
  const char* name;
  int64_t rows = 0, cols = 0;
  ScalarType type = at::kHalf;
  at::Device device{at::kCPU};
  armx_config cfg{};
  bool has_cfg = false;
};

// The tensor behind an argument; nullptr (nothing raised) if it is not one.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// The operand that the others must match: 2-D, on a GPU, of one of `types`.
const Tensor* first(Call& c, PyObject* o, const char* what, bool codes) {
  const Tensor* t = tensor(o);
  if (!t) {
    PyErr_Format(PyExc_TypeError, "%s: %s must be a torch.Tensor", c.name, what);
    return nullptr;
  }
  const ScalarType type = t->scalar_type();
  if (codes ? type != at::kChar : type != at::kHalf && type != at::kBFloat16) {
    PyErr_Format(PyExc_TypeError, "%s: %s must be %s, got %s", c.name, what,
                 codes ? "int8" : "float16 or bfloat16", c10::toString(type));
    return nullptr;
  }
  if (!t->is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s: %s must be on a GPU (HIP) device", c.name, what);
    return nullptr;
  }
  if (t->dim() != 2) {
    PyErr_Format(PyExc_ValueError, "%s: expected a 2-D %s, got %d-D", c.name, what,
                 int(t->dim()));
    return nullptr;
  }
  c.rows = t->size(0), c.cols = t->size(1);
  c.type = type;
  c.device = t->device();
  return t;
}

struct Rows {
  void* p = nullptr;
  size_t ld = 0;
};

// A rows x cols matrix of `type` with contiguous rows.
bool matrix(const Call& c, PyObject* o, const char* what, int64_t rows, int64_t cols,
            ScalarType type, Rows* out) {
  const Tensor* t = tensor(o);
  if (!t || t->scalar_type() != type || t->dim() != 2 || t->size(0) != rows ||
      t->size(1) != cols || t->device() != c.device) {
    PyErr_Format(PyExc_ValueError, "%s: %s must be a (%lld, %lld) %s tensor on %s", c.name, what,
                 (long long)rows, (long long)cols, c10::toString(type), c.device.str().c_str());
    return false;
  }
  if (cols > 1 && t->stride(1) != 1) {
    PyErr_Format(PyExc_ValueError, "%s: rows of %s must be contiguous (stride(1) == 1)", c.name,
                 what);
    return false;
  }
  out->p = t->data_ptr();
  out->ld = size_t(rows > 1 ? t->stride(0) : cols);
  return true;
}

// n contiguous values of `type`.
bool vector(const Call& c, PyObject* o, const char* what, int64_t n, ScalarType type, void** p) {
  const Tensor* t = tensor(o);
  if (!t || t->scalar_type() != type || t->numel() != n || t->device() != c.device ||
      !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s: %s must be %lld contiguous %s values on %s", c.name, what,
                 (long long)n, c10::toString(type), c.device.str().c_str());
    return false;
  }
  *p = t->data_ptr();
  return true;
}

Tensor make(const Call& c, at::IntArrayRef size, ScalarType type) {
  return at::empty(size, at::TensorOptions().dtype(type).device(c.device));
}

// A new matrix whose rows start at multiples of `multiple` values: allocated with its
// pitch as width, then given its own (a view of the wide one took 0.7 us more a call).
Tensor make_rows(const Call& c, int64_t multiple, ScalarType type, Rows* out) {
  const int64_t pitch = (c.cols + multiple - 1) / multiple * multiple;
  Tensor t = make(c, {c.rows, pitch}, type);
  out->p = t.data_ptr();
  out->ld = size_t(pitch);
  if (pitch != c.cols) {
    const int64_t sizes[] = {c.rows, c.cols}, strides[] = {pitch, 1};
    t.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(sizes), at::IntArrayRef(strides));
  }
  return t;
}

// Rows of codes made here: at least 16 codes apart in multiples of 16, which the
// product asks for, and from 512 codes on in whole 128-byte lines, which it reads
// them by (1024 x 4096 x 4112, a pitch of 4224 against 4112: 20.0 against 22.0 us).
int64_t code_multiple(int64_t cols) { return cols < 512 ? 16 : 128; }

// Writes that autograd does not see: what it saved of the tensor's old values is then
// refused.  (Inference tensors have no version, and nothing saves them.)
void written(PyObject* o) {
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Owned references that are released unless handed on; `given`: to the caller's own
// tensors.
struct Owned {
  PyObject* o[4] = {nullptr, nullptr, nullptr, nullptr};
  bool given[4] = {false, false, false, false};
  ~Owned() {
    for (PyObject* p : o) Py_XDECREF(p);
  }
  void give(int i, PyObject* tensor) {
    Py_INCREF(tensor);
    o[i] = tensor;
    given[i] = true;
  }
  // The tuple of `n` of them (None for those that are missing), or the status.
  PyObject* done(int status, int n) {
    if (status != ARMX_OK) return PyLong_FromLong(status);
    PyObject* t = PyTuple_New(n);
    if (!t) return nullptr;
    for (int i = 0; i < n; ++i) {
      if (!o[i]) {
        Py_INCREF(Py_None);
        o[i] = Py_None;
      }
      if (given[i]) written(o[i]);
      PyTuple_SET_ITEM(t, i, o[i]);
      o[i] = nullptr;
    }
    return t;
  }
};

// Output i of a call: the caller's (returned as it came) or a new one.
bool output(const Call& c, PyObject* given, const char* what, int64_t multiple, ScalarType type,
            Rows* out, Owned& r, int i) {
  if (given != Py_None) {
    if (!matrix(c, given, what, c.rows, c.cols, type, out)) return false;
    r.give(i, given);
    return true;
  }
  r.o[i] = THPVariable_Wrap(make_rows(c, multiple, type, out));
  return r.o[i] != nullptr;
}

bool vector_output(const Call& c, PyObject* given, const char* what, int64_t n, void** p, Owned& r,
                   int i) {
  if (given != Py_None) {
    if (!vector(c, given, what, n, at::kFloat, p)) return false;
    r.give(i, given);
    return true;
  }
  Tensor t = make(c, {n}, at::kFloat);
  *p = t.data_ptr();
  r.o[i] = THPVariable_Wrap(std::move(t));
  return r.o[i] != nullptr;
}

// hipEvent_t handles (ints or None) into the call's configuration.
bool events(Call& c, PyObject* start, PyObject* stop) {
  if (start == Py_None && stop == Py_None) return true;
  if (start != Py_None) c.cfg.start_event = PyLong_AsVoidPtr(start);
  if (stop != Py_None) c.cfg.stop_event = PyLong_AsVoidPtr(stop);
  c.has_cfg = true;
  return !PyErr_Occurred();
}

bool arity(const char* name, Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", name, want, got);
  return false;
}

void* stream_of(const Call& c) { return c10::hip::getCurrentHIPStream(c.device.index()).stream(); }

// A call's workspace: the caller's, or one from the allocator, which knows streams and
// graph captures (it needs no zeros, so nothing is gained by keeping one).
struct Workspace {
  Tensor space;
  void* p = nullptr;
  size_t bytes = 0;
  bool too_large = false;   // the call takes no such sizes
  bool take(const Call& c, PyObject* given, size_t need) {
    if (given == Py_None) {
      too_large = need == size_t(-1);
      if (too_large) return false;
      if (need) space = make(c, {int64_t(need)}, at::kByte);
      p = need ? space.data_ptr() : nullptr;
      bytes = need;
      return true;
    }
    const Tensor* t = tensor(given);
    if (!t || t->device() != c.device || !t->is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s: workspace must be a contiguous tensor on %s", c.name,
                   c.device.str().c_str());
      return false;
    }
    p = t->data_ptr();
    bytes = t->nbytes();
    return true;
  }
};

// (x, weight, residual, eps, keep_inv_rms | None, out, scales, sum_out, start, stop);
// codes: rms_norm_rows_int8, whose `out` is int8
PyObject* norm(const char* name, bool codes, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(name, n, 10)) return nullptr;
  Call c{name};
  Rows x, res, out, sum;
  void *w = nullptr, *side = nullptr;
  if (!first(c, a[0], "x", false) || !matrix(c, a[0], "x", c.rows, c.cols, c.type, &x) ||
      !vector(c, a[1], "weight", c.cols, c.type, &w))
    return nullptr;
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const int keep = codes ? 1 : PyObject_IsTrue(a[4]);
  if (keep < 0 || !events(c, a[8], a[9])) return nullptr;
  Owned r;   // out, sum, inv_rms; or codes, scales, sum
  const int sum_result = codes ? 2 : 1, side_result = codes ? 1 : 2;
  c10::DeviceGuard guard(c.device);
  if (a[2] != Py_None) {
    if (!matrix(c, a[2], "residual", c.rows, c.cols, c.type, &res) ||
        !output(c, a[7], "sum_out", 8, c.type, &sum, r, sum_result))
      return nullptr;
  } else if (a[7] != Py_None) {
    PyErr_Format(PyExc_ValueError, "%s: sum_out goes with a residual", name);
    return nullptr;
  }
  if (!output(c, a[5], "out", codes ? code_multiple(c.cols) : 8, codes ? at::kChar : c.type,
              &out, r, 0))
    return nullptr;
  if (keep && !vector_output(c, a[6], "scales", c.rows, &side, r, side_result)) return nullptr;
  const armx_config* cfg = c.has_cfg ? &c.cfg : nullptr;
  const int st =
      codes ? rms_norm_rows_int8(x.p, x.ld, res.p, res.ld, w, type_code(c.type), size_t(c.rows),
                                 size_t(c.cols), float(eps), static_cast<int8_t*>(out.p), out.ld,
                                 static_cast<float*>(side), sum.p, sum.ld, cfg, stream_of(c))
            : rms_norm_rows(x.p, x.ld, res.p, res.ld, w, type_code(c.type), size_t(c.rows),
                            size_t(c.cols), float(eps), out.p, out.ld, sum.p, sum.ld,
                            static_cast<float*>(side), cfg, stream_of(c));
  return r.done(st, 3);
  END_HANDLE_TH_ERRORS
}

PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return norm("rms_norm_rows", false, a, n);
}

PyObject* py_norm_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return norm("rms_norm_rows_int8", true, a, n);
}

// (x, out, scales, start, stop)
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"quantize_rows_int8"};
  Rows x, out;
  void* scales = nullptr;
  if (!arity(c.name, n, 5) || !first(c, a[0], "x", false) ||
      !matrix(c, a[0], "x", c.rows, c.cols, c.type, &x) || !events(c, a[3], a[4]))
    return nullptr;
  Owned r;
  c10::DeviceGuard guard(c.device);
  if (!output(c, a[1], "out", code_multiple(c.cols), at::kChar, &out, r, 0) ||
      !vector_output(c, a[2], "scales", c.rows, &scales, r, 1))
    return nullptr;
  const int st = quantize_rows_int8(x.p, x.ld, type_code(c.type), size_t(c.rows), size_t(c.cols),
                                    static_cast<int8_t*>(out.p), out.ld,
                                    static_cast<float*>(scales), c.has_cfg ? &c.cfg : nullptr,
                                    stream_of(c));
  return r.done(st, 2);
  END_HANDLE_TH_ERRORS
}

// (dy, h, weight, inv_rms, dsum, out, dweight, workspace, start, stop)
PyObject* py_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"rms_norm_rows_backward"};
  Rows dy, h, ds, dx;
  void *w = nullptr, *inv = nullptr, *dw = nullptr;
  if (!arity(c.name, n, 10) || !first(c, a[0], "dy", false) ||
      !matrix(c, a[0], "dy", c.rows, c.cols, c.type, &dy) ||
      !matrix(c, a[1], "h", c.rows, c.cols, c.type, &h) ||
      !vector(c, a[2], "weight", c.cols, c.type, &w) ||
      !vector(c, a[3], "inv_rms", c.rows, at::kFloat, &inv) ||
      (a[4] != Py_None && !matrix(c, a[4], "dsum", c.rows, c.cols, c.type, &ds)) ||
      !events(c, a[8], a[9]))
    return nullptr;
  Owned r;
  c10::DeviceGuard guard(c.device);
  if (!output(c, a[5], "out", 8, c.type, &dx, r, 0) ||
      !vector_output(c, a[6], "dweight", c.cols, &dw, r, 1))
    return nullptr;
  Workspace ws;
  if (!ws.take(c, a[7], armx_workspace_bytes(ARMX_OP_RMS_BACKWARD, size_t(c.rows), size_t(c.cols),
                                             nullptr)))
    return ws.too_large ? PyLong_FromLong(ARMX_ERR_SHAPE) : nullptr;
  const int st = rms_norm_rows_backward(
      dy.p, dy.ld, h.p, h.ld, w, static_cast<const float*>(inv), ds.p, ds.ld, type_code(c.type),
      size_t(c.rows), size_t(c.cols), dx.p, dx.ld, static_cast<float*>(dw), ws.p, ws.bytes,
      c.has_cfg ? &c.cfg : nullptr, stream_of(c));
  if (st == ARMX_OK && ws.bytes && a[7] != Py_None) written(a[7]);
  return r.done(st, 2);
  END_HANDLE_TH_ERRORS
}

// A Dropout (p, seed, offset, step, first_row), or None where `optional`: *given says
// which.
bool dropout(const Call& c, PyObject* o, bool optional, armx_dropout* d, bool* given) {
  *given = o != Py_None;
  if (!*given && optional) return true;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) {
    PyErr_Format(PyExc_TypeError, "%s: dropout must be a Dropout", c.name);
    return false;
  }
  d->p = PyFloat_AsDouble(PyTuple_GET_ITEM(o, 0));
  if (d->p == -1.0 && PyErr_Occurred()) return false;
  if (!(d->p >= 0.0 && d->p <= 1.0)) {
    PyErr_Format(PyExc_ValueError, "%s: dropout's p must be from 0 to 1", c.name);
    return false;
  }
  const char* names[] = {"seed", "offset", "first_row"};
  uint64_t* to[] = {&d->seed, &d->offset, &d->first_row};
  const int at[] = {1, 2, 4};
  for (int i = 0; i < 3; ++i) {
    PyObject* v = PyTuple_GET_ITEM(o, at[i]);
    if (!PyLong_Check(v)) {
      PyErr_Format(PyExc_TypeError, "%s: dropout's %s must be an int", c.name, names[i]);
      return false;
    }
    *to[i] = PyLong_AsUnsignedLongLong(v);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      PyErr_Format(PyExc_ValueError, "%s: dropout's %s must be from 0 to 2^64 - 1", c.name,
                   names[i]);
      return false;
    }
  }
  void* step = nullptr;
  if (PyTuple_GET_ITEM(o, 3) != Py_None &&
      !vector(c, PyTuple_GET_ITEM(o, 3), "dropout's step", 1, at::kLong, &step))
    return false;
  d->step = static_cast<const uint64_t*>(step);
  return true;
}

// (x, weight, bias, residual, dropout, eps, keep_stats, out, sum_out, start, stop)
PyObject* py_layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"layer_norm_rows"};
  Rows x, res, out, sum;
  void *w = nullptr, *b = nullptr, *mean = nullptr, *inv = nullptr;
  armx_dropout drop;
  bool drops = false;
  if (!arity(c.name, n, 11) || !first(c, a[0], "x", false) ||
      !matrix(c, a[0], "x", c.rows, c.cols, c.type, &x) ||
      !vector(c, a[1], "weight", c.cols, c.type, &w) ||
      (a[2] != Py_None && !vector(c, a[2], "bias", c.cols, c.type, &b)) ||
      (a[3] != Py_None && !matrix(c, a[3], "residual", c.rows, c.cols, c.type, &res)) ||
      !dropout(c, a[4], true, &drop, &drops))
    return nullptr;
  const double eps = PyFloat_AsDouble(a[5]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const int keep = PyObject_IsTrue(a[6]);
  if (keep < 0 || !events(c, a[9], a[10])) return nullptr;
  Owned r;   // out, sum, mean, inv_std
  c10::DeviceGuard guard(c.device);
  if (a[3] != Py_None || drops) {
    if (!output(c, a[8], "sum_out", 8, c.type, &sum, r, 1)) return nullptr;
  } else if (a[8] != Py_None) {
    PyErr_Format(PyExc_ValueError, "%s: sum_out goes with a residual or a dropout", c.name);
    return nullptr;
  }
  if (!output(c, a[7], "out", 8, c.type, &out, r, 0)) return nullptr;
  if (keep && (!vector_output(c, Py_None, "mean", c.rows, &mean, r, 2) ||
               !vector_output(c, Py_None, "inv_std", c.rows, &inv, r, 3)))
    return nullptr;
  const int st = layer_norm_rows(
      x.p, x.ld, res.p, res.ld, w, b, type_code(c.type), size_t(c.rows), size_t(c.cols),
      float(eps), drops ? &drop : nullptr, out.p, out.ld, sum.p, sum.ld,
      static_cast<float*>(mean), static_cast<float*>(inv), c.has_cfg ? &c.cfg : nullptr,
      stream_of(c));
  return r.done(st, 4);
  END_HANDLE_TH_ERRORS
}

// (dy, h, weight, mean, inv_std, dsum, dropout, out, dresidual, dweight, dbias, workspace,
// start, stop)
PyObject* py_layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"layer_norm_rows_backward"};
  Rows dy, h, ds, dx, dr;
  void *w = nullptr, *mean = nullptr, *inv = nullptr, *dw = nullptr, *db = nullptr;
  armx_dropout drop;
  bool drops = false;
  if (!arity(c.name, n, 14) || !first(c, a[0], "dy", false) ||
      !matrix(c, a[0], "dy", c.rows, c.cols, c.type, &dy) ||
      !matrix(c, a[1], "h", c.rows, c.cols, c.type, &h) ||
      !vector(c, a[2], "weight", c.cols, c.type, &w) ||
      !vector(c, a[3], "mean", c.rows, at::kFloat, &mean) ||
      !vector(c, a[4], "inv_std", c.rows, at::kFloat, &inv) ||
      (a[5] != Py_None && !matrix(c, a[5], "dsum", c.rows, c.cols, c.type, &ds)) ||
      !dropout(c, a[6], true, &drop, &drops) || !events(c, a[12], a[13]))
    return nullptr;
  if (!drops && a[8] != Py_None) {
    PyErr_Format(PyExc_ValueError, "%s: dresidual goes with a dropout (dx is both without)",
                 c.name);
    return nullptr;
  }
  Owned r;   // dx, dweight, dbias, dresidual
  c10::DeviceGuard guard(c.device);
  if (!output(c, a[7], "out", 8, c.type, &dx, r, 0) ||
      !vector_output(c, a[9], "dweight", c.cols, &dw, r, 1) ||
      !vector_output(c, a[10], "dbias", c.cols, &db, r, 2) ||
      (drops && !output(c, a[8], "dresidual", 8, c.type, &dr, r, 3)))
    return nullptr;
  Workspace ws;
  if (!ws.take(c, a[11], armx_workspace_bytes(ARMX_OP_LAYER_NORM_BACKWARD, size_t(c.rows),
                                              size_t(c.cols), nullptr)))
    return ws.too_large ? PyLong_FromLong(ARMX_ERR_SHAPE) : nullptr;
  const int st = layer_norm_rows_backward(
      dy.p, dy.ld, h.p, h.ld, w, static_cast<const float*>(mean), static_cast<const float*>(inv),
      ds.p, ds.ld, type_code(c.type), size_t(c.rows), size_t(c.cols), drops ? &drop : nullptr,
      dx.p, dx.ld, dr.p, dr.ld, static_cast<float*>(dw), static_cast<float*>(db), ws.p, ws.bytes,
      c.has_cfg ? &c.cfg : nullptr, stream_of(c));
  if (st == ARMX_OK && ws.bytes && a[11] != Py_None) written(a[11]);
  return r.done(st, 4);
  END_HANDLE_TH_ERRORS
}

// (x, dropout, residual, out, start, stop)
PyObject* py_dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"dropout_rows"};
  Rows x, res, out;
  armx_dropout drop;
  bool drops = false;
  if (!arity(c.name, n, 6) || !first(c, a[0], "x", false) ||
      !matrix(c, a[0], "x", c.rows, c.cols, c.type, &x) ||
      !dropout(c, a[1], false, &drop, &drops) ||
      (a[2] != Py_None && !matrix(c, a[2], "residual", c.rows, c.cols, c.type, &res)) ||
      !events(c, a[4], a[5]))
    return nullptr;
  Owned r;
  c10::DeviceGuard guard(c.device);
  if (!output(c, a[3], "out", 8, c.type, &out, r, 0)) return nullptr;
  const int st = dropout_rows(x.p, x.ld, res.p, res.ld, type_code(c.type), size_t(c.rows),
                              size_t(c.cols), &drop, out.p, out.ld, c.has_cfg ? &c.cfg : nullptr,
                              stream_of(c));
  return r.done(st, 1);
  END_HANDLE_TH_ERRORS
}

bool int64_arg(const Call& c, PyObject* o, const char* what, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  if (*v != -1 || !PyErr_Occurred()) return true;
  PyErr_Clear();
  PyErr_Format(PyExc_TypeError, "%s: %s must be an int of 64 bits", c.name, what);
  return false;
}

// (x, weight, targets, ignore_index, loss, lse, workspace, start, stop)
PyObject* py_cross_entropy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"cross_entropy_rows"}, other{"cross_entropy_rows"};
  Rows x, w;
  void *targets = nullptr, *loss = nullptr, *lse = nullptr;
  int64_t ignore = 0;
  if (!arity(c.name, n, 9) || !first(c, a[0], "x", false) || !first(other, a[1], "weight", false) ||
      !matrix(c, a[0], "x", c.rows, c.cols, c.type, &x) ||
      !matrix(c, a[1], "weight", other.rows, c.cols, c.type, &w) ||
      !vector(c, a[2], "targets", c.rows, at::kLong, &targets) ||
      !int64_arg(c, a[3], "ignore_index", &ignore) || !events(c, a[7], a[8]))
    return nullptr;
  const int64_t vocab = other.rows;
  Owned r;   // loss, lse
  c10::DeviceGuard guard(c.device);
  if (!vector_output(c, a[4], "loss", c.rows, &loss, r, 0) ||
      !vector_output(c, a[5], "lse", c.rows, &lse, r, 1))
    return nullptr;
  Workspace ws;
  if (!ws.take(c, a[6], armx_cross_entropy_workspace_bytes(size_t(c.rows), size_t(vocab),
                                                           size_t(c.cols))))
    return ws.too_large ? PyLong_FromLong(ARMX_ERR_SHAPE) : nullptr;
  const int st = cross_entropy_rows(
      x.p, x.ld, w.p, w.ld, static_cast<const int64_t*>(targets), type_code(c.type),
      size_t(c.rows), size_t(vocab), size_t(c.cols), ignore, static_cast<float*>(loss),
      static_cast<float*>(lse), ws.p, ws.bytes, c.has_cfg ? &c.cfg : nullptr, stream_of(c));
  if (st == ARMX_OK && ws.bytes && a[6] != Py_None) written(a[6]);
  return r.done(st, 2);
  END_HANDLE_TH_ERRORS
}

// (dloss, x, weight, targets, lse, ignore_index, need_dx, need_dweight, out, dweight,
// dweight's type code, workspace, start, stop)
PyObject* py_cross_entropy_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"cross_entropy_rows_backward"}, other{"cross_entropy_rows_backward"};
  Rows x, w, dx, dw;
  void *dloss = nullptr, *targets = nullptr, *lse = nullptr;
  int64_t ignore = 0;
  if (!arity(c.name, n, 14) || !first(c, a[1], "x", false) ||
      !first(other, a[2], "weight", false) ||
      !matrix(c, a[1], "x", c.rows, c.cols, c.type, &x) ||
      !matrix(c, a[2], "weight", other.rows, c.cols, c.type, &w) ||
      !vector(c, a[0], "dloss", c.rows, at::kFloat, &dloss) ||
      !vector(c, a[3], "targets", c.rows, at::kLong, &targets) ||
      !vector(c, a[4], "lse", c.rows, at::kFloat, &lse) ||
      !int64_arg(c, a[5], "ignore_index", &ignore) || !events(c, a[12], a[13]))
    return nullptr;
  const int need_dx = PyObject_IsTrue(a[6]), need_dw = PyObject_IsTrue(a[7]);
  if (need_dx < 0 || need_dw < 0) return nullptr;
  if ((!need_dx && a[8] != Py_None) || (!need_dw && a[9] != Py_None) || (!need_dx && !need_dw)) {
    PyErr_Format(PyExc_ValueError, "%s: a gradient that is not wanted takes no tensor, and one "
                 "is wanted", c.name);
    return nullptr;
  }
  ScalarType type = c.type;   // dweight's
  if (a[9] != Py_None) {
    if (const Tensor* given = tensor(a[9])) type = given->scalar_type();
  } else if (a[10] != Py_None) {
    const long code = PyLong_AsLong(a[10]);
    if (code == -1 && PyErr_Occurred()) return nullptr;
    type = code == ARMX_F16 ? at::kHalf : code == ARMX_BF16 ? at::kBFloat16
           : code == ARMX_F32 ? at::kFloat : at::kByte;
  }
  if (type != c.type && type != at::kFloat) {
    PyErr_Format(PyExc_TypeError, "%s: dweight is %s or float32", c.name, c10::toString(c.type));
    return nullptr;
  }
  other.type = type, other.device = c.device;
  other.cols = c.cols;
  Owned r;   // dx, dweight
  c10::DeviceGuard guard(c.device);
  if ((need_dx && !output(c, a[8], "out", 8, c.type, &dx, r, 0)) ||
      (need_dw && !output(other, a[9], "dweight", 8, type, &dw, r, 1)))
    return nullptr;
  Workspace ws;
  if (!ws.take(c, a[11], armx_cross_entropy_backward_workspace_bytes(
                             size_t(c.rows), size_t(other.rows), size_t(c.cols), need_dx, need_dw)))
    return ws.too_large ? PyLong_FromLong(ARMX_ERR_SHAPE) : nullptr;
  const int st = cross_entropy_rows_backward(
      static_cast<const float*>(dloss), x.p, x.ld, w.p, w.ld,
      static_cast<const int64_t*>(targets), static_cast<const float*>(lse), type_code(c.type),
      size_t(c.rows), size_t(other.rows), size_t(c.cols), ignore, dx.p, dx.ld, dw.p, dw.ld,
      type_code(type), ws.p, ws.bytes, c.has_cfg ? &c.cfg : nullptr, stream_of(c));
  if (st == ARMX_OK && ws.bytes && a[11] != Py_None) written(a[11]);
  return r.done(st, 2);
  END_HANDLE_TH_ERRORS
}

// A matrix of codes whose rows can be read in pieces of 16 to their end.
bool code_rows(const Call& c, PyObject* o, const char* what, int64_t rows, int64_t k, Rows* out) {
  if (!matrix(c, o, what, rows, k, at::kChar, out)) return false;
  if (k % 16 && rows && (out->ld % 16 == 0 || rows == 1)) {   // else the call reports the pitch
    const Tensor& t = *tensor(o);
    const int64_t end = t.storage_offset() + (rows - 1) * int64_t(out->ld) + (k + 15) / 16 * 16;
    if (end > int64_t(t.storage().nbytes())) {
      PyErr_Format(PyExc_ValueError,
                   "%s: the last row of %s must be readable to a multiple of 16 codes (allocate "
                   "rows with a pitch that is one)",
                   c.name, what);
      return false;
    }
  }
  return true;
}

// (a, a_scales, b, b_scales, bias, out, dtype code, start, stop)
PyObject* py_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c{"matmul_int8"}, other{"matmul_int8"};
  Rows ar, br, out;
  void *as = nullptr, *bs = nullptr, *bias = nullptr;
  if (!arity(c.name, n, 9) || !first(c, a[0], "a", true) || !first(other, a[2], "b", true))
    return nullptr;
  const int64_t m = c.rows, k = c.cols, cols = other.rows;
  if (!code_rows(c, a[0], "a", m, k, &ar) || !code_rows(c, a[2], "b", cols, k, &br) ||
      !vector(c, a[1], "a_scales", m, at::kFloat, &as) ||
      !vector(c, a[3], "b_scales", cols, at::kFloat, &bs) || !events(c, a[7], a[8]))
    return nullptr;
  long code = -1;
  const Tensor* given = tensor(a[5]);
  if (a[5] == Py_None) {
    code = PyLong_AsLong(a[6]);
    if (code == -1 && PyErr_Occurred()) return nullptr;
  } else if (given) {
    code = type_code(given->scalar_type());
  }
  if (code < 0 || code > 2) {
    PyErr_Format(PyExc_TypeError, "%s: the result is float16, bfloat16 or float32", c.name);
    return nullptr;
  }
  const ScalarType type = code == ARMX_F16 ? at::kHalf : code == ARMX_BF16 ? at::kBFloat16 : at::kFloat;
  if (a[4] != Py_None && !vector(c, a[4], "bias", cols, type, &bias)) return nullptr;
  Owned r;
  c10::DeviceGuard guard(c.device);
  c.cols = cols;
  // 16-bit rows as the norms and the quantiser read them
  if (!output(c, a[5], "out", type == at::kFloat ? 1 : 8, type, &out, r, 0)) return nullptr;
  const int st = matmul_int8(static_cast<const int8_t*>(ar.p), ar.ld, static_cast<const float*>(as),
                             static_cast<const int8_t*>(br.p), br.ld, static_cast<const float*>(bs),
                             bias, size_t(m), size_t(cols), size_t(k), out.p, out.ld, int(code),
                             c.has_cfg ? &c.cfg : nullptr, stream_of(c));
  return r.done(st, 1);
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {
    method<py_norm>("rms_norm_rows"),
    method<py_norm_int8>("rms_norm_rows_int8"),
    method<py_norm_backward>("rms_norm_rows_backward"),
    method<py_quantize>("quantize_rows_int8"),
    method<py_matmul>("matmul_int8"),
    method<py_layer_norm>("layer_norm_rows"),
    method<py_layer_norm_backward>("layer_norm_rows_backward"),
    method<py_dropout>("dropout_rows"),
    method<py_cross_entropy>("cross_entropy_rows"),
    method<py_cross_entropy_backward>("cross_entropy_rows_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
