// The layer entry points of include/armx.h for PyTorch tensors: a CPython module
// (arithmetic_reduction_matrix_amd._binding) that checks tensors, allocates
// results on the inputs' device, and calls the C ABI on the device's current
// stream.  The kernels of these calls take a few microseconds on small inputs;
// with the checks and allocations in Python the call took longer than they did
// (us per call on MI355X, Python / this: norm of 1 x 4096 with the residual and
// 1 / rms 11.0 / 6.3, product 1 x 4096 x 4096 8.5 / 4.7, backward 515 x 2056
// 15.6 / 9.5).
//
// Every function takes positional arguments (layer.py gives them names, defaults
// and documentation) and returns a tuple of tensors, or the library's status as an
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
  PyObject* o[3] = {nullptr, nullptr, nullptr};
  bool given[3] = {false, false, false};
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
  void *w = nullptr, *inv = nullptr, *dw = nullptr, *ws = nullptr;
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
  Tensor space;   // from the allocator, which knows streams and graph captures: it
                  // needs no zeros, so nothing is gained by keeping one
  size_t ws_bytes = 0;
  if (a[7] == Py_None) {
    ws_bytes = armx_workspace_bytes(ARMX_OP_RMS_BACKWARD, size_t(c.rows), size_t(c.cols), nullptr);
    if (ws_bytes == size_t(-1)) return PyLong_FromLong(ARMX_ERR_SHAPE);
    if (ws_bytes) space = make(c, {int64_t(ws_bytes)}, at::kByte);
    ws = ws_bytes ? space.data_ptr() : nullptr;
  } else {
    const Tensor* t = tensor(a[7]);
    if (!t || t->device() != c.device || !t->is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s: workspace must be a contiguous tensor on %s", c.name,
                   c.device.str().c_str());
      return nullptr;
    }
    ws = t->data_ptr();
    ws_bytes = t->nbytes();
  }
  const int st = rms_norm_rows_backward(
      dy.p, dy.ld, h.p, h.ld, w, static_cast<const float*>(inv), ds.p, ds.ld, type_code(c.type),
      size_t(c.rows), size_t(c.cols), dx.p, dx.ld, static_cast<float*>(dw), ws, ws_bytes,
      c.has_cfg ? &c.cfg : nullptr, stream_of(c));
  if (st == ARMX_OK && ws_bytes && a[7] != Py_None) written(a[7]);
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
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
