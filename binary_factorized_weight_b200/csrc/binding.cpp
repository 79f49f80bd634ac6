// Python side of the microscaled and norm calls: argument checks, output
// tensors and the C entry points of libdbf, in one C call each.
//
// A single token's norm or product takes the GPU 2 to 5 us; the same checks and
// torch.empty calls made from Python around ctypes took the host 9 to 13 us, and
// take it 4 to 6 here.  No computation happens here.
//
// The entry points are given as addresses by the module that loaded libdbf
// (init), so there is one library, the one that is loaded.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>

#include "../../include/dbf.h"

namespace {

// The entry points, in the order of init's arguments.
decltype(&dbf_mx_quantize) p_quantize;
decltype(&dbf_mx_dequantize) p_dequantize;
decltype(&dbf_mx_forward) p_forward;
decltype(&dbf_rmsnorm_forward) p_norm;
decltype(&dbf_rmsnorm_mx_forward) p_norm_mx;
decltype(&dbf_rmsnorm_backward) p_norm_backward;
decltype(&dbf_mx_code_bytes) p_code_bytes;
decltype(&dbf_mx_scale_bytes) p_scale_bytes;
decltype(&dbf_mx_forward_workspace_bytes) p_forward_ws;
decltype(&dbf_rmsnorm_backward_workspace_bytes) p_backward_ws;
PyObject* raise_status;  // callable(name, status)

struct Refused {  // the Python error is set
};
[[noreturn]] void refuse(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Refused{};
}

using OptTensor = std::optional<at::Tensor>;

at::Tensor tensor(PyObject* o) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "a torch.Tensor is wanted");
  return THPVariable_Unpack(o);
}
OptTensor optional_tensor(PyObject* o) {
  if (o == Py_None) return std::nullopt;
  return tensor(o);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
int format(PyObject* o) {
  const int64_t f = integer(o);
  if (f != DBF_MX_E2M1 && f != DBF_MX_E4M3) refuse(PyExc_ValueError, "fmt must be DBF_MX_E2M1 or DBF_MX_E4M3");
  return static_cast<int>(f);
}
at::ScalarType dtype(PyObject* o) {
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "a torch.dtype is wanted");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
dbf_dtype code_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return DBF_F16;
    case at::kBFloat16: return DBF_BF16;
    case at::kFloat: return DBF_F32;
    default: refuse(PyExc_TypeError, "unsupported dtype: float16, bfloat16 or float32");
  }
}

// Every tensor contiguous and on the current CUDA device.
void check_place(std::initializer_list<const at::Tensor*> list) {
  int device = -1;
  for (const at::Tensor* t : list) {
    if (!t) continue;
    if (t->is_cuda() && device < 0) device = c10::cuda::current_device();
    if (!t->is_cuda() || t->get_device() != device || !t->is_contiguous())
      refuse(PyExc_ValueError, "tensors must be contiguous and on the current CUDA device");
  }
}
const at::Tensor* ptr(const OptTensor& t) { return t ? &*t : nullptr; }
void* data(const OptTensor& t) { return t ? t->data_ptr() : nullptr; }

void check_like(const at::Tensor& t, at::ScalarType type, int64_t numel, const char* text) {
  if (t.scalar_type() != type || t.numel() != numel) refuse(PyExc_ValueError, text);
}
at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
  return at::empty(size, like.options().dtype(type).requires_grad(false));
}
// A C entry point (none throws), without the interpreter's lock: a launch may wait
// for room in the GPU's queue, and other Python threads run meanwhile.
template <typename... Want, typename... Given>
dbf_status unlocked(dbf_status (*call)(Want...), Given... args) {
  PyThreadState* const held = PyEval_SaveThread();
  const dbf_status st = call(args...);
  PyEval_RestoreThread(held);
  return st;
}
CUstream_st* stream() { return reinterpret_cast<CUstream_st*>(c10::cuda::getCurrentCUDAStream().stream()); }

void check_status(const char* name, dbf_status st) {
  if (st == DBF_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "si", name, static_cast<int>(st));
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
  throw Refused{};
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = PyTuple_Pack(2, a, b);
  Py_DECREF(a);
  Py_DECREF(b);
  return t;
}

// Codes and scales of a rows x cols matrix: given ones checked, missing ones made.
void mx_buffers(int64_t rows, int64_t cols, int fmt, const at::Tensor& like, OptTensor& codes, OptTensor& scales) {
  const int64_t nc = p_code_bytes(rows, cols, static_cast<dbf_mx_format>(fmt)), ns = p_scale_bytes(rows, cols);
  if (nc == 0) refuse(PyExc_ValueError, "rows or cols outside the MX contract");
  if (!codes) codes = empty({nc}, at::kByte, like);
  else if (codes->scalar_type() != at::kByte || codes->numel() < nc)
    refuse(PyExc_ValueError, "codes must be a uint8 tensor of dbf_mx_code_bytes");
  if (!scales) scales = empty({ns}, at::kByte, like);
  else if (scales->scalar_type() != at::kByte || scales->numel() < ns)
    refuse(PyExc_ValueError, "scales must be a uint8 tensor of dbf_mx_scale_bytes");
}
void check_mx(const at::Tensor& codes, const at::Tensor& scales, int64_t rows, int64_t cols, int fmt) {
  const int64_t nc = p_code_bytes(rows, cols, static_cast<dbf_mx_format>(fmt));
  if (nc == 0) refuse(PyExc_ValueError, "rows or cols outside the MX contract");
  if (codes.scalar_type() != at::kByte || scales.scalar_type() != at::kByte || codes.numel() < nc ||
      scales.numel() < p_scale_bytes(rows, cols))
    refuse(PyExc_ValueError, "codes and scales must be uint8 tensors of dbf_mx_code_bytes and dbf_mx_scale_bytes");
}

// Each function: arguments by position, as the Python functions pass them on.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception&) {  // the types that torch's own calls raise (OutOfMemoryError, ..)
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// (src, fmt, transpose, codes, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    const at::Tensor src = tensor(a[0]);
    const int fmt = format(a[1]), transpose = PyObject_IsTrue(a[2]);
    if (transpose < 0) throw Refused{};
    OptTensor codes = optional_tensor(a[3]), scales = optional_tensor(a[4]);
    if (src.dim() != 2) refuse(PyExc_ValueError, "src must be a 2-D tensor");
    const dbf_dtype t = code_of(src.scalar_type());
    check_place({&src, ptr(codes), ptr(scales)});
    const int64_t rows = src.size(0), cols = src.size(1);
    mx_buffers(transpose ? cols : rows, transpose ? rows : cols, fmt, src, codes, scales);
    check_status("dbf_mx_quantize",
                 unlocked(p_quantize, src.data_ptr(), t, rows, cols, static_cast<dbf_mx_format>(fmt),
                          transpose ? DBF_MX_TRANSPOSE : 0u, static_cast<uint8_t*>(codes->data_ptr()),
                          static_cast<uint8_t*>(scales->data_ptr()), stream()));
    return pair(wrap(*codes), wrap(*scales));
  });
}

// (codes, scales, rows, cols, fmt, dst, dtype)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const at::Tensor codes = tensor(a[0]), scales = tensor(a[1]);
    const int64_t rows = integer(a[2]), cols = integer(a[3]);
    const int fmt = format(a[4]);
    OptTensor dst = optional_tensor(a[5]);
    check_place({&codes, &scales, ptr(dst)});
    check_mx(codes, scales, rows, cols, fmt);
    const dbf_dtype t = code_of(dst ? dst->scalar_type() : dtype(a[6]));
    if (!dst) dst = empty({rows, cols}, dtype(a[6]), codes);
    else if (dst->numel() != rows * cols) refuse(PyExc_ValueError, "dst must have rows * cols elements");
    check_status("dbf_mx_dequantize",
                 unlocked(p_dequantize, static_cast<const uint8_t*>(codes.data_ptr()),
                          static_cast<const uint8_t*>(scales.data_ptr()), rows, cols, static_cast<dbf_mx_format>(fmt),
                          dst->data_ptr(), t, stream()));
    return wrap(*dst);
  });
}

// (x_codes, x_scales, w_codes, w_scales, n, m_in, batch, x_fmt, w_fmt, y, y_dtype, workspace, flags)
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 13, [&] {
    const at::Tensor xc = tensor(a[0]), xs = tensor(a[1]), wc = tensor(a[2]), ws = tensor(a[3]);
    const int64_t n = integer(a[4]), m_in = integer(a[5]), batch = integer(a[6]), flags = integer(a[12]);
    const int xf = format(a[7]), wf = format(a[8]);
    OptTensor y = optional_tensor(a[9]), work = optional_tensor(a[11]);
    if (flags < 0 || flags > 0xffffffffLL) refuse(PyExc_ValueError, "unknown flags");
    check_place({&xc, &xs, &wc, &ws, ptr(y), ptr(work)});
    check_mx(xc, xs, batch, m_in, xf);
    check_mx(wc, ws, n, m_in, wf);
    const dbf_dtype t = code_of(y ? y->scalar_type() : dtype(a[10]));
    if (!y) y = empty({batch, n}, dtype(a[10]), xc);
    else if (y->numel() != batch * n) refuse(PyExc_ValueError, "y must have batch * n elements");
    if (!work) work = at::zeros({static_cast<int64_t>(p_forward_ws(n, m_in, batch))}, xc.options());
    check_status("dbf_mx_forward",
                 unlocked(p_forward, static_cast<const uint8_t*>(xc.data_ptr()),
                          static_cast<const uint8_t*>(xs.data_ptr()), static_cast<dbf_mx_format>(xf),
                          static_cast<const uint8_t*>(wc.data_ptr()), static_cast<const uint8_t*>(ws.data_ptr()),
                          static_cast<dbf_mx_format>(wf), n, m_in, batch, y->data_ptr(), t, work->data_ptr(),
                          work->nbytes(), static_cast<uint32_t>(flags), stream()));
    return wrap(*y);
  });
}

// The norm's operands: x 2-D, weight, residual and h (made where a residual is given without it).
struct Norm {
  at::Tensor x, weight;
  OptTensor residual, h;
  int64_t rows, cols;
  dbf_dtype t;
  Norm(PyObject* x_, PyObject* w_, PyObject* r_, PyObject* h_)
      : x(tensor(x_)), weight(tensor(w_)), residual(optional_tensor(r_)), h(optional_tensor(h_)) {
    if (x.dim() != 2) refuse(PyExc_ValueError, "a 2-D tensor is wanted");
    rows = x.size(0), cols = x.size(1);
    t = code_of(x.scalar_type());
    check_place({&x, &weight, ptr(residual), ptr(h)});
    check_like(weight, x.scalar_type(), cols, "weight must have cols elements of x's type");
    if (!residual && h) refuse(PyExc_ValueError, "h is written only with a residual");
    if (residual) check_like(*residual, x.scalar_type(), rows * cols, "residual must be like x");
    if (h) check_like(*h, x.scalar_type(), rows * cols, "h must be like x");
  }
  void make_h() {
    if (residual && !h) h = empty({rows, cols}, x.scalar_type(), x);
  }
};

// (x, weight, eps, residual, h, y) -> (y, h)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    Norm m(a[0], a[1], a[3], a[4]);
    const float eps = static_cast<float>(number(a[2]));
    OptTensor y = optional_tensor(a[5]);
    check_place({ptr(y)});
    if (y) check_like(*y, m.x.scalar_type(), m.rows * m.cols, "y must be like x");
    else y = empty({m.rows, m.cols}, m.x.scalar_type(), m.x);
    m.make_h();
    check_status("dbf_rmsnorm_forward",
                 unlocked(p_norm, m.x.data_ptr(), data(m.residual), m.weight.data_ptr(), m.t, m.rows, m.cols, eps,
                          data(m.h), y->data_ptr(), stream()));
    PyObject* h = m.h ? wrap(*m.h) : (Py_INCREF(a[0]), a[0]);
    return pair(wrap(*y), h);
  });
}

// (x, weight, eps, fmt, residual, h, codes, scales) -> (codes, scales, h)
PyObject* norm_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    Norm m(a[0], a[1], a[4], a[5]);
    const float eps = static_cast<float>(number(a[2]));
    const int fmt = format(a[3]);
    OptTensor codes = optional_tensor(a[6]), scales = optional_tensor(a[7]);
    check_place({ptr(codes), ptr(scales)});
    mx_buffers(m.rows, m.cols, fmt, m.x, codes, scales);
    m.make_h();
    check_status("dbf_rmsnorm_mx_forward",
                 unlocked(p_norm_mx, m.x.data_ptr(), data(m.residual), m.weight.data_ptr(), m.t, m.rows, m.cols, eps,
                          static_cast<dbf_mx_format>(fmt), data(m.h), static_cast<uint8_t*>(codes->data_ptr()),
                          static_cast<uint8_t*>(scales->data_ptr()), stream()));
    PyObject* c = wrap(*codes);
    PyObject* s = wrap(*scales);
    PyObject* h = m.h ? wrap(*m.h) : (Py_INCREF(a[0]), a[0]);
    PyObject* out = PyTuple_Pack(3, c, s, h);
    Py_DECREF(c);
    Py_DECREF(s);
    Py_DECREF(h);
    return out;
  });
}

// (dy, h, weight, eps, dh, dx, dweight, workspace) -> (dx, dweight)
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    Norm m(a[1], a[2], Py_None, Py_None);
    const at::Tensor dy = tensor(a[0]);
    const float eps = static_cast<float>(number(a[3]));
    OptTensor dh = optional_tensor(a[4]), dx = optional_tensor(a[5]), dw = optional_tensor(a[6]), work = optional_tensor(a[7]);
    check_place({&dy, ptr(dh), ptr(dx), ptr(dw), ptr(work)});
    const int64_t numel = m.rows * m.cols;
    check_like(dy, m.x.scalar_type(), numel, "dy must be like h");
    if (dh) check_like(*dh, m.x.scalar_type(), numel, "dh must be like h");
    if (dx) check_like(*dx, m.x.scalar_type(), numel, "dx must be like h");
    else dx = empty({m.rows, m.cols}, m.x.scalar_type(), m.x);
    if (dw) check_like(*dw, at::kFloat, m.cols, "dweight must be a float32 tensor of cols elements");
    else dw = empty({m.cols}, at::kFloat, m.x);
    if (!work) work = empty({static_cast<int64_t>(p_backward_ws(m.rows, m.cols))}, at::kByte, m.x);
    check_status("dbf_rmsnorm_backward",
                 unlocked(p_norm_backward, dy.data_ptr(), m.x.data_ptr(), m.weight.data_ptr(), data(dh), m.t, m.rows,
                          m.cols, eps, dx->data_ptr(), static_cast<float*>(dw->data_ptr()), work->data_ptr(),
                          work->nbytes(), stream()));
    return pair(wrap(*dx), wrap(*dw));
  });
}

// init(raise_status, addresses of the entry points in the order above)
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long p[10];
  PyObject* raise = nullptr;
  if (!PyArg_ParseTuple(args, "OKKKKKKKKKK", &raise, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7], &p[8], &p[9]))
    return nullptr;
  p_quantize = reinterpret_cast<decltype(p_quantize)>(p[0]);
  p_dequantize = reinterpret_cast<decltype(p_dequantize)>(p[1]);
  p_forward = reinterpret_cast<decltype(p_forward)>(p[2]);
  p_norm = reinterpret_cast<decltype(p_norm)>(p[3]);
  p_norm_mx = reinterpret_cast<decltype(p_norm_mx)>(p[4]);
  p_norm_backward = reinterpret_cast<decltype(p_norm_backward)>(p[5]);
  p_code_bytes = reinterpret_cast<decltype(p_code_bytes)>(p[6]);
  p_scale_bytes = reinterpret_cast<decltype(p_scale_bytes)>(p[7]);
  p_forward_ws = reinterpret_cast<decltype(p_forward_ws)>(p[8]);
  p_backward_ws = reinterpret_cast<decltype(p_backward_ws)>(p[9]);
  Py_INCREF(raise);
  raise_status = raise;
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         FAST(quantize),
                         FAST(dequantize),
                         FAST(forward),
                         FAST(norm),
                         FAST(norm_mx),
                         FAST(norm_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mx_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx_binding() { return PyModule_Create(&module); }
