// The host side of the MXFP4 and gated feed-forward calls: argument checks,
// allocation on the current stream, the C call, and the autograd node of the
// gated projection.  These operators take a few microseconds on the GPU for
// one token; marshalled in Python a call took 11 to 18 us (here 4 to 5), and a
// training step of 777 tokens through a Python autograd node 145 us (here 82).
//
// The functions of the C ABI come as addresses from the library that the
// binding loaded (init), so that the checked build serves here too.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include <unordered_set>
#include <vector>

#include "nvfp4rac.h"

namespace {

using at::Tensor;

struct Api {
  decltype(&mxfp4_quantize) quantize;
  decltype(&mxfp4_dequantize) dequantize;
  decltype(&mxfp4_gemm_quantized) gemm;
  decltype(&mxfp4_gated_gemm) gated_gemm;
  decltype(&mxfp4_linear) linear;
  decltype(&mxfp4_gated_mlp) mlp;
  decltype(&gated_linear_forward) forward;
  decltype(&gated_linear_backward) backward;
  decltype(&gated_linear_saved_bytes) saved_bytes;
  decltype(&nvfp4_workspace_size) workspace;
  decltype(&weight_qdq) qdq;
  decltype(&nvfp4_status_string) status_string;
} api;
constexpr const char* kNames[] = {"mxfp4_quantize",       "mxfp4_dequantize",     "mxfp4_gemm_quantized",
                                  "mxfp4_gated_gemm",     "mxfp4_linear",         "mxfp4_gated_mlp",
                                  "gated_linear_forward", "gated_linear_backward", "gated_linear_saved_bytes",
                                  "nvfp4_workspace_size", "weight_qdq",            "nvfp4_status_string"};
PyObject* status_error;                // raises the binding's error for (status, where)
PyObject *s_codes, *s_scales, *s_rows, *s_cols, *s_layout;

// A status of the library on its way to the Python caller; where autograd's
// engine is between the two, it arrives there as a RuntimeError with this text.
struct Failed : std::runtime_error {
  int status;
  const char* where;
  Failed(int s, const char* w)
      : std::runtime_error(std::string(w) + ": " + api.status_string(static_cast<nvfp4_status>(s)) + " (status " +
                           std::to_string(s) + ")"),
        status(s), where(w) {}
};
void check(nvfp4_status st, const char* where) {
  if (st != NVFP4_OK) throw Failed(static_cast<int>(st), where);
}

#define HOST_BEGIN HANDLE_TH_ERRORS try {
#define HOST_END                                                              \
  }                                                                           \
  catch (const Failed& f) {                                                   \
    PyObject* r = PyObject_CallFunction(status_error, "is", f.status, f.where); \
    Py_XDECREF(r);                                                            \
    return nullptr;                                                           \
  }                                                                           \
  END_HANDLE_TH_ERRORS

const Tensor& tensor(PyObject* o, const char* what) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), what, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// bf16 [..., K] as rows the library can read (16-byte aligned, row stride a
// multiple of 8 and at least K), copied only if it must be.
struct Rows {
  Tensor t;                            // keeps the rows alive
  int64_t M, K, ld;
  const uint16_t* p() const { return static_cast<const uint16_t*>(t.const_data_ptr()); }
};
Rows rows(const Tensor& x, const char* where) {
  TORCH_CHECK_TYPE(x.scalar_type() == at::kBFloat16, where, ": expected a bf16 tensor, got ", x.scalar_type());
  TORCH_CHECK_VALUE(x.is_cuda(), where, ": expected CUDA tensors");
  TORCH_CHECK_VALUE(x.dim() >= 1, where, ": expected at least one dimension");
  Rows r;
  r.K = x.size(-1);
  if (x.dim() == 2) {
    r.t = x;
  } else {
    int64_t m = 1;
    for (int64_t d = 0; d + 1 < x.dim(); ++d) m *= x.size(d);
    r.t = x.reshape({m, r.K});
  }
  r.M = r.t.size(0);
  r.ld = r.M > 1 ? r.t.stride(0) : (r.K + 7) / 8 * 8;
  if (r.t.stride(1) != 1 || r.ld < r.K || r.ld % 8 != 0 ||
      (reinterpret_cast<uintptr_t>(r.t.const_data_ptr()) & 15u) != 0) {
    r.t = r.t.contiguous();
    if ((reinterpret_cast<uintptr_t>(r.t.const_data_ptr()) & 15u) != 0) r.t = r.t.clone();
    r.ld = r.K;
  }
  return r;
}

void on_device(const Tensor& t, const Tensor& like, const char* where) {
  TORCH_CHECK_VALUE(t.is_cuda(), where, ": expected CUDA tensors");
  TORCH_CHECK_VALUE(t.device() == like.device(), where, ": tensors on different devices");
}

// (straight from the CUDA allocator: the dispatcher's way costs as much again)
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

size_t scale_bytes(int64_t rows, int64_t cols, int layout) {
  return layout == 1 ? static_cast<size_t>((rows + 127) / 128 * ((cols + 127) / 128) * 512)
                     : static_cast<size_t>(rows * (cols / 32));
}

int64_t attr_int(PyObject* o, PyObject* name) {
  PyObject* v = PyObject_GetAttr(o, name);
  if (v == nullptr) throw python_error();
  const int64_t n = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (n == -1 && PyErr_Occurred()) throw python_error();
  return n;
}

// Integer and truth arguments: converted first of all in every call, since the
// conversion may run Python code or raise, for which the interpreter's lock has
// to be held.
int as_int(PyObject* o) {
  const long n = PyLong_AsLong(o);
  if (n == -1 && PyErr_Occurred()) throw python_error();
  if (n != static_cast<int>(n)) {
    PyErr_SetString(PyExc_OverflowError, "integer argument out of range");
    throw python_error();
  }
  return static_cast<int>(n);
}
bool as_bool(PyObject* o) {
  const int n = PyObject_IsTrue(o);
  if (n < 0) throw python_error();
  return n != 0;
}
Tensor attr_tensor(PyObject* o, PyObject* name, const char* where) {
  PyObject* v = PyObject_GetAttr(o, name);
  if (v == nullptr) throw python_error();
  if (!THPVariable_Check(v)) {
    Py_DECREF(v);
    TORCH_CHECK_TYPE(false, where, ": codes and scales must be tensors");
  }
  Tensor t = THPVariable_Unpack(v);
  Py_DECREF(v);
  return t;
}

// An MxFP4Tensor argument; its buffers must hold what its shape says.
struct Mx {
  Tensor codes, scales;
  mxfp4_tensor c{};
};
Mx mx(PyObject* o, const char* where) {
  Mx m;
  m.codes = attr_tensor(o, s_codes, where);
  m.scales = attr_tensor(o, s_scales, where);
  m.c.rows = attr_int(o, s_rows);
  m.c.cols = attr_int(o, s_cols);
  m.c.scale_layout = static_cast<int32_t>(attr_int(o, s_layout));
  TORCH_CHECK_VALUE(m.codes.is_cuda(), where, ": expected CUDA tensors");
  on_device(m.scales, m.codes, where);
  TORCH_CHECK_VALUE(m.c.rows >= 0 && m.c.cols >= 0 && m.codes.scalar_type() == at::kByte &&
                        m.scales.scalar_type() == at::kByte && m.codes.is_contiguous() && m.scales.is_contiguous() &&
                        m.codes.numel() >= m.c.rows * (m.c.cols / 2) &&
                        static_cast<size_t>(m.scales.numel()) >= scale_bytes(m.c.rows, m.c.cols, m.c.scale_layout),
                    where, ": an MxFP4Tensor's codes and scales must be contiguous uint8 buffers of its size");
  m.c.codes = static_cast<uint8_t*>(m.codes.data_ptr());
  m.c.scales = static_cast<uint8_t*>(m.scales.data_ptr());
  return m;
}
Mx mx_empty(int64_t rows, int64_t cols, int layout, const Tensor& like) {
  Mx m;
  m.codes = empty({rows, cols / 2}, at::kByte, like);
  m.scales = empty({static_cast<int64_t>(scale_bytes(rows, cols, layout))}, at::kByte, like);
  m.c = {static_cast<uint8_t*>(m.codes.data_ptr()), static_cast<uint8_t*>(m.scales.data_ptr()), rows, cols, layout};
  return m;
}
// An MxFP4Tensor's five fields.
PyObject* mx_fields(const Mx& m) {
  return Py_BuildValue("(NNLLi)", THPVariable_Wrap(m.codes), THPVariable_Wrap(m.scales),
                       static_cast<long long>(m.c.rows), static_cast<long long>(m.c.cols),
                       static_cast<int>(m.c.scale_layout));
}

// The output matrix [lead..., N]: new, or `out` after its checks.
struct Out {
  Tensor t;
  int code;
  int64_t ld;
};
Out output(PyObject* out, at::IntArrayRef lead, int64_t N, int code, const Tensor& like, const char* where) {
  Out o;
  o.code = code;
  c10::SmallVector<int64_t, 8> shape(lead.begin(), lead.end());
  shape.push_back(N);
  const at::ScalarType type = code == 0 ? at::kFloat : at::kBFloat16;
  if (out == Py_None) {
    o.t = empty(shape, type, like);
    o.ld = N > 0 ? N : 1;
    return o;
  }
  o.t = tensor(out, where);
  on_device(o.t, like, where);
  TORCH_CHECK_VALUE(o.t.sizes() == at::IntArrayRef(shape) && o.t.scalar_type() == type, where, ": out must be ", type,
                    " ", at::IntArrayRef(shape));
  int64_t m = 1;
  for (const int64_t d : lead) m *= d;
  const Tensor flat = o.t.dim() == 2 ? o.t : o.t.view({m, N});
  o.ld = m > 1 ? flat.stride(0) : (N > 0 ? N : 1);
  TORCH_CHECK_VALUE((N <= 1 || flat.stride(1) == 1) && o.ld >= N, where,
                    ": out must have contiguous rows that do not overlap");
  return o;
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

// Releases the interpreter around a call of the library.
struct NoGil {
  PyThreadState* s = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(s); }
};

#define WANT(n_)                                                                       \
  if (n != (n_)) {                                                                     \
    PyErr_Format(PyExc_TypeError, "%s: expected %d arguments, got %zd", __func__, n_, n); \
    return nullptr;                                                                    \
  }

// quantize(x, layout, out | None, want_values) -> fields, or (fields, values)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(4)
  const char* where = "mxfp4_quantize";
  const int layout = as_int(a[1]);
  const bool values = as_bool(a[3]);
  const Tensor& x = tensor(a[0], where);
  const Rows r = rows(x, where);
  const c10::cuda::CUDAGuard guard(x.device());
  Mx q = a[2] == Py_None ? mx_empty(r.M, r.K, layout, x) : mx(a[2], where);
  on_device(q.codes, x, where);
  Tensor v = values ? empty(x.sizes(), at::kBFloat16, x) : Tensor();
  nvfp4_status st;
  {
    NoGil g;
    st = api.quantize(r.p(), r.M, r.K, r.ld, &q.c, values ? static_cast<uint16_t*>(v.data_ptr()) : nullptr, r.K,
                      stream_of(x));
  }
  check(st, where);
  PyObject* fields = mx_fields(q);
  return values ? Py_BuildValue("(NN)", fields, THPVariable_Wrap(v)) : fields;
  HOST_END
}

Tensor qdq_mx(const Tensor& x, const char* where) {
  const Rows r = rows(x, where);
  Tensor v = empty(x.sizes(), at::kBFloat16, x);
  check(api.quantize(r.p(), r.M, r.K, r.ld, nullptr, static_cast<uint16_t*>(v.data_ptr()), r.K, stream_of(x)),
        "mxfp4_quantize");
  return v;
}

// qdq(x) -> values
PyObject* qdq(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(1)
  const Tensor& x = tensor(a[0], "mxfp4_qdq");
  TORCH_CHECK_VALUE(x.is_cuda(), "mxfp4_qdq: expected CUDA tensors");
  const c10::cuda::CUDAGuard guard(x.device());
  return THPVariable_Wrap(qdq_mx(x, "mxfp4_qdq"));
  HOST_END
}

// dequantize(q, dtype code, out | None) -> y
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(3)
  const char* where = "mxfp4_dequantize";
  const int code = as_int(a[1]);
  const Mx q = mx(a[0], where);
  const c10::cuda::CUDAGuard guard(q.codes.device());
  const Out y = output(a[2], {q.c.rows}, q.c.cols, code, q.codes, where);
  nvfp4_status st;
  {
    NoGil g;
    st = api.dequantize(&q.c, y.t.data_ptr(), y.code, y.ld, stream_of(q.codes));
  }
  check(st, where);
  return THPVariable_Wrap(y.t);
  HOST_END
}

// gemm(a, b, dtype code, out | None) -> y
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(4)
  const char* where = "mxfp4_gemm";
  const int code = as_int(a[2]);
  const Mx qa = mx(a[0], where), qb = mx(a[1], where);
  on_device(qb.codes, qa.codes, where);
  const c10::cuda::CUDAGuard guard(qa.codes.device());
  const Out y = output(a[3], {qa.c.rows}, qb.c.rows, code, qa.codes, where);
  nvfp4_status st;
  {
    NoGil g;
    st = api.gemm(&qa.c, &qb.c, y.t.data_ptr(), y.code, y.ld, stream_of(qa.codes));
  }
  check(st, "mxfp4_gemm_quantized");
  return THPVariable_Wrap(y.t);
  HOST_END
}

// gated_gemm(x, gate, up, act code, dtype code | 2 for MXFP4, out | None) -> y, or fields
PyObject* gated_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(6)
  const char* where = "mxfp4_gated_gemm";
  const int act = as_int(a[3]), code = as_int(a[4]);
  const Mx x = mx(a[0], where), g = mx(a[1], where), u = mx(a[2], where);
  on_device(g.codes, x.codes, where);
  on_device(u.codes, x.codes, where);
  const c10::cuda::CUDAGuard guard(x.codes.device());
  nvfp4_status st;
  if (code == 2) {
    Mx q = a[5] == Py_None ? mx_empty(x.c.rows, g.c.rows, 1, x.codes) : mx(a[5], where);
    on_device(q.codes, x.codes, where);
    {
      NoGil ng;
      st = api.gated_gemm(&x.c, &g.c, &u.c, act, nullptr, 0, 0, &q.c, stream_of(x.codes));
    }
    check(st, where);
    return mx_fields(q);
  }
  const Out y = output(a[5], {x.c.rows}, g.c.rows, code, x.codes, where);
  {
    NoGil ng;
    st = api.gated_gemm(&x.c, &g.c, &u.c, act, y.t.data_ptr(), y.code, y.ld, nullptr, stream_of(x.codes));
  }
  check(st, where);
  return THPVariable_Wrap(y.t);
  HOST_END
}

// linear(x, w, dtype code, out | None) -> y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(4)
  const char* where = "mxfp4_linear";
  const int code = as_int(a[2]);
  const Tensor& x = tensor(a[0], where);
  const Rows r = rows(x, where);
  const Mx w = mx(a[1], where);
  on_device(w.codes, x, where);
  const c10::cuda::CUDAGuard guard(x.device());
  const Out y = output(a[3], x.sizes().slice(0, x.dim() - 1), w.c.rows, code, x, where);
  const size_t bytes = api.workspace(NVFP4_OP_MXFP4_LINEAR, r.M, 0, r.K, 1);
  const Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, x);
  nvfp4_status st;
  {
    NoGil g;
    st = api.linear(r.p(), r.M, r.K, r.ld, &w.c, y.t.data_ptr(), y.code, y.ld, ws.data_ptr(), bytes, stream_of(x));
  }
  check(st, where);
  return THPVariable_Wrap(y.t);
  HOST_END
}

// mlp(x, gate, up, down, act code, dtype code, out | None) -> y
PyObject* mlp(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(7)
  const char* where = "mxfp4_gated_mlp";
  const int act = as_int(a[4]), code = as_int(a[5]);
  const Tensor& x = tensor(a[0], where);
  const Rows r = rows(x, where);
  const Mx g = mx(a[1], where), u = mx(a[2], where), d = mx(a[3], where);
  on_device(g.codes, x, where);
  on_device(u.codes, x, where);
  on_device(d.codes, x, where);
  const c10::cuda::CUDAGuard guard(x.device());
  const Out y = output(a[6], x.sizes().slice(0, x.dim() - 1), d.c.rows, code, x, where);
  const size_t bytes = api.workspace(NVFP4_OP_MXFP4_MLP, r.M, g.c.rows, r.K, 1);
  const Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, x);
  nvfp4_status st;
  {
    NoGil ng;
    st = api.mlp(r.p(), r.M, r.K, r.ld, &g.c, &u.c, &d.c, act, y.t.data_ptr(), y.code, y.ld, ws.data_ptr(), bytes,
                 stream_of(x));
  }
  check(st, where);
  return THPVariable_Wrap(y.t);
  HOST_END
}

// ---- the trainer's gated projection ----------------------------------------------
struct Gated {
  Rows x, g, u;
  int64_t F;
};
Gated gated_operands(const Tensor& x, const Tensor& wg, const Tensor& wu, const char* where) {
  Gated o{rows(x, where), rows(wg, where), rows(wu, where), wg.dim() == 2 ? wg.size(0) : -1};
  on_device(wg, x, where);
  on_device(wu, x, where);
  TORCH_CHECK_VALUE(wg.dim() == 2 && wu.dim() == 2 && wg.sizes() == wu.sizes() && o.g.K == o.x.K, where,
                    ": x [..., K] with two weights [F, K], got K = ", o.x.K, " and ", wg.sizes(), ", ", wu.sizes());
  if (o.g.ld != o.u.ld) {              // one row stride for both
    o.g.t = o.g.t.contiguous();
    o.u.t = o.u.t.contiguous();
    o.g.ld = o.u.ld = o.x.K;
  }
  return o;
}
c10::SmallVector<int64_t, 8> with_last(const Tensor& x, int64_t last) {
  c10::SmallVector<int64_t, 8> s(x.sizes().begin(), x.sizes().end());
  s.back() = last;
  return s;
}

Tensor forward_call(const Tensor& x, const Tensor& wg, const Tensor& wu, int act, bool save, Tensor* saved) {
  const char* where = "gated_linear_forward";
  const Gated o = gated_operands(x, wg, wu, where);
  Tensor h = empty(with_last(x, o.F), at::kBFloat16, x);
  if (save) *saved = empty({static_cast<int64_t>(api.saved_bytes(o.x.M, o.F) / 4)}, at::kFloat, x);
  check(api.forward(o.x.p(), o.x.M, o.x.K, o.x.ld, o.g.p(), o.u.p(), o.F, o.g.ld, act,
                    static_cast<uint16_t*>(h.data_ptr()), o.F, save ? static_cast<float*>(saved->data_ptr()) : nullptr,
                    stream_of(x)),
        where);
  return h;
}

void backward_call(const Tensor& x, const Tensor& wg, const Tensor& wu, const Tensor& dh, int act, const Tensor& saved,
                   const bool (&need)[3], Tensor (&grad)[3]) {
  const char* where = "gated_linear_backward";
  const Gated o = gated_operands(x, wg, wu, where);
  TORCH_CHECK_VALUE(dh.sizes() == at::IntArrayRef(with_last(x, o.F)), where, ": dh must be ",
                    at::IntArrayRef(with_last(x, o.F)), ", got ", dh.sizes());
  const Rows d = rows(dh, where);
  on_device(dh, x, where);
  if (saved.defined()) {
    on_device(saved, x, where);
    TORCH_CHECK_VALUE(saved.scalar_type() == at::kFloat && saved.is_contiguous() &&
                          static_cast<size_t>(saved.numel()) * 4 == api.saved_bytes(o.x.M, o.F),
                      where, ": saved is not the forward call's");
  }
  if (need[0]) grad[0] = empty(x.sizes(), at::kBFloat16, x);
  if (need[1]) grad[1] = empty({o.F, o.x.K}, at::kBFloat16, x);
  if (need[2]) grad[2] = empty({o.F, o.x.K}, at::kBFloat16, x);
  const size_t bytes =
      api.workspace(saved.defined() ? NVFP4_OP_GATED_BACKWARD : NVFP4_OP_GATED_RECOMPUTE, o.x.M, o.F, 0, 1);
  const Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, x);
  auto ptr = [](Tensor& t) { return t.defined() ? static_cast<uint16_t*>(t.data_ptr()) : nullptr; };
  check(api.backward(o.x.p(), o.x.M, o.x.K, o.x.ld, o.g.p(), o.u.p(), o.F, o.g.ld, act, d.p(), d.ld,
                     saved.defined() ? static_cast<const float*>(saved.const_data_ptr()) : nullptr, ptr(grad[0]), o.x.K,
                     ptr(grad[1]), ptr(grad[2]), ws.data_ptr(), bytes, stream_of(x)),
        where);
}

// gated_forward(x, w_gate, w_up, act code, save) -> h, or (h, saved)
PyObject* gated_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(5)
  const int act = as_int(a[3]);
  const bool save = as_bool(a[4]);
  const Tensor &x = tensor(a[0], "gated_linear_forward"), &g = tensor(a[1], "gated_linear_forward"),
               &u = tensor(a[2], "gated_linear_forward");
  TORCH_CHECK_VALUE(x.is_cuda(), "gated_linear_forward: expected CUDA tensors");
  const c10::cuda::CUDAGuard guard(x.device());
  const at::NoGradGuard no_grad;
  Tensor saved;
  Tensor h = forward_call(x, g, u, act, save, &saved);
  return save ? Py_BuildValue("(NN)", THPVariable_Wrap(h), THPVariable_Wrap(saved)) : THPVariable_Wrap(h);
  HOST_END
}

// gated_backward(x, w_gate, w_up, dh, act code, saved | None, (need x, gate, up)) -> (dx, dw_gate, dw_up)
PyObject* gated_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(7)
  const char* where = "gated_linear_backward";
  const int act = as_int(a[4]);
  TORCH_CHECK_VALUE(PyTuple_Check(a[6]) && PyTuple_GET_SIZE(a[6]) == 3, where, ": need is a tuple of three");
  bool need[3];
  for (int i = 0; i < 3; ++i) need[i] = as_bool(PyTuple_GET_ITEM(a[6], i));
  const Tensor &x = tensor(a[0], where), &g = tensor(a[1], where), &u = tensor(a[2], where), &dh = tensor(a[3], where);
  TORCH_CHECK_VALUE(x.is_cuda(), where, ": expected CUDA tensors");
  const c10::cuda::CUDAGuard guard(x.device());
  const at::NoGradGuard no_grad;
  const Tensor saved = a[5] == Py_None ? Tensor() : tensor(a[5], where);
  Tensor grad[3];
  backward_call(x, g, u, dh, act, saved, need, grad);
  PyObject* r = PyTuple_New(3);
  for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(grad[i]));   // (undefined: None)
  return r;
  HOST_END
}

// The fake-quantized form of t: fmt 1 NVFP4, 2 MXFP4.
Tensor fake_quantized(const Tensor& t, int64_t fmt) {
  if (fmt == 2) return qdq_mx(t, "mxfp4_qdq");
  TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16, "weight_qdq: expected a bf16 tensor");
  TORCH_CHECK_VALUE(t.is_cuda(), "weight_qdq: expected CUDA tensors");
  const int64_t K = t.size(-1);
  const Tensor w = t.contiguous();
  const int64_t N = K > 0 ? w.numel() / K : 0;
  Tensor out = at::empty_like(w);
  if (N == 0) return out;
  const size_t bytes = api.workspace(NVFP4_OP_WEIGHT_QDQ, 0, N, K, 1);
  const Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, t);
  check(api.qdq(static_cast<const uint16_t*>(w.const_data_ptr()), N, K, K, 1, static_cast<uint16_t*>(out.data_ptr()),
                nullptr, nullptr, ws.data_ptr(), bytes, stream_of(t)),
        "weight_qdq");
  return out;
}

// A leaf's gradient accumulator belongs to the stream on which the first graph
// that holds it was built.  If that is the default stream, which no capture can
// join, a captured backward pass that reaches it ends the process.
bool on_default_stream(torch::autograd::Node& accumulator) {
  const auto s = accumulator.stream();
  return s.has_value() && c10::cuda::CUDAStream(*s) == c10::cuda::getDefaultCUDAStream(s->device_index());
}
constexpr const char* kEagerGraph =
    ": captured while an eager graph of the same leaf, built on the default stream, lives; "
    "release it (its loss and outputs) before the capture";

// Called by a node of this package in its backward pass: refuses a captured one
// before the gradients it returns reach such an accumulator, directly or through
// the nodes between (a leaf's views, other layers).  Nodes that this pass does
// not run (torch.autograd.grad with respect to something nearer) do not count.
void check_backward(const char* where) {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
  const auto from = torch::autograd::get_current_node();
  if (from == nullptr) return;
  const auto* run = torch::autograd::get_current_graph_task_exec_info();
  std::vector<torch::autograd::Node*> todo{from.get()};
  std::unordered_set<torch::autograd::Node*> seen{from.get()};
  while (!todo.empty()) {
    torch::autograd::Node* n = todo.back();
    todo.pop_back();
    for (const auto& e : n->next_edges()) {
      torch::autograd::Node* f = e.function.get();
      if (f == nullptr || !seen.insert(f).second) continue;
      if (run != nullptr && !run->empty()) {
        const auto it = run->find(f);
        if (it == run->end() || !it->second.should_execute()) continue;
      }
      if (dynamic_cast<torch::autograd::AccumulateGrad*>(f) != nullptr)
        TORCH_CHECK(!on_default_stream(*f), where, kEagerGraph);
      todo.push_back(f);
    }
  }
}

// check_backward(name of the call)
PyObject* backward_capturable(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(1)
  const char* where = PyUnicode_AsUTF8(a[0]);
  if (where == nullptr) return nullptr;
  check_backward(where);
  Py_RETURN_NONE;
  HOST_END
}

// The gated projection as one autograd node: on fake-quantized weights with
// fmt, and activations with act_quant; the gradient crosses the fake quantizers
// unchanged.
struct GatedLinear : public torch::autograd::Function<GatedLinear> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x0, const Tensor& wg0, const Tensor& wu0,
                        int64_t act, bool keep, int64_t fmt, bool act_quant) {
    const Tensor x = act_quant ? fake_quantized(x0, fmt) : x0;
    const Tensor wg = fmt ? fake_quantized(wg0, fmt) : wg0, wu = fmt ? fake_quantized(wu0, fmt) : wu0;
    Tensor saved;
    Tensor h = forward_call(x, wg, wu, static_cast<int>(act), keep, &saved);
    ctx->save_for_backward({x, wg, wu, saved});
    ctx->saved_data["act"] = act;
    return h;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list dh) {
    torch::autograd::variable_list out(7);
    const auto s = ctx->get_saved_variables();
    const bool need[3] = {ctx->needs_input_grad(0), ctx->needs_input_grad(1), ctx->needs_input_grad(2)};
    if (!dh[0].defined() || !(need[0] || need[1] || need[2])) return out;
    Tensor grad[3];
    {
      const at::NoGradGuard no_grad;
      const c10::cuda::CUDAGuard guard(s[0].device());
      check_backward("gated_linear");
      backward_call(s[0], s[1], s[2], dh[0], static_cast<int>(ctx->saved_data["act"].toInt()), s[3], need, grad);
    }
    torch::autograd::variable_list given;
    for (const Tensor& t : grad)
      if (t.defined()) given.push_back(t);
    if (at::GradMode::is_enabled()) {
      // there is no second derivative: whoever asks for one gets an error
      auto node = std::make_shared<torch::autograd::DelayedError>("gated_linear has no second derivative",
                                                                  static_cast<int64_t>(given.size()));
      for (Tensor& t : given) t.set_requires_grad(true);
      given = (*node)(std::move(given));
    }
    size_t at = 0;
    for (int i = 0; i < 3; ++i)
      if (grad[i].defined()) out[i] = given[at++];
    return out;
  }
};

// Refuses a differentiable call on a leaf that is being captured while an eager
// graph of that leaf, built on the default stream, lives: before anything of it
// is captured, where check_backward would refuse its backward pass.
void check_capture(std::initializer_list<const Tensor*> leaves, const char* where) {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
  for (const Tensor* t : leaves) {
    if (!t->requires_grad() || !t->is_leaf()) continue;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
    TORCH_CHECK(node == nullptr || !on_default_stream(*node), where, kEagerGraph);
  }
}

// check_capture(leaf, name of the call)
PyObject* capturable(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(2)
  const char* where = PyUnicode_AsUTF8(a[1]);
  if (where == nullptr) return nullptr;
  const Tensor& t = tensor(a[0], where);
  if (t.is_cuda()) {
    const c10::cuda::CUDAGuard guard(t.device());
    check_capture({&t}, where);
  }
  Py_RETURN_NONE;
  HOST_END
}

// gated_linear(x, w_gate, w_up, act code, recompute, fmt code, act_quant, grad enabled) -> h
PyObject* gated_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HOST_BEGIN
  WANT(8)
  const char* where = "gated_linear";
  const int act = as_int(a[3]), fmt = as_int(a[5]);
  const bool recompute = as_bool(a[4]), act_quant = as_bool(a[6]), enabled = as_bool(a[7]);
  const Tensor &x = tensor(a[0], where), &g = tensor(a[1], where), &u = tensor(a[2], where);
  TORCH_CHECK_VALUE(x.is_cuda(), where, ": expected CUDA tensors");
  const c10::cuda::CUDAGuard guard(x.device());
  const bool grads = enabled && (x.requires_grad() || g.requires_grad() || u.requires_grad());
  if (grads) check_capture({&x, &g, &u}, where);
  return THPVariable_Wrap(GatedLinear::apply(x, g, u, act, grads && !recompute, fmt, act_quant));
  HOST_END
}

// init({name: address}, callable raising for (status, where))
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  WANT(2)
  void** slot = reinterpret_cast<void**>(&api);
  static_assert(sizeof(Api) == sizeof(kNames), "one address per name");
  for (const char* name : kNames) {
    PyObject* v = PyDict_GetItemString(a[0], name);
    if (v == nullptr) {
      PyErr_Format(PyExc_KeyError, "init: no address of %s", name);
      return nullptr;
    }
    *slot++ = PyLong_AsVoidPtr(v);
  }
  Py_INCREF(a[1]);
  status_error = a[1];
  s_codes = PyUnicode_InternFromString("codes");
  s_scales = PyUnicode_InternFromString("scales");
  s_rows = PyUnicode_InternFromString("rows");
  s_cols = PyUnicode_InternFromString("cols");
  s_layout = PyUnicode_InternFromString("layout");
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init),   METHOD(quantize), METHOD(qdq),           METHOD(dequantize),
                         METHOD(gemm),   METHOD(gated_gemm), METHOD(linear),      METHOD(mlp),
                         METHOD(gated_forward), METHOD(gated_backward), METHOD(gated_linear), METHOD(capturable),
                         METHOD(backward_capturable), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_against", HOST_BUILT_AGAINST) != 0) Py_CLEAR(m);
  return m;
}
