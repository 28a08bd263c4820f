// The feed-forward helpers of gptq.py as torch programs call them: checks of the tensors, output tensors,
// and the call of the C entry point.  Marshalling alone; the computation is the library's.
//
// Compiled because these run for every token: a Python helper reads about fifty tensor attributes and
// makes two to four tensors for a call, 16 to 27 us of host time (fp8_linear, fp8_gated), where the
// kernels of a small call take 2 to 19; here it is 4 to 6, and 5 to 8 for moe_route.
#include <Python.h>

#include <string>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gptq.h"

namespace {

constexpr int64_t kBlock = 128;

// Set by bind(): the library's entry points, and what raises for a status.
struct Entry {
  decltype(&gptq_fp8_linear) linear;
  decltype(&gptq_fp8_gated) gated;
  decltype(&gptq_fp8_experts) experts;
  decltype(&gptq_fp8_experts_gated) experts_gated;
  decltype(&gptq_moe_route) route;
  decltype(&gptq_moe_route_workspace_bytes) route_ws;
  decltype(&gptq_moe_combine) combine;
} g_entry;
PyObject *g_check = nullptr;

// Thrown with a Python error set.
struct Raised {};
[[noreturn]] void raise(PyObject *type, const std::string &what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}
[[noreturn]] void value_error(const std::string &what) { raise(PyExc_ValueError, what); }
[[noreturn]] void type_error(const std::string &what) { raise(PyExc_TypeError, what); }

// f() as a Python function: C++ exceptions end here, torch's as torch raises them.
template <typename F>
PyObject *guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
// None as an undefined tensor.
at::Tensor maybe(PyObject *o, const char *name) { return o == Py_None ? at::Tensor() : tensor(o, name); }

int gpu_of(const at::Tensor &t) { return t.is_cuda() ? (int)t.get_device() : -1; }
// Every tensor of a call has to be on one GPU, and that the current one (the kernels take addresses,
// and the default stream's handle means the current device's).
void on(const at::Tensor &t, int gpu) {
  if (gpu < 0 || gpu_of(t) != gpu) value_error("a call's tensors must be on one GPU");
}

std::string sizes_of(std::initializer_list<int64_t> sizes) {
  std::string s = "[";
  for (int64_t n : sizes) s += (s.size() > 1 ? ", " : "") + (n < 0 ? std::string("any") : std::to_string(n));
  return s + "]";
}

// Row pitch of a row-major matrix of the given size (-1: any).
int64_t rows_of(const char *name, const at::Tensor &t, int64_t rows = -1, int64_t d = -1) {
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (d >= 0 && t.size(1) != d) ||
      (t.stride(1) != 1 && t.size(1) != 1))
    value_error(std::string(name) + " must be a row-major " + sizes_of({rows, d}) + " matrix");
  return t.size(0) != 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
}

int dtype_code(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kHalf: return GPTQ_F16;
    case at::kBFloat16: return GPTQ_BF16;
    case at::kFloat: return GPTQ_F32;
    default: type_error("unsupported dtype " + std::string(c10::toString(t.scalar_type())));
  }
}

template <typename T>
T *ptr(const at::Tensor &t) { return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr; }
template <typename T>
const T *cptr(const at::Tensor &t) { return t.defined() ? static_cast<const T *>(t.const_data_ptr()) : nullptr; }
const uint8_t *bytes(const at::Tensor &t) { return static_cast<const uint8_t *>(t.const_data_ptr()); }

// A contiguous float32 vector (or [experts, n]); undefined is fine.
void floats(const at::Tensor &t, const std::string &name, at::IntArrayRef shape, int gpu) {
  if (!t.defined()) return;
  if (t.scalar_type() != at::kFloat || t.sizes() != shape || !t.is_contiguous()) {
    std::string s;
    for (int64_t n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
    value_error(name + " must be contiguous float32 [" + s + "]");
  }
  on(t, gpu);
}
void code_types(const at::Tensor &codes, const at::Tensor &exps) {
  if (codes.scalar_type() != at::kFloat8_e4m3fn || exps.scalar_type() != at::kByte)
    type_error("codes are float8_e4m3fn and exponents uint8");
}

// Activations: codes [m, k] and exponents.
struct Acts {
  at::Tensor codes, exps, scale;
  int64_t m, k, ld, lde;
  int gpu;
};
Acts acts(PyObject *a, PyObject *e, PyObject *scale) {
  Acts r{tensor(a, "a"), tensor(e, "a_exps"), maybe(scale, "a_scale"), 0, 0, 0, 0, -1};
  r.ld = rows_of("a", r.codes);
  r.m = r.codes.size(0);
  r.k = r.codes.size(1);
  r.lde = rows_of("a_exps", r.exps, r.m, (r.k + kBlock - 1) / kBlock);
  code_types(r.codes, r.exps);
  r.gpu = gpu_of(r.codes);
  on(r.exps, r.gpu);
  floats(r.scale, "a_scale", {r.m}, r.gpu);
  return r;
}

// Weights [n, k], or [experts, n, k] where experts > 0; n < 0: any.
struct Weights {
  int64_t n;
  gptq_fp8_weights w;
};
Weights weights(const char *name, const at::Tensor &w, const at::Tensor &e, const at::Tensor &scale,
                const at::Tensor &bias, int64_t k, int gpu, int64_t n = -1, int64_t experts = 0) {
  const int lead = experts > 0 ? 1 : 0;
  const int64_t kb = (k + kBlock - 1) / kBlock;
  if (w.dim() != 2 + lead || (lead && w.size(0) != experts) || w.size(lead + 1) != k || w.stride(lead + 1) != 1 ||
      (n >= 0 && w.size(lead) != n))
    value_error(std::string(name) + " must be row-major " + (lead ? sizes_of({experts, n, k}) : sizes_of({n, k})));
  const int64_t rows = w.size(lead), nb = (rows + kBlock - 1) / kBlock;
  if (e.dim() != 2 + lead || (lead && e.size(0) != experts) || e.size(lead) != nb || e.size(lead + 1) != kb ||
      (e.stride(lead + 1) != 1 && kb != 1))
    value_error("the exponents of " + std::string(name) + " must be row-major " +
                (lead ? sizes_of({experts, nb, kb}) : sizes_of({nb, kb})));
  code_types(w, e);
  on(w, gpu);
  on(e, gpu);
  const int64_t both[2] = {experts, rows};
  const at::IntArrayRef shape(both + 1 - lead, 1 + lead);
  floats(scale, "the scale of " + std::string(name), shape, gpu);
  floats(bias, "the bias of " + std::string(name), shape, gpu);
  Weights r{rows, {}};
  // (the step from the only row to the next has no meaning: any will do that the library takes)
  r.w.codes = bytes(w);
  r.w.ld = rows == 1 ? (k + 15) & ~(int64_t)15 : w.stride(lead);
  r.w.next_codes = lead ? w.stride(0) : 0;
  r.w.exps = bytes(e);
  r.w.ld_exps = nb == 1 ? (kb + 3) & ~(int64_t)3 : e.stride(lead);
  r.w.next_exps = lead ? e.stride(0) : 0;
  r.w.scale = cptr<float>(scale);
  r.w.bias = cptr<float>(bias);
  return r;
}
// From a sequence (codes, exps[, scale[, bias]]).
Weights weights(const char *name, PyObject *o, int64_t k, int gpu, int64_t n = -1, int64_t experts = 0) {
  if (!PyTuple_Check(o) && !PyList_Check(o))
    type_error(std::string(name) + " must be (codes, exps[, scale[, bias]])");
  const Py_ssize_t len = PySequence_Fast_GET_SIZE(o);
  if (len < 2 || len > 4) value_error(std::string(name) + " must be (codes, exps[, scale[, bias]])");
  PyObject **item = PySequence_Fast_ITEMS(o);
  return weights(name, tensor(item[0], name), tensor(item[1], name), len > 2 ? maybe(item[2], name) : at::Tensor(),
                 len > 3 ? maybe(item[3], name) : at::Tensor(), k, gpu, n, experts);
}

int act_code(PyObject *o) {
  if (o == Py_None) return GPTQ_ACT_NONE;
  const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  const std::string act = s ? s : "";
  if (act == "none") return GPTQ_ACT_NONE;
  if (act == "relu") return GPTQ_ACT_RELU;
  if (act == "silu") return GPTQ_ACT_SILU;
  if (act == "gelu") return GPTQ_ACT_GELU;
  value_error("act must be one of 'none', 'relu', 'silu', 'gelu' or None");
}

// What a call runs on, and the stream that its new tensors are lent to.
struct Run {
  gptq_stream_t stream;
  c10::optional<c10::cuda::CUDAStream> lent;
  void lend(const at::Tensor &t) const {
    if (lent) t.record_stream(lent->unwrap());
  }
};
Run run_on(PyObject *stream, int gpu) {
  if ((int)c10::cuda::current_device() != gpu) value_error("a call's tensors must be on the current device");
  if (stream == Py_None) return {(gptq_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)gpu).stream(), {}};
  PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
  if (!h) throw Raised{};
  void *raw = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!raw && PyErr_Occurred()) throw Raised{};
  return {(gptq_stream_t)raw, c10::cuda::getStreamFromExternal((cudaStream_t)raw, (c10::DeviceIndex)gpu)};
}

// Elements of a workspace are counted as its bytes: it has to hold them.
void holds(const at::Tensor &ws, int gpu) {
  if (!ws.is_contiguous()) value_error("ws must be contiguous");
  on(ws, gpu);
}

// The workspace given, or one block for each device: its status is not read back (serving_status tells
// of a wait that gave up).  Never freed: the process may end after CUDA has.
const at::Tensor &workspace(const at::Tensor &ws, const at::Tensor &like, int gpu) {
  static at::Tensor *blocks[128] = {};
  if (ws.defined()) {
    holds(ws, gpu);
    return ws;
  }
  if (gpu >= 128) value_error("more devices than a status block is kept for");
  if (!blocks[gpu]) blocks[gpu] = new at::Tensor(at::empty({256}, like.options().dtype(at::kByte)));
  return *blocks[gpu];
}

at::Tensor strided(int64_t rows, int64_t d, int64_t pitch, at::ScalarType type, const at::Tensor &like) {
  const int64_t size[2] = {rows, d}, stride[2] = {pitch, 1};
  return at::empty_strided(size, stride, like.options().dtype(type));
}

// The outputs of a call that has several, and a workspace, from one allocation: tensors of one storage, at
// multiples of 256 bytes.  (Each by itself takes 0.7 to 1.4 us: moe_route 6.9 and 10.6 us, now 4.8 and 7.6.)
class Together {
 public:
  // Room for `bytes`: where it begins.
  int64_t add(int64_t bytes) {
    const int64_t at = size_;
    size_ += (bytes + 255) & ~(int64_t)255;
    return at;
  }
  void allocate(const at::Tensor &like, const Run &run) {
    all_ = at::empty({size_}, like.options().dtype(at::kByte));
    run.lend(all_);
  }
  at::Tensor tensor(int64_t at, at::IntArrayRef size, at::IntArrayRef stride, at::ScalarType type) const {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all_.storage()), all_.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_and_strides(size, stride, at / (int64_t)c10::elementSize(type));
    return t;
  }
  void *address(int64_t at) const { return static_cast<uint8_t *>(all_.data_ptr()) + at; }

 private:
  int64_t size_ = 0;
  at::Tensor all_;
};

// Codes and exponents [rows, n] in the pitches that the library asks for, the last row's whole.
struct Coded {
  at::Tensor codes, exps;
  int64_t ldc, lde;
};
Coded coded(int64_t rows, int64_t n, const at::Tensor &like, const Run &run) {
  const int64_t ldc = (n + 15) & ~(int64_t)15, nb = (n + kBlock - 1) / kBlock, lde = (nb + 3) & ~(int64_t)3;
  Together both;
  const int64_t codes = both.add(rows * ldc), exps = both.add(rows * lde);
  both.allocate(like, run);
  return {both.tensor(codes, {rows, n}, {ldc, 1}, at::kFloat8_e4m3fn), both.tensor(exps, {rows, nb}, {lde, 1}, at::kByte),
          ldc, lde};
}

// A 16-bit output: the one given, or a new one.
struct Out {
  at::Tensor t;
  int64_t ld;
};
Out out16(PyObject *out, PyObject *dtype, int64_t rows, int64_t n, const at::Tensor &like, int gpu, const Run &run) {
  at::ScalarType type = at::kBFloat16;
  if (dtype != Py_None) {
    if (!THPDtype_Check(dtype)) type_error("out_dtype must be a torch dtype");
    type = reinterpret_cast<THPDtype *>(dtype)->scalar_type;
  }
  if (out == Py_None) {
    Out r{strided(rows, n, n, type, like), n};
    run.lend(r.t);
    return r;
  }
  Out r{tensor(out, "out"), 0};
  r.ld = rows_of("out", r.t, rows, n);
  if (dtype != Py_None && r.t.scalar_type() != type) type_error("out must have out_dtype");
  on(r.t, gpu);
  return r;
}

// moe_route's offsets and order of `rows` assignments: the number of experts.
int64_t plan(const at::Tensor &offsets, const at::Tensor &order, int64_t rows, int gpu) {
  if (offsets.scalar_type() != at::kInt || order.scalar_type() != at::kInt) type_error("offsets and order must be int32");
  if (offsets.dim() != 1 || offsets.size(0) < 2 || !offsets.is_contiguous() || order.dim() != 1 ||
      order.size(0) != rows || !order.is_contiguous())
    value_error("offsets [experts + 1] and order [" + std::to_string(rows) + "] as moe_route returns them");
  on(offsets, gpu);
  on(order, gpu);
  return offsets.size(0) - 1;
}

PyObject *wrap2(const at::Tensor &a, const at::Tensor &b) {
  return Py_BuildValue("(NN)", THPVariable_Wrap(a), THPVariable_Wrap(b));
}

// Raises for a status that is not OK.
bool fine(int status, const char *where) {
  if (status == GPTQ_OK) return true;
  PyObject *r = PyObject_CallFunction(g_check, "is", status, where);
  Py_XDECREF(r);
  return false;
}
#define CALL(where, status, ...)   \
  int status;                      \
  Py_BEGIN_ALLOW_THREADS status = __VA_ARGS__; \
  Py_END_ALLOW_THREADS             \
  if (!fine(status, where)) return nullptr

template <PyObject *(*F)(PyObject *const *), int COUNT>
PyObject *method(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
  if (nargs != COUNT) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected", COUNT);
    return nullptr;
  }
  return guarded([v] { return F(v); });
}
template <PyObject *(*F)(PyObject *const *), int COUNT>
PyMethodDef def(const char *name) {
  return {name, (PyCFunction)(void *)method<F, COUNT>, METH_FASTCALL, nullptr};
}

// (a, a_exps, w, w_exps, a_scale, w_scale, bias, act, residual, out_dtype, out, ws, stream)
PyObject *linear(PyObject *const *v) {
  const Acts a = acts(v[0], v[1], v[4]);
  const Weights w = weights("w", tensor(v[2], "w"), tensor(v[3], "w_exps"), maybe(v[5], "w_scale"), maybe(v[6], "bias"),
                            a.k, a.gpu);
  const int act = act_code(v[7]);
  const Run run = run_on(v[12], a.gpu);
  const Out out = out16(v[10], v[9], a.m, w.n, a.codes, a.gpu, run);
  const at::Tensor residual = maybe(v[8], "residual");
  int64_t ldr = 0;
  if (residual.defined()) {
    ldr = rows_of("residual", residual, a.m, w.n);
    if (residual.scalar_type() != out.t.scalar_type()) type_error("residual must have the output's dtype");
    on(residual, a.gpu);
  }
  const at::Tensor ws = workspace(maybe(v[11], "ws"), a.codes, a.gpu);
  CALL("gptq_fp8_linear", st, g_entry.linear(bytes(a.codes), a.ld, bytes(a.exps), a.lde, cptr<float>(a.scale), &w.w, act,
                                             cptr<void>(residual), ldr, a.m, w.n, a.k, ptr<void>(out.t),
                                             dtype_code(out.t), out.ld, ptr<void>(ws), ws.numel(), run.stream));
  return THPVariable_Wrap(out.t);
}

// (a, a_exps, gate, up, a_scale, act, ws, stream)
PyObject *gated(PyObject *const *v) {
  const Acts a = acts(v[0], v[1], v[4]);
  const Weights g = weights("gate", v[2], a.k, a.gpu), u = weights("up", v[3], a.k, a.gpu, g.n);
  const int act = act_code(v[5]);
  const Run run = run_on(v[7], a.gpu);
  const at::Tensor ws = workspace(maybe(v[6], "ws"), a.codes, a.gpu);
  const Coded out = coded(a.m, g.n, a.codes, run);
  CALL("gptq_fp8_gated", st, g_entry.gated(bytes(a.codes), a.ld, bytes(a.exps), a.lde, cptr<float>(a.scale), &g.w, &u.w,
                                           act, a.m, g.n, a.k, ptr<uint8_t>(out.codes), out.ldc, ptr<uint8_t>(out.exps),
                                           out.lde, ptr<void>(ws), ws.numel(), run.stream));
  return wrap2(out.codes, out.exps);
}

// (a, a_exps, gate, up, offsets, order, top_k, a_scale, act, ws, stream)
PyObject *experts_gated(PyObject *const *v) {
  const Acts a = acts(v[0], v[1], v[7]);
  const long top_k = PyLong_AsLong(v[6]);
  if (top_k == -1 && PyErr_Occurred()) return nullptr;
  if (top_k < 1 || top_k > 1 << 20) value_error("top_k must be at least 1");
  const at::Tensor &offsets = tensor(v[4], "offsets"), &order = tensor(v[5], "order");
  const int64_t experts = plan(offsets, order, a.m * top_k, a.gpu);
  const Weights g = weights("gate", v[2], a.k, a.gpu, -1, experts), u = weights("up", v[3], a.k, a.gpu, g.n, experts);
  const int act = act_code(v[8]);
  const Run run = run_on(v[10], a.gpu);
  const at::Tensor ws = workspace(maybe(v[9], "ws"), a.codes, a.gpu);
  const Coded out = coded(a.m * top_k, g.n, a.codes, run);
  CALL("gptq_fp8_experts_gated", st,
       g_entry.experts_gated(bytes(a.codes), a.ld, bytes(a.exps), a.lde, cptr<float>(a.scale), &g.w, &u.w, act,
                             (int)experts, cptr<int32_t>(offsets), cptr<int32_t>(order), (int)top_k, a.m, g.n, a.k,
                             ptr<uint8_t>(out.codes), out.ldc, ptr<uint8_t>(out.exps), out.lde, ptr<void>(ws), ws.numel(),
                             run.stream));
  return wrap2(out.codes, out.exps);
}

// (a, a_exps, w, w_exps, offsets, order, w_scale, bias, act, out_dtype, out, ws, stream)
PyObject *experts(PyObject *const *v) {
  const Acts a = acts(v[0], v[1], Py_None);
  const at::Tensor &offsets = tensor(v[4], "offsets"), &order = tensor(v[5], "order");
  const int64_t n_experts = plan(offsets, order, a.m, a.gpu);
  const Weights w = weights("w", tensor(v[2], "w"), tensor(v[3], "w_exps"), maybe(v[6], "w_scale"), maybe(v[7], "bias"),
                            a.k, a.gpu, -1, n_experts);
  const int act = act_code(v[8]);
  const Run run = run_on(v[12], a.gpu);
  const Out out = out16(v[10], v[9], a.m, w.n, a.codes, a.gpu, run);
  const at::Tensor ws = workspace(maybe(v[11], "ws"), a.codes, a.gpu);
  CALL("gptq_fp8_experts", st, g_entry.experts(bytes(a.codes), a.ld, bytes(a.exps), a.lde, &w.w, act, (int)n_experts,
                                               cptr<int32_t>(offsets), cptr<int32_t>(order), a.m, w.n, a.k,
                                               ptr<void>(out.t), dtype_code(out.t), out.ld, ptr<void>(ws), ws.numel(),
                                               run.stream));
  return THPVariable_Wrap(out.t);
}

// (logits, top_k, bias, scores, groups, top_groups, group_top, renormalize, scale, ws, stream)
PyObject *route(PyObject *const *v) {
  const at::Tensor &logits = tensor(v[0], "logits");
  const int64_t ld = rows_of("logits", logits), n = logits.size(0), n_experts = logits.size(1);
  const int gpu = gpu_of(logits);
  int number[5];   // top_k, scores, groups, top_groups, group_top
  const int at_arg[5] = {1, 3, 4, 5, 6};
  for (int i = 0; i < 5; ++i) {
    const long x = PyLong_AsLong(v[at_arg[i]]);
    if (x == -1 && PyErr_Occurred()) return nullptr;
    number[i] = (int)std::max(-1L, std::min(x, 1L << 20));
  }
  const int top_k = number[0], renormalize = PyObject_IsTrue(v[7]);
  const double scale = PyFloat_AsDouble(v[8]);
  if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  if (renormalize < 0) return nullptr;
  if (top_k < 1 || top_k > n_experts) value_error("top_k must be between 1 and the number of experts");
  const at::Tensor bias = maybe(v[2], "bias");
  floats(bias, "bias", {n_experts}, gpu);
  on(logits, gpu);
  const int dtype = dtype_code(logits);
  const Run run = run_on(v[10], gpu);
  const size_t need = g_entry.route_ws(n, (int)std::min(n_experts, (int64_t)INT32_MAX), top_k);
  const at::Tensor given = maybe(v[9], "ws");
  if (given.defined()) holds(given, gpu);
  const int64_t ws_bytes = given.defined() ? given.numel() : (int64_t)need;
  Together all;
  const int64_t at_ids = all.add(4 * n * top_k), at_w = all.add(4 * n * top_k), at_offsets = all.add(4 * (n_experts + 1));
  const int64_t at_order = all.add(4 * n * top_k), at_ws = all.add(given.defined() ? 0 : ws_bytes);
  all.allocate(logits, run);
  const at::Tensor ids = all.tensor(at_ids, {n, top_k}, {top_k, 1}, at::kInt);
  const at::Tensor w = all.tensor(at_w, {n, top_k}, {top_k, 1}, at::kFloat);
  const at::Tensor offsets = all.tensor(at_offsets, {n_experts + 1}, {1}, at::kInt);
  const at::Tensor order = all.tensor(at_order, {n * top_k}, {1}, at::kInt);
  void *const ws = given.defined() ? ptr<void>(given) : all.address(at_ws);
  CALL("gptq_moe_route", st,
       g_entry.route(cptr<void>(logits), dtype, ld, n, (int)n_experts, top_k, cptr<float>(bias), number[1], number[2],
                     number[3], number[4], renormalize, (float)scale, ptr<int32_t>(ids), ptr<float>(w),
                     ptr<int32_t>(offsets), ptr<int32_t>(order), ws, ws_bytes, run.stream));
  return Py_BuildValue("(NNNN)", THPVariable_Wrap(ids), THPVariable_Wrap(w), THPVariable_Wrap(offsets),
                       THPVariable_Wrap(order));
}

// (y, weights, residual, out, stream)
PyObject *combine(PyObject *const *v) {
  const at::Tensor &y = tensor(v[0], "y"), &w = tensor(v[1], "weights");
  if (w.scalar_type() != at::kFloat || w.dim() != 2 || !w.is_contiguous())
    value_error("weights must be a contiguous float32 [tokens, top_k] matrix");
  const int64_t n = w.size(0), top_k = w.size(1), ldy = rows_of("y", y, n * top_k), d = y.size(1);
  const at::Tensor residual = maybe(v[2], "residual");
  int64_t ldr = 0, ldo = d;
  if (residual.defined()) {
    ldr = rows_of("residual", residual, n, d);
    if (residual.scalar_type() != y.scalar_type()) type_error("residual must have y's dtype");
  }
  const int gpu = gpu_of(y);
  on(y, gpu);
  on(w, gpu);
  if (residual.defined()) on(residual, gpu);
  const int dtype = dtype_code(y);
  const Run run = run_on(v[4], gpu);
  at::Tensor out = maybe(v[3], "out");
  if (!out.defined()) {
    out = strided(n, d, d, y.scalar_type(), y);
    run.lend(out);
  } else {
    ldo = rows_of("out", out, n, d);
    if (out.scalar_type() != y.scalar_type()) type_error("out must have y's dtype");
    on(out, gpu);
  }
  CALL("gptq_moe_combine", st,
       g_entry.combine(cptr<void>(y), dtype, ldy, n, (int)std::min(top_k, (int64_t)INT32_MAX), d, cptr<float>(w),
                       cptr<void>(residual), ldr, ptr<void>(out), ldo, run.stream));
  return THPVariable_Wrap(out);
}

// (addresses of the entry points in Entry's order, the function that raises for (status, where))
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long p[7];
  PyObject *check;
  if (!PyArg_ParseTuple(args, "(KKKKKKK)O", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &check)) return nullptr;
  g_entry = {(decltype(g_entry.linear))p[0],  (decltype(g_entry.gated))p[1],    (decltype(g_entry.experts))p[2],
             (decltype(g_entry.experts_gated))p[3], (decltype(g_entry.route))p[4], (decltype(g_entry.route_ws))p[5],
             (decltype(g_entry.combine))p[6]};
  Py_INCREF(check);
  Py_XDECREF(g_check);
  g_check = check;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    def<linear, 13>("fp8_linear"),
    def<gated, 8>("fp8_gated"),
    def<experts, 13>("fp8_experts"),
    def<experts_gated, 11>("fp8_experts_gated"),
    def<route, 11>("moe_route"),
    def<combine, 5>("moe_combine"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
