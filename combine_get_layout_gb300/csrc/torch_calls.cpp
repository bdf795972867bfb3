// The torch layer's calls whose kernels take a few microseconds: checks of the
// tensors and the C ABI call in one step, for a Python wrapper each in
// __init__.py.  A call of ep_route for one token from Python, one after another:
// 2.9 to 3.0 us, and 5.4 with the same checks in Python and ctypes; of
// ep_route_backward for 4096, 4.0 and 7.4.
//
// Every function returns the entry point's status, or -1 where a tensor's
// type, shape, layout or place does not fit (nothing is called then).  The
// wrappers turn both into exceptions.  Tensors that may be absent are None.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <initializer_list>

#include "../../include/ep.h"

namespace {

using at::ScalarType;

constexpr long kUnfit = -1;

// A tensor argument: present, or absent where that is allowed.
struct Arg {
  const at::Tensor* t = nullptr;
  bool fits = true;

  explicit Arg(PyObject* o) {
    if (o == Py_None) return;
    fits = THPVariable_Check(o);
    if (fits) t = &THPVariable_Unpack(o);
  }
  // present, strided and on a GPU
  bool here() const { return t != nullptr && t->is_cuda() && t->layout() == at::kStrided; }
  // and contiguous, of this type and shape
  bool is(ScalarType type, at::IntArrayRef shape) const {
    return here() && t->scalar_type() == type && t->is_contiguous() && t->sizes() == shape;
  }
  bool is_or_absent(ScalarType type, at::IntArrayRef shape) const {
    return fits && (t == nullptr || is(type, shape));
  }
  bool is_mask_or_absent(int64_t n) const {
    return is_or_absent(ScalarType::Byte, {n}) || is_or_absent(ScalarType::Bool, {n});
  }
  // of so many bytes, whatever its type and shape
  bool holds(int64_t bytes) const {
    return here() && t->is_contiguous() && int64_t(t->nbytes()) >= bytes;
  }
  template <typename T>
  T* ptr() const {
    return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
  }
};

// Whether the present tensors are all on the current GPU: the one that the
// library launches on, and whose memory a launch may use.
bool on_current_gpu(std::initializer_list<const Arg*> args) {
  c10::DeviceIndex gpu = -1;
  if (c10::cuda::GetDevice(&gpu) != cudaSuccess) return false;
  for (const Arg* a : args)
    if (a->t != nullptr && (!a->t->is_cuda() || a->t->get_device() != gpu)) return false;
  return true;
}

// Router logits or their gradient: [T, E] of fp32 or bf16, columns of unit
// stride.
struct Logits {
  bool fits = false, bf16 = false;
  int64_t T = 0, ld = 0;

  Logits(const Arg& a, int64_t E) {
    if (!a.here() || a.t->dim() != 2 || a.t->size(1) != E) return;
    bf16 = a.t->scalar_type() == ScalarType::BFloat16;
    if (!bf16 && a.t->scalar_type() != ScalarType::Float) return;
    if (a.t->stride(1) != 1 && E != 1) return;
    T = a.t->size(0);
    ld = T > 1 ? a.t->stride(0) : E;
    fits = T <= INT32_MAX;
  }
};

// A stream handle, or the current stream for None.
bool stream_of(PyObject* o, void** stream) {
  if (o == Py_None) {
    *stream = c10::cuda::getCurrentCUDAStream().stream();
    return true;
  }
  *stream = PyLong_AsVoidPtr(o);
  return !PyErr_Occurred();
}

// The two forms (fp32, bf16 logits) of a router config, by their address.
const ep_router_config* router_config(PyObject* o) {
  return static_cast<const ep_router_config*>(PyLong_AsVoidPtr(o));
}

// Lets other host threads run, until the end of the scope by whatever way.
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(state); }
};

template <typename F>
PyObject* status_of(F&& call) {
  int32_t status;
  {
    Released others;
    status = call();
  }
  return PyLong_FromLong(status);
}

// A function as Python calls it; what torch throws (a tensor without
// storage, say) becomes a RuntimeError.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* unfit() { return PyLong_FromLong(kUnfit); }

bool arity(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, got);
  return false;
}

// route(configs, logits, bias, mask, idx, w, stream)
PyObject* route(PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  const ep_router_config* cfg = router_config(a[0]);
  if (cfg == nullptr) return nullptr;
  const int64_t E = cfg->num_experts, K = cfg->num_topk;
  const Arg logits(a[1]), bias(a[2]), mask(a[3]), idx(a[4]), w(a[5]);
  const Logits l(logits, E);
  if (!l.fits || !bias.is_or_absent(ScalarType::Float, {E}) || !mask.is_mask_or_absent(l.T) ||
      !idx.is(ScalarType::Long, {l.T, K}) || !w.is(ScalarType::Float, {l.T, K}) ||
      !on_current_gpu({&logits, &bias, &mask, &idx, &w}))
    return unfit();
  void* stream;
  if (!stream_of(a[6], &stream)) return nullptr;
  return status_of([&] {
    return ep_route(cfg + l.bf16, int32_t(l.T), logits.ptr<void>(), l.ld, bias.ptr<float>(),
                    mask.ptr<uint8_t>(), idx.ptr<int64_t>(), w.ptr<float>(), stream);
  });
}

// route_balance(configs, logits, bias, mask, seq_start, idx, w, count, prob,
// tokens, loss, workspace, workspace_bytes, stream)
PyObject* route_balance(PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 14)) return nullptr;
  const ep_router_config* cfg = router_config(a[0]);
  if (cfg == nullptr) return nullptr;
  const int64_t E = cfg->num_experts, K = cfg->num_topk;
  const Arg logits(a[1]), bias(a[2]), mask(a[3]), seq(a[4]), idx(a[5]), w(a[6]), count(a[7]),
      prob(a[8]), tokens(a[9]), loss(a[10]), workspace(a[11]);
  const int64_t bytes = PyLong_AsLongLong(a[12]);
  if (bytes == -1 && PyErr_Occurred()) return nullptr;
  const Logits l(logits, E);
  if (!l.fits || !seq.fits || (seq.t != nullptr && seq.t->dim() != 1)) return unfit();
  const int64_t B = seq.t == nullptr ? 1 : seq.t->size(0) - 1;
  if (B < 1 || B > INT32_MAX || !seq.is_or_absent(ScalarType::Int, {B + 1}) ||
      !bias.is_or_absent(ScalarType::Float, {E}) || !mask.is_mask_or_absent(l.T) ||
      !idx.is(ScalarType::Long, {l.T, K}) || !w.is(ScalarType::Float, {l.T, K}) ||
      !count.is(ScalarType::Int, {B, E}) || !prob.is(ScalarType::Float, {B, E}) ||
      !tokens.is(ScalarType::Int, {B + 2}) || !loss.is(ScalarType::Float, {2}) ||
      !workspace.holds(bytes) ||
      !on_current_gpu({&logits, &bias, &mask, &seq, &idx, &w, &count, &prob, &tokens, &loss,
                       &workspace}))
    return unfit();
  void* stream;
  if (!stream_of(a[13], &stream)) return nullptr;
  return status_of([&] {
    return ep_route_balance(cfg + l.bf16, int32_t(l.T), logits.ptr<void>(), l.ld,
                            bias.ptr<float>(), mask.ptr<uint8_t>(), int32_t(B),
                            seq.ptr<int32_t>(), idx.ptr<int64_t>(), w.ptr<float>(),
                            count.ptr<int32_t>(), prob.ptr<float>(), tokens.ptr<int32_t>(),
                            loss.ptr<float>(), workspace.ptr<void>(), stream);
  });
}

// route_backward(configs, logits, idx, grad_w, mask, seq_start, count, tokens,
// grad_loss, grad_logits, stream)
PyObject* route_backward(PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  const ep_router_config* cfg = router_config(a[0]);
  if (cfg == nullptr) return nullptr;
  const int64_t E = cfg->num_experts, K = cfg->num_topk;
  const Arg logits(a[1]), idx(a[2]), grad_w(a[3]), mask(a[4]), seq(a[5]), count(a[6]),
      tokens(a[7]), grad_loss(a[8]), grad(a[9]);
  const Logits l(logits, E), g(grad, E);
  if (!l.fits || !g.fits || l.bf16 != g.bf16 || l.T != g.T || !seq.fits ||
      (seq.t != nullptr && seq.t->dim() != 1))
    return unfit();
  const int64_t B = seq.t == nullptr ? 1 : seq.t->size(0) - 1;
  if (B < 1 || B > INT32_MAX || !seq.is_or_absent(ScalarType::Int, {B + 1}) ||
      !mask.is_mask_or_absent(l.T) || !idx.is_or_absent(ScalarType::Long, {l.T, K}) ||
      !grad_w.is_or_absent(ScalarType::Float, {l.T, K}) ||
      !count.is_or_absent(ScalarType::Int, {B, E}) ||
      !tokens.is_or_absent(ScalarType::Int, {B + 2}) ||
      !grad_loss.is_or_absent(ScalarType::Float, {2}) ||
      !on_current_gpu({&logits, &idx, &grad_w, &mask, &seq, &count, &tokens, &grad_loss, &grad}))
    return unfit();
  void* stream;
  if (!stream_of(a[10], &stream)) return nullptr;
  return status_of([&] {
    return ep_route_backward(cfg + l.bf16, int32_t(l.T), logits.ptr<void>(), l.ld,
                             mask.ptr<uint8_t>(), idx.ptr<int64_t>(), grad_w.ptr<float>(),
                             int32_t(B), seq.ptr<int32_t>(), count.ptr<int32_t>(),
                             tokens.ptr<int32_t>(), grad_loss.ptr<float>(), grad.ptr<void>(),
                             g.ld, stream);
  });
}

// A layout's segments: int32, at least E entries.
bool segments_of(const Arg& s, int64_t E) {
  return s.here() && s.t->scalar_type() == ScalarType::Int && s.t->is_contiguous() &&
         s.t->dim() == 1 && s.t->size(0) >= E;
}

// expert_w4(config, x, codes, scales, start, end, num_rows, zeros, x_scale,
// out, stream)
PyObject* expert_w4(PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  const auto* cfg = static_cast<const ep_w4_config*>(PyLong_AsVoidPtr(a[0]));
  if (cfg == nullptr) return nullptr;
  const Arg x(a[1]), codes(a[2]), scales(a[3]), start(a[4]), end(a[5]), zeros(a[7]),
      x_scale(a[8]), out(a[9]);
  const long long num_rows = PyLong_AsLongLong(a[6]);
  if (num_rows == -1 && PyErr_Occurred()) return nullptr;
  const int64_t E = cfg->num_experts, H = cfg->in_features;
  const int64_t N = cfg->gated ? cfg->out_features / 2 : cfg->out_features;
  if (x.t == nullptr || x.t->dim() != 2) return unfit();
  const int64_t cap = x.t->size(0);
  if (cap > INT32_MAX || num_rows > INT32_MAX || num_rows < INT32_MIN ||
      !x.is(cfg->x_fp8 ? ScalarType::Byte : ScalarType::BFloat16, {cap, H}) ||
      !x_scale.is_or_absent(ScalarType::Float, {cap, H / 128}) ||
      !out.is(ScalarType::BFloat16, {cap, N}) || !segments_of(start, E) || !segments_of(end, E) ||
      !codes.holds(ep_w4_codes_bytes(cfg)) || !scales.holds(ep_w4_scales_bytes(cfg)) ||
      scales.t->scalar_type() != ScalarType::BFloat16 || !zeros.fits ||
      (zeros.t != nullptr && !zeros.holds(ep_w4_zeros_bytes(cfg))) ||
      !on_current_gpu({&x, &codes, &scales, &start, &end, &zeros, &x_scale, &out}))
    return unfit();
  void* stream;
  if (!stream_of(a[10], &stream)) return nullptr;
  return status_of([&] {
    return ep_expert_w4(cfg, int32_t(cap), int32_t(num_rows), x.ptr<void>(),
                        x_scale.ptr<float>(), codes.ptr<void>(), scales.ptr<void>(),
                        zeros.ptr<uint8_t>(), start.ptr<int32_t>(), end.ptr<int32_t>(),
                        out.ptr<void>(), stream);
  });
}

// A layout's error word, or absent.
bool error_word(const Arg& err) {
  return err.fits &&
         (err.t == nullptr || (err.holds(4) && err.t->scalar_type() == ScalarType::Int));
}

// A number of rows that a 32-bit argument holds.
bool rows_of(PyObject* o, long long* rows) {
  *rows = PyLong_AsLongLong(o);
  return !(*rows == -1 && PyErr_Occurred());
}

bool in_32_bits(long long n) { return n <= INT32_MAX && n >= INT32_MIN; }

// expert_mm(config, x, w, start, end, num_rows, x_scale, out, err, stream)
PyObject* expert_mm(PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 10)) return nullptr;
  const auto* cfg = static_cast<const ep_expert_config*>(PyLong_AsVoidPtr(a[0]));
  if (cfg == nullptr) return nullptr;
  const Arg x(a[1]), w(a[2]), start(a[3]), end(a[4]), x_scale(a[6]), out(a[7]), err(a[8]);
  long long num_rows;
  if (!rows_of(a[5], &num_rows)) return nullptr;
  const int64_t E = cfg->num_experts, H = cfg->in_features, N = cfg->out_features;
  if (x.t == nullptr || x.t->dim() != 2) return unfit();
  const int64_t cap = x.t->size(0);
  if (cap > INT32_MAX || !in_32_bits(num_rows) ||
      !x.is(cfg->x_fp8 ? ScalarType::Byte : ScalarType::BFloat16, {cap, H}) ||
      !x_scale.is_or_absent(ScalarType::Float, {cap, H / 128}) ||
      !w.is(ScalarType::BFloat16, {E, N, H}) ||
      !out.is(ScalarType::BFloat16, {cap, cfg->gated ? N / 2 : N}) || !segments_of(start, E) ||
      !segments_of(end, E) || !error_word(err) ||
      !on_current_gpu({&x, &w, &start, &end, &x_scale, &out, &err}))
    return unfit();
  void* stream;
  if (!stream_of(a[9], &stream)) return nullptr;
  return status_of([&] {
    return ep_expert_mm(cfg, int32_t(cap), int32_t(num_rows), x.ptr<void>(), x_scale.ptr<float>(),
                        w.ptr<void>(), start.ptr<int32_t>(), end.ptr<int32_t>(), out.ptr<void>(),
                        err.ptr<int32_t>(), stream);
  });
}

// expert_mm_backward(config, grad_out, start, end, num_rows, w, x, x_scale,
// grad_x, grad_w, accumulate, err, stream)
PyObject* expert_mm_backward(PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 13)) return nullptr;
  const auto* cfg = static_cast<const ep_expert_config*>(PyLong_AsVoidPtr(a[0]));
  if (cfg == nullptr) return nullptr;
  const Arg dy(a[1]), start(a[2]), end(a[3]), w(a[5]), x(a[6]), x_scale(a[7]), dx(a[8]), dw(a[9]),
      err(a[11]);
  long long num_rows;
  if (!rows_of(a[4], &num_rows)) return nullptr;
  const int64_t E = cfg->num_experts, H = cfg->in_features, N = cfg->out_features;
  if (dy.t == nullptr || dy.t->dim() != 2) return unfit();
  const int64_t cap = dy.t->size(0);
  const bool f32 = dw.t != nullptr && dw.t->scalar_type() == ScalarType::Float;
  const bool add = a[10] == Py_True;
  if (cap > INT32_MAX || !in_32_bits(num_rows) || !dy.is(ScalarType::BFloat16, {cap, N}) ||
      !w.is_or_absent(ScalarType::BFloat16, {E, N, H}) ||
      !x.is_or_absent(cfg->x_fp8 ? ScalarType::Byte : ScalarType::BFloat16, {cap, H}) ||
      !x_scale.is_or_absent(ScalarType::Float, {cap, H / 128}) ||
      !dx.is_or_absent(ScalarType::BFloat16, {cap, H}) ||
      !dw.is_or_absent(f32 ? ScalarType::Float : ScalarType::BFloat16, {E, N, H}) ||
      (w.t == nullptr) != (dx.t == nullptr) || (x.t == nullptr) != (dw.t == nullptr) ||
      (add && !f32) || !segments_of(start, E) || !segments_of(end, E) || !error_word(err) ||
      !on_current_gpu({&dy, &start, &end, &w, &x, &x_scale, &dx, &dw, &err}))
    return unfit();
  void* stream;
  if (!stream_of(a[12], &stream)) return nullptr;
  return status_of([&] {
    return ep_expert_mm_backward(cfg, int32_t(cap), int32_t(num_rows), dy.ptr<void>(),
                                 w.ptr<void>(), x.ptr<void>(), x_scale.ptr<float>(),
                                 start.ptr<int32_t>(), end.ptr<int32_t>(), dx.ptr<void>(),
                                 dw.ptr<void>(),
                                 add ? EP_GRAD_FP32_ADD : f32 ? EP_GRAD_FP32 : EP_GRAD_BF16,
                                 err.ptr<int32_t>(), stream);
  });
}

// act_save(h, start, end, num_rows, a, q, scale, stream)
PyObject* act_save(PyObject* const* v, Py_ssize_t n) {
  if (!arity(n, 8)) return nullptr;
  const Arg h(v[0]), start(v[1]), end(v[2]), a(v[4]), q(v[5]), scale(v[6]);
  long long num_rows;
  if (!rows_of(v[3], &num_rows)) return nullptr;
  if (h.t == nullptr || h.t->dim() != 2 || end.t == nullptr || end.t->dim() != 1) return unfit();
  const int64_t cap = h.t->size(0), I = h.t->size(1) / 2, E = end.t->size(0);
  if (cap > INT32_MAX || E > INT32_MAX || I > INT32_MAX || !in_32_bits(num_rows) ||
      !h.is(ScalarType::BFloat16, {cap, 2 * I}) || !a.is(ScalarType::BFloat16, {cap, I}) ||
      !q.is(ScalarType::Byte, {cap, 2 * I}) ||
      !scale.is(ScalarType::Float, {cap, 2 * ((I + 127) / 128)}) || !segments_of(start, E) ||
      !segments_of(end, E) || !on_current_gpu({&h, &start, &end, &a, &q, &scale}))
    return unfit();
  void* stream;
  if (!stream_of(v[7], &stream)) return nullptr;
  return status_of([&] {
    return ep_act_save(int32_t(E), int32_t(I), int32_t(cap), int32_t(num_rows), h.ptr<void>(),
                       start.ptr<int32_t>(), end.ptr<int32_t>(), a.ptr<void>(), q.ptr<uint8_t>(),
                       scale.ptr<float>(), stream);
  });
}

// act_backward(grad_a, q, scale, start, end, num_rows, grad_h, a, stream)
PyObject* act_backward(PyObject* const* v, Py_ssize_t n) {
  if (!arity(n, 9)) return nullptr;
  const Arg da(v[0]), q(v[1]), scale(v[2]), start(v[3]), end(v[4]), dh(v[6]), a(v[7]);
  long long num_rows;
  if (!rows_of(v[5], &num_rows)) return nullptr;
  if (da.t == nullptr || da.t->dim() != 2 || end.t == nullptr || end.t->dim() != 1)
    return unfit();
  const int64_t cap = da.t->size(0), I = da.t->size(1), E = end.t->size(0);
  if (cap > INT32_MAX || E > INT32_MAX || I > INT32_MAX || !in_32_bits(num_rows) ||
      !da.is(ScalarType::BFloat16, {cap, I}) || !q.is(ScalarType::Byte, {cap, 2 * I}) ||
      !scale.is(ScalarType::Float, {cap, 2 * ((I + 127) / 128)}) ||
      !dh.is(ScalarType::BFloat16, {cap, 2 * I}) ||
      !a.is_or_absent(ScalarType::BFloat16, {cap, I}) || !segments_of(start, E) ||
      !segments_of(end, E) || !on_current_gpu({&da, &q, &scale, &start, &end, &dh, &a}))
    return unfit();
  void* stream;
  if (!stream_of(v[8], &stream)) return nullptr;
  return status_of([&] {
    return ep_act_backward(int32_t(E), int32_t(I), int32_t(cap), int32_t(num_rows),
                           da.ptr<void>(), q.ptr<uint8_t>(), scale.ptr<float>(),
                           start.ptr<int32_t>(), end.ptr<int32_t>(), dh.ptr<void>(),
                           a.ptr<void>(), stream);
  });
}

#define EP_CALL(f)                                                                      \
  {                                                                                     \
    #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>)),        \
        METH_FASTCALL, nullptr                                                          \
  }
PyMethodDef methods[] = {EP_CALL(route), EP_CALL(route_balance), EP_CALL(route_backward),
                         EP_CALL(expert_w4), EP_CALL(expert_mm), EP_CALL(expert_mm_backward),
                         EP_CALL(act_save), EP_CALL(act_backward), {nullptr, nullptr, 0, nullptr}};
#undef EP_CALL

PyModuleDef module = {PyModuleDef_HEAD_INIT, "ep_torch_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ep_torch_calls() { return PyModule_Create(&module); }
