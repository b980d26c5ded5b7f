// mixer_binding.cpp -- the Python binding of the mixer's and a hybrid block's operators: argument
// marshalling only.
//
// A single-token call costs the GPU a few microseconds; describing its tensors from Python cost
// three times that.  Here descriptors point straight at the tensors' sizes and strides, outputs
// come from PyTorch's allocator, and the work goes to libgdr's C entry points on torch's current
// stream.  Arguments are positional and complete: the Python functions in mixer.py and block.py
// give them names, defaults and documentation.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "gdr.h"

namespace {

PyObject *g_error = nullptr;  // GdrError(status, where)

[[noreturn]] void refuse(PyObject *type, const char *what) {
  PyErr_SetString(type, what);
  throw python_error();
}

// Descriptors of one call's tensors.  All must be on the first one's CUDA device.
struct Call {
  gdr_tensor_t d[24];
  int n = 0, index = -1;

  explicit Call(const at::Tensor &first) {
    index = first.is_cuda() ? first.get_device() : -1;
    if (index < 0) refuse(PyExc_ValueError, "tensors must be on a CUDA device");
  }
  gdr_tensor_t *add(const at::Tensor &t) {
    if (!t.defined()) return nullptr;
    if (!t.is_cuda() || t.get_device() != index)
      refuse(PyExc_ValueError, "tensors must be on one CUDA device");
    gdr_tensor_t &g = d[n++];
    switch (t.scalar_type()) {
      case at::kBFloat16: g.dtype = GDR_BF16; break;
      case at::kFloat: g.dtype = GDR_F32; break;
      default: refuse(PyExc_TypeError, "unsupported dtype: tensors are bfloat16 or float32");
    }
    if (t.dim() < 1 || t.dim() > 4) refuse(PyExc_ValueError, "tensors must have 1..4 dims");
    g.data = t.numel() ? t.data_ptr() : nullptr;
    g.ndim = (int32_t)t.dim();
    for (int i = 0; i < 4; ++i) g.shape[i] = i < t.dim() ? t.size(i) : 0;
    g.strides = t.strides().data();
    return &g;
  }
  // int32 [rows, any], rows of any stride
  gdr_tensor_t *table(const at::Tensor &t, const char *name) {
    if (t.scalar_type() != at::kInt)
      refuse(PyExc_TypeError, (std::string(name) + " must be int32").c_str());
    if (!t.is_cuda() || t.get_device() != index)
      refuse(PyExc_ValueError, "tensors must be on one CUDA device");
    gdr_tensor_t &g = d[n++];
    g.dtype = GDR_I32;
    g.data = t.numel() ? t.data_ptr() : nullptr;
    g.ndim = (int32_t)t.dim();
    for (int i = 0; i < 4; ++i) g.shape[i] = i < t.dim() ? t.size(i) : 0;
    g.strides = t.strides().data();
    return &g;
  }
  // a compact int32 array on the call's device (None: null); n < 0: of any length
  const int32_t *ints(const at::Tensor &t, int64_t count, const char *name) const {
    if (!t.defined()) return nullptr;
    if (t.scalar_type() != at::kInt)
      refuse(PyExc_TypeError, (std::string(name) + " must be int32").c_str());
    if (t.dim() != 1 || (count >= 0 && t.size(0) != count) || !t.is_contiguous())
      refuse(PyExc_ValueError,
             (std::string(name) + " must be compact, one-dimensional and of the call's length")
                 .c_str());
    if (!t.is_cuda() || t.get_device() != index)
      refuse(PyExc_ValueError, (std::string(name) + " must be on the call's device").c_str());
    return t.numel() ? t.data_ptr<int32_t>() : nullptr;
  }
  cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(index).stream(); }
};

// cu_seqlens: its address and the number of segments (None: one segment of all tokens)
struct Segments {
  const int32_t *cu = nullptr;
  int32_t n = 1;
  Segments(const Call &c, const at::Tensor &t) {
    if (!t.defined()) return;
    if (t.dim() != 1 || t.size(0) < 1)
      refuse(PyExc_ValueError, "cu_seqlens must hold n_seq + 1 offsets");
    cu = c.ints(t, -1, "cu_seqlens");
    n = (int32_t)(t.size(0) - 1);
  }
};

at::Tensor tensor(PyObject *o) {  // None: undefined
  if (o == Py_None) return at::Tensor();
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "a tensor or None was expected");
  return THPVariable_Unpack(o);
}
at::Tensor required(PyObject *o, int dims, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, (std::string(name) + " must be a tensor").c_str());
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.dim() != dims)
    refuse(PyExc_ValueError,
           (std::string(name) + " must have " + std::to_string(dims) + " dims").c_str());
  return t;
}
at::Tensor empty(at::IntArrayRef sizes, const at::Tensor &like) {
  return at::empty(sizes, at::TensorOptions().dtype(like.scalar_type()).device(like.device()));
}
at::Tensor empty32(at::IntArrayRef sizes, const at::Tensor &like) {
  return at::empty(sizes, at::TensorOptions().dtype(at::kFloat).device(like.device()));
}
// Several compact tensors of `like`'s type out of one allocation (256 bytes apart): allocating each costs
// the host a microsecond.
struct Parts {
  at::Tensor all;
  int64_t at = 0;
  Parts(int64_t count, const at::Tensor &like)
      : all(at::empty({count}, at::TensorOptions().dtype(like.scalar_type()).device(like.device()))) {}
  at::Tensor next(int64_t n) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::TensorImpl::VIEW, c10::Storage(all.storage()), all.key_set(), all.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    at += (n + 63) / 64 * 64;
    return t;
  }
};
PyObject *wrap(const at::Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject *tuple(std::initializer_list<at::Tensor> ts) {
  PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor &t : ts) PyTuple_SET_ITEM(out, i++, wrap(t));
  return out;
}
bool truth(PyObject *o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t activation(PyObject *o) {
  if (o == Py_None) return GDR_ACT_NONE;
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return GDR_ACT_SILU;
    if (PyUnicode_CompareWithASCIIString(o, "none") == 0) return GDR_ACT_NONE;
  }
  refuse(PyExc_ValueError, "activation must be 'silu', 'none' or None");
}
int32_t norm_of(PyObject *o) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "rms") == 0) return GDR_NORM_RMS;
    if (PyUnicode_CompareWithASCIIString(o, "l2") == 0) return GDR_NORM_L2;
  }
  refuse(PyExc_ValueError, "norm must be 'rms' or 'l2'");
}

int32_t gate_activation(PyObject *o) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return GDR_ACT_SILU;
    if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0) return GDR_ACT_SIGMOID;
  }
  refuse(PyExc_ValueError, "activation must be 'silu' or 'sigmoid'");
}
int32_t whole(PyObject *o, const char *name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < -0x7ff00000L || v > 0x7ff00000L)
    refuse(PyExc_ValueError, (std::string(name) + " is out of range").c_str());
  return (int32_t)v;
}

struct Scratch {
  at::Tensor t;
  void *p = nullptr;
  size_t n = 0;
  Scratch(const Call &c, const at::Tensor &given, size_t need, const at::Tensor &like) {
    if (given.defined()) {
      if (!given.is_cuda() || given.get_device() != c.index || !given.is_contiguous())
        refuse(PyExc_ValueError, "workspace must be compact and on the call's device");
      t = given;
    } else if (need) {
      t = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(like.device()));
    }
    if (t.defined()) {
      p = t.data_ptr();
      n = (size_t)t.nbytes();
    }
  }
};

void check(int status, const char *where) {
  if (status == GDR_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", status, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

// Makes the tensors' device current while it lives, where it is not.
using Guard = c10::cuda::OptionalCUDAGuard;
void enter(Guard &g, const Call &c) {
  if (c10::cuda::current_device() != c.index) g.set_index((c10::DeviceIndex)c.index);
}

#define ENTRY(name, count)                                                          \
  PyObject *name(PyObject *, PyObject *const *args, Py_ssize_t nargs) {             \
    HANDLE_TH_ERRORS                                                                \
    if (nargs != count) refuse(PyExc_TypeError, #name ": wrong number of arguments"); \
    Guard guard;
#define EXIT END_HANDLE_TH_ERRORS }

// The library only enqueues work; other Python threads may run meanwhile.
template <typename F>
int run(F f) {
  PyThreadState *s = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(s);
  return status;
}

// x, weight, bias, h0, cu, activation, want_ht, out, ht (a given one is written, wanted or not)
ENTRY(conv_fwd, 9)
  const at::Tensor x = required(args[0], 2, "x"), w = required(args[1], 2, "weight");
  const at::Tensor b = tensor(args[2]), h0 = tensor(args[3]), cu = tensor(args[4]);
  Call c(x);
  enter(guard, c);
  const Segments s(c, cu);
  at::Tensor y = tensor(args[7]), ht = tensor(args[8]);
  if (!y.defined()) y = empty(x.sizes(), x);
  if (truth(args[6]) && !ht.defined()) ht = empty({s.n, w.size(1) - 1, x.size(1)}, x);
  const int32_t act = activation(args[5]);
  gdr_tensor_t *dx = c.add(x), *dw = c.add(w), *db = c.add(b), *dh = c.add(h0), *dy = c.add(y),
               *dt = c.add(ht);
  const cudaStream_t st = c.stream();
  check(run([&] { return gdr_conv_fwd(dx, dw, db, dh, s.cu, s.n, act, dy, dt, st); }),
        "gdr_conv_fwd");
  return tuple({y, ht});
EXIT

// x, weight, dy, bias, h0, cu, activation, dht, want_dh0, workspace
ENTRY(conv_bwd, 10)
  const at::Tensor x = required(args[0], 2, "x"), w = required(args[1], 2, "weight"),
                   dy = required(args[2], 2, "dy");
  const at::Tensor b = tensor(args[3]), h0 = tensor(args[4]), cu = tensor(args[5]),
                   dht = tensor(args[7]);
  Call c(x);
  enter(guard, c);
  const Segments s(c, cu);
  const int32_t act = activation(args[6]);
  at::Tensor dx = empty(x.sizes(), x), dw = empty32(w.sizes(), x), db, dh0;
  if (b.defined()) db = empty32({x.size(1)}, x);
  if (truth(args[8])) dh0 = empty({s.n, w.size(1) - 1, x.size(1)}, x);
  const Scratch ws(c, tensor(args[9]),
                   gdr_conv_bwd_workspace_bytes(x.size(0), (int32_t)x.size(1), (int32_t)w.size(1)),
                   x);
  gdr_tensor_t *p[] = {c.add(x), c.add(w), c.add(b), c.add(h0), c.add(dy), c.add(dht),
                       c.add(dx), c.add(dw), c.add(db), c.add(dh0)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_conv_bwd(p[0], p[1], p[2], p[3], s.cu, s.n, act, p[4], p[5], p[6], p[7], p[8],
                              p[9], ws.p, ws.n, st);
        }),
        "gdr_conv_bwd");
  return tuple({dx, dw, db, dh0});
EXIT

// x, weight, state, bias, activation, idx, out
ENTRY(conv_step, 7)
  const at::Tensor x = required(args[0], 2, "x"), w = required(args[1], 2, "weight"),
                   state = required(args[2], 3, "state");
  const at::Tensor b = tensor(args[3]), idx = tensor(args[5]);
  Call c(x);
  enter(guard, c);
  const int32_t act = activation(args[4]);
  const int32_t *ix = c.ints(idx, x.size(0), "state_indices");
  at::Tensor y = tensor(args[6]);
  if (!y.defined()) y = empty(x.sizes(), x);
  gdr_tensor_t *dx = c.add(x), *dw = c.add(w), *db = c.add(b), *ds = c.add(state), *dy = c.add(y);
  const cudaStream_t st = c.stream();
  check(run([&] { return gdr_conv_step(dx, dw, db, ds, ix, act, dy, st); }), "gdr_conv_step");
  return wrap(y);
EXIT

// x, dt, A, B, C, D, z, dt_bias, softplus, h0, cu, want_ht, out, ht (as above), workspace
ENTRY(ssm_fwd, 15)
  const at::Tensor x = required(args[0], 2, "x"), B = required(args[3], 3, "B");
  const at::Tensor dt = tensor(args[1]), A = tensor(args[2]), C = tensor(args[4]),
                   D = tensor(args[5]), z = tensor(args[6]), bias = tensor(args[7]),
                   h0 = tensor(args[9]), cu = tensor(args[10]);
  Call c(x);
  enter(guard, c);
  const Segments s(c, cu);
  const int32_t sp = truth(args[8]);
  at::Tensor y = tensor(args[12]), ht = tensor(args[13]);
  if (!y.defined()) y = empty(x.sizes(), x);
  if (truth(args[11]) && !ht.defined()) ht = empty32({s.n, x.size(1), B.size(2)}, x);
  const Scratch ws(c, tensor(args[14]),
                   gdr_ssm_fwd_workspace_bytes(x.size(0), (int32_t)x.size(1), (int32_t)B.size(2),
                                               (int32_t)B.size(1)),
                   x);
  gdr_tensor_t *p[] = {c.add(x), c.add(dt), c.add(A), c.add(B), c.add(C), c.add(D),
                       c.add(z), c.add(bias), c.add(h0), c.add(y), c.add(ht)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_ssm_fwd(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], sp, p[8], s.cu, s.n,
                             p[9], p[10], ws.p, ws.n, st);
        }),
        "gdr_ssm_fwd");
  return tuple({y, ht});
EXIT

// x, dt, A, B, C, dy, D, z, dt_bias, softplus, h0, cu, dht, want_dh0, workspace
ENTRY(ssm_bwd, 15)
  const at::Tensor x = required(args[0], 2, "x"), B = required(args[3], 3, "B"),
                   dt = required(args[1], 2, "dt"), C = required(args[4], 3, "C");
  const at::Tensor A = tensor(args[2]), dy = tensor(args[5]), D = tensor(args[6]),
                   z = tensor(args[7]), bias = tensor(args[8]), h0 = tensor(args[10]),
                   cu = tensor(args[11]), dht = tensor(args[12]);
  Call c(x);
  enter(guard, c);
  const Segments s(c, cu);
  const int32_t sp = truth(args[9]);
  at::Tensor dx = empty(x.sizes(), x), ddt = empty(dt.sizes(), x), dB = empty(B.sizes(), x),
             dC = empty(C.sizes(), x), dA = empty32({x.size(1), B.size(2)}, x), dD, dz, dbias, dh0;
  if (D.defined()) dD = empty32({x.size(1)}, x);
  if (z.defined()) dz = empty(x.sizes(), x);
  if (bias.defined()) dbias = empty32({x.size(1)}, x);
  if (truth(args[13])) dh0 = empty32({s.n, x.size(1), B.size(2)}, x);
  const Scratch ws(c, tensor(args[14]),
                   gdr_ssm_bwd_workspace_bytes(x.size(0), (int32_t)x.size(1), (int32_t)B.size(2),
                                               (int32_t)B.size(1)),
                   x);
  gdr_tensor_t *p[] = {c.add(x), c.add(dt), c.add(A), c.add(B), c.add(C), c.add(D), c.add(z),
                       c.add(bias), c.add(h0), c.add(dy), c.add(dht), c.add(dx), c.add(ddt),
                       c.add(dA), c.add(dB), c.add(dC), c.add(dD), c.add(dz), c.add(dbias),
                       c.add(dh0)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_ssm_bwd(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], sp, p[8], s.cu, s.n,
                             p[9], p[10], p[11], p[12], p[13], p[14], p[15], p[16], p[17], p[18],
                             p[19], ws.p, ws.n, st);
        }),
        "gdr_ssm_bwd");
  return tuple({dx, ddt, dA, dB, dC, dD, dz, dbias, dh0});
EXIT

// x, dt, A, B, C, state, D, z, dt_bias, softplus, idx, out
ENTRY(ssm_step, 12)
  const at::Tensor x = required(args[0], 2, "x");
  const at::Tensor dt = tensor(args[1]), A = tensor(args[2]), B = tensor(args[3]),
                   C = tensor(args[4]), state = tensor(args[5]), D = tensor(args[6]),
                   z = tensor(args[7]), bias = tensor(args[8]), idx = tensor(args[10]);
  Call c(x);
  enter(guard, c);
  const int32_t sp = truth(args[9]);
  const int32_t *ix = c.ints(idx, x.size(0), "state_indices");
  at::Tensor y = tensor(args[11]);
  if (!y.defined()) y = empty(x.sizes(), x);
  gdr_tensor_t *p[] = {c.add(x), c.add(dt), c.add(A), c.add(B), c.add(C),
                       c.add(D), c.add(z), c.add(bias), c.add(state), c.add(y)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_ssm_step(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], sp, p[8], ix, p[9],
                              st);
        }),
        "gdr_ssm_step");
  return wrap(y);
EXIT

// q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved, q_out, k_out
ENTRY(qk_fwd, 12)
  const at::Tensor q = required(args[0], 3, "q"), k = required(args[1], 3, "k");
  const at::Tensor qw = tensor(args[2]), kw = tensor(args[3]), cos = tensor(args[6]),
                   sin = tensor(args[7]), pos = tensor(args[8]);
  Call c(q);
  enter(guard, c);
  const int32_t norm = norm_of(args[4]), inter = truth(args[9]);
  const float eps = (float)real(args[5]);
  const int32_t *ps = c.ints(pos, q.size(0), "positions");
  at::Tensor qo = tensor(args[10]), ko = tensor(args[11]);
  if (!qo.defined()) qo = empty(q.sizes(), q);
  if (!ko.defined()) ko = empty(k.sizes(), k);
  gdr_tensor_t *p[] = {c.add(q), c.add(k), c.add(qw), c.add(kw),
                       c.add(cos), c.add(sin), c.add(qo), c.add(ko)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_qk_fwd(p[0], p[1], p[2], p[3], norm, eps, p[4], p[5], ps, inter, p[6], p[7],
                            st);
        }),
        "gdr_qk_fwd");
  return tuple({qo, ko});
EXIT

// q, k, dq_out, dk_out, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved, workspace
ENTRY(qk_bwd, 13)
  const at::Tensor q = required(args[0], 3, "q"), k = required(args[1], 3, "k");
  const at::Tensor dqo = tensor(args[2]), dko = tensor(args[3]), qw = tensor(args[4]),
                   kw = tensor(args[5]), cos = tensor(args[8]), sin = tensor(args[9]),
                   pos = tensor(args[10]);
  Call c(q);
  enter(guard, c);
  const int32_t norm = norm_of(args[6]), inter = truth(args[11]);
  const float eps = (float)real(args[7]);
  const int32_t *ps = c.ints(pos, q.size(0), "positions");
  at::Tensor dq = empty(q.sizes(), q), dk = empty(k.sizes(), k), dqw, dkw;
  if (qw.defined()) dqw = empty32({q.size(2)}, q);
  if (kw.defined()) dkw = empty32({q.size(2)}, q);
  const Scratch ws(c, tensor(args[12]),
                   gdr_qk_bwd_workspace_bytes(q.size(0), (int32_t)q.size(1), (int32_t)k.size(1),
                                              (int32_t)q.size(2)),
                   q);
  gdr_tensor_t *p[] = {c.add(q), c.add(k), c.add(qw), c.add(kw), c.add(cos), c.add(sin),
                       c.add(dqo), c.add(dko), c.add(dq), c.add(dk), c.add(dqw), c.add(dkw)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_qk_bwd(p[0], p[1], p[2], p[3], norm, eps, p[4], p[5], ps, inter, p[6], p[7],
                            p[8], p[9], p[10], p[11], ws.p, ws.n, st);
        }),
        "gdr_qk_bwd");
  return tuple({dq, dk, dqw, dkw});
EXIT

// q, k, v, g, beta, state, scale (None: dk^-1/2), idx, out
ENTRY(delta_step, 9)
  const at::Tensor q = required(args[0], 3, "q"), v = required(args[2], 3, "v");
  const at::Tensor k = tensor(args[1]), g = tensor(args[3]), beta = tensor(args[4]),
                   state = tensor(args[5]), idx = tensor(args[7]);
  Call c(q);
  enter(guard, c);
  const float scale = args[6] == Py_None ? 1.f / std::sqrt((float)q.size(2)) : (float)real(args[6]);
  const int32_t *ix = c.ints(idx, q.size(0), "state_indices");
  at::Tensor o = tensor(args[8]);
  if (!o.defined()) o = empty(v.sizes(), v);
  gdr_tensor_t *p[] = {c.add(q), c.add(k), c.add(v), c.add(g), c.add(beta), c.add(state),
                       c.add(o)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_delta_step(p[0], p[1], p[2], p[3], p[4], scale, p[5], ix, p[6], st);
        }),
        "gdr_delta_step");
  return wrap(o);
EXIT

// x, r, A, i, normalize, h0, cu, want_ht, want_checkpoints, out, ht, checkpoints
ENTRY(rec_fwd, 12)
  const at::Tensor x = required(args[0], 2, "x");
  const at::Tensor r = tensor(args[1]), A = tensor(args[2]), i = tensor(args[3]),
                   h0 = tensor(args[5]), cu = tensor(args[6]);
  Call c(x);
  enter(guard, c);
  const Segments s(c, cu);
  const int32_t normalize = truth(args[4]);
  at::Tensor y = tensor(args[9]), ht = tensor(args[10]), kept = tensor(args[11]);
  if (!y.defined()) y = empty(x.sizes(), x);
  if (truth(args[7]) && !ht.defined()) ht = empty32({s.n, x.size(1)}, x);
  if (truth(args[8]) && !kept.defined())
    kept = empty32({gdr_rec_checkpoint_rows(x.size(0)), x.size(1)}, x);
  gdr_tensor_t *p[] = {c.add(x), c.add(r), c.add(i), c.add(A), c.add(h0), c.add(y), c.add(ht),
                       c.add(kept)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_rec_fwd(p[0], p[1], p[2], p[3], normalize, p[4], s.cu, s.n, p[5], p[6], p[7],
                             st);
        }),
        "gdr_rec_fwd");
  return tuple({y, ht, kept});
EXIT

// x, r, A, dy, i, normalize, h0, cu, dht, want_dh0, checkpoints, workspace
ENTRY(rec_bwd, 12)
  const at::Tensor x = required(args[0], 2, "x"), r = required(args[1], 2, "r");
  const at::Tensor A = tensor(args[2]), dy = tensor(args[3]), i = tensor(args[4]),
                   h0 = tensor(args[6]), cu = tensor(args[7]), dht = tensor(args[8]),
                   kept = tensor(args[10]);
  Call c(x);
  enter(guard, c);
  const Segments s(c, cu);
  const int32_t normalize = truth(args[5]);
  at::Tensor dx = empty(x.sizes(), x), dr = empty(r.sizes(), x), dA = empty32({x.size(1)}, x), di,
             dh0;
  if (i.defined()) di = empty(x.sizes(), x);
  if (truth(args[9])) dh0 = empty32({s.n, x.size(1)}, x);
  const Scratch ws(c, tensor(args[11]),
                   gdr_rec_bwd_workspace_bytes(x.size(0), (int32_t)x.size(1), s.n, kept.defined()),
                   x);
  gdr_tensor_t *p[] = {c.add(x),  c.add(r),   c.add(i),  c.add(A),  c.add(h0), c.add(kept),
                       c.add(dy), c.add(dht), c.add(dx), c.add(dr), c.add(di), c.add(dA),
                       c.add(dh0)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_rec_bwd(p[0], p[1], p[2], p[3], normalize, p[4], s.cu, s.n, p[5], p[6], p[7],
                             p[8], p[9], p[10], p[11], p[12], ws.p, ws.n, st);
        }),
        "gdr_rec_bwd");
  return tuple({dx, dr, dA, di, dh0});
EXIT

// x, r, A, state, i, normalize, idx, out
ENTRY(rec_step, 8)
  const at::Tensor x = required(args[0], 2, "x");
  const at::Tensor r = tensor(args[1]), A = tensor(args[2]), state = tensor(args[3]),
                   i = tensor(args[4]), idx = tensor(args[6]);
  Call c(x);
  enter(guard, c);
  const int32_t normalize = truth(args[5]);
  const int32_t *ix = c.ints(idx, x.size(0), "state_indices");
  at::Tensor y = tensor(args[7]);
  if (!y.defined()) y = empty(x.sizes(), x);
  gdr_tensor_t *p[] = {c.add(x), c.add(r), c.add(i), c.add(A), c.add(state), c.add(y)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_rec_step(p[0], p[1], p[2], p[3], normalize, p[4], ix, p[5], st);
        }),
        "gdr_rec_step");
  return wrap(y);
EXIT

// x, z, weight, activation, eps, out
ENTRY(gated_norm_fwd, 6)
  const at::Tensor x = required(args[0], 3, "x");
  const at::Tensor z = tensor(args[1]), w = tensor(args[2]);
  Call c(x);
  enter(guard, c);
  const int32_t act = gate_activation(args[3]);
  const float eps = (float)real(args[4]);
  at::Tensor y = tensor(args[5]);
  if (!y.defined()) y = empty(x.sizes(), x);
  gdr_tensor_t *p[] = {c.add(x), c.add(z), c.add(w), c.add(y)};
  const cudaStream_t st = c.stream();
  check(run([&] { return gdr_gated_norm_fwd(p[0], p[1], p[2], act, eps, p[3], st); }),
        "gdr_gated_norm_fwd");
  return wrap(y);
EXIT

// x, z, dy, weight, activation, eps, workspace
ENTRY(gated_norm_bwd, 7)
  const at::Tensor x = required(args[0], 3, "x"), z = required(args[1], 3, "z");
  const at::Tensor dy = tensor(args[2]), w = tensor(args[3]);
  Call c(x);
  enter(guard, c);
  const int32_t act = gate_activation(args[4]);
  const float eps = (float)real(args[5]);
  at::Tensor dx = empty(x.sizes(), x), dz = empty(z.sizes(), x), dw;
  if (w.defined()) dw = empty32({x.size(2)}, x);
  const Scratch ws(c, tensor(args[6]),
                   gdr_gated_norm_bwd_workspace_bytes(x.size(0), (int32_t)x.size(1),
                                                      (int32_t)x.size(2)),
                   x);
  gdr_tensor_t *p[] = {c.add(x), c.add(z), c.add(w), c.add(dy), c.add(dx), c.add(dz), c.add(dw)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_gated_norm_bwd(p[0], p[1], p[2], act, eps, p[3], p[4], p[5], p[6], ws.p, ws.n,
                                    st);
        }),
        "gdr_gated_norm_bwd");
  return tuple({dx, dz, dw});
EXIT

// x, residual, weight, post, post_weight, gate, scale, eps, out, residual_out
ENTRY(residual_norm_fwd, 10)
  const at::Tensor x = required(args[0], 2, "x");
  const at::Tensor res = tensor(args[1]), w = tensor(args[2]), wp = tensor(args[4]),
                   g = tensor(args[5]);
  Call c(x);
  enter(guard, c);
  const int32_t post = truth(args[3]);
  const float scale = (float)real(args[6]), eps = (float)real(args[7]);
  at::Tensor y = tensor(args[8]), h = tensor(args[9]);
  if (!y.defined()) y = empty(x.sizes(), x);
  if (!h.defined()) h = empty(x.sizes(), res.defined() ? res : x);
  gdr_tensor_t *p[] = {c.add(x), c.add(res), c.add(w), c.add(wp), c.add(g), c.add(y), c.add(h)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_residual_norm_fwd(p[0], p[1], p[2], post, p[3], p[4], scale, eps, p[5], p[6],
                                       st);
        }),
        "gdr_residual_norm_fwd");
  return tuple({y, h});
EXIT

// x, residual, dy, dh, weight, post, post_weight, gate, scale, eps, workspace
ENTRY(residual_norm_bwd, 11)
  const at::Tensor x = required(args[0], 2, "x");
  const at::Tensor res = tensor(args[1]), dy = tensor(args[2]), dh = tensor(args[3]),
                   w = tensor(args[4]), wp = tensor(args[6]), g = tensor(args[7]);
  Call c(x);
  enter(guard, c);
  const int32_t post = truth(args[5]);
  const float scale = (float)real(args[8]), eps = (float)real(args[9]);
  at::Tensor dx = empty(x.sizes(), x), dres, dw, dwp, dg;
  if (res.defined()) dres = empty(x.sizes(), res);
  if (w.defined()) dw = empty32({x.size(1)}, x);
  if (wp.defined()) dwp = empty32({x.size(1)}, x);
  if (g.defined()) dg = empty32({x.size(1)}, x);
  const Scratch ws(c, tensor(args[10]),
                   gdr_residual_norm_bwd_workspace_bytes(x.size(0), (int32_t)x.size(1)), x);
  gdr_tensor_t *p[] = {c.add(x),  c.add(res), c.add(w),    c.add(wp), c.add(g),   c.add(dy),
                       c.add(dh), c.add(dx),  c.add(dres), c.add(dw), c.add(dwp), c.add(dg)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_residual_norm_bwd(p[0], p[1], p[2], post, p[3], p[4], scale, eps, p[5], p[6],
                                       p[7], p[8], p[9], p[10], p[11], ws.p, ws.n, st);
        }),
        "gdr_residual_norm_bwd");
  return tuple({dx, dres, dw, dwp, dg});
EXIT

// q, k_cache, v_cache, block_table, lengths, scale (None: d^-1/2), window, out, workspace
ENTRY(attn_step, 9)
  const at::Tensor q = required(args[0], 3, "q"), kc = required(args[1], 4, "k_cache"),
                   table = required(args[3], 2, "block_table"),
                   lens = required(args[4], 1, "lengths");
  const at::Tensor vc = tensor(args[2]);
  Call c(q);
  enter(guard, c);
  const float scale = args[5] == Py_None ? 1.f / std::sqrt((float)q.size(2)) : (float)real(args[5]);
  const int32_t window = whole(args[6], "window");
  const int32_t *ln = c.ints(lens, q.size(0), "lengths");
  at::Tensor o = tensor(args[7]);
  if (!o.defined()) o = empty(q.sizes(), q);
  const Scratch ws(c, tensor(args[8]),
                   gdr_attn_step_workspace_bytes((int32_t)q.size(0), (int32_t)q.size(1),
                                                 (int32_t)kc.size(2), (int32_t)q.size(2)),
                   q);
  gdr_tensor_t *p[] = {c.add(q), c.add(kc), c.add(vc), c.table(table, "block_table"), c.add(o)};
  const cudaStream_t st = c.stream();
  check(run([&] {
          return gdr_attn_step(p[0], p[1], p[2], p[3], ln, scale, window, p[4], ws.p, ws.n, st);
        }),
        "gdr_attn_step");
  return wrap(o);
EXIT

// lengths, new_tokens, block_table, free_pages, taken, page_size, max_tokens, lengths_out, taken_out
ENTRY(cache_plan, 9)
  const at::Tensor lens = required(args[0], 1, "lengths"), fresh = required(args[1], 1, "new_tokens"),
                   table = required(args[2], 2, "block_table"),
                   pages = required(args[3], 1, "free_pages"), taken = required(args[4], 1, "taken");
  Call c(lens);
  enter(guard, c);
  const int64_t B = lens.size(0);
  const int32_t page = whole(args[5], "page_size"), most = whole(args[6], "max_tokens");
  if (B > 0x7ff00000) refuse(PyExc_ValueError, "too many requests");
  if (most < 0) refuse(PyExc_ValueError, "max_tokens must not be negative");
  const int32_t *ln = c.ints(lens, B, "lengths"), *nw = c.ints(fresh, B, "new_tokens"),
                *tk = c.ints(taken, 1, "taken");
  c.ints(pages, -1, "free_pages");
  at::Tensor lens_out = tensor(args[7]), taken_out = tensor(args[8]);
  // the results in one allocation
  Parts parts(2 * (int64_t)most + 2 * B + 2 + 5 * 64, lens);
  const at::Tensor slots = parts.next(most), pos = parts.next(most), cu = parts.next(B + 1);
  if (!lens_out.defined()) lens_out = parts.next(B);
  if (!taken_out.defined()) taken_out = parts.next(1);
  const int32_t *lo = c.ints(lens_out, B, "lengths_out"), *to = c.ints(taken_out, 1, "taken_out");
  gdr_tensor_t *p[] = {c.table(table, "block_table"), c.table(pages, "free_pages")};
  const cudaStream_t st = c.stream();
  int32_t *sp = most ? slots.data_ptr<int32_t>() : nullptr, *pp = most ? pos.data_ptr<int32_t>() : nullptr;
  int32_t *cp = cu.data_ptr<int32_t>();
  check(run([&] {
          return gdr_cache_plan(ln, nw, (int32_t)B, p[0], p[1], tk, page, sp, pp, most, cp,
                                const_cast<int32_t *>(lo), const_cast<int32_t *>(to), st);
        }),
        "gdr_cache_plan");
  return tuple({slots, pos, cu, lens_out, taken_out});
EXIT

// k, v, k_cache, v_cache, slots
ENTRY(cache_write, 5)
  const at::Tensor k = required(args[0], 3, "k");
  const at::Tensor v = tensor(args[1]), kc = tensor(args[2]), vc = tensor(args[3]),
                   slots = required(args[4], 1, "slots");
  Call c(k);
  enter(guard, c);
  const int32_t *sl = c.ints(slots, k.size(0), "slots");
  gdr_tensor_t *p[] = {c.add(k), c.add(v), c.add(kc), c.add(vc)};
  const cudaStream_t st = c.stream();
  check(run([&] { return gdr_cache_write(p[0], p[1], p[2], p[3], sl, st); }), "gdr_cache_write");
  Py_RETURN_NONE;
EXIT

PyObject *set_error(PyObject *, PyObject *type) {
  Py_XINCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD(conv_fwd),  METHOD(conv_bwd), METHOD(conv_step),
                          METHOD(ssm_fwd),   METHOD(ssm_bwd),  METHOD(ssm_step),
                          METHOD(qk_fwd),    METHOD(qk_bwd),   METHOD(delta_step),
                          METHOD(rec_fwd),   METHOD(rec_bwd),  METHOD(rec_step),
                          METHOD(gated_norm_fwd),    METHOD(gated_norm_bwd),
                          METHOD(residual_norm_fwd), METHOD(residual_norm_bwd),
                          METHOD(attn_step), METHOD(cache_plan), METHOD(cache_write),
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_mixer", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mixer(void) { return PyModule_Create(&kModule); }
