// Direct calls of the hybrid block's forward and serving entry points.
//
// A decoded token's kernels run for a few microseconds, less than Python
// needs to check eight tensors and marshal their addresses (glr_step 9.7 us a
// call that way, 3.6 of them the launch). These functions do both in C++ for
// the ordinary call: every argument a torch.Tensor of the right type, shape
// and device, dense where it has to be, outputs to be allocated, the current
// stream. For any other call they return None and have done nothing; the
// Python wrapper then takes its own path, which accepts the rest of what is
// valid and says what is wrong with what is not.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPStream.h>

#include <cstring>
#include <initializer_list>

#include "ssm_hybrid.h"

namespace {

struct Calls {
  decltype(&ssm_glr_step) glr_step;
  decltype(&ssm_glr_fwd) glr_fwd;
  decltype(&ssm_glr_workspace_bytes) glr_bytes;
  decltype(&ssm_qk_rope_fwd) rope_fwd;
  decltype(&ssm_qk_rope_append) rope_append;
  decltype(&ssm_swa_fwd) swa_fwd;
  decltype(&ssm_swa_decode) swa_decode;
  decltype(&ssm_swa_decode_workspace_bytes) decode_bytes;
} calls;

struct NotOrdinary {};
void need(bool ok) {
  if (!ok) throw NotOrdinary{};
}

const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_CheckExact(o));
  return THPVariable_Unpack(o);
}

bool shape_is(const at::Tensor& t, std::initializer_list<int64_t> shape) {
  return t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
}

// The call's device and type, from its first argument.
struct Call {
  c10::Device device;
  at::ScalarType type;
  int code;
  explicit Call(const at::Tensor& t, int64_t dims) : device(t.device()), type(t.scalar_type()) {
    need(t.dim() == dims && device.is_cuda());
    need(type == at::kFloat || type == at::kBFloat16);
    code = type == at::kFloat ? SSM_F32 : SSM_BF16;
    need(c10::hip::current_device() == device.index());
  }
  void* dense(PyObject* o, at::ScalarType want, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == want && t.device() == device && shape_is(t, shape) && t.is_contiguous());
    return t.data_ptr();
  }
  void* maybe(PyObject* o, at::ScalarType want, std::initializer_list<int64_t> shape) const {
    return o == Py_None ? nullptr : dense(o, want, shape);
  }
  // (batch, token, head, D) whose last dimension is contiguous
  void* strided(PyObject* o, std::initializer_list<int64_t> shape, ssm_strides* s) const {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.device() == device && t.layout() == at::kStrided && shape_is(t, shape));
    need(t.numel() > 0 && t.stride(3) == 1);
    *s = ssm_strides{t.stride(0), t.stride(1), t.stride(2)};
    return t.data_ptr();
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType want) const {
    return at::empty(shape, at::TensorOptions().dtype(want).device(device));
  }
  void* stream() const { return c10::hip::getCurrentHIPStream(device.index()).stream(); }
};

int64_t integer(PyObject* o) {
  need(PyLong_Check(o));
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotOrdinary{};
  }
  return v;
}
double number(PyObject* o) {
  need(PyFloat_Check(o));
  return PyFloat_AS_DOUBLE(o);
}
void none(PyObject* o) { need(o == Py_None); }

PyObject* pair(at::Tensor a, at::Tensor b) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(a)));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(b)));
  return t;
}

// f(args), or None where it is not an ordinary call (or the library refuses).
template <typename F>
PyObject* ordinary(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) Py_RETURN_NONE;
  try {
    return f();
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// x, gr, gi, A, h, y, h_out, stream
PyObject* glr_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 8, [&] {
    none(a[5]), none(a[6]), none(a[7]);
    const at::Tensor& x = tensor(a[0]);
    const Call c(x, 2);
    const int64_t Bs = x.size(0), ED = x.size(1);
    const void* px = c.dense(a[0], c.type, {Bs, ED});
    const void* pr = c.dense(a[1], c.type, {Bs, ED});
    const void* pi = c.dense(a[2], c.type, {Bs, ED});
    const auto pA = static_cast<const float*>(c.dense(a[3], at::kFloat, {ED}));
    const auto ph = static_cast<const float*>(c.dense(a[4], at::kFloat, {Bs, ED}));
    at::Tensor y = c.make({Bs, ED}, c.type), h = c.make({Bs, ED}, at::kFloat);
    need(calls.glr_step(px, pr, pi, pA, ph, y.data_ptr(), h.data_ptr<float>(), Bs, ED, c.code, c.stream()) == SSM_OK);
    return pair(std::move(y), std::move(h));
  });
}

// x, gr, gi, A, y, h_last, ckpt, h0, workspace, stream
PyObject* glr_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 10, [&] {
    none(a[4]), none(a[8]), none(a[9]);
    const at::Tensor& x = tensor(a[0]);
    const Call c(x, 3);
    const int64_t Bs = x.size(0), L = x.size(1), ED = x.size(2);
    const void* px = c.dense(a[0], c.type, {Bs, L, ED});
    const void* pr = c.dense(a[1], c.type, {Bs, L, ED});
    const void* pi = c.dense(a[2], c.type, {Bs, L, ED});
    const auto pA = static_cast<const float*>(c.dense(a[3], at::kFloat, {ED}));
    const auto pl = static_cast<float*>(c.maybe(a[5], at::kFloat, {Bs, ED}));
    const auto pc = static_cast<float*>(
        c.maybe(a[6], at::kFloat, {Bs, (L + SSM_GLR_CKPT_STEPS - 1) / SSM_GLR_CKPT_STEPS, ED}));
    const auto p0 = static_cast<const float*>(c.maybe(a[7], at::kFloat, {Bs, ED}));
    at::Tensor y = c.make({Bs, L, ED}, c.type), ws;
    const size_t bytes = calls.glr_bytes(Bs, L, ED, c.code);
    if (bytes) ws = c.make({static_cast<int64_t>(bytes)}, at::kByte);
    need(calls.glr_fwd(px, pr, pi, pA, p0, y.data_ptr(), pl, pc, Bs, L, ED, c.code, bytes ? ws.data_ptr() : nullptr,
                       bytes, c.stream()) == SSM_OK);
    return THPVariable_Wrap(std::move(y));
  });
}

struct Rope {
  int64_t Bs, L, Hq, Hk, D, R;
  ssm_strides sq, sk;
  const void *q, *k;
  const float *wq, *wk;
  const double* freq;
  // q, k, wq, wk, freq at a[0 .. 1], a[w .. w + 2]
  Rope(const Call& c, PyObject* const* a, int w) {
    const at::Tensor &tq = tensor(a[0]), &tk = tensor(a[1]);
    need(tk.dim() == 4);
    Bs = tq.size(0), L = tq.size(1), Hq = tq.size(2), D = tq.size(3), Hk = tk.size(2);
    q = c.strided(a[0], {Bs, L, Hq, D}, &sq);
    k = c.strided(a[1], {Bs, L, Hk, D}, &sk);
    wq = static_cast<const float*>(c.maybe(a[w], at::kFloat, {D}));
    wk = static_cast<const float*>(c.maybe(a[w + 1], at::kFloat, {D}));
    const at::Tensor& tf = tensor(a[w + 2]);
    need(tf.dim() == 1);
    R = 2 * tf.size(0);
    freq = static_cast<const double*>(c.dense(a[w + 2], at::kDouble, {R / 2}));
  }
};

// q, k, wq, wk, freq, pos, eps, q_out, k_out, stream
PyObject* rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 10, [&] {
    none(a[7]), none(a[8]), none(a[9]);
    const Call c(tensor(a[0]), 4);
    const Rope r(c, a, 2);
    const auto pos = static_cast<const int32_t*>(c.maybe(a[5], at::kInt, {r.Bs, r.L}));
    const double eps = number(a[6]);
    at::Tensor qo = c.make({r.Bs, r.L, r.Hq, r.D}, c.type), ko = c.make({r.Bs, r.L, r.Hk, r.D}, c.type);
    need(calls.rope_fwd(r.q, &r.sq, r.k, &r.sk, r.wq, r.wk, r.freq, pos, eps, qo.data_ptr(), ko.data_ptr(), r.Bs, r.L,
                        r.Hq, r.Hk, r.D, r.R, c.code, c.stream()) == SSM_OK);
    return pair(std::move(qo), std::move(ko));
  });
}

// q, k, v, wq, wk, freq, pos, k_cache, v_cache, sinks, eps, q_out, stream
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 13, [&] {
    none(a[11]), none(a[12]);
    const Call c(tensor(a[0]), 4);
    const Rope r(c, a, 3);
    ssm_strides sv;
    const void* v = c.strided(a[2], {r.Bs, r.L, r.Hk, r.D}, &sv);
    const auto pos = static_cast<const int32_t*>(c.dense(a[6], at::kInt, {r.Bs}));
    const at::Tensor& tc = tensor(a[7]);
    need(tc.dim() == 4);
    const int64_t C = tc.size(2), sinks = integer(a[9]);
    need(sinks >= 0 && sinks < C);
    void* kc = c.dense(a[7], c.type, {r.Bs, r.Hk, C, r.D});
    void* vc = c.dense(a[8], c.type, {r.Bs, r.Hk, C, r.D});
    const double eps = number(a[10]);
    at::Tensor qo = c.make({r.Bs, r.L, r.Hq, r.D}, c.type);
    need(calls.rope_append(r.q, &r.sq, r.k, &r.sk, v, &sv, r.wq, r.wk, r.freq, pos, eps, qo.data_ptr(), kc, vc, r.Bs,
                           r.L, r.Hq, r.Hk, r.D, r.R, C - sinks, sinks, c.code, c.stream()) == SSM_OK);
    return THPVariable_Wrap(std::move(qo));
  });
}

// q, k, v, window, sinks, scale, lens, o, lse, stream
PyObject* swa_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 10, [&] {
    none(a[7]), none(a[9]);
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]);
    const Call c(q, 4);
    need(k.dim() == 4);
    const int64_t Bs = q.size(0), Lq = q.size(1), Hq = q.size(2), D = q.size(3), Lk = k.size(1), Hk = k.size(2);
    ssm_strides sq, sk, sv;
    const void* pq = c.strided(a[0], {Bs, Lq, Hq, D}, &sq);
    const void* pk = c.strided(a[1], {Bs, Lk, Hk, D}, &sk);
    const void* pv = c.strided(a[2], {Bs, Lk, Hk, D}, &sv);
    const int64_t window = integer(a[3]), sinks = integer(a[4]);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : number(a[5]);
    const auto lens = static_cast<const int32_t*>(c.maybe(a[6], at::kInt, {Bs}));
    const auto lse = static_cast<float*>(c.maybe(a[8], at::kFloat, {Bs, Hq, Lq}));
    at::Tensor o = c.make({Bs, Lq, Hq, D}, c.type);
    need(calls.swa_fwd(pq, &sq, pk, &sk, pv, &sv, lens, scale, o.data_ptr(), lse, Bs, Lq, Lk, Hq, Hk, D, window, sinks,
                       c.code, c.stream()) == SSM_OK);
    return THPVariable_Wrap(std::move(o));
  });
}

// q, k_cache, v_cache, pos, scale, o, workspace, stream
PyObject* swa_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 8, [&] {
    none(a[5]), none(a[6]), none(a[7]);
    const at::Tensor &q = tensor(a[0]), &tc = tensor(a[1]);
    const Call c(q, 3);
    need(tc.dim() == 4 && q.layout() == at::kStrided && q.numel() > 0 && q.stride(2) == 1);
    const int64_t Bs = q.size(0), Hq = q.size(1), D = q.size(2), Hk = tc.size(1), C = tc.size(2);
    const ssm_strides sq{q.stride(0), 0, q.stride(1)};
    const void* kc = c.dense(a[1], c.type, {Bs, Hk, C, D});
    const void* vc = c.dense(a[2], c.type, {Bs, Hk, C, D});
    const auto pos = static_cast<const int32_t*>(c.dense(a[3], at::kInt, {Bs}));
    const double scale = a[4] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : number(a[4]);
    at::Tensor o = c.make({Bs, Hq, D}, c.type), ws;
    const size_t bytes = calls.decode_bytes(Bs, C, Hq, Hk, D, c.code);
    if (bytes) ws = c.make({static_cast<int64_t>(bytes)}, at::kByte);
    need(calls.swa_decode(q.data_ptr(), &sq, kc, vc, pos, scale, o.data_ptr(), Bs, C, Hq, Hk, D, c.code,
                          bytes ? ws.data_ptr() : nullptr, bytes, c.stream()) == SSM_OK);
    return THPVariable_Wrap(std::move(o));
  });
}

// bind(name, address): an entry point of the loaded library
PyObject* bind(PyObject*, PyObject* args) {
  const char* name;
  unsigned long long at;
  if (!PyArg_ParseTuple(args, "sK", &name, &at)) return nullptr;
  const auto p = reinterpret_cast<void*>(static_cast<uintptr_t>(at));
  const struct {
    const char* name;
    void** to;
  } table[] = {{"ssm_glr_step", reinterpret_cast<void**>(&calls.glr_step)},
               {"ssm_glr_fwd", reinterpret_cast<void**>(&calls.glr_fwd)},
               {"ssm_glr_workspace_bytes", reinterpret_cast<void**>(&calls.glr_bytes)},
               {"ssm_qk_rope_fwd", reinterpret_cast<void**>(&calls.rope_fwd)},
               {"ssm_qk_rope_append", reinterpret_cast<void**>(&calls.rope_append)},
               {"ssm_swa_fwd", reinterpret_cast<void**>(&calls.swa_fwd)},
               {"ssm_swa_decode", reinterpret_cast<void**>(&calls.swa_decode)},
               {"ssm_swa_decode_workspace_bytes", reinterpret_cast<void**>(&calls.decode_bytes)}};
  for (const auto& t : table)
    if (!std::strcmp(t.name, name)) {
      *t.to = p;
      Py_RETURN_NONE;
    }
  PyErr_Format(PyExc_KeyError, "%s", name);
  return nullptr;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"glr_step", fast<glr_step>(), METH_FASTCALL, nullptr},
                         {"glr_fwd", fast<glr_fwd>(), METH_FASTCALL, nullptr},
                         {"rope_fwd", fast<rope_fwd>(), METH_FASTCALL, nullptr},
                         {"rope_append", fast<rope_append>(), METH_FASTCALL, nullptr},
                         {"swa_fwd", fast<swa_fwd>(), METH_FASTCALL, nullptr},
                         {"swa_decode", fast<swa_decode>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_calls() { return PyModule_Create(&module); }
