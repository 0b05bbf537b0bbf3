// CPython entry to the calls of pkv.h whose kernels run for a few microseconds: checks of the tensors
// and marshalling without interpreter time (a rotary append of 64 tokens takes 2.3 us on the GPU; its
// checks in Python and the conversions of ctypes took 7 us; the whole call is now 3.6 us of host time).
//
// Every function takes what the binding of the same name was given, with outputs and workspace
// present, and a stream's address or None for the current stream.  It returns the call's pkv_status,
// or 1 when an argument is not what the call takes: nothing was called then, and the binding names the
// mistake.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>

#include "../../include/pkv.h"

namespace {

constexpr long kNotTaken = 1;
constexpr auto BF16 = at::kBFloat16;
constexpr auto F32 = at::kFloat;
constexpr auto I32 = at::kInt;
constexpr auto I64 = at::kLong;
constexpr auto U8 = at::kByte;

// The arguments of one call; `ok` turns false at the first that is not taken.
struct Args {
  PyObject* const* a;
  int dev = -1;                                                // device of the first tensor
  bool ok = true;
  explicit Args(PyObject* const* args) : a(args) {}

  const at::Tensor& any(int i, at::ScalarType type, at::ScalarType other) {
    static const at::Tensor none;
    if (!ok || !THPVariable_Check(a[i])) {
      ok = false;
      return none;
    }
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    const int d = t.is_cuda() ? (int)t.get_device() : -1;
    if (dev < 0) dev = d;
    ok = d >= 0 && d == dev && (t.scalar_type() == type || t.scalar_type() == other);
    return t;
  }
  const at::Tensor& any(int i, at::ScalarType type) { return any(i, type, type); }
  bool shaped(const at::Tensor& t, std::initializer_list<int64_t> shape) {
    if (ok) ok = t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
    return ok;
  }
  const at::Tensor& dense(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor& t = any(i, type);
    if (shaped(t, shape)) ok = t.is_contiguous();
    return t;
  }
  const at::Tensor& dense(int i, at::ScalarType type, int64_t dims) {
    const at::Tensor& t = any(i, type);
    if (ok) ok = t.dim() == dims && t.is_contiguous();
    return t;
  }
  // [tokens][heads][d] with dense heads; the stride between tokens goes to `stride`
  const at::Tensor& tokens(int i, int64_t n, int64_t heads, int64_t d, int64_t& stride) {
    const at::Tensor& t = any(i, BF16);
    if (shaped(t, {n, heads, d})) {
      const auto s = t.strides();
      ok = t.numel() == 0 || (s[2] == 1 && (heads == 1 || s[1] == d));
      stride = n > 1 ? s[0] : heads * d;                      // one token has no stride
    }
    return t;
  }
  int32_t* err(int i) {
    if (!ok || a[i] == Py_None) return nullptr;
    const at::Tensor& t = any(i, I32);
    if (ok) ok = t.numel() > 0;
    return ok ? static_cast<int32_t*>(t.data_ptr()) : nullptr;
  }
  int integer(int i) {
    const long v = PyLong_AsLong(a[i]);
    if ((v == -1 && PyErr_Occurred()) || v != (long)(int)v) ok = false;
    return (int)v;
  }
  float number(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return (float)v;
  }
  pkv_rope_table table(int i) {                                // a copy of the binding's structure
    pkv_rope_table t = {};
    Py_buffer view;
    if (PyObject_GetBuffer(a[i], &view, PyBUF_SIMPLE) != 0) {
      ok = false;
      return t;
    }
    if (view.len == (Py_ssize_t)sizeof(t)) memcpy(&t, view.buf, sizeof(t));
    else ok = false;
    PyBuffer_Release(&view);
    return t;
  }
  void size(int64_t v) { ok = ok && v >= 0 && v <= 0x7fffffff; }
  template <class... T>
  void sizes(T... v) {                                         // what the C calls take as int
    (size(v), ...);
  }
  // the stream of the call; its tensors are on the current device
  void* stream(int i) {
    if (ok) ok = c10::cuda::current_device() == dev;
    if (!ok) return nullptr;
    if (a[i] == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    void* p = PyLong_AsVoidPtr(a[i]);
    if (p == nullptr && PyErr_Occurred()) ok = false;
    return p;
  }
};

PyObject* result(long status) { return PyLong_FromLong(status); }

// The C call without the interpreter's lock: a launch may wait for room in the stream's queue.
struct NoLock {
  PyThreadState* state = PyEval_SaveThread();
  ~NoLock() { PyEval_RestoreThread(state); }
};
template <class F>
PyObject* unlocked(F call) {
  pkv_status st;
  {
    const NoLock none;
    st = call();
  }
  return result(st);
}

int32_t* ints(const at::Tensor& t) { return t.data_ptr<int32_t>(); }

// a workspace of any type and shape, or none
void workspace(Args& x, int i, void*& ptr, size_t& bytes) {
  if (!x.ok || x.a[i] == Py_None) return;
  const at::Tensor& t = x.any(i, THPVariable_Check(x.a[i]) ? THPVariable_Unpack(x.a[i]).scalar_type() : U8);
  if (x.ok) x.ok = t.is_contiguous();
  if (x.ok) ptr = t.data_ptr(), bytes = t.nbytes();
}

// q, k, v, positions, slot_mapping, table, k_pool, v_pool, q_out, err, stream
PyObject* rope_append(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 11) return result(kNotTaken);
  Args x(a);
  const at::Tensor &q = x.any(0, BF16), &kp = x.dense(6, BF16, 4);
  if (!x.ok || q.dim() != 3) return result(kNotTaken);
  const int64_t n = q.size(0), n_h = q.size(1), d = q.size(2), nb = kp.size(0), n_kv = kp.size(1), bs = kp.size(2);
  int64_t sq = 0, sk = 0, sv = 0, so = 0;
  x.tokens(0, n, n_h, d, sq);
  x.shaped(kp, {nb, n_kv, bs, d});
  const at::Tensor &k = x.tokens(1, n, n_kv, d, sk), &v = x.tokens(2, n, n_kv, d, sv), &out = x.tokens(8, n, n_h, d, so);
  const at::Tensor &pos = x.dense(3, I32, {n}), &slots = x.dense(4, I64, {n}), &vp = x.dense(7, BF16, {nb, n_kv, bs, d});
  const pkv_rope_table table = x.table(5);
  int32_t* err = x.err(9);
  void* stream = x.stream(10);
  x.sizes(n, n_h, nb, n_kv, bs, d);
  if (!x.ok) return result(kNotTaken);
  return unlocked([&] {
    return pkv_rope_append(q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, ints(pos), slots.data_ptr<int64_t>(), (int)n,
                           &table, out.data_ptr(), so, kp.data_ptr(), vp.data_ptr(), (int)nb, (int)bs, (int)n_h, (int)n_kv,
                           (int)d, err, stream);
  });
}

// q, k, positions, table, q_out, k_out, stream
PyObject* rope_qk(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 7) return result(kNotTaken);
  Args x(a);
  const at::Tensor &q = x.any(0, BF16), &k = x.any(1, BF16);
  if (!x.ok || q.dim() != 3 || k.dim() != 3) return result(kNotTaken);
  const int64_t n = q.size(0), n_h = q.size(1), d = q.size(2), n_kv = k.size(1);
  int64_t sq = 0, sk = 0, so = 0, ko = 0;
  x.tokens(0, n, n_h, d, sq);
  x.tokens(1, n, n_kv, d, sk);
  const at::Tensor &qo = x.tokens(4, n, n_h, d, so), &kout = x.tokens(5, n, n_kv, d, ko), &pos = x.dense(2, I32, {n});
  const pkv_rope_table table = x.table(3);
  void* stream = x.stream(6);
  x.sizes(n, n_h, n_kv, d);
  if (!x.ok) return result(kNotTaken);
  return unlocked([&] {
    return pkv_rope_qk(q.data_ptr(), sq, k.data_ptr(), sk, ints(pos), (int)n, &table, qo.data_ptr(), so, kout.data_ptr(), ko,
                       (int)n_h, (int)n_kv, (int)d, stream);
  });
}

// An 8-bit cache's records, k_tail and v_tail at a[i .. i + 2].
struct Cache {
  const at::Tensor &records, &k_tail;
  const at::Tensor* v_tail = nullptr;
  int64_t rows = 0, n_kv = 0, bs = 0, d = 0, nb = 0;
  Cache(Args& x, int i) : records(x.dense(i, U8, 3)), k_tail(x.dense(i + 1, BF16, 4)) {
    if (!x.ok) return;
    rows = k_tail.size(0), n_kv = k_tail.size(1), bs = k_tail.size(2), d = k_tail.size(3), nb = records.size(0);
    x.sizes(rows, n_kv, bs, d, nb);
    x.shaped(records, {nb, n_kv, 2 * bs * d + 16});
    v_tail = &x.dense(i + 2, BF16, {rows, n_kv, bs, d});
  }
};

// k, v, slot_mapping, tail_seq, records, k_tail, v_tail, format, err, stream
PyObject* kv_quant_append_q8(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 10) return result(kNotTaken);
  Args x(a);
  const at::Tensor& k = x.any(0, BF16);
  const Cache c(x, 4);
  if (!x.ok || k.dim() != 3) return result(kNotTaken);
  const int64_t n = k.size(0);
  int64_t sk = 0, sv = 0;
  x.tokens(0, n, c.n_kv, c.d, sk);
  const at::Tensor &v = x.tokens(1, n, c.n_kv, c.d, sv), &slots = x.dense(2, I64, {n}), &seq = x.dense(3, I32, {n});
  const int format = x.integer(7);
  int32_t* err = x.err(8);
  void* stream = x.stream(9);
  x.sizes(n);
  if (!x.ok) return result(kNotTaken);
  return unlocked([&] {
    return pkv_kv_quant_append_q8(k.data_ptr(), sk, v.data_ptr(), sv, slots.data_ptr<int64_t>(), ints(seq), (int)n, format,
                                  c.records.data_ptr<uint8_t>(), c.k_tail.data_ptr(), c.v_tail->data_ptr(), (int)c.rows,
                                  (int)c.nb, (int)c.bs, (int)c.n_kv, (int)c.d, err, stream);
  });
}

// What the attention calls share: q, block tables, context lengths, output and workspace (None for none).
struct Decode {
  const at::Tensor& q;
  const at::Tensor *bt = nullptr, *ctx = nullptr, *out = nullptr;
  int64_t B = 0, n_h = 0, mb = 0;
  int out_type = PKV_OUT_BF16;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  Decode(Args& x, int iq, int ibt, int ictx, int iout, int iws, int64_t d) : q(x.dense(iq, BF16, 3)) {
    if (!x.ok) return;
    B = q.size(0), n_h = q.size(1);
    x.shaped(q, {B, n_h, d});
    bt = &x.dense(ibt, I32, 2);
    if (!x.ok) return;
    mb = bt->size(1);
    x.shaped(*bt, {B, mb});
    ctx = &x.dense(ictx, I32, {B});
    out = &x.any(iout, BF16, F32);
    if (x.shaped(*out, {B, n_h, d})) x.ok = out->is_contiguous();
    workspace(x, iws, ws, ws_bytes);
    x.sizes(B, n_h, mb);
    if (x.ok && out->scalar_type() == F32) out_type = PKV_OUT_F32;
  }
};

// q, records, k_tail, v_tail, format, block_tables, context_lens, scale, window, out, workspace, err, stream
PyObject* paged_decode_attn_q8(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 13) return result(kNotTaken);
  Args x(a);
  const Cache c(x, 1);
  const Decode t(x, 0, 5, 6, 9, 10, c.d);
  const int format = x.integer(4), window = x.integer(8);
  const float scale = x.number(7);
  int32_t* err = x.err(11);
  void* stream = x.stream(12);
  if (!x.ok) return result(kNotTaken);
  return unlocked([&] {
    return pkv_paged_decode_attn_q8(t.q.data_ptr(), c.records.data_ptr<uint8_t>(), format, ints(*t.bt), (int)t.mb, ints(*t.ctx),
                                    scale, window, (int)t.B, (int)t.n_h, (int)c.n_kv, (int)c.d, (int)c.bs, (int)c.nb,
                                    t.out->data_ptr(), t.out_type, t.ws, t.ws_bytes, err, stream);
  });
}

// q, k_pool, v_pool, block_tables, context_lens, scale, mass, out, workspace, err, stream
PyObject* paged_decode_attn_mass(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 11) return result(kNotTaken);
  Args x(a);
  const at::Tensor &kp = x.dense(1, BF16, 4), &mass = x.dense(6, F32, 3);
  if (!x.ok) return result(kNotTaken);
  const int64_t nb = kp.size(0), n_kv = kp.size(1), bs = kp.size(2), d = kp.size(3), T = mass.size(2);
  const at::Tensor& vp = x.dense(2, BF16, {nb, n_kv, bs, d});
  const Decode t(x, 0, 3, 4, 7, 8, d);
  x.shaped(mass, {t.B, n_kv, T});
  const float scale = x.number(5);
  int32_t* err = x.err(9);
  void* stream = x.stream(10);
  x.sizes(nb, n_kv, bs, d);
  if (!x.ok) return result(kNotTaken);
  return unlocked([&] {
    return pkv_paged_decode_attn_mass(t.q.data_ptr(), kp.data_ptr(), vp.data_ptr(), ints(*t.bt), (int)t.mb, ints(*t.ctx), scale,
                                      (int)t.B, (int)t.n_h, (int)n_kv, (int)d, (int)bs, (int)nb, t.out->data_ptr(), t.out_type,
                                      mass.data_ptr<float>(), T, t.ws, t.ws_bytes, err, stream);
  });
}

// One state of an eviction, mass, positions, kept and dropped at a[i .. i + 3].
struct State {
  float* mass = nullptr;
  int32_t *positions = nullptr, *kept = nullptr, *dropped = nullptr;
  State(Args& x, int i, int64_t B, int64_t n_kv, int64_t T) {
    const at::Tensor &m = x.dense(i, F32, {B, n_kv, T}), &p = x.dense(i + 1, I32, {B, n_kv, T}), &k = x.dense(i + 2, I32, {B}),
                     &r = x.dense(i + 3, I32, {B});
    if (x.ok) mass = m.data_ptr<float>(), positions = ints(p), kept = ints(k), dropped = ints(r);
  }
};

// k_pool, v_pool, block_tables, context_lens, keep, recent, 4 tensors of the state, 4 of the new state, new_lens, workspace,
// err, stream
PyObject* kv_evict(PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 18) return result(kNotTaken);
  Args x(a);
  const at::Tensor &kp = x.dense(0, BF16, 4), &bt = x.dense(2, I32, 2), &mass = x.dense(6, F32, 3);
  if (!x.ok) return result(kNotTaken);
  const int64_t nb = kp.size(0), n_kv = kp.size(1), bs = kp.size(2), d = kp.size(3), B = bt.size(0), mb = bt.size(1), T = mass.size(2);
  const at::Tensor &vp = x.dense(1, BF16, {nb, n_kv, bs, d}), &ctx = x.dense(3, I32, {B}), &keep = x.dense(4, I32, {B}),
                   &new_lens = x.dense(14, I32, {B});
  const State from(x, 6, B, n_kv, T), to(x, 10, B, n_kv, T);
  const int recent = x.integer(5);
  void* ws = nullptr;
  size_t ws_bytes = 0;
  workspace(x, 15, ws, ws_bytes);
  int32_t* err = x.err(16);
  void* stream = x.stream(17);
  x.sizes(nb, n_kv, bs, d, B, mb);
  if (!x.ok) return result(kNotTaken);
  return unlocked([&] {
    return pkv_kv_evict(kp.data_ptr(), vp.data_ptr(), ints(bt), (int)mb, ints(ctx), ints(keep), recent, from.mass, from.positions,
                        from.kept, from.dropped, to.mass, to.positions, to.kept, to.dropped, T, ints(new_lens), (int)B, (int)n_kv,
                        (int)d, (int)bs, (int)nb, ws, ws_bytes, err, stream);
  });
}

// No C++ exception leaves a call: one inside, before the C call, counts as "not taken".
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  PyObject* r = nullptr;
  try {
    r = F(a, n);
  } catch (...) {
    r = result(kNotTaken);
  }
  if (PyErr_Occurred()) PyErr_Clear();                         // a number that is none was not taken
  return r;
}

#define PKV_CALL(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PKV_CALL(rope_append),
                         PKV_CALL(rope_qk),
                         PKV_CALL(kv_quant_append_q8),
                         PKV_CALL(paged_decode_attn_q8),
                         PKV_CALL(paged_decode_attn_mass),
                         PKV_CALL(kv_evict),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
