// Marshalling of the calls that a decode step makes once or more a layer, as a Python module:
// checks of tensor arguments, outputs from PyTorch's allocator, and the call of the C ABI.
//
// The same in Python costs more than these calls' kernels: 1.6 us for an output and 0.3 us for
// the checks of an argument, 14 us for a pool's step of which the launch is 3; here it is 0.7 and
// below 0.1 us.  The functions of libqgemm are given by address (bind), so that this module and
// ctypes call the one library that was loaded.
//
// Nothing is thrown into Python but its own exceptions: ValueError for a wrong tensor, the
// class given to bind for a status of the library, and what PyTorch makes of its own errors.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/as_strided.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "qgemm.h"

namespace {

struct Library {
  decltype(&qgemm_kv_append_norm) append_norm;
  decltype(&qgemm_norm_rotate) norm_rotate;
  decltype(&qgemm_norm_rotate_backward_workspace) norm_rotate_backward_workspace;
  decltype(&qgemm_norm_rotate_backward) norm_rotate_backward;
  decltype(&qgemm_kv_extend_workspace) extend_workspace;
  decltype(&qgemm_kv_extend) extend;
  decltype(&qgemm_attention_window) attention_window;
} lib;
PyObject* status_error = nullptr;  // class of (status, name of the call)

struct Status {  // thrown where the library refuses a call
  qgemm_status status;
  const char* where;
};
struct Raised {};  // a Python exception is set already

void check(qgemm_status s, const char* where) {
  if (s != QGEMM_OK) throw Status{s, where};
}

// the body of a module function: its result, or null with an exception set
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const Status& s) {
    PyObject* e = PyObject_CallFunction(status_error, "is", (int)s.status, s.where);
    if (e) PyErr_SetObject(status_error, e);
    Py_XDECREF(e);
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// ---- arguments

// positional arguments one after the other, for tensors that lie on one device
struct Args {
  PyObject* const* next;
  int64_t device;

  PyObject* object() { return *next++; }
  int64_t integer() {
    const int64_t v = PyLong_AsLongLong(object());
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
  }
  double real() {
    const double v = PyFloat_AsDouble(object());
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
  }
  bool truth() {
    const int v = PyObject_IsTrue(object());
    if (v < 0) throw Raised();
    return v != 0;
  }
  // None where `optional`, else a tensor on the device
  const at::Tensor* tensor(const char* name, bool optional = false) {
    PyObject* o = object();
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + ": a tensor expected");
    return &THPVariable_Unpack(o);
  }
};

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

void on_device(const at::Tensor& t, const char* name, int64_t device) {
  if (t.get_device() != device)
    throw std::invalid_argument(std::string(name) + ": a tensor on device " + std::to_string(device) + " expected, got one on " +
                                t.device().str());
}

// a contiguous tensor of this shape and type on the device; its address (null for null)
void* whole(const at::Tensor* t, const char* name, at::IntArrayRef shape, at::ScalarType type, int64_t device) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->sizes() != shape)
    throw std::invalid_argument(std::string(name) + ": " + c10::toString(type) + " " + shape_of(shape) + " expected, got " +
                                c10::toString(t->scalar_type()) + " " + shape_of(t->sizes()));
  on_device(*t, name, device);
  if (!t->is_contiguous()) throw std::invalid_argument(std::string(name) + ": a contiguous tensor expected");
  return t->data_ptr();
}

// fp16 [T, width] whose rows may be slices of wider ones; the step of a single row says nothing
struct Rows {
  void* at;
  int64_t step;
};
Rows rows(const at::Tensor* t, const char* name, int64_t T, int64_t width, int64_t device) {
  if (t->dim() != 2 || t->scalar_type() != at::kHalf || t->size(0) != T || t->size(1) != width ||
      (t->stride(1) != 1 && width > 1) || (t->stride(0) < width && T > 1))
    throw std::invalid_argument(std::string(name) + ": fp16 " + shape_of({T, width}) + " with contiguous rows expected, got " +
                                c10::toString(t->scalar_type()) + " " + shape_of(t->sizes()));
  on_device(*t, name, device);
  return {t->data_ptr(), T > 1 ? t->stride(0) : width};
}

// a number that the library takes in 32 bits
int32_t narrow(int64_t v, const char* name) {
  if (v != (int32_t)v) throw std::invalid_argument(std::string(name) + ": " + std::to_string(v) + " is too large");
  return (int32_t)v;
}

// the places of a head, by which widths are divided
int64_t head_dim(int64_t D) {
  if (D < 1) throw std::invalid_argument("head_dim: at least 1 expected");
  return D;
}

// address and bytes of a workspace (null for null)
struct Scratch {
  void* at;
  size_t bytes;
};
Scratch scratch(const at::Tensor* t, int64_t device) {
  if (!t) return {nullptr, 0};
  on_device(*t, "ws", device);
  if (!t->is_contiguous()) throw std::invalid_argument("ws: a contiguous tensor expected");
  return {t->data_ptr(), (size_t)t->nbytes()};
}

void two(const at::Tensor* t, const char* name) {
  if (t->dim() != 2) throw std::invalid_argument(std::string(name) + ": two dimensions expected, got " + shape_of(t->sizes()));
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int64_t device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
}

// the argument if there is one (a new reference), else a new tensor
PyObject* result(PyObject* given, at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(std::move(made));
}

// places [from, from + count) of a contiguous tensor.  Results have no history: past the dispatch that
// keeps one the four views of a pool's step take 0.3 us instead of 2 (the call 8.1 -> 5.7 to 6.4 us)
PyObject* part(const at::Tensor& t, int64_t from, int64_t count) {
  at::AutoDispatchBelowADInplaceOrView guard;
  return THPVariable_Wrap(at::as_strided(t, {count}, {1}, t.storage_offset() + from));
}

void device_only(int64_t device) {
  if (device < 0) throw std::invalid_argument("qgemm takes device tensors only");
}

// ---- normed and rotated heads

struct Norm {
  void *q_weight, *k_weight;
  float eps;
  float *cos, *sin;
  int64_t n_positions;
  int32_t rot, interleaved;
  int32_t* positions;
};
// (cos, sin, positions, q_weight, k_weight, eps, interleaved)
Norm norm_args(Args& a, int64_t T, int64_t D) {
  const at::Tensor *cos = a.tensor("cos"), *sin = a.tensor("sin"), *pos = a.tensor("positions");
  const at::Tensor *qw = a.tensor("q_weight", true), *kw = a.tensor("k_weight", true);
  two(cos, "cos");
  Norm n;
  n.eps = (float)a.real();
  n.interleaved = a.truth();
  n.n_positions = cos->size(0);
  const int64_t half = cos->size(1);
  n.rot = narrow(2 * half, "rot_dim");
  n.cos = (float*)whole(cos, "cos", {n.n_positions, half}, at::kFloat, a.device);
  n.sin = (float*)whole(sin, "sin", {n.n_positions, half}, at::kFloat, a.device);
  n.positions = (int32_t*)whole(pos, "positions", {T}, at::kInt, a.device);
  n.q_weight = whole(qw, "q_weight", {D}, at::kHalf, a.device);
  n.k_weight = whole(kw, "k_weight", {D}, at::kHalf, a.device);
  return n;
}

// append_norm(device, stream, cache, kv_heads, head_dim, q, k, v, cos, sin, positions, q_weight, k_weight, eps, interleaved, slots,
// q_out or None) -> q_out
PyObject* append_norm(PyObject*, PyObject* const* args, Py_ssize_t) {
  return guarded([&] {
    Args a{args, -1};
    a.device = a.integer();
    void* stream = (void*)a.integer();
    const qgemm_kv_cache* cache = (const qgemm_kv_cache*)a.integer();
    const int64_t kv_heads = a.integer(), D = head_dim(a.integer());
    const at::Tensor *q = a.tensor("q"), *k = a.tensor("k"), *v = a.tensor("v");
    two(q, "q");
    const int64_t T = q->size(0), heads = q->size(1) / D;
    const Rows rq = rows(q, "q", T, heads * D, a.device), rk = rows(k, "k", T, kv_heads * D, a.device),
               rv = rows(v, "v", T, kv_heads * D, a.device);
    const Norm n = norm_args(a, T, D);
    const int64_t* slots = (const int64_t*)whole(a.tensor("slots"), "slots", {T}, at::kLong, a.device);
    PyObject* given = *a.next;
    const at::Tensor* out = a.tensor("q_out", true);
    device_only(a.device);
    at::Tensor made;
    if (!out) out = &(made = empty({T, heads, D}, at::kHalf, a.device));
    void* to = whole(out, "q_out", {T, heads, D}, at::kHalf, a.device);
    check(lib.append_norm(cache, T, narrow(heads, "q_heads"), rq.at, rq.step, rk.at, rk.step, rv.at, rv.step, n.q_weight, n.k_weight, n.eps,
                          n.cos, n.sin, n.n_positions, n.rot, n.interleaved, n.positions, slots, to, stream),
          "qgemm_kv_append_norm");
    return result(given, made);
  });
}

// norm_rotate(device, stream, head_dim, q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, q_out or None, k_out or None)
// -> (q_out, k_out)
PyObject* norm_rotate(PyObject*, PyObject* const* args, Py_ssize_t) {
  return guarded([&] {
    Args a{args, -1};
    a.device = a.integer();
    void* stream = (void*)a.integer();
    const int64_t D = head_dim(a.integer());
    const at::Tensor *q = a.tensor("q"), *k = a.tensor("k");
    two(q, "q");
    two(k, "k");
    const int64_t T = q->size(0), hq = q->size(1) / D, hk = k->size(1) / D;
    const int32_t nq = narrow(hq, "q_heads"), nk = narrow(hk, "kv_heads");
    const Norm n = norm_args(a, T, D);
    const Rows rq = rows(q, "q", T, hq * D, a.device), rk = rows(k, "k", T, hk * D, a.device);
    PyObject *gq = a.next[0], *gk = a.next[1];
    const at::Tensor *qo = a.tensor("q_out", true), *ko = a.tensor("k_out", true);
    device_only(a.device);
    at::Tensor mq, mk;
    if (!qo) qo = &(mq = empty({T, hq, D}, at::kHalf, a.device));
    if (!ko) ko = &(mk = empty({T, hk, D}, at::kHalf, a.device));
    void *to_q = whole(qo, "q_out", {T, hq, D}, at::kHalf, a.device), *to_k = whole(ko, "k_out", {T, hk, D}, at::kHalf, a.device);
    check(lib.norm_rotate(T, nq, nk, narrow(D, "head_dim"), rq.at, rq.step, rk.at, rk.step, n.q_weight, n.k_weight, n.eps, n.cos,
                          n.sin, n.n_positions, n.rot, n.interleaved, n.positions, to_q, to_k, stream),
          "qgemm_norm_rotate");
    PyObject *a0 = result(gq, mq), *a1 = result(gk, mk);
    return Py_BuildValue("NN", a0, a1);
  });
}

// norm_rotate_backward(device, stream, q, k, dq_out, dk_out, cos, sin, positions, q_weight, k_weight, eps, interleaved, weight_grads,
// dq or None, dk or None, (2, head_dim) weight gradients or None, workspace or None) -> (dq, dk, dq_weight, dk_weight)
PyObject* norm_rotate_backward(PyObject*, PyObject* const* args, Py_ssize_t) {
  return guarded([&] {
    Args a{args, -1};
    a.device = a.integer();
    void* stream = (void*)a.integer();
    const at::Tensor *q = a.tensor("q"), *k = a.tensor("k"), *dqo = a.tensor("dq_out"), *dko = a.tensor("dk_out");
    if (dqo->dim() != 3 || dko->dim() != 3) throw std::invalid_argument("dq_out, dk_out: three dimensions expected");
    const int64_t T = dqo->size(0), hq = dqo->size(1), hk = dko->size(1), D = dqo->size(2);
    const int32_t nq = narrow(hq, "q_heads"), nk = narrow(hk, "kv_heads");
    const Norm n = norm_args(a, T, D);
    const Rows rq = rows(q, "q", T, hq * D, a.device), rk = rows(k, "k", T, hk * D, a.device);
    const void *gq = whole(dqo, "dq_out", {T, hq, D}, at::kHalf, a.device), *gk = whole(dko, "dk_out", {T, hk, D}, at::kHalf, a.device);
    const bool weights = a.truth() && (n.q_weight || n.k_weight);
    PyObject *given_q = a.next[0], *given_k = a.next[1];
    const at::Tensor *dq = a.tensor("dq", true), *dk = a.tensor("dk", true), *dw = a.tensor("weights", true), *ws = a.tensor("ws", true);
    device_only(a.device);
    at::Tensor mq, mk, mw, ms;
    if (!dq) dq = &(mq = empty({T, hq * D}, at::kHalf, a.device));
    if (!dk) dk = &(mk = empty({T, hk * D}, at::kHalf, a.device));
    const Rows to_q = rows(dq, "dq", T, hq * D, a.device), to_k = rows(dk, "dk", T, hk * D, a.device);
    float *wq = nullptr, *wk = nullptr;
    Scratch held{nullptr, 0};
    if (weights) {
      size_t bytes = 0;
      check(lib.norm_rotate_backward_workspace(T, nq, nk, narrow(D, "head_dim"), 1, &bytes), "qgemm_norm_rotate_backward_workspace");
      if (!dw) dw = &(mw = empty({2, D}, at::kFloat, a.device));
      if (!ws) ws = &(ms = empty({(int64_t)bytes}, at::kByte, a.device));
      float* w = (float*)whole(dw, "weights", {2, D}, at::kFloat, a.device);
      wq = n.q_weight ? w : nullptr;
      wk = n.k_weight ? w + D : nullptr;
      held = scratch(ws, a.device);
    }
    check(lib.norm_rotate_backward(T, nq, nk, narrow(D, "head_dim"), rq.at, rq.step, rk.at, rk.step, n.q_weight, n.k_weight, n.eps,
                                   n.cos, n.sin, n.n_positions, n.rot, n.interleaved, n.positions, gq, gk, to_q.at, to_q.step, to_k.at,
                                   to_k.step, wq, wk, held.at, held.bytes, stream),
          "qgemm_norm_rotate_backward");
    auto weight = [&](float* w, int64_t i) {
      if (w) return part(*dw, i * D, D);
      Py_RETURN_NONE;
    };
    PyObject *a0 = result(given_q, mq), *a1 = result(given_k, mk), *a2 = weight(wq, 0), *a3 = weight(wk, 1);
    return Py_BuildValue("NNNN", a0, a1, a2, a3);
  });
}

// ---- block tables

// extend(device, stream, page_size, prefix_len, window, sinks, T, new_tokens, state, ring, tables, state_out or None, workspace or None,
// int32 results or None, slots or None) -> (q_starts, kv_lens, positions, slots, refused)
PyObject* extend(PyObject*, PyObject* const* args, Py_ssize_t) {
  return guarded([&] {
    Args a{args, -1};
    a.device = a.integer();
    void* stream = (void*)a.integer();
    const int32_t page = narrow(a.integer(), "page_size");
    const int64_t prefix = a.integer(), window = a.integer(), sinks = a.integer(), T = a.integer();
    const at::Tensor *news = a.tensor("new_tokens"), *state = a.tensor("state"), *ring = a.tensor("ring"), *tables = a.tensor("tables");
    const at::Tensor *out = a.tensor("state_out", true), *ws = a.tensor("ws", true), *res = a.tensor("results", true);
    PyObject* given = *a.next;
    const at::Tensor* slots = a.tensor("slots", true);
    two(tables, "tables");
    if (T < 0) throw std::invalid_argument("T: at least 0 expected");
    const int64_t B = tables->size(0), width = tables->size(1), R = ring->numel(), n = 2 * B + 2;
    if (!out) out = state;
    int32_t* table = (int32_t*)whole(tables, "tables", {B, width}, at::kInt, a.device);
    const int32_t* asked = (const int32_t*)whole(news, "new_tokens", {B}, at::kInt, a.device);
    const int32_t* before = (const int32_t*)whole(state, "state", {n}, at::kInt, a.device);
    int32_t* after = (int32_t*)whole(out, "state_out", {n}, at::kInt, a.device);
    int32_t* pages = (int32_t*)whole(ring, "ring", {R}, at::kInt, a.device);
    device_only(a.device);
    at::Tensor mr, ms, mw;
    size_t bytes = 0;
    check(lib.extend_workspace(B, T, &bytes), "qgemm_kv_extend_workspace");
    if (bytes && !ws) ws = &(mw = empty({(int64_t)bytes}, at::kByte, a.device));
    const Scratch held = scratch(ws, a.device);
    // one allocation for the three int32 arrays: q_starts, refused, positions
    if (!res) res = &(mr = empty({2 * B + 1 + T}, at::kInt, a.device));
    if (!slots) slots = &(ms = empty({T}, at::kLong, a.device));
    int32_t* to = (int32_t*)whole(res, "results", {2 * B + 1 + T}, at::kInt, a.device);
    int64_t* to_slots = (int64_t*)whole(slots, "slots", {T}, at::kLong, a.device);
    check(lib.extend(B, T, page, asked, before, before + B, before + 2 * B, pages, R, table, width, prefix, window, sinks, to, after,
                     after + B, after + 2 * B, to + 2 * B + 1, to_slots, to + B + 1, held.at, held.bytes, stream),
          "qgemm_kv_extend");
    PyObject *a0 = part(*res, 0, B + 1), *a1 = part(*out, 0, B), *a2 = part(*res, 2 * B + 1, T), *a3 = result(given, ms),
             *a4 = part(*res, B + 1, B);
    return Py_BuildValue("NNNNN", a0, a1, a2, a3, a4);
  });
}

// ---- attention with a window

// attend_window(device, stream, cache, head_dim, q, q_starts, kv_lens, tables, max_q, max_len, prefix_table or None, prefix_len, scale or
// None, window, sinks, out or None, lse or None, workspace or None) -> out
PyObject* attend_window(PyObject*, PyObject* const* args, Py_ssize_t) {
  return guarded([&] {
    Args a{args, -1};
    a.device = a.integer();
    void* stream = (void*)a.integer();
    const qgemm_kv_cache* cache = (const qgemm_kv_cache*)a.integer();
    const int64_t D = a.integer();
    const at::Tensor *q = a.tensor("q"), *starts = a.tensor("q_starts"), *lens = a.tensor("kv_lens"), *tables = a.tensor("tables");
    const int64_t max_q = a.integer(), max_len = a.integer();
    const at::Tensor* prefix = a.tensor("prefix_table", true);
    const int64_t prefix_len = a.integer();
    const double scale = *a.next == Py_None ? (++a.next, 1.0 / std::sqrt((double)D)) : a.real();
    const int64_t window = a.integer(), sinks = a.integer();
    PyObject* given = *a.next;
    const at::Tensor *out = a.tensor("out", true), *lse = a.tensor("lse", true), *ws = a.tensor("ws", true);
    if (q->dim() != 3 || q->size(2) != D || q->scalar_type() != at::kHalf || (q->stride(2) != 1 && D > 1) ||
        (q->stride(1) != D && q->size(1) > 1) || (q->stride(0) < q->size(1) * D && q->size(0) > 1))
      throw std::invalid_argument("q: fp16 [T, q_heads, " + std::to_string(D) + "] with contiguous rows on the device expected, got " +
                                  c10::toString(q->scalar_type()) + " " + shape_of(q->sizes()));
    on_device(*q, "q", a.device);
    const int64_t T = q->size(0), heads = q->size(1), step = T > 1 ? q->stride(0) : heads * D;
    two(tables, "tables");
    const int64_t B = tables->size(0), width = tables->size(1);
    const int32_t* s = (const int32_t*)whole(starts, "q_starts", {B + 1}, at::kInt, a.device);
    const int32_t* l = (const int32_t*)whole(lens, "kv_lens", {B}, at::kInt, a.device);
    const int32_t* t = (const int32_t*)whole(tables, "tables", {B, width}, at::kInt, a.device);
    const int32_t* p = nullptr;
    if (prefix_len) {
      if (!prefix || prefix->numel() * cache->page_size < prefix_len)
        throw std::invalid_argument("prefix_table holds the pages of prefix_len tokens");
      p = (const int32_t*)whole(prefix, "prefix_table", {prefix->numel()}, at::kInt, a.device);
    }
    device_only(a.device);
    at::Tensor made;
    if (!out) out = &(made = empty({T, heads, D}, at::kHalf, a.device));
    void* to = whole(out, "out", {T, heads, D}, at::kHalf, a.device);
    float* sums = (float*)whole(lse, "lse", {T, heads}, at::kFloat, a.device);
    const Scratch held = scratch(ws, a.device);
    check(lib.attention_window(cache, T, narrow(heads, "q_heads"), q->data_ptr(), step, B, s, l, t, width, p, prefix_len, max_q, max_len, window, sinks,
                               (float)scale, to, sums, held.at, held.bytes, stream),
          "qgemm_attention_window");
    return result(given, made);
  });
}

// bind({name: address} of libqgemm's functions, class of its errors)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    auto take = [&](auto& to, const char* name) {
      PyObject* v = PyDict_GetItemString(args[0], name);
      void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
      if (!p) throw std::invalid_argument(std::string(name) + ": an address expected");
      to = reinterpret_cast<std::remove_reference_t<decltype(to)>>(p);
    };
    take(lib.append_norm, "qgemm_kv_append_norm");
    take(lib.norm_rotate, "qgemm_norm_rotate");
    take(lib.norm_rotate_backward_workspace, "qgemm_norm_rotate_backward_workspace");
    take(lib.norm_rotate_backward, "qgemm_norm_rotate_backward");
    take(lib.extend_workspace, "qgemm_kv_extend_workspace");
    take(lib.extend, "qgemm_kv_extend");
    take(lib.attention_window, "qgemm_attention_window");
    Py_INCREF(args[1]);
    Py_XDECREF(status_error);
    status_error = args[1];
    Py_RETURN_NONE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  if (F != bind && !status_error) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  return F(self, args, n);
}
#define ENTRY(f, n) {#f, (PyCFunction)(void (*)(void))counted<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind, 2), ENTRY(append_norm, 17), ENTRY(norm_rotate, 14), ENTRY(norm_rotate_backward, 18), ENTRY(extend, 15),
                         ENTRY(attend_window, 18), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
