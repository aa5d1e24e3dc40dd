// Python binding of the operators around the window attention, over torch tensors: argument checks
// and marshalling only, as the ctypes binding does for the rest of the library.
//
// Why these in C++: the kernels of a small call (one window's rotation: 3 us, a verification: 8 us)
// take less time than checking and converting a dozen tensors from Python (10 to 15 us). Here a
// call costs about what its launches cost.
//
// Every function takes positional arguments, None for what is left out, the addresses of the
// configuration and the plan, and last the stream (None: the current one, or its handle). It
// returns the library's status, raises TypeError for a wrong type and ValueError for a wrong shape,
// layout or device.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>

#include "la_pbd.h"

namespace {

struct WrongType : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct WrongValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};

template <typename E, typename... A>
[[noreturn]] void fail(const A&... a) {
  std::ostringstream o;
  (o << ... << a);
  throw E(o.str());
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bf16";
    case at::kHalf: return "fp16";
    case at::kFloat: return "fp32";
    case at::kInt: return "i32";
    default: return c10::toString(t);
  }
}

// The arguments of one call, in order.
class Args {
 public:
  Args(PyObject* const* v, Py_ssize_t n, Py_ssize_t want, const char* where) : v_(v) {
    if (n != want) fail<WrongType>(where, ": expected ", want, " arguments, got ", n);
  }
  const at::Tensor* maybe(int i, const char* name) const {
    if (v_[i] == Py_None) return nullptr;
    if (!THPVariable_Check(v_[i])) fail<WrongType>(name, ": expected a tensor, got ", Py_TYPE(v_[i])->tp_name);
    return &THPVariable_Unpack(v_[i]);
  }
  const at::Tensor& tensor(int i, const char* name) const {
    const at::Tensor* t = maybe(i, name);
    if (!t) fail<WrongType>(name, ": expected a tensor, got None");
    return *t;
  }
  long long integer(int i) const {
    const long long x = PyLong_AsLongLong(v_[i]);
    if (x == -1 && PyErr_Occurred()) throw 0;   // (Python's own error stands)
    return x;
  }
  int32_t int32(int i, const char* name) const {
    const long long x = integer(i);
    if (x != (int32_t)x) fail<WrongValue>(name, ": ", x, " does not fit 32 bits");
    return (int32_t)x;
  }
  float number(int i) const {
    const double x = PyFloat_AsDouble(v_[i]);
    if (x == -1.0 && PyErr_Occurred()) throw 0;
    return (float)x;
  }
  template <typename T> const T* address(int i) const {
    return reinterpret_cast<const T*>(static_cast<intptr_t>(integer(i)));
  }
  // The stream to use: tensors must be on the current device.
  void* stream(int i) const {
    if (v_[i] != Py_None) return reinterpret_cast<void*>(static_cast<intptr_t>(integer(i)));
    return c10::cuda::getCurrentCUDAStream().stream();
  }

 private:
  PyObject* const* v_;
};

void on_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) fail<WrongValue>(name, ": must be a CUDA tensor");
  const int dev = c10::cuda::current_device();
  if (t.get_device() != dev)
    fail<WrongValue>(name, ": must be on the current device (cuda:", dev, "), is on ", t.device().str());
}
void of_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type) fail<WrongType>(name, ": expected ", type_name(type), ", got ", type_name(t.scalar_type()));
}
void of_shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape) {
  if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
    fail<WrongValue>(name, ": expected shape ", at::IntArrayRef(shape.begin(), shape.size()), ", got ", t.sizes());
}
// A dense tensor of a type and shape on the current device: its address.
void* dense(const at::Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
  of_type(t, name, type);
  on_device(t, name);
  if (!t.is_contiguous()) fail<WrongValue>(name, ": must be contiguous");
  of_shape(t, name, shape);
  return t.data_ptr();
}
template <typename T>
T* dense_maybe(const at::Tensor* t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
  return t ? static_cast<T*>(dense(*t, name, type, shape)) : nullptr;
}
int32_t dtype_number(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return LA_DTYPE_BF16;
    case at::kHalf: return LA_DTYPE_F16;
    case at::kFloat: return LA_DTYPE_F32;
    default: fail<WrongType>(name, ": expected bf16, fp16 or fp32, got ", type_name(t.scalar_type()));
  }
}

// K and V caches, contiguous or (with a block table) page pools; `slots` = key slots of a sequence.
struct Caches {
  void *k, *v;
  const int32_t* table = nullptr;
  int32_t pages_per_seq = 0, page_size = 0, num_pages = 0;
  int64_t slots;
};
Caches caches(const la_pbd_cfg& c, const at::Tensor& k, const at::Tensor& v, const at::Tensor* table) {
  Caches r;
  if (!table) {
    r.slots = c.max_seq;
    r.k = dense(k, "k_cache", at::kBFloat16, {c.batch, c.num_kv_heads, c.max_seq, c.head_dim});
    r.v = dense(v, "v_cache", at::kBFloat16, {c.batch, c.num_kv_heads, c.max_seq, c.head_dim});
    return r;
  }
  of_type(*table, "block_table", at::kInt);
  if (k.dim() != 4 || table->dim() != 2)
    fail<WrongValue>("k_pool: expected [num_pages, ", c.num_kv_heads, ", page_size, ", c.head_dim,
                     "], block_table: [", c.batch, ", pages_per_seq], got ", k.sizes(), " and ", table->sizes());
  r.num_pages = (int32_t)k.size(0);
  r.page_size = (int32_t)k.size(2);
  r.pages_per_seq = (int32_t)table->size(1);
  r.slots = (int64_t)r.pages_per_seq * r.page_size;
  r.k = dense(k, "k_pool", at::kBFloat16, {k.size(0), c.num_kv_heads, k.size(2), c.head_dim});
  r.v = dense(v, "v_pool", at::kBFloat16, {k.size(0), c.num_kv_heads, k.size(2), c.head_dim});
  r.table = static_cast<const int32_t*>(dense(*table, "block_table", at::kInt, {c.batch, table->size(1)}));
  return r;
}

// Elements between consecutive rows of a [B, T, H, D] tensor whose heads are dense and whose batch is
// evenly strided (a part of a fused projection's output, or contiguous).
int64_t token_stride(const at::Tensor& t, const char* name, int64_t B, int64_t T, int64_t H, int64_t D) {
  of_type(t, name, at::kBFloat16);
  on_device(t, name);
  of_shape(t, name, {B, T, H, D});
  const int64_t tok = T > 1 ? t.stride(1) : B > 1 ? t.stride(0) : H * D;
  if (t.stride(3) != 1 || (H > 1 && t.stride(2) != D) || (B > 1 && t.stride(0) != T * tok))
    fail<WrongValue>(name, ": heads must be dense and rows evenly strided, got strides ", t.strides());
  return tok;
}

// ---- rope(plan, x, positions, out, inverse, stream)
la_status rope(PyObject* const* v, Py_ssize_t n) {
  const Args a(v, n, 6, "la_rope");
  const at::Tensor &x = a.tensor(1, "x"), &pos = a.tensor(2, "positions"), &out = a.tensor(3, "out");
  const int32_t type = dtype_number(x, "x");
  on_device(x, "x");
  of_type(out, "out", x.scalar_type());
  on_device(out, "out");
  if (x.dim() != 3) fail<WrongValue>("x: expected [T, H, D], got ", x.sizes());
  of_shape(out, "out", {x.size(0), x.size(1), x.size(2)});
  if (x.size(2) > 1 && (x.stride(2) != 1 || out.stride(2) != 1))
    fail<WrongValue>("x, out: channels must be contiguous");
  const void* p = dense(pos, "positions", at::kInt, {x.size(0)});
  if (x.size(1) > INT32_MAX || x.size(2) > INT32_MAX) fail<WrongValue>("x: too large, ", x.sizes());
  return la_rope(a.address<la_rope_plan>(0), type, x.data_ptr(), x.stride(0), x.stride(1),
                 static_cast<const int32_t*>(p), x.size(0), (int32_t)x.size(1), (int32_t)x.size(2),
                 (int32_t)a.integer(4), out.data_ptr(), out.stride(0), out.stride(1), a.stream(5));
}

// ---- rope_append(cfg, plan, q, k_new, v_new, block_table, seq_lens, q_out, k, v, row_lens, pos0,
//                  key_pos, stream)
la_status rope_append(PyObject* const* v, Py_ssize_t n) {
  const Args a(v, n, 14, "la_rope_append");
  const la_pbd_cfg& c = *a.address<la_pbd_cfg>(0);
  const at::Tensor &q = a.tensor(2, "q"), &kn = a.tensor(3, "k_new"), &vn = a.tensor(4, "v_new");
  if (q.dim() != 4) fail<WrongValue>("q: expected [B, T, Hq, D], got ", q.sizes());
  const int64_t B = c.batch, T = q.size(1), D = c.head_dim;
  if (T > INT32_MAX) fail<WrongValue>("q: too many rows, ", T);
  const int64_t sq = token_stride(q, "q", B, T, c.num_q_heads, D);
  const int64_t sk = token_stride(kn, "k_new", B, T, c.num_kv_heads, D);
  const int64_t sv = token_stride(vn, "v_new", B, T, c.num_kv_heads, D);
  void* q_out = dense(a.tensor(7, "q_out"), "q_out", at::kBFloat16, {B, T, c.num_q_heads, D});
  const Caches kv = caches(c, a.tensor(8, "k_cache"), a.tensor(9, "v_cache"), a.maybe(5, "block_table"));
  const int32_t* lens = dense_maybe<int32_t>(a.maybe(6, "seq_lens"), "seq_lens", at::kInt, {B});
  const int32_t* rows = dense_maybe<int32_t>(a.maybe(10, "row_lens"), "row_lens", at::kInt, {B});
  const int32_t* pos0 = dense_maybe<int32_t>(a.maybe(11, "pos0"), "pos0", at::kInt, {B});
  int32_t* key_pos = dense_maybe<int32_t>(a.maybe(12, "key_pos"), "key_pos", at::kInt, {B, c.num_kv_heads, kv.slots});
  const la_rope_plan* plan = a.address<la_rope_plan>(1);
  void* stream = a.stream(13);
  if (kv.table)
    return la_rope_append_paged(&c, plan, q.data_ptr(), sq, kn.data_ptr(), sk, vn.data_ptr(), sv, kv.table,
                                kv.pages_per_seq, kv.page_size, kv.num_pages, lens, rows, pos0, (int32_t)T, q_out,
                                kv.k, kv.v, key_pos, stream);
  return la_rope_append(&c, plan, q.data_ptr(), sq, kn.data_ptr(), sk, vn.data_ptr(), sv, lens, rows, pos0,
                        (int32_t)T, q_out, kv.k, kv.v, key_pos, stream);
}

// ---- attn_weights(cfg, q, k, v, block_table, seq_lens, window_len, out, weights_out, workspace,
//                   weights_in, decay, window_lens, stream)
la_status attn_weights(PyObject* const* v, Py_ssize_t n) {
  const Args a(v, n, 14, "la_pbd_attn_weights");
  const la_pbd_cfg& c = *a.address<la_pbd_cfg>(0);
  const int64_t B = c.batch, D = c.head_dim;
  const int32_t W = a.int32(6, "window_len");
  const void* q = dense(a.tensor(1, "q"), "q", at::kBFloat16, {B, W, c.num_q_heads, D});
  const Caches kv = caches(c, a.tensor(2, "k_cache"), a.tensor(3, "v_cache"), a.maybe(4, "block_table"));
  const int32_t* lens = static_cast<int32_t*>(dense(a.tensor(5, "seq_lens"), "seq_lens", at::kInt, {B}));
  void* out = dense(a.tensor(7, "out"), "out", at::kBFloat16, {B, W, c.num_q_heads, D});
  float* w_out = static_cast<float*>(
      dense(a.tensor(8, "weights_out"), "weights_out", at::kFloat, {B, c.num_kv_heads, kv.slots}));
  const at::Tensor& ws = a.tensor(9, "workspace");
  on_device(ws, "workspace");
  const float* w_in =
      dense_maybe<float>(a.maybe(10, "weights_in"), "weights_in", at::kFloat, {B, c.num_kv_heads, kv.slots});
  const float decay = a.number(11);
  const int32_t* wl = dense_maybe<int32_t>(a.maybe(12, "window_lens"), "window_lens", at::kInt, {B});
  void* stream = a.stream(13);
  if (kv.table)
    return la_pbd_attn_weights_paged(&c, q, kv.k, kv.v, kv.table, kv.pages_per_seq, kv.page_size, kv.num_pages,
                                     lens, wl, W, out, w_in, decay, w_out, ws.data_ptr(), ws.nbytes(), stream);
  return la_pbd_attn_weights(&c, q, kv.k, kv.v, lens, wl, W, out, w_in, decay, w_out, ws.data_ptr(), ws.nbytes(),
                             stream);
}

// ---- kv_evict(cfg, weights, block_table, seq_lens, budget, k, v, weights_out, new_lens, workspace,
//               key_pos, next_pos, sink, recent, key_pos_out, kept_slots, stream)
la_status kv_evict(PyObject* const* v, Py_ssize_t n) {
  const Args a(v, n, 17, "la_kv_evict");
  const la_pbd_cfg& c = *a.address<la_pbd_cfg>(0);
  const int64_t B = c.batch, H = c.num_kv_heads;
  const int32_t budget = a.int32(4, "budget"), sink = a.int32(12, "sink"), recent = a.int32(13, "recent");
  const Caches kv = caches(c, a.tensor(5, "k_cache"), a.tensor(6, "v_cache"), a.maybe(2, "block_table"));
  const float* w = static_cast<float*>(dense(a.tensor(1, "weights"), "weights", at::kFloat, {B, H, kv.slots}));
  const int32_t* lens = static_cast<int32_t*>(dense(a.tensor(3, "seq_lens"), "seq_lens", at::kInt, {B}));
  float* w_out = static_cast<float*>(dense(a.tensor(7, "weights_out"), "weights_out", at::kFloat, {B, H, kv.slots}));
  int32_t* new_lens = static_cast<int32_t*>(dense(a.tensor(8, "new_lens"), "new_lens", at::kInt, {B}));
  const at::Tensor& ws = a.tensor(9, "workspace");
  on_device(ws, "workspace");
  const int32_t* pos = dense_maybe<int32_t>(a.maybe(10, "key_pos"), "key_pos", at::kInt, {B, H, kv.slots});
  const int32_t* next = dense_maybe<int32_t>(a.maybe(11, "next_pos"), "next_pos", at::kInt, {B});
  int32_t* pos_out = dense_maybe<int32_t>(a.maybe(14, "key_pos_out"), "key_pos_out", at::kInt, {B, H, kv.slots});
  int32_t* kept = dense_maybe<int32_t>(a.maybe(15, "kept_slots"), "kept_slots", at::kInt, {B, H, budget});
  void* stream = a.stream(16);
  if (kv.table)
    return la_kv_evict_paged(&c, w, pos, kv.table, kv.pages_per_seq, kv.page_size, kv.num_pages, lens, next, budget,
                             sink, recent, kv.k, kv.v, w_out, pos_out, kept, new_lens, ws.data_ptr(), ws.nbytes(),
                             stream);
  return la_kv_evict(&c, w, pos, lens, next, budget, sink, recent, kv.k, kv.v, w_out, pos_out, kept, new_lens,
                     ws.data_ptr(), ws.nbytes(), stream);
}

// ---- verify(p, q, drafts, u, sample_u, tokens, accepted, draft_lens, seq_lens, seq_lens_out, stream)
la_status verify(PyObject* const* v, Py_ssize_t n) {
  const Args a(v, n, 11, "la_pbd_verify");
  const at::Tensor& p = a.tensor(0, "p");
  const int32_t type = dtype_number(p, "p");
  on_device(p, "p");
  if (p.dim() != 3 || p.size(1) < 1 || (p.size(2) > 1 && p.stride(2) != 1))
    fail<WrongValue>("p: expected [B, K + 1, V] with contiguous entries, got ", p.sizes(), " strides ", p.strides());
  const int64_t B = p.size(0), K = p.size(1) - 1, V = p.size(2);
  if (B > INT32_MAX || K > INT32_MAX || V > INT32_MAX) fail<WrongValue>("p: too large, ", p.sizes());
  const at::Tensor* q = a.maybe(1, "q");
  if (q) {
    of_type(*q, "q", p.scalar_type());
    on_device(*q, "q");
    of_shape(*q, "q", {B, K, V});
    if (V > 1 && q->stride(2) != 1) fail<WrongValue>("q: entries must be contiguous, got strides ", q->strides());
  }
  const void* x = dense(a.tensor(2, "drafts"), "drafts", at::kInt, {B, K});
  const void* u = dense(a.tensor(3, "u"), "u", at::kFloat, {B, K});
  const void* su = dense(a.tensor(4, "sample_u"), "sample_u", at::kFloat, {B});
  void* tokens = dense(a.tensor(5, "tokens"), "tokens", at::kInt, {B, K + 1});
  void* accepted = dense(a.tensor(6, "accepted"), "accepted", at::kInt, {B});
  const int32_t* dl = dense_maybe<int32_t>(a.maybe(7, "draft_lens"), "draft_lens", at::kInt, {B});
  const int32_t* sl = dense_maybe<int32_t>(a.maybe(8, "seq_lens"), "seq_lens", at::kInt, {B});
  int32_t* slo = dense_maybe<int32_t>(a.maybe(9, "seq_lens_out"), "seq_lens_out", at::kInt, {B});
  return la_pbd_verify(type, p.data_ptr(), p.stride(0), p.stride(1), q ? q->data_ptr() : nullptr,
                       q ? q->stride(0) : 0, q ? q->stride(1) : 0, static_cast<const int32_t*>(x), dl,
                       static_cast<const float*>(u), static_cast<const float*>(su), (int32_t)B, (int32_t)K, (int32_t)V,
                       static_cast<int32_t*>(tokens), static_cast<int32_t*>(accepted), sl, slo, a.stream(10));
}

// Python's errors for the exceptions above: none of them leaves the module.
template <la_status (*F)(PyObject* const*, Py_ssize_t)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return PyLong_FromLong((long)F(args, n));
  } catch (const WrongType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const WrongValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <la_status (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(call<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<rope>("rope"),         method<rope_append>("rope_append"), method<attn_weights>("attn_weights"),
    method<kv_evict>("kv_evict"), method<verify>("verify"),           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_la_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__la_torch() { return PyModule_Create(&g_module); }
