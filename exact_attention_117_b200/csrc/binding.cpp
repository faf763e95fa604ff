// binding.cpp -- the part of the Python binding that a serving step calls many
// times a layer: argument checks, output allocation and the call of the C ABI
// for the rotary and 4-bit cache entry points, without ctypes (a call of ten
// tensors costs about 20 us through ctypes and torch's Python surface, a few
// here, against 3 to 10 us on the GPU for a decode step's kernels).
//
// No computation happens here: the functions check tensor properties, take
// device pointers and the current stream, and return the C status in front of
// their outputs.  The C functions are the ones of the library that fa.py has
// loaded; bind() receives their addresses.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/fa.h"

namespace {

struct Api {
  decltype(&fa_rotary) rotary;
  decltype(&fa_kv4_plan) plan;
  decltype(&fa_kv4_append) append;
  decltype(&fa_kv4_gather) gather;
  decltype(&fa_kv4_attention_workspace_size) workspace_size;
  decltype(&fa_kv4_attention) attention;
} g_api = {};

// A refused argument: Python's ValueError.
struct Refused : std::invalid_argument {
  using std::invalid_argument::invalid_argument;
};
void require(bool ok, const char* what) {
  if (!ok) throw Refused(what);
}

using Tensor = at::Tensor;

const Tensor& tensor(PyObject* o, const char* what) {
  require(THPVariable_Check(o), what);
  return THPVariable_Unpack(o);
}
std::optional<Tensor> maybe(PyObject* o, const char* what) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, what);
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int narrow(long long v) {
  require(v >= INT32_MIN && v <= INT32_MAX, "an integer does not fit 32 bits");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// The current device, on which every tensor of a call lies; asked for with the
// first tensor that is on a CUDA device at all.
struct Here {
  mutable c10::DeviceIndex index = -1;
  void check(const Tensor& t) const {
    const bool ok = t.is_cuda();
    if (ok && index < 0) index = c10::cuda::current_device();
    require(ok && t.get_device() == index, "tensors must be on the current CUDA device");
  }
  at::Device device() const { return at::Device(at::kCUDA, index); }
  // None: the current stream.  `made`: what this call allocated, on the current
  // stream; on another one it must not be handed out again before the call's
  // work there is done.
  void* stream(PyObject* o, std::initializer_list<const Tensor*> made = {}) const {
    const auto current = c10::cuda::getCurrentCUDAStream(index);
    if (o == Py_None) return current.stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw python_error();
    if (p != static_cast<void*>(current.stream())) {
      const auto other = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), index);
      for (const Tensor* t : made)
        if (t && t->numel() > 0)
          c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), other);
    }
    return p;
  }
};

Tensor empty(const Here& here, at::IntArrayRef size, at::ScalarType type) {
  return at::detail::empty_cuda(size, type, here.device(), std::nullopt);
}
// Dense, its axes in memory in the order of t's.
Tensor empty_like_dense(const Here& here, const Tensor& t) {
  const int n = static_cast<int>(t.dim());
  int order[8];
  for (int i = 0; i < n; ++i) order[i] = i;
  std::stable_sort(order, order + n, [&](int a, int b) { return t.stride(a) < t.stride(b); });
  // the contiguous last axis innermost, also where an axis of length 1 ties
  std::stable_partition(order, order + n, [&](int a) { return a == n - 1; });
  int64_t strides[8], step = 1;
  for (int i = 0; i < n; ++i) {
    strides[order[i]] = step;
    step *= std::max<int64_t>(t.size(order[i]), 1);
  }
  return at::detail::empty_strided_cuda(t.sizes(), at::IntArrayRef(strides, n), t.scalar_type(),
                                        here.device());
}

// Vectors of int32 and int64 that share one allocation, each 16-byte aligned (an
// allocation of its own costs a vector of a few numbers as much time as a launch).
struct Carved {
  Tensor base;
  int64_t used = 0;  // bytes
  static int64_t padded(int64_t bytes) { return (bytes + 15) / 16 * 16; }
  Carved(const Here& here, int64_t bytes) : base(empty(here, {bytes}, at::kByte)) {}
  Tensor take(int64_t n, at::ScalarType type) {
    const int64_t size = type == at::kLong ? 8 : 4;
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(base.storage()), base.key_set(), c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl* impl = t.unsafeGetTensorImpl();
    impl->set_storage_offset(used / size);
    impl->set_sizes_contiguous({n});
    used += padded(n * size);
    return t;
  }
};

// The stride of an axis; one of length 1 has none that matters.
long long step(const Tensor& t, int axis) { return t.size(axis) > 1 ? t.stride(axis) : 0; }

bool overlaps_itself(const Tensor& t, int axes) {
  for (int i = 0; i < axes; ++i)
    if (t.stride(i) == 0 && t.size(i) > 1) return true;
  return false;
}
int type_code(at::ScalarType t) {
  return t == at::kBFloat16 ? FA_BF16 : t == at::kHalf ? FA_FP16 : t == at::kFloat ? FA_FP32 : -1;
}
void vector_of(const Tensor& t, at::ScalarType type, int64_t n, const char* what) {
  require(t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && (n < 2 || t.stride(0) == 1),
          what);
}
// A zero-size last axis aside, its stride is 1.
bool unit(const Tensor& t) { return t.stride(t.dim() - 1) == 1; }

void put(PyObject* tuple, int i, PyObject* item) {
  if (!item) throw python_error();
  PyTuple_SET_ITEM(tuple, i, item);
}
struct Tuple {
  PyObject* p;
  explicit Tuple(int n, int status) : p(PyTuple_New(n)) {
    if (!p) throw python_error();
    put(p, 0, PyLong_FromLong(status));
  }
  ~Tuple() { Py_XDECREF(p); }
  void set(int i, Tensor t) { put(p, i, THPVariable_Wrap(std::move(t))); }
  PyObject* release() {
    PyObject* r = p;
    p = nullptr;
    return r;
  }
};

struct Cache {
  int pages, heads, page_size;
  Cache(const Tensor& c, int64_t d) {
    require(c.scalar_type() == at::kByte && c.dim() == 4 && c.is_contiguous() && c.size(3) == 18 * d,
            "the cache must be contiguous uint8 [pages, kv_heads, page / 16, 18 d]");
    pages = narrow(c.size(0));
    heads = narrow(c.size(1));
    page_size = narrow(c.size(2) * 16);
  }
};

using Args = PyObject* const*;
void count(Py_ssize_t n, Py_ssize_t want) { require(n == want, "wrong number of arguments"); }

// (q, k, positions, inv_freq, interleaved, amplitude, out_q, out_k, stream, inverse)
PyObject* rotary(Args a, Py_ssize_t n) {
  count(n, 10);
  const Here here;
  const Tensor& q = tensor(a[0], "q must be a tensor");
  const auto k = maybe(a[1], "k must be a tensor or None");
  const Tensor& pos = tensor(a[2], "positions must be a tensor");
  const Tensor& freq = tensor(a[3], "inv_freq must be a tensor");
  auto oq = maybe(a[6], "out_q must be a tensor or None"), ok = maybe(a[7], "out_k must be a tensor or None");
  require(q.dim() == 4 && unit(q) && type_code(q.scalar_type()) >= 0,
          "expected bf16, fp16 or fp32 [B, H, N, d] tensors, d contiguous");
  const int64_t B = q.size(0), N = q.size(2), d = q.size(3);
  require(k || !ok, "an output for k without k");
  if (k)
    require(k->dim() == 4 && k->scalar_type() == q.scalar_type() && k->size(0) == B &&
                k->size(2) == N && k->size(3) == d && unit(*k),
            "k must match q's [B, ., N, d], dtype and layout");
  require((pos.scalar_type() == at::kInt || pos.scalar_type() == at::kLong) &&
              ((pos.dim() == 1 && pos.size(0) == N) ||
               (pos.dim() == 2 && pos.size(0) == B && pos.size(1) == N)) &&
              (N < 2 || unit(pos)),
          "positions must be int32 or int64 [N] or [B, N], N contiguous");
  require(freq.scalar_type() == at::kDouble && freq.dim() == 1 && (freq.size(0) < 2 || unit(freq)),
          "inv_freq must be a contiguous fp64 vector");
  for (const Tensor* t : {&q, &pos, &freq}) here.check(*t);
  if (k) here.check(*k);
  const bool made_q = !oq, made_k = k && !ok;
  if (made_q) oq = empty_like_dense(here, q);
  if (made_k) ok = empty_like_dense(here, *k);
  auto output = [&](const Tensor& o, const Tensor& x) {
    here.check(o);
    require(o.sizes() == x.sizes() && o.scalar_type() == x.scalar_type() && unit(o),
            "an output must have its input's shape, dtype and a contiguous d");
    require(!overlaps_itself(o, 3), "outputs must not overlap themselves");
  };
  output(*oq, q);
  if (k) output(*ok, *k);
  long long strides[12] = {};
  for (int i = 0; i < 3; ++i) {
    strides[i] = step(q, i);
    strides[3 + i] = step(*oq, i);
    if (k) {
      strides[6 + i] = step(*k, i);
      strides[9 + i] = step(*ok, i);
    }
  }
  const int st = g_api.rotary(
      q.data_ptr(), k ? k->data_ptr() : nullptr, oq->data_ptr(), k ? ok->data_ptr() : nullptr,
      narrow(B), narrow(q.size(1)), k ? narrow(k->size(1)) : 0, narrow(N), narrow(d), strides,
      pos.data_ptr(), pos.scalar_type() == at::kLong, pos.dim() == 2 ? pos.stride(0) : 0,
      static_cast<const double*>(freq.data_ptr()), narrow(2 * freq.size(0)), truth(a[4]),
      static_cast<float>(number(a[5])), truth(a[9]), type_code(q.scalar_type()),
      here.stream(a[8], {made_q ? &*oq : nullptr, made_k ? &*ok : nullptr}));
  Tuple r(3, st);
  r.set(1, *oq);
  if (k) {
    r.set(2, *ok);
  } else {
    Py_INCREF(Py_None);
    put(r.p, 2, Py_None);
  }
  return r.release();
}

// (lengths, new_lengths, block_table, free_pages, free_range, page_size, max_tokens,
//  lengths_out, free_range_out, stream)
PyObject* plan(Args a, Py_ssize_t n) {
  count(n, 10);
  const Here here;
  const Tensor& len = tensor(a[0], "lengths must be a tensor");
  const Tensor& want = tensor(a[1], "new_lengths must be a tensor");
  const Tensor& table = tensor(a[2], "block_table must be a tensor");
  const Tensor& ring = tensor(a[3], "free_pages must be a tensor");
  const Tensor& range = tensor(a[4], "free_range must be a tensor");
  const int page_size = narrow(integer(a[5])), most = narrow(integer(a[6]));
  auto len_out = maybe(a[7], "lengths_out must be a tensor or None");
  auto range_out = maybe(a[8], "free_range_out must be a tensor or None");
  const int64_t R = len.dim() == 1 ? len.size(0) : -1;
  require(R >= 0, "lengths must be int32 [requests]");
  vector_of(len, at::kInt, R, "lengths must be contiguous int32 [requests]");
  vector_of(want, at::kInt, R, "new_lengths must be contiguous int32 [requests]");
  require(table.scalar_type() == at::kInt && table.dim() == 2 && table.size(0) == R &&
              (unit(table) || table.size(1) < 2) && (R < 2 || table.stride(0) >= table.size(1)),
          "block_table must be int32 [requests, width] with contiguous rows");
  require(ring.dim() == 1, "free_pages must be contiguous int32 [pages]");
  vector_of(ring, at::kInt, ring.size(0), "free_pages must be contiguous int32 [pages]");
  vector_of(range, at::kLong, 2, "free_range must be contiguous int64 [2]");
  require(most >= 0, "max_tokens must not be negative");
  for (const Tensor* t : {&len, &want, &table, &ring, &range}) here.check(*t);
  auto pad = [](int64_t bytes) { return Carved::padded(bytes); };
  Carved from(here, pad(4 * R) + pad(16) + pad(4 * (R + 1)) + pad(8LL * most) + pad(4LL * most) + pad(4));
  if (!len_out) len_out = from.take(R, at::kInt);
  if (!range_out) range_out = from.take(2, at::kLong);
  vector_of(*len_out, at::kInt, R, "lengths_out must be contiguous int32 [requests]");
  vector_of(*range_out, at::kLong, 2, "free_range_out must be contiguous int64 [2]");
  here.check(*len_out);
  here.check(*range_out);
  Tensor cu = from.take(R + 1, at::kInt), slots = from.take(most, at::kLong),
         positions = from.take(most, at::kInt), status = from.take(1, at::kInt);
  auto ints = [](const Tensor& t) { return static_cast<int*>(t.data_ptr()); };
  auto longs = [](const Tensor& t) { return static_cast<long long*>(t.data_ptr()); };
  const int st = g_api.plan(ints(len), ints(want), ints(table),
                            R < 2 ? std::max(table.stride(0), table.size(1)) : table.stride(0),
                            narrow(table.size(1)), ints(ring), narrow(ring.size(0)), longs(range),
                            narrow(R), page_size, most, ints(*len_out), longs(*range_out),
                            ints(cu), longs(slots), ints(positions), ints(status),
                            here.stream(a[9], {&from.base}));
  Tuple r(7, st);
  r.set(1, *len_out);
  r.set(2, std::move(cu));
  r.set(3, std::move(slots));
  r.set(4, std::move(positions));
  r.set(5, std::move(status));
  r.set(6, *range_out);
  return r.release();
}

void check_rows(const Here& here, const Tensor& k, const Tensor& v, const Tensor& slots) {
  require(k.dim() == 3 && k.scalar_type() == at::kBFloat16 && v.scalar_type() == at::kBFloat16 &&
              v.sizes() == k.sizes() && unit(k) && unit(v),
          "keys and values must be bf16 [tokens, kv_heads, d], d contiguous");
  vector_of(slots, at::kLong, k.size(0), "slots must be contiguous int64 [tokens]");
  for (const Tensor* t : {&k, &v, &slots}) here.check(*t);
}

// (k, v, cache, slots, stream)
PyObject* append(Args a, Py_ssize_t n) {
  count(n, 5);
  const Here here;
  const Tensor &k = tensor(a[0], "k must be a tensor"), &v = tensor(a[1], "v must be a tensor");
  const Tensor &cache = tensor(a[2], "cache must be a tensor"), &slots = tensor(a[3], "slots must be a tensor");
  check_rows(here, k, v, slots);
  const Cache c(cache, k.size(2));
  require(c.heads == k.size(1), "keys and the cache differ in kv_heads");
  here.check(cache);
  const long long strides[4] = {step(k, 0), step(k, 1), step(v, 0), step(v, 1)};
  return PyLong_FromLong(g_api.append(k.data_ptr(), v.data_ptr(), cache.data_ptr(),
                                      static_cast<const long long*>(slots.data_ptr()), k.size(0),
                                      c.heads, narrow(k.size(2)), c.pages, c.page_size, strides,
                                      here.stream(a[4])));
}

// (cache, slots, out_k, out_v, stream)
PyObject* gather(Args a, Py_ssize_t n) {
  count(n, 5);
  const Here here;
  const Tensor &cache = tensor(a[0], "cache must be a tensor"), &slots = tensor(a[1], "slots must be a tensor");
  auto k = maybe(a[2], "out_k must be a tensor or None"), v = maybe(a[3], "out_v must be a tensor or None");
  require(cache.dim() == 4 && cache.size(3) % 18 == 0,
          "the cache must be contiguous uint8 [pages, kv_heads, page / 16, 18 d]");
  const int64_t d = cache.size(3) / 18;
  const Cache c(cache, d);
  require(slots.dim() == 1, "slots must be contiguous int64 [tokens]");
  here.check(cache);
  here.check(slots);
  const int64_t T = slots.size(0);
  const bool made_k = !k, made_v = !v;
  if (made_k) k = empty(here, {T, c.heads, d}, at::kBFloat16);
  if (made_v) v = empty(here, {T, c.heads, d}, at::kBFloat16);
  check_rows(here, *k, *v, slots);
  require(k->size(1) == c.heads && k->size(2) == d, "outputs must be bf16 [tokens, kv_heads, d]");
  require(!overlaps_itself(*k, 2) && !overlaps_itself(*v, 2), "outputs must not overlap themselves");
  const long long strides[4] = {step(*k, 0), step(*k, 1), step(*v, 0), step(*v, 1)};
  const int st = g_api.gather(cache.data_ptr(), static_cast<const long long*>(slots.data_ptr()),
                              k->data_ptr(), v->data_ptr(), T, c.heads, narrow(d), c.pages,
                              c.page_size, strides,
                              here.stream(a[4], {made_k ? &*k : nullptr, made_v ? &*v : nullptr}));
  Tuple r(3, st);
  r.set(1, *k);
  r.set(2, *v);
  return r.release();
}

// (q, cache, block_table, lengths, cu_tokens, max_tokens, causal, scale, out, lse,
//  workspace, stream)
PyObject* attention(Args a, Py_ssize_t n) {
  count(n, 12);
  const Here here;
  const Tensor &q = tensor(a[0], "q must be a tensor"), &cache = tensor(a[1], "cache must be a tensor");
  const Tensor& table = tensor(a[2], "block_table must be a tensor");
  const Tensor& len = tensor(a[3], "lengths must be a tensor");
  const Tensor& cu = tensor(a[4], "cu_tokens must be a tensor");
  auto out = maybe(a[8], "out must be a tensor or None"), lse = maybe(a[9], "lse must be a tensor or None");
  auto ws = maybe(a[10], "workspace must be a tensor or None");
  require(q.dim() == 3 && unit(q) && (q.scalar_type() == at::kBFloat16 || q.scalar_type() == at::kHalf),
          "queries must be bf16 or fp16 [tokens, heads, d], d contiguous");
  const int64_t T = q.size(0), heads = q.size(1), d = q.size(2);
  const Cache c(cache, d);
  require(c.heads > 0 && heads % c.heads == 0,
          "the number of heads must be a multiple of the cache's");
  require(table.scalar_type() == at::kInt && table.dim() == 2 && (unit(table) || table.size(1) < 2),
          "block_table must be int32 [requests, width] with contiguous rows");
  const int64_t R = table.size(0);
  vector_of(len, at::kInt, R, "lengths must be contiguous int32 [requests]");
  vector_of(cu, at::kInt, R + 1, "cu_tokens must be contiguous int32 [requests + 1]");
  for (const Tensor* t : {&q, &cache, &table, &len, &cu}) here.check(*t);
  const int most = narrow(integer(a[5]));
  const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[7]);
  const bool made_out = !out, made_lse = !lse, made_ws = !ws;
  if (made_out) out = empty_like_dense(here, q);
  if (made_lse) lse = empty(here, {T, heads}, at::kFloat);
  require(out->sizes() == q.sizes() && out->scalar_type() == q.scalar_type() && unit(*out) &&
              !overlaps_itself(*out, 2),
          "the output must have q's shape, dtype, a contiguous d and rows of its own");
  require(lse->scalar_type() == at::kFloat && lse->dim() == 2 && lse->size(0) == T &&
              lse->size(1) == heads && lse->is_contiguous(),
          "lse must be a contiguous fp32 [tokens, heads] tensor");
  if (made_ws) {
    const size_t need = g_api.workspace_size(narrow(heads), c.heads, narrow(d), most);
    ws = empty(here, {static_cast<int64_t>(std::max<size_t>(need, 16))}, at::kByte);
  }
  require(ws->is_contiguous(), "the workspace must be contiguous");
  for (const Tensor* t : {&*out, &*lse, &*ws}) here.check(*t);
  const long long strides[4] = {step(q, 0), step(q, 1), step(*out, 0), step(*out, 1)};
  const int st = g_api.attention(
      q.data_ptr(), cache.data_ptr(), static_cast<const int*>(table.data_ptr()),
      static_cast<const int*>(len.data_ptr()), static_cast<const int*>(cu.data_ptr()),
      out->data_ptr(), static_cast<float*>(lse->data_ptr()), narrow(R), narrow(T), narrow(heads),
      c.heads, narrow(d), c.pages, c.page_size, narrow(table.size(1)),
      R < 2 ? std::max(table.stride(0), table.size(1)) : table.stride(0), strides, most, truth(a[6]),
      static_cast<float>(scale), type_code(q.scalar_type()), ws->data_ptr(), ws->nbytes(),
      here.stream(a[11], {made_out ? &*out : nullptr, made_lse ? &*lse : nullptr,
                          made_ws ? &*ws : nullptr}));
  Tuple r(3, st);
  r.set(1, *out);
  r.set(2, *lse);
  return r.release();
}

// bind(addresses of fa_rotary, fa_kv4_plan, fa_kv4_append, fa_kv4_gather,
//      fa_kv4_attention_workspace_size, fa_kv4_attention)
PyObject* bind(Args a, Py_ssize_t n) {
  count(n, 6);
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) throw Refused("bind needs six function addresses");
  }
  g_api = {reinterpret_cast<decltype(Api::rotary)>(p[0]),
           reinterpret_cast<decltype(Api::plan)>(p[1]),
           reinterpret_cast<decltype(Api::append)>(p[2]),
           reinterpret_cast<decltype(Api::gather)>(p[3]),
           reinterpret_cast<decltype(Api::workspace_size)>(p[4]),
           reinterpret_cast<decltype(Api::attention)>(p[5])};
  Py_RETURN_NONE;
}

// No C++ exception leaves an entry: refusals become ValueError, torch's errors
// theirs.
template <PyObject* (*F)(Args, Py_ssize_t)>
PyObject* entry(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (F != bind && !g_api.rotary) throw Refused("the CUDA library is not loaded");
    return F(a, n);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(Args, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<bind>("bind"),     method<rotary>("rotary"),
                           method<plan>("plan"),     method<append>("append"),
                           method<gather>("gather"), method<attention>("attention"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_binding() { return PyModule_Create(&g_module); }
