// serve_binding.cpp - the serving operators' Python calls on torch tensors:
// checks, outputs, workspace, the current stream, one C call each
// (include/dsatopk.h). Compiled, because a call on a few rows takes the GPU
// less time than the interpreter needs to look at its 10 to 25 arguments
// (16 to 21 us a call by way of ctypes).

#include <Python.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <initializer_list>
#include <string>
#include <utility>

#include "dsatopk.h"

namespace {

PyObject* g_error;      // DsatopkError(status, what)
PyObject* g_page_maps;  // PageMaps

struct Failed {};  // a Python error is set

// A reference of one's own.
struct Ref {
  PyObject* is;
  explicit Ref(PyObject* o) : is(o) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(is); }
};

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Failed{};
}

void check_status(int status, const char* what) {
  if (status == DSATOPK_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", status, what)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Failed{};
}

// A call's arguments by position and name. `names`: all of them, the first
// `required` without a default.
template <int kMost>
struct Args {
  PyObject* at[kMost] = {};

  Args(const char* fn, const char* const (&names)[kMost], int required, PyObject* const* args,
       Py_ssize_t n, PyObject* kw) {
    if (n > kMost) {
      PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, kMost, n);
      throw Failed{};
    }
    for (Py_ssize_t i = 0; i < n; ++i) at[i] = args[i];
    const Py_ssize_t more = kw ? PyTuple_GET_SIZE(kw) : 0;
    for (Py_ssize_t i = 0; i < more; ++i) {
      PyObject* name = PyTuple_GET_ITEM(kw, i);
      int k = 0;
      while (k < kMost && PyUnicode_CompareWithASCIIString(name, names[k]) != 0) ++k;
      if (k == kMost || at[k]) {
        PyErr_Format(PyExc_TypeError, "%s() got %s argument '%U'", fn,
                     k == kMost ? "an unexpected keyword" : "a second value for", name);
        throw Failed{};
      }
      at[k] = args[n + i];
    }
    for (int k = 0; k < required; ++k)
      if (!at[k]) {
        PyErr_Format(PyExc_TypeError, "%s() needs '%s'", fn, names[k]);
        throw Failed{};
      }
  }
  bool given(int k) const { return at[k] && at[k] != Py_None; }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  // results would be without their history, and without a word
  const c10::AutogradState& state = c10::AutogradState::get_tls_state();
  if ((state.get_grad_mode() && t.requires_grad()) ||
      (state.get_fw_grad_mode() && t._fw_grad(/*level=*/0).defined()))
    refuse(std::string(name) + " has gradients to keep, which this call does not compute (detach it, or "
                               "call under torch.no_grad())");
  return t;
}

int64_t integer(PyObject* o, const char* name) {
  PyObject* i = PyNumber_Index(o);
  if (!i) {
    PyErr_Format(PyExc_TypeError, "%s must be an integer", name);
    throw Failed{};
  }
  const int64_t v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return (int32_t)v;
}

int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + " has too many entries");
  return (int32_t)v;
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Format(PyExc_TypeError, "%s must be a number", name);
    throw Failed{};
  }
  return (float)v;
}

// A device tensor, on like's device if there is one.
void on_device(const at::Tensor& t, const at::Tensor* like, const char* name) {
  if (!t.is_cuda() || (like && t.device() != like->device()))
    refuse(std::string(name) + " must be a device tensor" +
           (like && like->is_cuda() ? " on " + like->device().str() : ""));
}

// A device tensor of `dims` dimensions with a contiguous last one.
const at::Tensor& shaped(PyObject* o, int dims, const at::Tensor* like, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims || (dims && t.size(dims - 1) > 1 && t.stride(dims - 1) != 1))
    refuse(std::string(name) + " must have " + std::to_string(dims) + " dimensions, the last one contiguous");
  on_device(t, like, name);
  return t;
}

const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }

// A contiguous int32 vector of length n (any length where n < 0).
const at::Tensor& vector(PyObject* o, int64_t n, const at::Tensor* like, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous int32 vector" +
           (n >= 0 ? " of length " + std::to_string(n) : ""));
  on_device(t, like, name);
  return t;
}

const int32_t* vector_or_null(PyObject* o, int64_t n, const at::Tensor* like, const char* name) {
  return o && o != Py_None ? ints(vector(o, n, like, name)) : nullptr;
}

const at::Tensor& table(PyObject* o, const at::Tensor* like) {
  const at::Tensor& t = tensor(o, "page_table");
  if (t.scalar_type() != at::kInt) refuse("page_table must be int32");
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("page_table must be [rows, width] with contiguous columns");
  on_device(t, like, "page_table");
  return t;
}

// Elements between entries of a dimension; 0 where one entry makes it meaningless.
int64_t stride(const at::Tensor& t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

// Elements between the rows of a matrix: a row at least, whatever one row's stride says.
int64_t row_stride(const at::Tensor& t) {
  return t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
}

int32_t element_type(const at::Tensor& t, const char* name, bool fp8) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return DSATOPK_BF16;
    case at::kHalf: return DSATOPK_FP16;
    case at::kFloat8_e4m3fn:
      if (fp8) return DSATOPK_FP8;
      [[fallthrough]];
    default:
      refuse(std::string(name) + (fp8 ? " must be bfloat16, float16 or float8_e4m3fn"
                                      : " must be bfloat16 or float16"));
  }
}

// Where a call goes: its tensors' device, and that device's current stream
// unless one is given. A given stream is the current one while this lives, so
// that what the call allocates is of that stream: memory that earlier work of
// the current stream may still use is not written by the other, and a
// workspace that the call frees goes back to work behind its kernels only.
class On {
 public:
  void* stream;

  On(const at::Tensor& like, PyObject* given)
      : device_(like.get_device()),
        before_(c10::hip::getCurrentHIPStream((c10::DeviceIndex)device_)) {
    stream = given && given != Py_None ? handle(given) : before_.stream();
    other_ = stream != before_.stream();
    if (other_)
      c10::hip::setCurrentHIPStream(
          c10::hip::getStreamFromExternal((hipStream_t)stream, (c10::DeviceIndex)device_));
    int now = -1;
    if (hipGetDevice(&now) == hipSuccess && now != device_ && hipSetDevice(device_) == hipSuccess)
      device_before_ = now;
  }
  On(const On&) = delete;
  On& operator=(const On&) = delete;
  ~On() {
    if (other_) c10::hip::setCurrentHIPStream(before_);
    if (device_before_ >= 0) (void)hipSetDevice(device_before_);
  }

  // What only this call uses.
  at::Tensor room(int64_t bytes, const at::Tensor& like) const {
    return at::detail::empty_cuda({bytes}, at::kByte, like.device(), c10::nullopt);
  }
  // What the caller gets, who may read and drop it on the stream that was current.
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) const {
    at::Tensor t = at::detail::empty_cuda(size, type, like.device(), c10::nullopt);
    if (other_) c10::hip::HIPCachingAllocator::recordStream(t.storage().data_ptr(), before_);
    return t;
  }

 private:
  int device_, device_before_ = -1;
  c10::hip::HIPStream before_;
  bool other_;

  static void* handle(PyObject* given) {
    unsigned long long h;
    if (PyLong_Check(given)) {
      h = PyLong_AsUnsignedLongLong(given);
    } else {
      PyObject* s = PyObject_GetAttrString(given, "cuda_stream");
      if (!s) throw Failed{};
      h = PyLong_AsUnsignedLongLong(s);
      Py_DECREF(s);
    }
    if (PyErr_Occurred()) throw Failed{};
    return reinterpret_cast<void*>(h);
  }
};

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

// ---------------------------------------------------------------------------

PyObject* page_maps(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"seq_lens", "page_table", "page_size", "free_pages",
                                      "num_tokens", "new_lens", "out", "stream"};
  const Args<8> a("page_maps", names, 5, args, n, kw);
  const at::Tensor& lens = vector(a.at[0], -1, nullptr, "seq_lens");
  const int32_t requests = size32(lens.size(0), "seq_lens");
  const at::Tensor& tab = table(a.at[1], &lens);
  if (tab.size(0) != requests) refuse("page_table must have one row per request");
  const int32_t page = integer32(a.at[2], "page_size");
  const at::Tensor& free = vector(a.at[3], -1, &lens, "free_pages");
  const int32_t tokens = integer32(a.at[4], "num_tokens");
  if (tokens < 0) refuse("num_tokens must not be negative");
  const int32_t* fresh = vector_or_null(a.at[5], requests, &lens, "new_lens");
  const On on(lens, a.at[7]);
  static const char* const fields[] = {"token_starts", "slots", "table_rows", "row_lens", "counts"};
  const int64_t sizes[] = {requests + int64_t(1), tokens, tokens, tokens, 2};
  // Held until the call is made: an attribute of `out` may be made when it is
  // asked for, and be nobody else's.
  at::Tensor to[5];
  for (int i = 0; i < 5; ++i) {
    if (!a.given(6)) {
      to[i] = on.empty({sizes[i]}, at::kInt, lens);
      continue;
    }
    const Ref o(PyObject_GetAttrString(a.at[6], fields[i]));
    if (!o.is) throw Failed{};
    to[i] = vector(o.is, sizes[i], &lens, fields[i]);
  }
  auto at = [&](int i) { return const_cast<int32_t*>(ints(to[i])); };
  check_status(dsatopk_page_maps(ints(lens), fresh, requests, const_cast<int32_t*>(ints(tab)),
                                 row_stride(tab), size32(tab.size(1), "page_table"), page,
                                 ints(free), size32(free.size(0), "free_pages"), tokens, at(0),
                                 at(1), at(2), at(3), at(4), on.stream),
               "dsatopk_page_maps");
  if (a.given(6)) {
    Py_INCREF(a.at[6]);
    return a.at[6];
  }
  const Ref made[5] = {Ref(THPVariable_Wrap(to[0])), Ref(THPVariable_Wrap(to[1])),
                       Ref(THPVariable_Wrap(to[2])), Ref(THPVariable_Wrap(to[3])),
                       Ref(THPVariable_Wrap(to[4]))};
  PyObject* fields_of[5];
  for (int i = 0; i < 5; ++i)
    if (!(fields_of[i] = made[i].is)) throw Failed{};
  return PyObject_Vectorcall(g_page_maps, fields_of, 5, nullptr);
}

// What both cache writes know of the tokens.
struct Tokens {
  const at::Tensor &slots, &lens, &angles;
  int32_t count, positions;
  float eps;
  int near;
  Tokens(const at::Tensor& x, PyObject* slots_, PyObject* lens_, PyObject* angles_, PyObject* eps_, PyObject* near_)
      : slots(vector(slots_, x.size(0), &x, "slots")),
        lens(vector(lens_, x.size(0), &x, "row_lens")),
        angles(shaped(angles_, 2, &x, "cos_sin")),
        count(size32(x.size(0), "slots")),
        positions(size32(angles.size(0), "cos_sin")),
        eps(eps_ ? number(eps_, "eps") : 1e-6f),
        near(near_ ? PyObject_IsTrue(near_) : 0) {
    if (near < 0) throw Failed{};
    if (angles.scalar_type() != at::kFloat || angles.size(1) != 64)
      refuse("cos_sin must be float32 [positions, 64]");
  }
};

// A contiguous float32 vector of length n, or null.
const float* floats_or_null(PyObject* o, int64_t n, const at::Tensor& like, const char* name) {
  if (!o || o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous float32 vector of length " + std::to_string(n));
  on_device(t, &like, name);
  return static_cast<const float*>(t.data_ptr());
}

// The caller's output of x's shape, or a new one.
at::Tensor result_like(const On& on, PyObject* o, const at::Tensor& x, at::ScalarType type, const char* name) {
  if (!o || o == Py_None) return on.empty(x.sizes(), type, x);
  const at::Tensor& t = shaped(o, (int)x.dim(), &x, name);
  if (t.scalar_type() != type || t.sizes() != x.sizes())
    refuse(std::string(name) + " does not have the type and shape of what it is to hold");
  return t;
}

// A written tensor's rows must not share memory: from the closest ones on, every
// dimension steps over all of those inside it.
void apart(const at::Tensor& t, const char* name) {
  if (!t.numel()) return;
  std::pair<int64_t, int64_t> outer[2];  // strides and sizes of the others than the last
  int n = 0;
  for (int64_t d = 0; d + 1 < t.dim() && n < 2; ++d)
    if (t.size(d) > 1) outer[n++] = {t.stride(d), t.size(d)};
  std::sort(outer, outer + n);
  int64_t extent = t.size(t.dim() - 1);
  for (int i = 0; i < n; ++i) {
    if (outer[i].first < extent)
      refuse(std::string(name) + " must not be expanded, nor its rows overlap: it is written");
    extent += outer[i].first * (outer[i].second - 1);
  }
}

PyObject* append_latent(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"latent", "cache", "slots", "row_lens", "cos_sin", "weight", "eps",
                                      "q_rope", "q_out", "out", "interleaved", "stream"};
  const Args<12> a("append_latent", names, 5, args, n, kw);
  const at::Tensor& x = shaped(a.at[0], 2, nullptr, "latent");
  const int32_t type = element_type(x, "latent", false);
  const at::Tensor& cache = shaped(a.at[1], 3, &x, "cache");
  if (cache.scalar_type() != x.scalar_type() || cache.size(2) != x.size(1))
    refuse("cache must have latent's type and last dimension");
  apart(cache, "cache");
  const Tokens t(x, a.at[2], a.at[3], a.at[4], a.at[6], a.at[10]);
  const int32_t dim = size32(x.size(1) - 64, "latent");
  const float* weight = floats_or_null(a.at[5], dim, x, "weight");
  const On on(x, a.at[11]);
  const at::Tensor* q = nullptr;
  at::Tensor q_out, out;
  if (a.given(7)) {
    q = &shaped(a.at[7], 3, &x, "q_rope");
    if (q->scalar_type() != x.scalar_type() || q->size(0) != x.size(0) || q->size(2) != 64)
      refuse("q_rope must have latent's type and shape (" + std::to_string(x.size(0)) + ", heads, 64)");
    q_out = result_like(on, a.at[8], *q, q->scalar_type(), "q_out");
    apart(q_out, "q_out");
  } else if (a.given(8)) {
    refuse("q_out is for q_rope");
  }
  if (a.given(9)) {
    out = result_like(on, a.at[9], x, x.scalar_type(), "out");
    apart(out, "out");
  }
  check_status(
      dsatopk_append_latent(
          x.data_ptr(), stride(x, 0), ints(t.slots), ints(t.lens), t.count,
          static_cast<const float*>(t.angles.data_ptr()), row_stride(t.angles), t.positions, t.near, weight,
          t.eps, type, dim, 64, cache.data_ptr(), cache.size(0), stride(cache, 0), stride(cache, 1),
          size32(cache.size(1), "cache"), out.defined() ? out.data_ptr() : nullptr,
          out.defined() ? stride(out, 0) : 0, q ? q->data_ptr() : nullptr, q ? stride(*q, 0) : 0,
          q ? stride(*q, 1) : 0, q ? q_out.data_ptr() : nullptr, q ? stride(q_out, 0) : 0,
          q ? stride(q_out, 1) : 0, q ? size32(q->size(1), "q_rope") : 0, on.stream),
      "dsatopk_append_latent");
  if (!q) Py_RETURN_NONE;
  return THPVariable_Wrap(q_out);
}

PyObject* append_index(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"keys", "index_keys", "slots", "row_lens", "cos_sin", "key_scales",
                                      "weight", "bias", "eps", "q", "weights", "q_out", "weights_out",
                                      "interleaved", "stream"};
  const Args<15> a("append_index", names, 5, args, n, kw);
  const at::Tensor& x = shaped(a.at[0], 2, nullptr, "keys");
  const int32_t type = element_type(x, "keys", false);
  const at::Tensor& cache = shaped(a.at[1], 3, &x, "index_keys");
  const int32_t to = element_type(cache, "index_keys", true);
  if ((to != DSATOPK_FP8 && to != type) || cache.size(2) != x.size(1))
    refuse("index_keys must be float8_e4m3fn or of keys' type, with keys' last dimension");
  apart(cache, "index_keys");
  const Tokens t(x, a.at[2], a.at[3], a.at[4], a.at[8], a.at[13]);
  const at::Tensor* scales = nullptr;
  if (a.given(5)) {
    scales = &shaped(a.at[5], 2, &x, "key_scales");
    if (to != DSATOPK_FP8 || scales->scalar_type() != at::kFloat ||
        scales->sizes() != cache.sizes().slice(0, 2))
      refuse("key_scales must be float32, one per key, of float8_e4m3fn index_keys");
    apart(*scales, "key_scales");
  } else if (to == DSATOPK_FP8) {
    refuse("float8_e4m3fn index_keys need key_scales");
  }
  const float* weight = floats_or_null(a.at[6], x.size(1), x, "weight");
  const float* bias = floats_or_null(a.at[7], x.size(1), x, "bias");
  if (!weight != !bias) refuse("weight and bias are given together");
  const On on(x, a.at[14]);
  const at::Tensor *q = nullptr, *weights = nullptr;
  at::Tensor q_out, weights_out;
  if (a.given(9)) {
    q = &shaped(a.at[9], 3, &x, "q");
    if (q->scalar_type() != x.scalar_type() || q->size(0) != x.size(0) || q->size(2) != x.size(1))
      refuse("q must have keys' type and shape (" + std::to_string(x.size(0)) + ", heads, " +
             std::to_string(x.size(1)) + ")");
    q_out = result_like(on, a.at[11], *q, cache.scalar_type(), "q_out");
    apart(q_out, "q_out");
    if (to == DSATOPK_FP8) {
      if (!a.given(10)) refuse("8-bit queries need weights");
      weights = &shaped(a.at[10], 2, &x, "weights");
      if (weights->scalar_type() != at::kFloat || weights->size(0) != q->size(0) || weights->size(1) != q->size(1))
        refuse("weights must be float32 of shape (" + std::to_string(q->size(0)) + ", " +
               std::to_string(q->size(1)) + ")");
      weights_out = result_like(on, a.at[12], *weights, at::kFloat, "weights_out");
      apart(weights_out, "weights_out");
    }
  }
  if ((a.given(10) || a.given(12)) && !weights) refuse("weights and weights_out are for 8-bit queries");
  if (a.given(11) && !q) refuse("q_out is for q");
  check_status(
      dsatopk_append_index(
          x.data_ptr(), stride(x, 0), ints(t.slots), ints(t.lens), t.count,
          static_cast<const float*>(t.angles.data_ptr()), row_stride(t.angles), t.positions, 64, t.near,
          weight, bias, t.eps, type, size32(x.size(1), "keys"), cache.data_ptr(), to, cache.size(0),
          stride(cache, 0), stride(cache, 1), size32(cache.size(1), "index_keys"),
          scales ? static_cast<float*>(scales->data_ptr()) : nullptr, scales ? stride(*scales, 0) : 0,
          q ? q->data_ptr() : nullptr, q ? stride(*q, 0) : 0, q ? stride(*q, 1) : 0,
          q ? q_out.data_ptr() : nullptr, q ? stride(q_out, 0) : 0, q ? stride(q_out, 1) : 0,
          weights ? static_cast<const float*>(weights->data_ptr()) : nullptr,
          weights ? stride(*weights, 0) : 0,
          weights ? static_cast<float*>(weights_out.data_ptr()) : nullptr,
          weights ? stride(weights_out, 0) : 0, q ? size32(q->size(1), "q") : 0, on.stream),
      "dsatopk_append_index");
  if (!q) Py_RETURN_NONE;
  if (weights) return pair(q_out, weights_out);
  const Ref made(THPVariable_Wrap(q_out));
  if (!made.is) throw Failed{};
  return PyTuple_Pack(2, made.is, Py_None);
}

struct Scores {
  const at::Tensor &q, &weights, &keys;
  const at::Tensor* scales = nullptr;
  int32_t type, rows, heads, dim;
  Scores(PyObject* q_, PyObject* w_, PyObject* k_, PyObject* s_, int key_dims)
      : q(shaped(q_, 3, nullptr, "q")),
        weights(shaped(w_, 2, &q, "weights")),
        keys(shaped(k_, key_dims, &q, "keys")),
        type(element_type(q, "q", true)),
        rows(size32(q.size(0), "q")),
        heads(size32(q.size(1), "q")),
        dim(size32(q.size(2), "q")) {
    if (weights.scalar_type() != at::kFloat || weights.size(0) != rows || weights.size(1) != heads)
      refuse("weights must be float32 of shape (" + std::to_string(rows) + ", " + std::to_string(heads) + ")");
    if (keys.scalar_type() != q.scalar_type() || keys.size(key_dims - 1) != dim)
      refuse("keys must have q's type and head dimension");
    if (s_ && s_ != Py_None) {
      scales = &shaped(s_, key_dims - 1, &q, "key_scales");
      if (scales->scalar_type() != at::kFloat || scales->sizes() != keys.sizes().slice(0, key_dims - 1))
        refuse("key_scales must be float32, one per key");
    }
  }
  at::Tensor out(const On& on, PyObject* o, int64_t columns) const {
    // a top-k's score buffer: a row stride that is a multiple of 4
    if (!o || o == Py_None)
      return on.empty({rows, std::max<int64_t>(4, (columns + 3) / 4 * 4)}, at::kFloat, q);
    const at::Tensor& t = shaped(o, 2, &q, "out");
    if (t.scalar_type() != at::kFloat || t.size(0) != rows)
      refuse("out must be float32 with " + std::to_string(rows) + " rows");
    return t;
  }
};

PyObject* scores_paged(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "weights", "keys", "seq_lens", "page_table",
                                      "key_scales", "table_rows", "out", "stream"};
  const Args<9> a("scores_paged", names, 5, args, n, kw);
  const Scores s(a.at[0], a.at[1], a.at[2], a.at[5], 3);
  const at::Tensor& lens = vector(a.at[3], s.rows, &s.q, "seq_lens");
  const int32_t* rows = vector_or_null(a.at[6], s.rows, &s.q, "table_rows");
  const at::Tensor& tab = table(a.at[4], &s.q);
  if (!rows && tab.size(0) != s.rows)
    refuse("page_table must have one row per query row without table_rows");
  const int32_t page = size32(s.keys.size(1), "keys");
  const On on(s.q, a.at[8]);
  const at::Tensor out = s.out(on, a.at[7], tab.size(1) * page);
  check_status(
      dsatopk_scores_paged(s.q.data_ptr(), stride(s.q, 0), stride(s.q, 1),
                           static_cast<const float*>(s.weights.data_ptr()), stride(s.weights, 0),
                           s.keys.data_ptr(), s.keys.size(0), stride(s.keys, 0), stride(s.keys, 1),
                           s.scales ? static_cast<const float*>(s.scales->data_ptr()) : nullptr,
                           s.scales ? stride(*s.scales, 0) : 0, s.type, s.heads, s.dim, ints(lens),
                           ints(tab), row_stride(tab), size32(tab.size(1), "page_table"), page, rows,
                           s.rows, static_cast<float*>(out.data_ptr()), row_stride(out), out.size(1),
                           on.stream),
      "dsatopk_scores_paged");
  return THPVariable_Wrap(out);
}

PyObject* scores_ragged(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "weights", "keys", "seq_lens", "row_starts",
                                      "key_scales", "out", "stream"};
  const Args<8> a("scores_ragged", names, 5, args, n, kw);
  const Scores s(a.at[0], a.at[1], a.at[2], a.at[5], 2);
  const at::Tensor& lens = vector(a.at[3], s.rows, &s.q, "seq_lens");
  const at::Tensor& starts = vector(a.at[4], s.rows, &s.q, "row_starts");
  const On on(s.q, a.at[7]);
  const at::Tensor out = s.out(on, a.at[6], s.keys.size(0));
  check_status(
      dsatopk_scores_ragged(s.q.data_ptr(), stride(s.q, 0), stride(s.q, 1),
                            static_cast<const float*>(s.weights.data_ptr()), stride(s.weights, 0),
                            s.keys.data_ptr(), s.keys.size(0), stride(s.keys, 0),
                            s.scales ? static_cast<const float*>(s.scales->data_ptr()) : nullptr,
                            s.type, s.heads, s.dim, ints(lens), ints(starts), s.rows,
                            static_cast<float*>(out.data_ptr()), row_stride(out), out.size(1),
                            on.stream),
      "dsatopk_scores_ragged");
  return THPVariable_Wrap(out);
}

// Attention's results: out (q's type) of rows x heads x dim, lse (float32) of rows x heads.
struct Results {
  at::Tensor out, lse;
  Results(const On& on, PyObject* o, PyObject* l, const at::Tensor& q, int64_t dim) {
    if (o && o != Py_None) {
      out = tensor(o, "out");
      if (out.scalar_type() != q.scalar_type() || out.dim() != 3 || out.size(0) != q.size(0) ||
          out.size(1) != q.size(1) || out.size(2) != dim || !out.is_contiguous())
        refuse("out must be contiguous, of q's type and shape (" + std::to_string(q.size(0)) + ", " +
               std::to_string(q.size(1)) + ", " + std::to_string(dim) + ")");
      on_device(out, &q, "out");
    } else {
      if (dim < 0) refuse("latent_dim must not be negative");
      out = on.empty({q.size(0), q.size(1), dim}, q.scalar_type(), q);
    }
    if (l && l != Py_None) {
      lse = tensor(l, "lse");
      if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != q.size(0) ||
          lse.size(1) != q.size(1) || !lse.is_contiguous())
        refuse("lse must be contiguous float32 of shape (" + std::to_string(q.size(0)) + ", " +
               std::to_string(q.size(1)) + ")");
      on_device(lse, &q, "lse");
    } else {
      lse = on.empty({q.size(0), q.size(1)}, at::kFloat, q);
    }
  }
};

// The given workspace, or one of `need` bytes.
at::Tensor workspace_of(const On& on, PyObject* given, size_t need, const at::Tensor& q) {
  if (given && given != Py_None) {
    const at::Tensor& t = tensor(given, "workspace");
    if (t.scalar_type() != at::kByte || !t.is_contiguous())
      refuse("workspace must be a contiguous uint8 tensor");
    on_device(t, &q, "workspace");
    return t;
  }
  return need ? on.room((int64_t)need, q) : at::Tensor();
}
void* room_ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t room_bytes(const at::Tensor& t) { return t.defined() ? (size_t)t.numel() : 0; }

// The absorbed forms' common arguments.
struct Absorbed {
  const at::Tensor &q, &cache;
  int32_t type, rows, heads, latent;
  On on;
  Results results;
  at::Tensor workspace;
  Absorbed(PyObject* q_, PyObject* c_, PyObject* latent_, PyObject* out, PyObject* lse, PyObject* stream)
      : q(shaped(q_, 3, nullptr, "q")),
        cache(shaped(c_, 3, &q, "cache")),
        type(element_type(q, "q", false)),
        rows(size32(q.size(0), "q")),
        heads(size32(q.size(1), "q")),
        latent(integer32(latent_, "latent_dim")),
        on((check(), q), stream),
        results(on, out, lse, q, latent) {}
  void check() const {
    if (cache.scalar_type() != q.scalar_type() || cache.size(2) != q.size(2))
      refuse("cache must have q's type and last dimension");
  }
  void room(PyObject* given, int64_t tokens) {
    workspace = workspace_of(on, given, dsatopk_attend_bytes(rows, heads, latent, tokens), q);
  }
  // A bound on a row's tokens; a table may have more positions than the largest, 2^31 - 65.
  int64_t bound(PyObject* given, const at::Tensor& tab, const char* name) const {
    return given && given != Py_None ? integer(given, name)
                                     : std::min<int64_t>(tab.size(1) * cache.size(1), INT32_MAX - 64);
  }
};

PyObject* attend_selected(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "cache", "slots", "latent_dim", "scale",
                                      "out", "lse", "workspace", "stream"};
  const Args<9> a("attend_selected", names, 5, args, n, kw);
  Absorbed s(a.at[0], a.at[1], a.at[3], a.at[5], a.at[6], a.at[8]);
  const at::Tensor& slots = shaped(a.at[2], 2, &s.q, "slots");
  if (slots.scalar_type() != at::kInt || slots.size(0) != s.rows)
    refuse("slots must be int32 with one row per query row");
  const int32_t k = size32(slots.size(1), "slots");
  const float scale = number(a.at[4], "scale");
  s.room(a.at[7], k);
  check_status(
      dsatopk_attend_selected(s.q.data_ptr(), stride(s.q, 0), stride(s.q, 1), s.cache.data_ptr(),
                              s.cache.size(0), stride(s.cache, 0), stride(s.cache, 1),
                              size32(s.cache.size(1), "cache"), s.type, s.heads, s.latent,
                              size32(s.q.size(2) - s.latent, "q"), scale, ints(slots),
                              row_stride(slots), k, s.rows, s.results.out.data_ptr(),
                              static_cast<float*>(s.results.lse.data_ptr()), room_ptr(s.workspace),
                              room_bytes(s.workspace), s.on.stream),
      "dsatopk_attend_selected");
  return pair(s.results.out, s.results.lse);
}

PyObject* attend_paged(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "cache", "seq_lens", "page_table", "latent_dim", "scale",
                                      "table_rows", "max_seq_len", "out", "lse", "workspace", "stream"};
  const Args<12> a("attend_paged", names, 6, args, n, kw);
  Absorbed s(a.at[0], a.at[1], a.at[4], a.at[8], a.at[9], a.at[11]);
  const at::Tensor& lens = vector(a.at[2], s.rows, &s.q, "seq_lens");
  const int32_t* rows = vector_or_null(a.at[6], s.rows, &s.q, "table_rows");
  const at::Tensor& tab = table(a.at[3], &s.q);
  if (!rows && tab.size(0) != s.rows)
    refuse("page_table must have one row per query row without table_rows");
  const float scale = number(a.at[5], "scale");
  const int64_t longest = s.bound(a.at[7], tab, "max_seq_len");
  s.room(a.at[10], longest);
  check_status(
      dsatopk_attend_paged(s.q.data_ptr(), stride(s.q, 0), stride(s.q, 1), s.cache.data_ptr(),
                           s.cache.size(0), stride(s.cache, 0), stride(s.cache, 1),
                           size32(s.cache.size(1), "cache"), s.type, s.heads, s.latent,
                           size32(s.q.size(2) - s.latent, "q"), scale, ints(lens), ints(tab),
                           row_stride(tab), size32(tab.size(1), "page_table"), rows, longest, s.rows,
                           s.results.out.data_ptr(), static_cast<float*>(s.results.lse.data_ptr()),
                           room_ptr(s.workspace), room_bytes(s.workspace), s.on.stream),
      "dsatopk_attend_paged");
  return pair(s.results.out, s.results.lse);
}

PyObject* attend_shared(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "cache", "seq_lens", "page_table", "group_starts", "shared_lens",
                                      "latent_dim", "scale", "table_rows", "max_shared_len", "max_own_len",
                                      "out", "lse", "workspace", "stream"};
  const Args<15> a("attend_shared", names, 8, args, n, kw);
  Absorbed s(a.at[0], a.at[1], a.at[6], a.at[11], a.at[12], a.at[14]);
  const at::Tensor& lens = vector(a.at[2], s.rows, &s.q, "seq_lens");
  const int32_t* rows = vector_or_null(a.at[8], s.rows, &s.q, "table_rows");
  const at::Tensor& tab = table(a.at[3], &s.q);
  if (!rows && tab.size(0) != s.rows)
    refuse("page_table must have one row per query row without table_rows");
  const at::Tensor& starts = vector(a.at[4], -1, &s.q, "group_starts");
  if (starts.size(0) < 1 || (s.rows && starts.size(0) < 2))
    refuse("group_starts must have an entry more than there are groups, one group at least");
  const int32_t groups = size32(starts.size(0) - 1, "group_starts");
  const at::Tensor& shared = vector(a.at[5], groups, &s.q, "shared_lens");
  const float scale = number(a.at[7], "scale");
  const int64_t most_shared = s.bound(a.at[9], tab, "max_shared_len");
  const int64_t most_own = s.bound(a.at[10], tab, "max_own_len");
  s.workspace = workspace_of(s.on, a.at[13],
                             dsatopk_shared_bytes(s.rows, s.heads, s.latent, groups, most_shared, most_own), s.q);
  check_status(
      dsatopk_attend_shared(s.q.data_ptr(), stride(s.q, 0), stride(s.q, 1), s.cache.data_ptr(),
                            s.cache.size(0), stride(s.cache, 0), stride(s.cache, 1),
                            size32(s.cache.size(1), "cache"), s.type, s.heads, s.latent,
                            size32(s.q.size(2) - s.latent, "q"), scale, ints(lens), ints(tab),
                            row_stride(tab), size32(tab.size(1), "page_table"), rows, ints(starts),
                            ints(shared), groups, most_shared, most_own, s.rows,
                            s.results.out.data_ptr(), static_cast<float*>(s.results.lse.data_ptr()),
                            room_ptr(s.workspace), room_bytes(s.workspace), s.on.stream),
      "dsatopk_attend_shared");
  return pair(s.results.out, s.results.lse);
}

// The expanded forms' common tensors.
struct Expanded {
  const at::Tensor &q, &k, &v, &rope;
  int32_t type, heads, queries, keys;
  Expanded(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* rope_)
      : q(shaped(q_, 3, nullptr, "q")),
        k(shaped(k_, 3, &q, "k")),
        v(shaped(v_, 3, &q, "v")),
        rope(shaped(rope_, 2, &q, "k_rope")),
        type(element_type(q, "q", false)) {
    for (const at::Tensor* t : {&k, &v, &rope})
      if (t->scalar_type() != q.scalar_type() || t->size(0) != k.size(0) ||
          (t != &rope && t->size(1) != q.size(1)))
        refuse("k, v and k_rope must have q's type, as many rows as k, and q's heads");
    if (q.size(2) != k.size(2) + rope.size(1))
      refuse("q's last dimension must be k's and k_rope's together");
    heads = size32(q.size(1), "q");
    queries = size32(q.size(0), "q");
    keys = size32(k.size(0), "k");
  }
};

int truth(PyObject* o, int otherwise) {
  const int is = o ? PyObject_IsTrue(o) : otherwise;
  if (is < 0) throw Failed{};
  return is;
}

PyObject* attend_expanded(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "k", "v", "k_rope", "q_starts", "k_starts", "max_queries",
                                      "scale", "causal", "out", "lse", "workspace", "stream"};
  const Args<13> a("attend_expanded", names, 8, args, n, kw);
  const Expanded e(a.at[0], a.at[1], a.at[2], a.at[3]);
  const at::Tensor &q = e.q, &k = e.k, &v = e.v, &rope = e.rope;
  const at::Tensor& qs = vector(a.at[4], -1, &q, "q_starts");
  if (qs.size(0) < 1) refuse("q_starts must have an entry more than there are requests");
  const at::Tensor& ks = vector(a.at[5], qs.size(0), &q, "k_starts");
  const int32_t longest = integer32(a.at[6], "max_queries");
  const float scale = number(a.at[7], "scale");
  const int causal = truth(a.at[8], 1);
  const On on(q, a.at[12]);
  const Results r(on, a.at[9], a.at[10], q, v.size(2));
  const int32_t requests = size32(qs.size(0) - 1, "q_starts");
  const at::Tensor room = workspace_of(
      on, a.at[11], dsatopk_expanded_bytes(requests, e.heads, e.queries, e.keys, longest), q);
  check_status(
      dsatopk_attend_expanded(q.data_ptr(), stride(q, 0), stride(q, 1), k.data_ptr(), stride(k, 0),
                              stride(k, 1), v.data_ptr(), stride(v, 0), stride(v, 1),
                              rope.data_ptr(), stride(rope, 0), e.type, e.heads,
                              size32(k.size(2), "k"), size32(rope.size(1), "k_rope"),
                              size32(v.size(2), "v"), scale, causal, ints(qs), ints(ks),
                              requests, e.queries, e.keys, longest, r.out.data_ptr(),
                              static_cast<float*>(r.lse.data_ptr()), room_ptr(room),
                              room_bytes(room), on.stream),
      "dsatopk_attend_expanded");
  return pair(r.out, r.lse);
}

PyObject* attend_expanded_shared(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "k", "v", "k_rope", "q_starts", "k_starts", "shared_starts",
                                      "shared_lens", "scale", "max_keys", "causal", "out", "lse",
                                      "workspace", "stream"};
  const Args<15> a("attend_expanded_shared", names, 9, args, n, kw);
  const Expanded e(a.at[0], a.at[1], a.at[2], a.at[3]);
  const at::Tensor &q = e.q, &k = e.k, &v = e.v, &rope = e.rope;
  const at::Tensor& qs = vector(a.at[4], -1, &q, "q_starts");
  if (qs.size(0) < 1) refuse("q_starts must have an entry more than there are requests");
  const at::Tensor& ks = vector(a.at[5], qs.size(0), &q, "k_starts");
  const int32_t requests = size32(qs.size(0) - 1, "q_starts");
  const at::Tensor& ss = vector(a.at[6], requests, &q, "shared_starts");
  const at::Tensor& sl = vector(a.at[7], requests, &q, "shared_lens");
  const float scale = number(a.at[8], "scale");
  const int32_t longest = a.given(9) ? integer32(a.at[9], "max_keys") : e.keys;
  const int causal = truth(a.at[10], 1);
  const On on(q, a.at[14]);
  const Results r(on, a.at[11], a.at[12], q, v.size(2));
  const at::Tensor room =
      workspace_of(on, a.at[13], dsatopk_expanded_shared_bytes(e.heads, e.queries, longest), q);
  check_status(
      dsatopk_attend_expanded_shared(
          q.data_ptr(), stride(q, 0), stride(q, 1), k.data_ptr(), stride(k, 0), stride(k, 1), v.data_ptr(),
          stride(v, 0), stride(v, 1), rope.data_ptr(), stride(rope, 0), e.type, e.heads,
          size32(k.size(2), "k"), size32(rope.size(1), "k_rope"), size32(v.size(2), "v"), scale, causal,
          ints(qs), ints(ks), ints(ss), ints(sl), requests, e.queries, e.keys, longest, r.out.data_ptr(),
          static_cast<float*>(r.lse.data_ptr()), room_ptr(room), room_bytes(room), on.stream),
      "dsatopk_attend_expanded_shared");
  return pair(r.out, r.lse);
}

// No C++ exception leaves a call: torch's become the Python errors that its own
// calls raise.
template <PyObject* (*fn)(PyObject* const*, Py_ssize_t, PyObject*)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  try {
    return fn(args, n, kw);
  } catch (const Failed&) {
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

PyObject* setup(PyObject*, PyObject* args) {
  PyObject *error, *maps;
  if (!PyArg_ParseTuple(args, "OO", &error, &maps)) return nullptr;
  Py_INCREF(error);
  Py_INCREF(maps);
  Py_XDECREF(g_error);
  Py_XDECREF(g_page_maps);
  g_error = error;
  g_page_maps = maps;
  Py_RETURN_NONE;
}

const char page_maps_doc[] = R"doc(page_maps(seq_lens, page_table, page_size, free_pages, num_tokens, new_lens=None, out=None, stream=None)
--

The pages, slots and top-k row arguments of a serving step.

Requests of seq_lens tokens after the step, new_lens of them new (None: one
each), take the pages that they lack from free_pages: these are written into
page_table in place. Returns PageMaps, whose slots, table_rows and row_lens
have num_tokens rows (empty ones behind the step's tokens). out: a PageMaps
to write into.

stream (here and in the other calls): a stream, or its handle, to go to
instead of the current one, as if it were the current one: inputs have to be
ready on it, and what the call allocates is of it. None of the calls has a
gradient: tensors that require one are refused where gradients are recorded.)doc";

const char append_latent_doc[] = R"doc(append_latent(latent, cache, slots, row_lens, cos_sin, weight=None, eps=1e-6, q_rope=None, q_out=None, out=None, interleaved=False, stream=None)
--

New tokens' latent vectors into the paged cache, normalised and turned.

latent [tokens, latent_dim + 64] in bfloat16 or float16, as the projection
leaves it: its latent part is divided by its root mean square and multiplied
by weight (float32 [latent_dim]; None: left as it is), its last 64 elements are
turned by the angles of position row_lens - 1 (cos_sin float32 [positions, 64]:
32 cosines, then 32 sines; pairs of neighbours if interleaved, else of halves).
slots and row_lens are page_maps'; a token without a slot in the cache or a
position in the table is not cached. out: like latent, also receives the
vectors (may be latent). q_rope [tokens, heads, 64]: the queries' rotary parts,
turned likewise into q_out (a view of absorbed queries, or q_rope itself;
allocated when None), which is returned; None without q_rope.)doc";

const char append_index_doc[] = R"doc(append_index(keys, index_keys, slots, row_lens, cos_sin, key_scales=None, weight=None, bias=None, eps=1e-6, q=None, weights=None, q_out=None, weights_out=None, interleaved=False, stream=None)
--

New tokens' indexer keys into their paged cache, as scores_paged() reads it.

keys [tokens, dim] in bfloat16 or float16: normalised (layer norm with weight
and bias, float32 [dim]; None: left as they are), their first 64 elements turned
as by append_latent. index_keys [pages, page_size, dim] of the same type, or
float8_e4m3fn with key_scales float32 [pages, page_size], which get the largest
element / 448. q [tokens, heads, dim]: the indexer's queries, turned and rounded
likewise, with their scales multiplied into weights (float32 [tokens, heads],
8 bits only). Returns (q_out, weights_out), None without q; weights_out is None
with 16 bits.)doc";

const char scores_paged_doc[] = R"doc(scores_paged(q, weights, keys, seq_lens, page_table, key_scales=None, table_rows=None, out=None, stream=None)
--

Indexer scores over a paged key cache, as paged() reads them.

q [rows, heads, dim] and keys [pages, page_size, dim] in bfloat16, float16 or
float8_e4m3fn, weights float32 [rows, heads], key_scales float32 [pages,
page_size] or None. Column j < seq_len of row b of out gets key_scale[j] *
sum_h weights[b, h] * max(0, q[b, h] . key[j]); other columns are not written.
Returns out (allocated with a column per table position when None).)doc";

const char scores_ragged_doc[] = R"doc(scores_ragged(q, weights, keys, seq_lens, row_starts, key_scales=None, out=None, stream=None)
--

Indexer scores over flattened keys [tokens, dim], as ragged() reads them.

Row b's window is columns row_starts[b] .. row_starts[b] + seq_lens[b] - 1 of
out; other columns are not written. Arguments as for scores_paged, key_scales
float32 [tokens].)doc";

const char attend_selected_doc[] = R"doc(attend_selected(q, cache, slots, latent_dim, scale, out=None, lse=None, workspace=None, stream=None)
--

Absorbed latent attention over selected cache slots.

q [rows, heads, latent_dim + 64] and cache [pages, page_size, latent_dim + 64]
in bfloat16 or float16; slots int32 [rows, k] as paged() returns them (-1:
none). Returns (out, lse): q's type [rows, heads, latent_dim], and float32
[rows, heads]. workspace: uint8 of attend_bytes(rows, heads, latent_dim, k)
(allocated when None).)doc";

const char attend_paged_doc[] = R"doc(attend_paged(q, cache, seq_lens, page_table, latent_dim, scale, table_rows=None, max_seq_len=None, out=None, lse=None, workspace=None, stream=None)
--

Absorbed latent attention over the first seq_lens positions of each row's
page table.

Arguments as for attend_selected and paged(); max_seq_len bounds seq_lens (the
table's positions when None) and sets how rows are split.)doc";

const char attend_shared_doc[] = R"doc(attend_shared(q, cache, seq_lens, page_table, group_starts, shared_lens, latent_dim, scale, table_rows=None, max_shared_len=None, max_own_len=None, out=None, lse=None, workspace=None, stream=None)
--

attend_paged for rows in groups whose first tokens are the same cached ones,
read once for all rows of a group.

group_starts int32 [groups + 1]: a group's first row (the first one is taken as
0, the last as the number of rows); shared_lens int32 [groups]: how many
positions its rows share, those of its first row's page table. A row reads what
it sees of them there and its other positions in its own table. max_shared_len
and max_own_len bound the shared positions and those that a row reads by
itself (the table's positions when None; 0: there are none). workspace: uint8 of
shared_bytes(rows, heads, latent_dim, groups, max_shared_len, max_own_len)
(allocated when None).)doc";

const char attend_expanded_doc[] = R"doc(attend_expanded(q, k, v, k_rope, q_starts, k_starts, max_queries, scale, causal=True, out=None, lse=None, workspace=None, stream=None)
--

Expanded latent attention over a ragged batch of prompts.

q [queries, heads, 192], k and v [keys, heads, 128] and k_rope [keys, 64] in
bfloat16 or float16 (k and v may be parts of one tensor); q_starts and
k_starts int32 [requests + 1]; max_queries bounds a request's queries, which
are its last tokens. Returns (out, lse): q's type [queries, heads, 128], and
float32 [queries, heads]. workspace: uint8 of expanded_bytes(requests, heads,
queries, keys, max_queries) (allocated when None).)doc";

const char attend_expanded_shared_doc[] = R"doc(attend_expanded_shared(q, k, v, k_rope, q_starts, k_starts, shared_starts, shared_lens, scale, max_keys=None, causal=True, out=None, lse=None, workspace=None, stream=None)
--

attend_expanded for prompts behind keys that several of them share, which are
there once.

Request r's keys are rows shared_starts[r] .. shared_starts[r] + shared_lens[r]
- 1 of k, v and k_rope (int32 [requests] each), which all of its queries see, and
then its own, k_starts[r] .. k_starts[r + 1] - 1. Neighbouring requests with the
same shared rows share the work on them. max_keys bounds a request's keys (the
rows of k when None) and sets how few queries of many keys are split.
workspace: uint8 of expanded_shared_bytes(heads, queries, max_keys) (allocated
when None).)doc";

#define SERVE_CALL(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), \
   METH_FASTCALL | METH_KEYWORDS, name##_doc}

PyMethodDef methods[] = {
    SERVE_CALL(page_maps),       SERVE_CALL(append_latent), SERVE_CALL(append_index),
    SERVE_CALL(scores_paged),    SERVE_CALL(scores_ragged),
    SERVE_CALL(attend_selected), SERVE_CALL(attend_paged), SERVE_CALL(attend_shared),
    SERVE_CALL(attend_expanded), SERVE_CALL(attend_expanded_shared),
    {"setup", setup, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__serve(void) { return PyModule_Create(&module); }
