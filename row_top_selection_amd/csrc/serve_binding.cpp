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
  // a table may have more positions than the largest bound, 2^31 - 65
  const int64_t longest =
      a.given(7) ? integer(a.at[7], "max_seq_len")
                 : std::min<int64_t>(tab.size(1) * s.cache.size(1), INT32_MAX - 64);
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

PyObject* attend_expanded(PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const char* const names[] = {"q", "k", "v", "k_rope", "q_starts", "k_starts", "max_queries",
                                      "scale", "causal", "out", "lse", "workspace", "stream"};
  const Args<13> a("attend_expanded", names, 8, args, n, kw);
  const at::Tensor& q = shaped(a.at[0], 3, nullptr, "q");
  const at::Tensor& k = shaped(a.at[1], 3, &q, "k");
  const at::Tensor& v = shaped(a.at[2], 3, &q, "v");
  const at::Tensor& rope = shaped(a.at[3], 2, &q, "k_rope");
  const int32_t type = element_type(q, "q", false);
  for (const at::Tensor* t : {&k, &v, &rope})
    if (t->scalar_type() != q.scalar_type() || t->size(0) != k.size(0) ||
        (t != &rope && t->size(1) != q.size(1)))
      refuse("k, v and k_rope must have q's type, as many rows as k, and q's heads");
  if (q.size(2) != k.size(2) + rope.size(1))
    refuse("q's last dimension must be k's and k_rope's together");
  const at::Tensor& qs = vector(a.at[4], -1, &q, "q_starts");
  if (qs.size(0) < 1) refuse("q_starts must have an entry more than there are requests");
  const at::Tensor& ks = vector(a.at[5], qs.size(0), &q, "k_starts");
  const int32_t longest = integer32(a.at[6], "max_queries");
  const float scale = number(a.at[7], "scale");
  const int causal = a.at[8] ? PyObject_IsTrue(a.at[8]) : 1;
  if (causal < 0) throw Failed{};
  const On on(q, a.at[12]);
  const Results r(on, a.at[9], a.at[10], q, v.size(2));
  const int32_t requests = size32(qs.size(0) - 1, "q_starts"), heads = size32(q.size(1), "q");
  const int32_t queries = size32(q.size(0), "q"), keys = size32(k.size(0), "k");
  const at::Tensor room = workspace_of(
      on, a.at[11], dsatopk_expanded_bytes(requests, heads, queries, keys, longest), q);
  check_status(
      dsatopk_attend_expanded(q.data_ptr(), stride(q, 0), stride(q, 1), k.data_ptr(), stride(k, 0),
                              stride(k, 1), v.data_ptr(), stride(v, 0), stride(v, 1),
                              rope.data_ptr(), stride(rope, 0), type, heads,
                              size32(k.size(2), "k"), size32(rope.size(1), "k_rope"),
                              size32(v.size(2), "v"), scale, causal, ints(qs), ints(ks),
                              requests, queries, keys, longest, r.out.data_ptr(),
                              static_cast<float*>(r.lse.data_ptr()), room_ptr(room),
                              room_bytes(room), on.stream),
      "dsatopk_attend_expanded");
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

const char attend_expanded_doc[] = R"doc(attend_expanded(q, k, v, k_rope, q_starts, k_starts, max_queries, scale, causal=True, out=None, lse=None, workspace=None, stream=None)
--

Expanded latent attention over a ragged batch of prompts.

q [queries, heads, 192], k and v [keys, heads, 128] and k_rope [keys, 64] in
bfloat16 or float16 (k and v may be parts of one tensor); q_starts and
k_starts int32 [requests + 1]; max_queries bounds a request's queries, which
are its last tokens. Returns (out, lse): q's type [queries, heads, 128], and
float32 [queries, heads]. workspace: uint8 of expanded_bytes(requests, heads,
queries, keys, max_queries) (allocated when None).)doc";

#define SERVE_CALL(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), \
   METH_FASTCALL | METH_KEYWORDS, name##_doc}

PyMethodDef methods[] = {
    SERVE_CALL(page_maps),       SERVE_CALL(scores_paged), SERVE_CALL(scores_ragged),
    SERVE_CALL(attend_selected), SERVE_CALL(attend_paged), SERVE_CALL(attend_expanded),
    {"setup", setup, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__serve(void) { return PyModule_Create(&module); }
