// binding.cpp -- the torch-facing half of cache16.py: tensors into the C structs
// of bsfa_rotary, bsfa_cache16_write and bsfa_decode16 (argument marshalling only).
//
// Compiled because a decode step's calls are short: reading forty tensor attributes
// from Python costs more than the call.  cache16.py names and documents the
// arguments; here they come by position.  Everything that can be told from shapes,
// types, strides and devices is checked before anything is allocated or launched.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <optional>
#include <string>

#include "bsfa.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw python_error();
}
void want(bool ok, const char* what) {
  if (!ok) refuse(PyExc_ValueError, what);
}

// A tensor argument; nullptr for None.
const Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& needed(PyObject* o, const char* name) {
  const Tensor* t = tensor(o, name);
  if (t == nullptr) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return *t;
}

// Whether autograd is to record what is made of one of these.
template <class... T>
bool recorded(const T*... t) {
  return c10::GradMode::is_enabled() && ((t != nullptr && t->requires_grad()) || ...);
}

// A caller's tensor that a call has written: counted, so that a graph that keeps its old
// contents is told (tensors made for inference carry no count).
void written(const Tensor* t) {
  if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// A layout by name; `otherwise` for None.
const char* layout_of(PyObject* o, const char* otherwise) {
  if (o == Py_None) return otherwise;
  for (const char* name : {"bhld", "blhd", "htd", "thd", "phtd", "pthd"})
    if (PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, name) == 0) return name;
  PyErr_SetObject(PyExc_ValueError, o);
  throw python_error();
}
bool is(const char* layout, const char* name) { return std::strcmp(layout, name) == 0; }

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}

int dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return BSFA_DTYPE_BF16;
  if (t.scalar_type() == at::kHalf) return BSFA_DTYPE_F16;
  refuse(PyExc_TypeError, "expected a bfloat16 or float16 tensor");
}

int to_int(int64_t x) {
  want(x >= INT32_MIN && x <= INT32_MAX, "a size beyond 32 bits");
  return static_cast<int>(x);
}

void on_device(const Tensor& t, const at::Device& device, const char* name) {
  if (t.device() != device)
    refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " +
                                 device.str());
}

// Where a call runs: on `stream` (None: the device's current one) of its tensors'
// device.  Made when all other arguments have been found good.
class Place {
 public:
  Place(const at::Device& device, PyObject* stream) : device_(device) {
    if (!device.is_cuda())
      refuse(PyExc_ValueError, "the tensors must be CUDA tensors, not on " + device.str());
    if (stream != Py_None) {
      const int64_t id = number(stream, "stream_id"), index = number(stream, "device_index");
      const int64_t type = number(stream, "device_type");
      other_ = c10::cuda::CUDAStream::unpack3(id, static_cast<c10::DeviceIndex>(index),
                                              static_cast<c10::DeviceType>(type));
    }
    guard_.emplace(device);
  }
  bsfa_stream_t stream() const {
    return reinterpret_cast<bsfa_stream_t>(
        (other_ ? *other_ : c10::cuda::getCurrentCUDAStream(device_.index())).stream());
  }
  // Memory that the call's stream may write at once, and that is not handed out again
  // while the caller's stream reads it.
  template <class Make>
  Tensor fresh(Make make) const {
    if (!other_) return make();
    const auto mine = c10::cuda::getCurrentCUDAStream(device_.index());
    Tensor t;
    {
      c10::cuda::CUDAStreamGuard on(*other_);
      t = make();
    }
    t.record_stream(mine);
    return t;
  }
  // (Straight from the allocator: a fifth of a short call's time was torch's dispatch.)
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return fresh(
        [&] { return Tensor(at::detail::empty_cuda(size, type, device_, std::nullopt)); });
  }
  Tensor like(const Tensor& t) const {
    if (t.is_contiguous()) return empty(t.sizes(), t.scalar_type());
    return fresh([&] { return at::empty_like(t); });
  }

 private:
  static int64_t number(PyObject* o, const char* name) {
    PyObject* x = PyObject_GetAttrString(o, name);
    if (x == nullptr) throw python_error();
    const int64_t v = PyLong_AsLongLong(x);
    Py_DECREF(x);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
  }
  at::Device device_;
  std::optional<c10::cuda::CUDAStream> other_;
  std::optional<c10::cuda::CUDAGuard> guard_;
};

// A status other than BSFA_OK becomes the package's BsfaError.
void check(bsfa_status s, const char* what) {
  if (s == BSFA_OK) return;
  PyObject* api = PyImport_ImportModule("block_sparse_gated_gb300.api");
  if (api != nullptr) {
    PyObject* r = PyObject_CallMethod(api, "_check", "is", static_cast<int>(s), what);
    Py_XDECREF(r);
    Py_DECREF(api);
  }
  throw python_error();
}

// Strides {batch, head, token}, heads and tokens of 16-bit rows.
struct Rows {
  int64_t stride[3];
  int64_t heads, tokens;
};
Rows rows_of(const Tensor& t, const char* layout, bool varlen) {
  const auto size = t.sizes(), s = t.strides();
  const int dims = static_cast<int>(size.size());
  want(dims == 3 || (dims == 4 && !varlen), varlen ? "varlen tensors are 3-D"
                                                   : "batched tensors are 4-D");
  want(s[dims - 1] == 1, "the head dimension must be contiguous");
  if (dims == 3 && !varlen) return {{size[0] * s[0], s[0], s[1]}, size[0], size[1]};
  if (varlen) {
    want(is(layout, "htd") || is(layout, "thd"), "packed rows are \"htd\" or \"thd\"");
    if (is(layout, "htd")) return {{0, s[0], s[1]}, size[0], size[1]};
    return {{0, s[1], s[0]}, size[1], size[0]};
  }
  want(is(layout, "bhld") || is(layout, "blhd"), "batched rows are \"bhld\" or \"blhd\"");
  if (is(layout, "bhld")) return {{s[0], s[1], s[2]}, size[1], size[2]};
  return {{s[0], s[2], s[1]}, size[2], size[1]};
}
void set(int64_t (&to)[3], const Rows& r) {
  for (int i = 0; i < 3; ++i) to[i] = r.stride[i];
}

const int32_t* int32_vector(const Tensor& t, int64_t n, const at::Device& device,
                            const char* name) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be a contiguous int32 [" +
                                 std::to_string(n) + "] tensor");
  on_device(t, device, name);
  return static_cast<const int32_t*>(t.const_data_ptr());
}

// The pools and the block table of a call with `batch` sequences.
bsfa_cache16 cache_of(const Tensor& k, const Tensor& v, const char* layout, const Tensor& table,
                      int64_t batch, const at::Device& device) {
  want(k.dim() == 4, "page pools are 4-D");
  want(is(layout, "phtd") || is(layout, "pthd"), "the pools' layout is \"phtd\" or \"pthd\"");
  const int h = is(layout, "phtd") ? 1 : 2, t = 3 - h;
  bsfa_cache16 c{};
  c.dtype = dtype_code(k);
  if (v.scalar_type() != k.scalar_type())
    refuse(PyExc_TypeError, "page pools are bfloat16 or float16, both of one type");
  want(v.sizes() == k.sizes() && k.stride(3) == 1 && v.stride(3) == 1,
       "K and V pools must have one shape, with the head dimension contiguous");
  on_device(k, device, "cache.k");
  on_device(v, device, "cache.v");
  want(table.scalar_type() == at::kInt && table.dim() == 2 &&
           (table.stride(1) == 1 || table.size(1) <= 1),
       "block_table must be an int32 [batch, pages_per_sequence] tensor");
  want(table.size(0) >= batch, "block_table has fewer rows than sequences");
  on_device(table, device, "block_table");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  const int order[3] = {0, h, t};
  for (int i = 0; i < 3; ++i) {
    c.k_stride[i] = k.stride(order[i]);
    c.v_stride[i] = v.stride(order[i]);
  }
  c.num_pages = to_int(k.size(0));
  c.num_heads_kv = to_int(k.size(h));
  c.page_size = to_int(k.size(t));
  c.head_dim = to_int(k.size(3));
  c.block_table = static_cast<const int32_t*>(table.const_data_ptr());
  c.block_table_width = to_int(table.size(1));
  c.block_table_stride = table.size(0) > 1 ? to_int(table.stride(0)) : c.block_table_width;
  return c;
}

// A call's rows; any of q, k, v, q_out and k_out may be absent, but not both q and k.
// An output that the call makes itself is filled in later.
bsfa_rows16 rows_fields(const Tensor* q, const Tensor* k, const Tensor* v, const Tensor* q_out,
                        const Tensor* k_out, PyObject* layout_name, const Tensor* cu,
                        const Tensor* start, const at::Device& device) {
  const bool varlen = cu != nullptr;
  const char* layout = layout_of(layout_name, varlen ? "htd" : "bhld");
  const Tensor& one = k != nullptr ? *k : *q;
  bsfa_rows16 r{};
  r.dtype = dtype_code(one);
  std::optional<Rows> first;
  // (One tensor may be given twice, as queries and keys.)
  auto take = [&](const Tensor* t, const Tensor* like, int64_t (&stride)[3], int* heads) -> void* {
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != one.scalar_type())
      refuse(PyExc_TypeError, "all rows must share one element type");
    const Rows x = rows_of(*t, layout, varlen);
    if (like != nullptr) want(t->sizes() == like->sizes(), "tensors of one kind must have one shape");
    want(t->dim() == one.dim() && t->size(-1) == one.size(-1) &&
             (t->dim() == 3 || t->size(0) == one.size(0)) &&
             (!first || first->tokens == x.tokens),
         "Q, K and V shapes disagree");
    if (!first) first = x;
    on_device(*t, device, "a row tensor");
    set(stride, x);
    if (heads != nullptr) *heads = to_int(x.heads);
    return t->data_ptr();
  };
  r.q = take(q, nullptr, r.q_stride, &r.num_heads_q);
  r.k = take(k, nullptr, r.k_stride, &r.num_heads_kv);
  r.v = take(v, k, r.v_stride, nullptr);
  r.q_out = take(q_out, q, r.q_out_stride, nullptr);
  r.k_out = take(k_out, k, r.k_out_stride, nullptr);
  r.seqlen = to_int(first->tokens);
  r.head_dim = to_int(one.size(-1));
  if (varlen) {
    want(cu->scalar_type() == at::kInt && cu->dim() == 1 && cu->is_contiguous() && cu->numel() >= 1,
         "cu_seqlens must be a contiguous int32 [batch + 1] tensor");
    on_device(*cu, device, "cu_seqlens");
    r.batch = to_int(cu->numel() - 1);
    r.cu_seqlens = static_cast<const int32_t*>(cu->const_data_ptr());
  } else {
    r.batch = one.dim() == 3 ? 1 : to_int(one.size(0));
  }
  if (start != nullptr) r.start = int32_vector(*start, r.batch, device, "start");
  return r;
}

void out_of(const Tensor& t, PyObject* layout_name, bool varlen, void*& to, int64_t (&stride)[3]) {
  set(stride, rows_of(t, layout_of(layout_name, varlen ? "htd" : "bhld"), varlen));
  to = t.data_ptr();
}

// A rotation of these rows.
bsfa_rope rope_of(const Tensor& f, PyObject* axes, PyObject* interleaved, const Tensor* positions,
                  bool inverse, const bsfa_rows16& rows, const at::Device& device) {
  bsfa_rope p{};
  want(f.scalar_type() == at::kFloat && f.dim() == 1 && f.is_contiguous(),
       "inv_freq must be a contiguous float32 [pairs] tensor");
  want(f.numel() > 0 && f.numel() <= 64, "inv_freq must have 1 to 64 pairs");
  on_device(f, device, "inv_freq");
  p.inv_freq = static_cast<const float*>(f.const_data_ptr());
  p.pairs = static_cast<int>(f.numel());
  p.interleaved = truth(interleaved);
  p.inverse = inverse;
  p.num_axes = 1;
  if (axes != Py_None) {
    PyObject* seq = PySequence_Fast(axes, "axes must be a sequence");
    if (seq == nullptr) throw python_error();
    bool ok = PySequence_Fast_GET_SIZE(seq) == p.pairs;
    for (int j = 0; ok && j < p.pairs; ++j) {
      const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, j));
      ok = x >= 0 && x < BSFA_ROPE_MAX_AXES;
      p.axis[j] = static_cast<uint8_t>(x);
      if (ok && x >= p.num_axes) p.num_axes = static_cast<int>(x) + 1;
    }
    Py_DECREF(seq);
    if (PyErr_Occurred()) throw python_error();
    want(ok, "axes must name one of at most 4 axes for each pair");
  }
  if (positions != nullptr) {
    const bool varlen = rows.cu_seqlens != nullptr;
    const int64_t n = rows.seqlen, inner = varlen ? 1 : 2, dims = positions->dim();
    const int64_t axes_given = dims == inner + 1 ? positions->size(0) : 1;
    bool ok = (dims == inner && p.num_axes == 1) ||
              (dims == inner + 1 && axes_given >= p.num_axes && axes_given <= BSFA_ROPE_MAX_AXES);
    ok = ok && positions->size(-1) == n && (varlen || positions->size(-2) == rows.batch);
    if (!ok)
      refuse(PyExc_ValueError,
             "positions must be an int32 [axes, " +
                 (varlen ? "" : std::to_string(rows.batch) + ", ") + std::to_string(n) +
                 "] tensor");
    want(positions->scalar_type() == at::kInt && (positions->stride(-1) == 1 || n <= 1),
         "positions must be int32 with the positions of a sequence contiguous");
    on_device(*positions, device, "positions");
    p.positions = static_cast<const int32_t*>(positions->const_data_ptr());
    p.position_stride[0] = dims == inner + 1 ? positions->stride(0) : 0;
    p.position_stride[1] = varlen ? 0 : positions->stride(-2);
  }
  return p;
}

void arguments(Py_ssize_t got, Py_ssize_t expected) {
  if (got != expected) refuse(PyExc_TypeError, "wrong number of arguments");
}

// The same call as a node of the autograd graph, which calls back without recording.
PyObject* rotary_recorded(PyObject* const* a, Py_ssize_t n) {
  PyObject* m = PyImport_ImportModule("block_sparse_gated_gb300.cache16");
  if (m == nullptr) throw python_error();
  PyObject* f = PyObject_GetAttrString(m, "_rotary_recorded");
  Py_DECREF(m);
  if (f == nullptr) throw python_error();
  PyObject* r = PyObject_Vectorcall(f, a, n, nullptr);
  Py_DECREF(f);
  if (r == nullptr) throw python_error();
  return r;
}

// inv_freq, axes, interleaved, q, k, positions, start, cu_seqlens, layout, inverse, q_out, k_out,
// stream -> (q_out, k_out)
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 13);
  const Tensor &f = needed(a[0], "inv_freq"), &q = needed(a[3], "q");
  const Tensor *k = tensor(a[4], "k"), *positions = tensor(a[5], "positions");
  const Tensor *start = tensor(a[6], "start"), *cu = tensor(a[7], "cu_seqlens");
  const Tensor *q_out = tensor(a[10], "out"), *k_out = tensor(a[11], "out");
  const at::Device device = q.device();
  want(!recorded(&f), "inv_freq has no gradient");
  if (recorded(&q, k, q_out, k_out)) {
    want(q_out == nullptr && k_out == nullptr,
         "out has no gradient: leave it out, or call rotary under torch.no_grad()");
    return rotary_recorded(a, n);
  }
  want(q_out == nullptr ? k_out == nullptr : (k_out == nullptr) == (k == nullptr),
       "out must be a pair, with None where there is no k");
  want(k_out == nullptr || q_out->const_data_ptr() != k_out->const_data_ptr() || q.numel() == 0,
       "out must be a pair of two tensors");
  bsfa_rows16 r = rows_fields(&q, k, nullptr, q_out, k_out, a[8], cu, start, device);
  const bsfa_rope p = rope_of(f, a[1], a[2], positions, truth(a[9]), r, device);
  const Place place(device, a[12]);
  Tensor made_q, made_k;
  if (q_out == nullptr) {
    made_q = place.like(q);
    out_of(made_q, a[8], cu != nullptr, r.q_out, r.q_out_stride);
    if (k != nullptr) {
      made_k = place.like(*k);
      out_of(made_k, a[8], cu != nullptr, r.k_out, r.k_out_stride);
    }
  }
  check(bsfa_rotary(&p, &r, place.stream()), "bsfa_rotary");
  written(q_out);
  written(k_out);
  PyObject* first = q_out ? Py_NewRef(a[10]) : THPVariable_Wrap(made_q);
  PyObject* second = k_out ? Py_NewRef(a[11]) : k ? THPVariable_Wrap(made_k) : Py_NewRef(Py_None);
  return Py_BuildValue("NN", first, second);
  END_HANDLE_TH_ERRORS
}

// k pool, v pool, pool layout, k, v, block_table, inv_freq, axes, interleaved, q, positions,
// start, cu_seqlens, layout, q_out, stream -> q_out
PyObject* py_cache16_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 16);
  const Tensor &k = needed(a[3], "k"), &v = needed(a[4], "v");
  const Tensor *f = tensor(a[6], "inv_freq"), *q = tensor(a[9], "q");
  const Tensor *positions = tensor(a[10], "positions"), *start = tensor(a[11], "start");
  const Tensor *cu = tensor(a[12], "cu_seqlens"), *q_out = tensor(a[14], "q_out");
  const Tensor &k_pool = needed(a[0], "cache.k"), &v_pool = needed(a[1], "cache.v");
  const at::Device device = k.device();
  want(!recorded(&k, &v, q, q_out, f, &k_pool, &v_pool),
       "cache16_write records no gradient: call it under torch.no_grad()");
  want(q != nullptr || q_out == nullptr, "q_out without q");
  want(q == nullptr || f != nullptr, "q is only rotated: it needs a rope");
  want(positions == nullptr || f != nullptr, "positions without a rope");
  bsfa_rows16 r = rows_fields(q, &k, &v, q_out, nullptr, a[13], cu, start, device);
  const bsfa_cache16 c =
      cache_of(k_pool, v_pool, layout_of(a[2], "phtd"), needed(a[5], "block_table"), r.batch,
               device);
  want(c.num_heads_kv == r.num_heads_kv && c.head_dim == r.head_dim && c.dtype == r.dtype,
       "K and V must have the cache's heads, head dimension and type");
  bsfa_rope p{};
  if (f != nullptr) p = rope_of(*f, a[7], a[8], positions, false, r, device);
  const Place place(device, a[15]);
  Tensor made;
  if (q != nullptr && q_out == nullptr) {
    made = place.like(*q);
    out_of(made, a[13], cu != nullptr, r.q_out, r.q_out_stride);
  }
  check(bsfa_cache16_write(&c, f ? &p : nullptr, &r, place.stream()), "bsfa_cache16_write");
  for (const Tensor* t : {&k_pool, &v_pool, q_out}) written(t);
  if (q == nullptr) Py_RETURN_NONE;
  return q_out ? Py_NewRef(a[14]) : THPVariable_Wrap(made);
  END_HANDLE_TH_ERRORS
}

// The structs of a decode call, without its output and workspace.
struct Decode {
  bsfa_cache16 cache;
  bsfa_decode4_params p;
};
Decode decode_of(const Tensor& q, PyObject* const* pool, PyObject* seqlens, PyObject* max_seqlen,
                 const char* layout, const at::Device& device) {
  Decode d{};
  d.p.dtype = dtype_code(q);
  const Rows r = rows_of(q, layout, false);
  set(d.p.q_stride, r);
  d.p.q = q.data_ptr();
  d.p.batch = q.dim() == 3 ? 1 : to_int(q.size(0));
  d.p.num_heads_q = to_int(r.heads);
  d.p.q_len = to_int(r.tokens);
  d.cache = cache_of(needed(pool[0], "cache.k"), needed(pool[1], "cache.v"),
                     layout_of(pool[2], "phtd"), needed(pool[3], "block_table"), d.p.batch, device);
  want(q.size(-1) == d.cache.head_dim && d.cache.num_heads_kv > 0 &&
           d.p.num_heads_q % d.cache.num_heads_kv == 0 && d.p.dtype == d.cache.dtype,
       "q must have the cache's head dimension and type and a multiple of its heads");
  d.p.seqlens = int32_vector(needed(seqlens, "seqlens"), d.p.batch, device, "seqlens");
  const int64_t most = static_cast<int64_t>(d.cache.block_table_width) * d.cache.page_size;
  int64_t bound = most;
  if (max_seqlen != Py_None) {
    bound = PyLong_AsLongLong(max_seqlen);
    if (bound == -1 && PyErr_Occurred()) throw python_error();
    want(bound <= most, "block_table has too few pages per row for max_seqlen");
  }
  d.p.max_seqlen = to_int(bound);
  return d;
}

// q, k pool, v pool, pool layout, block_table, seqlens, max_seqlen, softmax_scale, causal, layout,
// out, return_lse, workspace, stream -> {"out": .., "lse": ..}
PyObject* py_decode16(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 14);
  const Tensor& q = needed(a[0], "q");
  const Tensor *out = tensor(a[10], "out"), *workspace = tensor(a[12], "workspace");
  const at::Device device = q.device();
  const char* layout = layout_of(a[9], "bhld");
  Decode d = decode_of(q, a + 1, a[5], a[6], layout, device);
  if (a[7] != Py_None) {
    d.p.softmax_scale = static_cast<float>(PyFloat_AsDouble(a[7]));
    if (PyErr_Occurred()) throw python_error();
  }
  d.p.causal = truth(a[8]);
  if (out != nullptr) {
    want(out->sizes() == q.sizes() && out->scalar_type() == q.scalar_type(),
         "q and out must have one shape and type");
    on_device(*out, device, "out");
  }
  if (workspace != nullptr) {
    want(workspace->is_contiguous(), "the workspace must be contiguous");
    on_device(*workspace, device, "workspace");
  }
  const Place place(device, a[13]);
  const Tensor o = out ? *out : place.like(q);
  set(d.p.o_stride, rows_of(o, layout, false));
  d.p.o = o.data_ptr();
  Tensor lse, scratch;
  if (truth(a[11])) {
    lse = place.empty({d.p.num_heads_q, static_cast<int64_t>(d.p.batch) * d.p.q_len}, at::kFloat);
    d.p.lse = static_cast<float*>(lse.data_ptr());
  }
  if (workspace != nullptr) {
    d.p.workspace = workspace->data_ptr();
    d.p.workspace_bytes = workspace->nbytes();
  } else if (const size_t need = bsfa_decode16_workspace_size(&d.cache, &d.p)) {
    scratch = place.empty({static_cast<int64_t>(need)}, at::kByte);
    d.p.workspace = scratch.data_ptr();
    d.p.workspace_bytes = need;
  }
  check(bsfa_decode16(&d.cache, &d.p, place.stream()), "bsfa_decode16");
  written(out);
  PyObject* first = out ? Py_NewRef(a[10]) : THPVariable_Wrap(o);
  if (!lse.defined()) return Py_BuildValue("{sN}", "out", first);
  return Py_BuildValue("{sNsN}", "out", first, "lse", THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

// q, k pool, v pool, pool layout, block_table, seqlens, max_seqlen, layout -> bytes
PyObject* py_decode16_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const Tensor& q = needed(a[0], "q");
  const Decode d = decode_of(q, a + 1, a[5], a[6], layout_of(a[7], "bhld"), q.device());
  return PyLong_FromSize_t(bsfa_decode16_workspace_size(&d.cache, &d.p));
  END_HANDLE_TH_ERRORS
}

#define BSFA_METHOD(name, function) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(function)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {BSFA_METHOD("rotary", py_rotary),
                         BSFA_METHOD("cache16_write", py_cache16_write),
                         BSFA_METHOD("decode16", py_decode16),
                         BSFA_METHOD("decode16_workspace", py_decode16_workspace),
                         {nullptr, nullptr, 0, nullptr}};
#undef BSFA_METHOD
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr) PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION);
  return m;
}
