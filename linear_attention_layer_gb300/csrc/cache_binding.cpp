// cache_binding.cpp -- the Python side of the cache calls (include/kda.h), for
// __init__.py: argument checks, outputs and workspace from torch's allocator, the
// device's current stream.
//
// A decode step makes these calls once a layer and each takes the GPU some
// microseconds; checked and marshalled in Python (ctypes) they took the host 23 to 28,
// most of it in attribute lookups and torch.empty.  Nothing is computed here.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>
#include <vector>

#include "../../include/kda.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// A refusal, raised as ValueError.
#define REFUSE(...)                                    \
  do {                                                 \
    std::ostringstream s_;                             \
    s_ << __VA_ARGS__;                                 \
    throw c10::ValueError({__func__, __FILE__, 0}, s_.str()); \
  } while (0)

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) REFUSE(name << " must be a tensor");
  return THPVariable_Unpack(o);
}

void on(const char* name, const Tensor& t, c10::Device dev) {
  if (t.device() != dev || !t.is_cuda()) REFUSE(name << " must be on " << dev << ", got " << t.device());
}

void typed(const char* name, const Tensor& t, ScalarType type, IntArrayRef shape, c10::Device dev) {
  on(name, t, dev);
  if (t.scalar_type() != type) REFUSE(name << " must be " << type << ", got " << t.scalar_type());
  if (t.sizes() != shape) REFUSE(name << " must have shape " << shape << ", got " << t.sizes());
}

// A contiguous argument.
template <typename P>
P* need(PyObject* o, const char* name, ScalarType type, IntArrayRef shape, c10::Device dev) {
  const Tensor& t = tensor(o, name);
  typed(name, t, type, shape, dev);
  if (!t.is_contiguous()) REFUSE(name << " must be contiguous");
  return static_cast<P*>(t.data_ptr());
}

// An output: the caller's, or a new one when it gave none.
template <typename P>
P* output(PyObject* o, const char* name, ScalarType type, IntArrayRef shape, c10::Device dev,
          Tensor& keep) {
  if (o == Py_None) {
    keep = at::detail::empty_cuda(shape, type, dev, std::nullopt);
  } else {
    need<P>(o, name, type, shape, dev);
    keep = THPVariable_Unpack(o);
  }
  return static_cast<P*>(keep.data_ptr());
}

int32_t io_code(ScalarType t) {
  if (t == ScalarType::Float) return KDA_F32;
  if (t == ScalarType::BFloat16) return KDA_BF16;
  REFUSE("q/k/v must be float32 or bfloat16, got " << t);
}

// [T, heads, channels] with strides; the channels contiguous.
const Tensor& rows(PyObject* o, const char* name, ScalarType type, IntArrayRef shape,
                   c10::Device dev) {
  const Tensor& t = tensor(o, name);
  typed(name, t, type, shape, dev);
  if (t.numel() > 0 && t.stride(2) != 1) REFUSE(name << "'s channels must be contiguous");
  return t;
}

// Token and head stride of t [T, heads, channels].  The stride of a dimension of one element
// says nothing (torch leaves any number there) and gives way to the packed one.
void outer_strides(const Tensor& t, int64_t* strides) {
  strides[0] = t.size(0) == 1 ? t.size(1) * t.size(2) : t.stride(0);
  strides[1] = t.size(1) == 1 ? t.size(2) : t.stride(1);
}

// The same of q.  Zeros mean "packed" to the C call, so a q broadcast over tokens or heads is
// refused: it would be read as the T heads channels elements that it does not have.
void query_strides(const Tensor& q, int64_t (&strides)[2]) {
  if (q.numel() == 0) return;  // not read
  outer_strides(q, strides);
  if (strides[0] == 0 || strides[1] == 0)
    REFUSE("q must not be broadcast over tokens or heads, got strides " << q.strides()
           << " of shape " << q.sizes());
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT32_MIN || v > INT32_MAX) REFUSE(name << " is out of range: " << v);
  return v;
}

c10::Device cache_struct(PyObject* cache, PyObject* k_exp, PyObject* v_exp, kda_cache_t& c) {
  const Tensor& t = tensor(cache, "cache");
  if (!t.is_cuda()) REFUSE("cache must be on a CUDA device, got " << t.device());
  if (t.dim() != 4 || t.size(3) % 18 != 0)
    REFUSE("cache must be uint8 [num_pages, kv heads, page_size / 16, 18 head_dim], got "
           << t.sizes());
  for (int i = 0; i < 4; ++i)
    if (t.size(i) > (1 << 30)) REFUSE("cache is too large: " << t.sizes());
  const c10::Device dev = t.device();
  c.pages = need<void>(cache, "cache", ScalarType::Byte, t.sizes(), dev);
  c.num_pages = (int32_t)t.size(0);
  c.num_kv_heads = (int32_t)t.size(1);
  c.page_size = (int32_t)(t.size(2) > 4096 ? -1 : t.size(2) * 16);
  c.head_dim = (int32_t)(t.size(3) / 18);
  const int64_t heads[] = {t.size(1)};
  c.k_exponent = k_exp == Py_None
                     ? nullptr
                     : need<int32_t>(k_exp, "k_exponent", ScalarType::Int, heads, dev);
  c.v_exponent = v_exp == Py_None
                     ? nullptr
                     : need<int32_t>(v_exp, "v_exponent", ScalarType::Int, heads, dev);
  return dev;
}

kda_stream_t stream_of(c10::Device dev) {
  return reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

void arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) REFUSE("expected " << want << " arguments, got " << n);
}

PyObject* status_object(int st) { return PyLong_FromLong(st); }

// A tuple of the tensors that are defined.
PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// Every function returns its outputs, or a kda_status_t when the call was refused.

PyObject* tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 12);
  const Tensor& held = tensor(a[0], "held_lens");
  if (!held.is_cuda()) REFUSE("held_lens must be on a CUDA device, got " << held.device());
  const c10::Device dev = held.device();
  const Tensor &table = tensor(a[3], "block_table"), &ring = tensor(a[4], "free_pages");
  if (table.dim() != 2) REFUSE("block_table must be [B, max_blocks]");
  const int64_t B = held.numel(), blocks = table.size(1), pages = ring.numel();
  if (B > INT32_MAX || blocks > INT32_MAX || pages > INT32_MAX)
    REFUSE("more requests, columns or pages than 32 bits count");
  const int64_t page_size = integer(a[6], "page_size"), cap = integer(a[7], "max_tokens");
  if (cap < 0) REFUSE("max_tokens must not be negative, got " << cap);
  const int64_t lens[] = {B}, cu_shape[] = {B + 1}, cap_shape[] = {cap}, two[] = {2},
                table_shape[] = {B, blocks}, ring_shape[] = {pages};
  constexpr ScalarType I = ScalarType::Int, L = ScalarType::Long;
  const int32_t* held_p = need<int32_t>(a[0], "held_lens", I, lens, dev);
  const int32_t* seq_p = need<int32_t>(a[1], "seq_lens", I, lens, dev);
  const int32_t* new_p = need<int32_t>(a[2], "new_lens", I, lens, dev);
  int32_t* table_p = need<int32_t>(a[3], "block_table", I, table_shape, dev);
  int32_t* ring_p = need<int32_t>(a[4], "free_pages", I, ring_shape, dev);
  const int64_t* span_p = need<int64_t>(a[5], "free_range", L, two, dev);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor kv, cu, slots, span;
  int32_t* kv_p = output<int32_t>(a[8], "kv_lens", I, lens, dev, kv);
  int32_t* cu_p = output<int32_t>(a[9], "cu_new", I, cu_shape, dev, cu);
  int64_t* slots_p = output<int64_t>(a[10], "slots", L, cap_shape, dev, slots);
  int64_t* out_p = output<int64_t>(a[11], "free_range_out", L, two, dev, span);
  const kda_status_t st = kda_cache_tables(
      (int32_t)page_size, (int32_t)B, (int32_t)blocks, (int32_t)cap, (int32_t)pages, held_p, seq_p,
      new_p, table_p, ring_p, span_p, out_p, kv_p, cu_p, slots_p, stream_of(dev));
  if (st != KDA_OK) return status_object(st);
  return tuple_of({kv, cu, slots, span});
  END_HANDLE_TH_ERRORS
}

// k, v, slots, cache, k_exponent, v_exponent
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 6);
  kda_cache_t c;
  const c10::Device dev = cache_struct(a[3], a[4], a[5], c);
  const int64_t T = tensor(a[2], "slots").numel();
  const int64_t shape[] = {T, c.num_kv_heads, c.head_dim}, slots_shape[] = {T};
  if (T > INT32_MAX) REFUSE("more tokens than 32 bits count");
  const ScalarType type = tensor(a[0], "k").scalar_type();
  const int32_t io = io_code(type);
  const Tensor &k = rows(a[0], "k", type, shape, dev), &v = rows(a[1], "v", type, shape, dev);
  const int64_t* slots = need<int64_t>(a[2], "slots", ScalarType::Long, slots_shape, dev);
  int64_t strides[4];
  outer_strides(k, strides);
  outer_strides(v, strides + 2);
  const c10::cuda::CUDAGuard guard(dev);
  return status_object(kda_cache_append(&c, io, (int32_t)T, k.data_ptr(), v.data_ptr(), strides,
                                        slots, stream_of(dev)));
  END_HANDLE_TH_ERRORS
}

// slots, cache, is_bf16, k_exponent, v_exponent, k, v
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 7);
  kda_cache_t c;
  const c10::Device dev = cache_struct(a[1], a[3], a[4], c);
  const ScalarType type = a[2] == Py_True ? ScalarType::BFloat16 : ScalarType::Float;
  const int64_t T = tensor(a[0], "slots").numel();
  if (T > INT32_MAX) REFUSE("more tokens than 32 bits count");
  const int64_t shape[] = {T, c.num_kv_heads, c.head_dim}, slots_shape[] = {T};
  const int64_t* slots = need<int64_t>(a[0], "slots", ScalarType::Long, slots_shape, dev);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor k, v;
  void* kp = output<void>(a[5], "k", type, shape, dev, k);
  void* vp = output<void>(a[6], "v", type, shape, dev, v);
  const kda_status_t st =
      kda_cache_read(&c, io_code(type), (int32_t)T, slots, kp, vp, stream_of(dev));
  if (st != KDA_OK) return status_object(st);
  return tuple_of({k, v});
  END_HANDLE_TH_ERRORS
}

// q, cache, block_table, kv_lens, cu_new, max_new, scale (or None), k_exponent, v_exponent,
// out, lse, want_lse, workspace (None: allocated here)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 13);
  const Tensor &q = tensor(a[0], "q"), &table = tensor(a[2], "block_table");
  if (q.dim() != 3 || table.dim() != 2)
    REFUSE("q must be [T, heads, head_dim] and block_table [B, max_blocks]");
  kda_attention_t d = {};
  query_strides(q, d.q_strides);
  kda_cache_t c;
  const c10::Device dev = cache_struct(a[1], a[7], a[8], c);
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2), blocks = table.size(1),
                B = tensor(a[3], "kv_lens").numel();
  if (D != c.head_dim || c.num_kv_heads <= 0 || H % c.num_kv_heads != 0)
    REFUSE("q " << q.sizes() << " does not fit a cache of " << c.num_kv_heads << " heads of "
                << c.head_dim << " channels");
  if (T > INT32_MAX || H > INT32_MAX || B > INT32_MAX || blocks > INT32_MAX)
    REFUSE("more tokens, heads, requests or columns than 32 bits count");
  const int64_t shape[] = {T, H, D}, table_shape[] = {B, blocks}, lens[] = {B}, cu_shape[] = {B + 1},
                lse_shape[] = {T, H};
  const ScalarType type = q.scalar_type();
  constexpr ScalarType I = ScalarType::Int;
  d.io_dtype = io_code(type);
  rows(a[0], "q", type, shape, dev);
  d.num_seqs = (int32_t)B;
  d.total_tokens = (int32_t)T;
  d.num_heads = (int32_t)H;
  d.max_new = (int32_t)integer(a[5], "max_new");
  d.max_blocks = (int32_t)blocks;
  if (a[6] == Py_None) {
    d.scale = (float)(1.0 / std::sqrt((double)D));
  } else {
    const double s = PyFloat_AsDouble(a[6]);
    if (s == -1.0 && PyErr_Occurred()) throw python_error();
    d.scale = (float)s;
  }
  const int32_t* table_p = need<int32_t>(a[2], "block_table", I, table_shape, dev);
  const int32_t* kv_p = need<int32_t>(a[3], "kv_lens", I, lens, dev);
  const int32_t* cu_p = need<int32_t>(a[4], "cu_new", I, cu_shape, dev);
  const c10::cuda::CUDAGuard guard(dev);
  size_t bytes = 0;
  kda_status_t st = kda_cache_attention_workspace_size(&c, &d, &bytes);
  if (st != KDA_OK) return status_object(st);
  Tensor out, lse, ws;
  void* out_p = output<void>(a[9], "out", type, shape, dev, out);
  const bool with_lse = a[11] == Py_True || a[10] != Py_None;
  float* lse_p =
      with_lse ? output<float>(a[10], "lse", ScalarType::Float, lse_shape, dev, lse) : nullptr;
  if (a[12] == Py_None) {
    const int64_t size[] = {(int64_t)bytes};
    ws = at::detail::empty_cuda(size, ScalarType::Byte, dev, std::nullopt);
  } else {
    ws = tensor(a[12], "workspace");
    const int64_t size[] = {ws.numel()};
    need<void>(a[12], "workspace", ScalarType::Byte, size, dev);
  }
  d.workspace = ws.data_ptr();
  d.workspace_bytes = (size_t)ws.numel();
  st = kda_cache_attention(&c, &d, q.data_ptr(), table_p, kv_p, cu_p, out_p, lse_p, stream_of(dev));
  if (st != KDA_OK) return status_object(st);
  if (a[11] == Py_True) return tuple_of({out, lse});
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// A cache of the 8-bit form.
c10::Device byte_cache_struct(PyObject* cache, kda_byte_cache_t& c) {
  const Tensor& t = tensor(cache, "cache");
  if (!t.is_cuda()) REFUSE("cache must be on a CUDA device, got " << t.device());
  if (t.dim() != 4 || t.size(3) % 32 != 16)
    REFUSE("cache must be uint8 [num_pages, kv heads, page_size / 16, 32 head_dim + 16], got "
           << t.sizes());
  for (int i = 0; i < 4; ++i)
    if (t.size(i) > (1 << 30)) REFUSE("cache is too large: " << t.sizes());
  c.pages = need<void>(cache, "cache", ScalarType::Byte, t.sizes(), t.device());
  c.num_pages = (int32_t)t.size(0);
  c.num_kv_heads = (int32_t)t.size(1);
  c.page_size = (int32_t)(t.size(2) > 4096 ? -1 : t.size(2) * 16);
  c.head_dim = (int32_t)(t.size(3) / 32);
  return t.device();
}

// k, v, slots, cache
PyObject* append8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 4);
  kda_byte_cache_t c;
  const c10::Device dev = byte_cache_struct(a[3], c);
  const int64_t T = tensor(a[2], "slots").numel();
  const int64_t shape[] = {T, c.num_kv_heads, c.head_dim}, slots_shape[] = {T};
  if (T > INT32_MAX) REFUSE("more tokens than 32 bits count");
  const ScalarType type = tensor(a[0], "k").scalar_type();
  const int32_t io = io_code(type);
  const Tensor &k = rows(a[0], "k", type, shape, dev), &v = rows(a[1], "v", type, shape, dev);
  const int64_t* slots = need<int64_t>(a[2], "slots", ScalarType::Long, slots_shape, dev);
  int64_t strides[4];
  outer_strides(k, strides);
  outer_strides(v, strides + 2);
  const c10::cuda::CUDAGuard guard(dev);
  return status_object(kda_byte_cache_append(&c, io, (int32_t)T, k.data_ptr(), v.data_ptr(), strides,
                                         slots, stream_of(dev)));
  END_HANDLE_TH_ERRORS
}

// slots, cache, is_bf16, k, v
PyObject* read8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 5);
  kda_byte_cache_t c;
  const c10::Device dev = byte_cache_struct(a[1], c);
  const ScalarType type = a[2] == Py_True ? ScalarType::BFloat16 : ScalarType::Float;
  const int64_t T = tensor(a[0], "slots").numel();
  if (T > INT32_MAX) REFUSE("more tokens than 32 bits count");
  const int64_t shape[] = {T, c.num_kv_heads, c.head_dim}, slots_shape[] = {T};
  const int64_t* slots = need<int64_t>(a[0], "slots", ScalarType::Long, slots_shape, dev);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor k, v;
  void* kp = output<void>(a[3], "k", type, shape, dev, k);
  void* vp = output<void>(a[4], "v", type, shape, dev, v);
  const kda_status_t st =
      kda_byte_cache_read(&c, io_code(type), (int32_t)T, slots, kp, vp, stream_of(dev));
  if (st != KDA_OK) return status_object(st);
  return tuple_of({k, v});
  END_HANDLE_TH_ERRORS
}

// Device scratch: the caller's, or new when it gave none.
void* scratch(PyObject* o, size_t bytes, c10::Device dev, Tensor& keep, size_t& have) {
  if (o == Py_None) {
    const int64_t size[] = {(int64_t)bytes};
    keep = at::detail::empty_cuda(size, ScalarType::Byte, dev, std::nullopt);
  } else {
    keep = tensor(o, "workspace");
    const int64_t size[] = {keep.numel()};
    need<void>(o, "workspace", ScalarType::Byte, size, dev);
  }
  have = (size_t)keep.numel();
  return keep.data_ptr();
}

// The same over the 8-bit form: q, cache, block_table, kv_lens, cu_new, max_new, scale (or None),
// out, lse, want_lse, workspace (None: allocated here)
PyObject* attention8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 11);
  const Tensor &q = tensor(a[0], "q"), &table = tensor(a[2], "block_table");
  if (q.dim() != 3 || table.dim() != 2)
    REFUSE("q must be [T, heads, head_dim] and block_table [B, max_blocks]");
  kda_attention_t d = {};
  query_strides(q, d.q_strides);
  kda_byte_cache_t c;
  const c10::Device dev = byte_cache_struct(a[1], c);
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2), blocks = table.size(1),
                B = tensor(a[3], "kv_lens").numel();
  if (D != c.head_dim || c.num_kv_heads <= 0 || H % c.num_kv_heads != 0)
    REFUSE("q " << q.sizes() << " does not fit a cache of " << c.num_kv_heads << " heads of "
                << c.head_dim << " channels");
  if (T > INT32_MAX || H > INT32_MAX || B > INT32_MAX || blocks > INT32_MAX)
    REFUSE("more tokens, heads, requests or columns than 32 bits count");
  const int64_t shape[] = {T, H, D}, table_shape[] = {B, blocks}, lens[] = {B}, cu_shape[] = {B + 1},
                lse_shape[] = {T, H};
  const ScalarType type = q.scalar_type();
  constexpr ScalarType I = ScalarType::Int;
  d.io_dtype = io_code(type);
  rows(a[0], "q", type, shape, dev);
  d.num_seqs = (int32_t)B;
  d.total_tokens = (int32_t)T;
  d.num_heads = (int32_t)H;
  d.max_new = (int32_t)integer(a[5], "max_new");
  d.max_blocks = (int32_t)blocks;
  if (a[6] == Py_None) {
    d.scale = (float)(1.0 / std::sqrt((double)D));
  } else {
    const double s = PyFloat_AsDouble(a[6]);
    if (s == -1.0 && PyErr_Occurred()) throw python_error();
    d.scale = (float)s;
  }
  const int32_t* table_p = need<int32_t>(a[2], "block_table", I, table_shape, dev);
  const int32_t* kv_p = need<int32_t>(a[3], "kv_lens", I, lens, dev);
  const int32_t* cu_p = need<int32_t>(a[4], "cu_new", I, cu_shape, dev);
  const c10::cuda::CUDAGuard guard(dev);
  size_t bytes = 0;
  kda_status_t st = kda_byte_cache_attention_workspace_size(&c, &d, &bytes);
  if (st != KDA_OK) return status_object(st);
  Tensor out, lse, ws;
  void* out_p = output<void>(a[7], "out", type, shape, dev, out);
  const bool with_lse = a[9] == Py_True || a[8] != Py_None;
  float* lse_p =
      with_lse ? output<float>(a[8], "lse", ScalarType::Float, lse_shape, dev, lse) : nullptr;
  d.workspace = scratch(a[10], bytes, dev, ws, d.workspace_bytes);
  st = kda_byte_cache_attention(&c, &d, q.data_ptr(), table_p, kv_p, cu_p, out_p, lse_p, stream_of(dev));
  if (st != KDA_OK) return status_object(st);
  if (a[9] == Py_True) return tuple_of({out, lse});
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// Small outputs out of one allocation, which costs the host most of a microsecond each: the
// caller's where it gave one, else a piece of `room`, made large enough for all that follow.
struct Pieces {
  c10::Device dev;
  size_t bytes;  // of all pieces, each rounded up to 16
  Tensor room;
  size_t used = 0;
  template <typename P>
  P* output(PyObject* o, const char* name, ScalarType type, IntArrayRef shape, Tensor& keep) {
    if (o != Py_None) {
      need<P>(o, name, type, shape, dev);
      keep = THPVariable_Unpack(o);
      return static_cast<P*>(keep.data_ptr());
    }
    if (!room.defined()) {
      const int64_t size[] = {(int64_t)bytes};
      room = at::detail::empty_cuda(size, ScalarType::Byte, dev, std::nullopt);
    }
    keep = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(room.storage()), room.key_set(),
                                                    c10::scalarTypeToTypeMeta(type));
    keep.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    keep.unsafeGetTensorImpl()->set_storage_offset((int64_t)(used / sizeof(P)));
    used += ((size_t)keep.numel() * sizeof(P) + 15) / 16 * 16;
    return static_cast<P*>(keep.data_ptr());
  }
};

// held_lens, block_table, parents, keep_lens, free_pages, free_range, page_size, num_pages,
// kv_lens, block_table_out, copies, free_range_out, workspace (None: allocated here)
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 13);
  const Tensor& held = tensor(a[0], "held_lens");
  if (!held.is_cuda()) REFUSE("held_lens must be on a CUDA device, got " << held.device());
  const c10::Device dev = held.device();
  const Tensor &table = tensor(a[1], "block_table"), &ring = tensor(a[4], "free_pages");
  if (table.dim() != 2) REFUSE("block_table must be [B, max_blocks]");
  const int64_t B = held.numel(), R = tensor(a[2], "parents").numel(), blocks = table.size(1),
                cap = ring.numel();
  if (B > INT32_MAX || R > INT32_MAX || blocks > INT32_MAX || cap > INT32_MAX)
    REFUSE("more requests, columns or pages than 32 bits count");
  const int64_t page_size = integer(a[6], "page_size"), pages = integer(a[7], "num_pages");
  const int64_t old_lens[] = {B}, lens[] = {R}, table_shape[] = {B, blocks},
                out_shape[] = {R, blocks}, ring_shape[] = {cap}, two[] = {2}, three[] = {R, 3};
  constexpr ScalarType I = ScalarType::Int, L = ScalarType::Long;
  const int32_t* held_p = need<int32_t>(a[0], "held_lens", I, old_lens, dev);
  const int32_t* table_p = need<int32_t>(a[1], "block_table", I, table_shape, dev);
  const int32_t* parents_p = need<int32_t>(a[2], "parents", I, lens, dev);
  const int32_t* keep_p = need<int32_t>(a[3], "keep_lens", I, lens, dev);
  int32_t* ring_p = need<int32_t>(a[4], "free_pages", I, ring_shape, dev);
  const int64_t* span_p = need<int64_t>(a[5], "free_range", L, two, dev);
  const c10::cuda::CUDAGuard guard(dev);
  size_t bytes = 0, have = 0;
  kda_status_t st = kda_cache_fork_workspace_size((int32_t)pages, (int32_t)R, &bytes);
  if (st != KDA_OK) return status_object(st);
  Tensor kv, out, copies, span, ws;
  Pieces pieces{dev, (size_t)(16 * R + 64), {}};
  int64_t* span_out = pieces.output<int64_t>(a[11], "free_range_out", L, two, span);
  int32_t* kv_p = pieces.output<int32_t>(a[8], "kv_lens", I, lens, kv);
  int32_t* copies_p = pieces.output<int32_t>(a[10], "copies", I, three, copies);
  int32_t* out_p = output<int32_t>(a[9], "block_table_out", I, out_shape, dev, out);
  void* ws_p = scratch(a[12], bytes, dev, ws, have);
  st = kda_cache_fork((int32_t)page_size, (int32_t)pages, (int32_t)B, (int32_t)R, (int32_t)blocks,
                      (int32_t)cap, held_p, table_p, parents_p, keep_p, ring_p, span_p, span_out,
                      kv_p, out_p, copies_p, ws_p, have, stream_of(dev));
  if (st != KDA_OK) return status_object(st);
  return tuple_of({kv, out, copies, span});
  END_HANDLE_TH_ERRORS
}

// held_lens, block_table, free_pages, page_size, num_pages, block_table_out, copies,
// free_range_out, workspace (None: allocated here)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 9);
  const Tensor& held = tensor(a[0], "held_lens");
  if (!held.is_cuda()) REFUSE("held_lens must be on a CUDA device, got " << held.device());
  const c10::Device dev = held.device();
  const Tensor &table = tensor(a[1], "block_table"), &ring = tensor(a[2], "free_pages");
  if (table.dim() != 2) REFUSE("block_table must be [B, max_blocks]");
  const int64_t B = held.numel(), blocks = table.size(1), cap = ring.numel();
  if (B > INT32_MAX || blocks > INT32_MAX || cap > INT32_MAX)
    REFUSE("more requests, columns or pages than 32 bits count");
  const int64_t page_size = integer(a[3], "page_size"), pages = integer(a[4], "num_pages");
  if (pages < 0) REFUSE("num_pages must not be negative, got " << pages);
  const int64_t lens[] = {B}, table_shape[] = {B, blocks}, ring_shape[] = {cap}, two[] = {2},
                moves[] = {pages / 2, 3};
  constexpr ScalarType I = ScalarType::Int, L = ScalarType::Long;
  const int32_t* held_p = need<int32_t>(a[0], "held_lens", I, lens, dev);
  const int32_t* table_p = need<int32_t>(a[1], "block_table", I, table_shape, dev);
  int32_t* ring_p = need<int32_t>(a[2], "free_pages", I, ring_shape, dev);
  const c10::cuda::CUDAGuard guard(dev);
  size_t bytes = 0, have = 0;
  kda_status_t st = kda_cache_compact_workspace_size((int32_t)pages, &bytes);
  if (st != KDA_OK) return status_object(st);
  Tensor out, copies, span, ws;
  Pieces pieces{dev, (size_t)(12 * moves[0] + 48), {}};
  int64_t* span_p = pieces.output<int64_t>(a[7], "free_range_out", L, two, span);
  int32_t* copies_p = pieces.output<int32_t>(a[6], "copies", I, moves, copies);
  int32_t* out_p = output<int32_t>(a[5], "block_table_out", I, table_shape, dev, out);
  void* ws_p = scratch(a[8], bytes, dev, ws, have);
  st = kda_cache_compact((int32_t)page_size, (int32_t)pages, (int32_t)B, (int32_t)blocks,
                         (int32_t)cap, held_p, table_p, out_p, copies_p, ring_p, span_p, ws_p,
                         have, stream_of(dev));
  if (st != KDA_OK) return status_object(st);
  return tuple_of({out, copies, span});
  END_HANDLE_TH_ERRORS
}

// caches (a tuple of tensors of one shape), copies
PyObject* copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 2);
  const Tensor& copies = tensor(a[1], "copies");
  if (!copies.is_cuda()) REFUSE("copies must be on a CUDA device, got " << copies.device());
  const c10::Device dev = copies.device();
  const int64_t shape[] = {copies.numel() / 3, 3};
  const int32_t* copies_p = need<int32_t>(a[1], "copies", ScalarType::Int, shape, dev);
  if (shape[0] > INT32_MAX) REFUSE("more copies than 32 bits count");
  const Py_ssize_t layers = PyTuple_Size(a[0]);
  if (layers < 0) throw python_error();
  if (layers == 0) return status_object(KDA_OK);
  std::vector<void*> pages((size_t)layers);
  const Tensor& first = tensor(PyTuple_GET_ITEM(a[0], 0), "cache");
  if (first.dim() != 4)
    REFUSE("cache must be uint8 [num_pages, kv heads, page_size / 16, bytes], got "
           << first.sizes());
  for (int i = 0; i < 4; ++i)
    if (first.size(i) > (1 << 30)) REFUSE("cache is too large: " << first.sizes());
  const std::vector<int64_t> sizes = first.sizes().vec();
  for (Py_ssize_t i = 0; i < layers; ++i)
    pages[(size_t)i] =
        need<void>(PyTuple_GET_ITEM(a[0], i), "cache", ScalarType::Byte, sizes, dev);
  const c10::cuda::CUDAGuard guard(dev);
  return status_object(kda_cache_copy(
      (int32_t)layers, pages.data(), (int32_t)sizes[0], (int32_t)sizes[1],
      (int32_t)(sizes[2] > 4096 ? -1 : sizes[2] * 16), (int32_t)sizes[3], (int32_t)shape[0],
      copies_p, stream_of(dev)));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"tables", (PyCFunction)(void (*)())tables, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
    {"read", (PyCFunction)(void (*)())read, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)())attention, METH_FASTCALL, nullptr},
    {"append8", (PyCFunction)(void (*)())append8, METH_FASTCALL, nullptr},
    {"read8", (PyCFunction)(void (*)())read8, METH_FASTCALL, nullptr},
    {"attention8", (PyCFunction)(void (*)())attention8, METH_FASTCALL, nullptr},
    {"fork", (PyCFunction)(void (*)())fork, METH_FASTCALL, nullptr},
    {"compact", (PyCFunction)(void (*)())compact, METH_FASTCALL, nullptr},
    {"copy", (PyCFunction)(void (*)())copy, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, methods,
                      nullptr,               nullptr,          nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding() { return PyModule_Create(&module); }
