// The Python side of the calls whose device time is a few microseconds
// (cp_qk_norm_rope, cp_qk_norm_rope_bwd, cp_paged_append, cp_paged_attn_decode,
// cp_packed_attn_fwd, cp_packed_attn_bwd): a Python extension that checks torch tensors, allocates
// outputs where none are given, and calls the C ABI.  It computes nothing.
// Against the same checks in Python over ctypes a call's host side fell from
// 24 to 6.5 us (norm and rotation), 41 to 12.5 (its backward), 21 to 4.3 (append) and 33
// to 10 (decode).
#include <ATen/ATen.h>
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <climits>
#include <cstdint>

#include "../../include/cpring.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // the package's CpError(function, status)

void check(const char* fn, cp_status st) {
  if (st == CP_OK) return;
  PyObject* const e = PyObject_CallFunction(g_error, "si", fn, static_cast<int>(st));
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

// An operand, or null for None.
const Tensor* given(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch.Tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& needed(PyObject* o, const char* name) {
  const Tensor* const t = given(o, name);
  TORCH_CHECK_TYPE(t != nullptr, name, " must be a torch.Tensor");
  return *t;
}
const Tensor& rows4(PyObject* o, const char* name) {
  const Tensor& t = needed(o, name);
  TORCH_CHECK_VALUE(t.dim() == 4, name, " must be a tensor of four dimensions");
  return t;
}

int device_of(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must live on a CUDA device");
  return t.get_device();
}

// t's address, after checking its type, device and shape, and that its last
// dimension is contiguous.
void* operand(const Tensor& t, const char* name, at::ScalarType type, int dev,
              at::IntArrayRef shape) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == dev, name, " must live on cuda:", dev,
                    ", got ", t.device());
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
  TORCH_CHECK_VALUE(t.dim() == 0 || t.size(-1) <= 1 || t.stride(-1) == 1, name,
                    " must be contiguous in its last dimension");
  return t.data_ptr();
}
void* dense(const Tensor& t, const char* name, at::ScalarType type, int dev,
            at::IntArrayRef shape) {
  void* const at = operand(t, name, type, dev, shape);
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return at;
}
template <typename T>
T* dense_or_null(PyObject* o, const char* name, at::ScalarType type, int dev,
                 at::IntArrayRef shape) {
  const Tensor* const t = given(o, name);
  return t ? static_cast<T*>(dense(*t, name, type, dev, shape)) : nullptr;
}
float* floats(PyObject* o, const char* name, int dev, int64_t n) {
  return dense_or_null<float>(o, name, at::kFloat, dev, {n});
}

// The three leading strides of [a, b, c, d]; the stride of a dimension of one
// entry is never used and passed as 0.
struct Steps {
  int64_t v[3];
  bool dense = true;
  explicit Steps(const Tensor* t) {
    if (t == nullptr || (dense = t->is_contiguous())) return;
    for (int i = 0; i < 3; ++i) v[i] = t->size(i) > 1 ? t->stride(i) : 0;
  }
  const int64_t* get() const { return dense ? nullptr : v; }
};

int to_int(int64_t n, const char* name) {
  TORCH_CHECK_VALUE(n >= 0 && n <= INT_MAX, name, " is too large");
  return static_cast<int>(n);
}

float to_float(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}

bool to_bool(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x != 0;
}

// The stream that a call runs on: None is the device's current one, otherwise a
// torch.cuda.Stream of that device or a raw handle.
cudaStream_t stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  THPObjectPtr raw;
  if (!PyLong_Check(o)) {
    THPObjectPtr index(PyObject_GetAttrString(o, "device_index"));
    if (!index) throw python_error();
    const long of = PyLong_AsLong(index.get());
    if (of == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(of == dev, "stream belongs to cuda:", of, ", the tensors to cuda:", dev);
    raw = PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) throw python_error();
    o = raw.get();
  }
  const unsigned long long h = PyLong_AsUnsignedLongLong(o);
  if (h == static_cast<unsigned long long>(-1) && PyErr_Occurred()) throw python_error();
  return reinterpret_cast<cudaStream_t>(h);
}

void arity(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// The stream that a call runs on, made torch's current one while the call's own
// tensors are made: the allocator hands a block to the stream that it was made for,
// and takes it back in that stream's order.  On another stream a workspace that
// the call drops could be given away while the kernels still use it, and an output
// be a block that the other stream's work still writes.
class Home {
 public:
  Home(PyObject* o, int dev)
      : caller_(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev))),
        stream_(stream_of(o, dev)) {
    if (stream_ == caller_.stream()) return;
    // The handle 1 is the default stream under another name; torch knows it as 0.
    const cudaStream_t known = stream_ == cudaStreamLegacy ? nullptr : stream_;
    guard_.reset_stream(
        c10::cuda::getStreamFromExternal(known, static_cast<c10::DeviceIndex>(dev)));
  }
  cudaStream_t get() const { return stream_; }
  // An output made here goes to the caller, whose current stream may use it too.
  void hand_over(const Tensor& t, bool made) const {
    if (made && t.defined() && guard_.current_stream()) t.record_stream(caller_.unwrap());
  }

 private:
  c10::cuda::CUDAStream caller_;
  cudaStream_t stream_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};

template <class F>
void run(const char* name, int dev, F&& call) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  cp_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  check(name, st);
}

PyObject* wrap(const Tensor* t) {
  if (t == nullptr || !t->defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}
PyObject* tuple_of(std::initializer_list<const Tensor*> ts) {
  THPObjectPtr r(PyTuple_New(static_cast<Py_ssize_t>(ts.size())));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* const o = wrap(t);
    if (o == nullptr) throw python_error();
    PyTuple_SET_ITEM(r.get(), i++, o);
  }
  return r.release();
}

// An output: the caller's, or a new contiguous one like `t`.
Tensor output(PyObject* o, const char* name, const Tensor& t) {
  const Tensor* const x = given(o, name);
  return x ? *x : at::empty(t.sizes(), t.options());
}

at::ScalarType rows_type(const Tensor& q) {
  const at::ScalarType t = q.scalar_type();
  TORCH_CHECK_TYPE(t == at::kBFloat16 || t == at::kFloat, "q must be bf16 or fp32");
  return t;
}

int rotated(const Tensor* inv_freq) {
  return inv_freq ? to_int(2 * inv_freq->numel(), "inv_freq") : 0;
}

// (q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, eps, interleaved, stream)
// -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 11);
  const Tensor& q = rows4(a[0], "q");
  const int dev = device_of(q, "q");
  const Home home(a[10], dev);
  const at::ScalarType type = rows_type(q);
  const int B = to_int(q.size(0), "q"), S = to_int(q.size(1), "q"), Hq = to_int(q.size(2), "q"),
            d = to_int(q.size(3), "q");
  const void* const q_at = operand(q, "q", type, dev, q.sizes());
  Tensor q_out = output(a[6], "q_out", q), k_out;
  void* const qo_at = dense(q_out, "q_out", type, dev, q.sizes());
  const Tensor* const k = a[1] == Py_None ? nullptr : &rows4(a[1], "k");
  int Hk = 0;
  const void* k_at = nullptr;
  void* ko_at = nullptr;
  if (k) {
    Hk = to_int(k->size(2), "k");
    k_at = operand(*k, "k", type, dev, {B, S, Hk, d});
    k_out = output(a[7], "k_out", *k);
    ko_at = dense(k_out, "k_out", type, dev, k->sizes());
  }
  const float* const qw = floats(a[2], "q_weight", dev, d);
  const float* const kw = floats(a[3], "k_weight", dev, d);
  const int rot = rotated(given(a[4], "inv_freq"));
  const float* const freq = floats(a[4], "inv_freq", dev, rot / 2);
  const int32_t* const pos = dense_or_null<int32_t>(a[5], "positions", at::kInt, dev, {B, S});
  const float eps = to_float(a[8]);
  const bool pairs = to_bool(a[9]);
  const Steps qs(&q), ks(k);
  run("cp_qk_norm_rope", dev, [&] {
    return cp_qk_norm_rope(q_at, qs.get(), k_at, ks.get(), qw, kw, eps, freq, rot, pairs, pos,
                           qo_at, ko_at, B, S, Hq, Hk, d, type == at::kBFloat16, home.get());
  });
  home.hand_over(q_out, a[6] == Py_None);
  home.hand_over(k_out, a[7] == Py_None);
  return tuple_of({&q_out, &k_out});
  END_HANDLE_TH_ERRORS
}

// (dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, positions, dq, dk, dq_weight, dk_weight,
//  eps, interleaved, workspace, stream, allocate) -> (dq, dk, dq_weight, dk_weight)
// allocate: outputs that are None are made, where their operand is there.
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 17);
  const Tensor& q = rows4(a[2], "q");
  const int dev = device_of(q, "q");
  const Home home(a[15], dev);
  const at::ScalarType type = rows_type(q);
  const int B = to_int(q.size(0), "q"), S = to_int(q.size(1), "q"), Hq = to_int(q.size(2), "q"),
            d = to_int(q.size(3), "q");
  const bool allocate = to_bool(a[16]);
  const void* const q_at = operand(q, "q", type, dev, q.sizes());
  const void* const dqo_at = dense(needed(a[0], "dq_out"), "dq_out", type, dev, q.sizes());
  Tensor dq = allocate ? output(a[8], "dq", q) : needed(a[8], "dq");
  void* const dq_at = operand(dq, "dq", type, dev, q.sizes());
  const Tensor* const k = a[3] == Py_None ? nullptr : &rows4(a[3], "k");
  int Hk = 0;
  const void *k_at = nullptr, *dko_at = nullptr;
  void* dk_at = nullptr;
  Tensor dk;
  if (k) {
    Hk = to_int(k->size(2), "k");
    k_at = operand(*k, "k", type, dev, {B, S, Hk, d});
    dko_at = dense(needed(a[1], "dk_out"), "dk_out", type, dev, k->sizes());
    dk = allocate ? output(a[9], "dk", *k) : needed(a[9], "dk");
    dk_at = operand(dk, "dk", type, dev, k->sizes());
  }
  const float* const qw = floats(a[4], "q_weight", dev, d);
  const float* const kw = floats(a[5], "k_weight", dev, d);
  const int rot = rotated(given(a[6], "inv_freq"));
  const float* const freq = floats(a[6], "inv_freq", dev, rot / 2);
  const int32_t* const pos = dense_or_null<int32_t>(a[7], "positions", at::kInt, dev, {B, S});
  Tensor dw[2];
  float* dw_at[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i) {
    const char* const name = i ? "dk_weight" : "dq_weight";
    const Tensor* const x = given(a[10 + i], name);
    if (x)
      dw[i] = *x;
    else if (allocate && (i ? kw != nullptr && k != nullptr : qw != nullptr))
      dw[i] = at::empty({d}, q.options().dtype(at::kFloat));
    if (dw[i].defined()) dw_at[i] = static_cast<float*>(dense(dw[i], name, at::kFloat, dev, {d}));
  }
  const float eps = to_float(a[12]);
  const bool pairs = to_bool(a[13]);
  const Tensor* const ws_given = given(a[14], "workspace");
  Tensor ws;
  if (ws_given) {
    ws = *ws_given;
  } else {
    const int64_t need = cp_qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hk, d);
    if (need < 0) check("cp_qk_norm_rope_bwd_workspace_bytes", CP_ERR_SHAPE);
    ws = at::empty({need}, q.options().dtype(at::kByte));
  }
  void* const ws_at = dense(ws, "workspace", at::kByte, dev, ws.sizes());
  const Steps qs(&q), ks(k), dqs(&dq), dks(k ? &dk : nullptr);
  run("cp_qk_norm_rope_bwd", dev, [&] {
    return cp_qk_norm_rope_bwd(dqo_at, dko_at, q_at, qs.get(), k_at, ks.get(), qw, kw, eps, freq,
                               rot, pairs, pos, dq_at, dqs.get(), dk_at, dks.get(), dw_at[0],
                               dw_at[1], B, S, Hq, Hk, d, type == at::kBFloat16, ws_at,
                               ws.numel(), home.get());
  });
  home.hand_over(dq, a[8] == Py_None);
  home.hand_over(dk, a[9] == Py_None);
  for (int i = 0; i < 2; ++i) home.hand_over(dw[i], a[10 + i] == Py_None);
  return tuple_of({&dq, &dk, &dw[0], &dw[1]});
  END_HANDLE_TH_ERRORS
}

// The strides of a cache tensor's pages, tokens and heads, in its elements.
void cache_strides(const Tensor& t, int64_t (&to)[3]) {
  for (int i = 0; i < 3; ++i) to[i] = t.size(i) > 1 ? t.stride(i) : 0;
}

// The cache of caches [pages, page_size, Hk, d] (bf16, or E4M3 with fp32 [Hk]
// descales; with scales [pages, page_size, Hk, d / 16], codes in 4 bits [pages,
// page_size, Hk, d / 2]) and an int32 table [B, max_pages].
cp_paged_cache cache_of(PyObject* ko, PyObject* vo, PyObject* to, PyObject* kdo, PyObject* vdo,
                        PyObject* kso, PyObject* vso, int64_t B, int dev) {
  const Tensor& k = rows4(ko, "k_cache");
  const at::ScalarType type = k.scalar_type();
  const bool int4 = kso != Py_None || vso != Py_None;
  const bool e4m3 = !int4 && (type == at::kByte || type == at::kFloat8_e4m3fn);
  if (int4) {
    TORCH_CHECK_TYPE(type == at::kByte, "k_cache must be uint8 (two codes a byte) with k_scale");
  } else {
    TORCH_CHECK_TYPE(e4m3 || type == at::kBFloat16,
                     "k_cache must be bf16, or E4M3 (float8_e4m3fn, or its codes as uint8)");
  }
  const Tensor& v = needed(vo, "v_cache");
  const Tensor& table = needed(to, "page_table");
  cp_paged_cache c{};
  c.k = operand(k, "k_cache", type, dev, k.sizes());
  c.v = operand(v, "v_cache", type, dev, k.sizes());
  TORCH_CHECK_VALUE(table.dim() == 2, "page_table must have two dimensions");
  TORCH_CHECK_VALUE(table.size(0) == B, "page_table must have ", B, " rows, got ", table.size(0));
  c.page_table = static_cast<const int32_t*>(
      operand(table, "page_table", at::kInt, dev, table.sizes()));
  c.n_pages = to_int(k.size(0), "k_cache");
  c.page_size = to_int(k.size(1), "k_cache");
  c.Hk = to_int(k.size(2), "k_cache");
  c.d = to_int(int4 ? 2 * k.size(3) : k.size(3), "k_cache");
  c.max_pages = to_int(table.size(1), "page_table");
  c.table_stride = B > 1 ? table.stride(0) : c.max_pages;
  c.elem_bytes = int4 ? -2 : e4m3 ? 1 : 2;
  if (int4) {
    const int64_t shape[4] = {c.n_pages, c.page_size, c.Hk, c.d / 16};
    const Tensor* const scale[2] = {&needed(kso, "k_scale"), &needed(vso, "v_scale")};
    const at::ScalarType of = scale[0]->scalar_type();
    TORCH_CHECK_TYPE(of == at::kByte || of == at::kFloat8_e4m3fn,
                     "k_scale must be float8_e4m3fn, or its codes as uint8");
    c.k_scale = operand(*scale[0], "k_scale", of, dev, shape);
    c.v_scale = operand(*scale[1], "v_scale", of, dev, shape);
    cache_strides(*scale[0], c.k_scale_strides);
    cache_strides(*scale[1], c.v_scale_strides);
    c.k_descale = floats(kdo, "k_descale", dev, c.Hk);
    c.v_descale = floats(vdo, "v_descale", dev, c.Hk);
  } else if (e4m3) {
    c.k_descale = static_cast<const float*>(
        dense(needed(kdo, "k_descale"), "k_descale", at::kFloat, dev, {c.Hk}));
    c.v_descale = static_cast<const float*>(
        dense(needed(vdo, "v_descale"), "v_descale", at::kFloat, dev, {c.Hk}));
  } else {
    TORCH_CHECK_VALUE(kdo == Py_None && vdo == Py_None,
                      "k_descale and v_descale go with an E4M3 cache");
  }
  cache_strides(k, c.k_strides);
  cache_strides(v, c.v_strides);
  return c;
}

// (q, k, v, k_cache, v_cache, page_table, cache_lens, new_lens, q_weight, k_weight, inv_freq,
//  q_out, eps, interleaved, k_descale, v_descale, stream, k_scale, v_scale) -> q_out
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 19);
  const Tensor& k = rows4(a[1], "k");
  const int dev = device_of(k, "k");
  const Home home(a[16], dev);
  const int B = to_int(k.size(0), "k"), S = to_int(k.size(1), "k");
  const cp_paged_cache cache = cache_of(a[3], a[4], a[5], a[14], a[15], a[17], a[18], B, dev);
  const int64_t shape[4] = {B, S, cache.Hk, cache.d};
  const void* const k_at = operand(k, "k", at::kBFloat16, dev, shape);
  const Tensor& v = needed(a[2], "v");
  const void* const v_at = operand(v, "v", at::kBFloat16, dev, shape);
  const Tensor* const q = a[0] == Py_None ? nullptr : &rows4(a[0], "q");
  int Hq = 0;
  const void* q_at = nullptr;
  void* qo_at = nullptr;
  Tensor q_out;
  if (q) {
    Hq = to_int(q->size(2), "q");
    q_at = operand(*q, "q", at::kBFloat16, dev, {B, S, Hq, cache.d});
    q_out = output(a[11], "q_out", *q);
    qo_at = dense(q_out, "q_out", at::kBFloat16, dev, q->sizes());
  }
  const int32_t* const lens = static_cast<const int32_t*>(
      dense(needed(a[6], "cache_lens"), "cache_lens", at::kInt, dev, {B}));
  const int32_t* const fresh = dense_or_null<int32_t>(a[7], "new_lens", at::kInt, dev, {B});
  const float* const qw = floats(a[8], "q_weight", dev, cache.d);
  const float* const kw = floats(a[9], "k_weight", dev, cache.d);
  const int rot = rotated(given(a[10], "inv_freq"));
  const float* const freq = floats(a[10], "inv_freq", dev, rot / 2);
  const float eps = to_float(a[12]);
  const bool pairs = to_bool(a[13]);
  const Steps qs(q), ks(&k), vs(&v);
  run("cp_paged_append", dev, [&] {
    return cp_paged_append(&cache, q_at, qs.get(), k_at, ks.get(), v_at, vs.get(), lens, fresh, qw,
                           kw, eps, freq, rot, pairs, qo_at, B, S, Hq, home.get());
  });
  home.hand_over(q_out, a[11] == Py_None);
  return wrap(&q_out);
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, page_table, seq_lens, out, lse, prefix_pages, prefix_len, k_descale,
//  v_descale, workspace, stream, k_scale, v_scale) -> (out, lse)
PyObject* paged_attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 15);
  const Tensor& q = rows4(a[0], "q");
  const int dev = device_of(q, "q");
  const Home home(a[12], dev);
  const int B = to_int(q.size(0), "q"), n_q = to_int(q.size(1), "q"), Hq = to_int(q.size(2), "q");
  const cp_paged_cache cache = cache_of(a[1], a[2], a[3], a[9], a[10], a[13], a[14], B, dev);
  const void* const q_at = operand(q, "q", at::kBFloat16, dev, {B, n_q, Hq, cache.d});
  const Tensor out = output(a[5], "out", q);
  void* const out_at = dense(out, "out", at::kBFloat16, dev, q.sizes());
  const Tensor* const lse_given = given(a[6], "lse");
  const Tensor lse =
      lse_given ? *lse_given : at::empty({B, Hq, n_q}, q.options().dtype(at::kFloat));
  float* const lse_at = static_cast<float*>(dense(lse, "lse", at::kFloat, dev, {B, Hq, n_q}));
  const int32_t* const lens = static_cast<const int32_t*>(
      dense(needed(a[4], "seq_lens"), "seq_lens", at::kInt, dev, {B}));
  const long prefix = PyLong_AsLong(a[8]);
  if (prefix == -1 && PyErr_Occurred()) throw python_error();
  TORCH_CHECK_VALUE(prefix >= INT_MIN && prefix <= INT_MAX, "prefix_len is too large");
  const int prefix_len = static_cast<int>(prefix);
  const Tensor* const pages = given(a[7], "prefix_pages");
  const int32_t* pages_at = nullptr;
  if (pages) {
    pages_at = static_cast<const int32_t*>(
        dense(*pages, "prefix_pages", at::kInt, dev, {pages->numel()}));
    TORCH_CHECK_VALUE(pages->numel() * cache.page_size >= prefix_len,
                      "prefix_pages holds fewer tokens than prefix_len");
  }
  const Tensor* const ws_given = given(a[11], "workspace");
  Tensor ws;
  if (ws_given) {
    ws = *ws_given;
  } else {
    const int64_t need =
        cp_paged_attn_decode_workspace_bytes(B, n_q, Hq, cache.Hk, cache.d, prefix_len);
    if (need < 0) check("cp_paged_attn_decode_workspace_bytes", CP_ERR_SHAPE);
    ws = at::empty({need}, q.options().dtype(at::kByte));
  }
  void* const ws_at = dense(ws, "workspace", at::kByte, dev, ws.sizes());
  const Steps qs(&q);
  run("cp_paged_attn_decode", dev, [&] {
    return cp_paged_attn_decode(&cache, q_at, qs.get(), lens, pages_at, prefix_len, out_at, lse_at,
                                B, n_q, Hq, ws_at, ws.numel(), home.get());
  });
  home.hand_over(out, a[5] == Py_None);
  home.hand_over(lse, a[6] == Py_None);
  return tuple_of({&out, &lse});
  END_HANDLE_TH_ERRORS
}

const Tensor& rows3(PyObject* o, const char* name) {
  const Tensor& t = needed(o, name);
  TORCH_CHECK_VALUE(t.dim() == 3, name, " must be a tensor of three dimensions");
  return t;
}

// The (row, head) strides of [T, H, d]; the stride of a dimension of one entry is never used:
// what a contiguous tensor has is passed.
struct PackedSteps {
  int64_t v[2];
  bool dense = true;
  explicit PackedSteps(const Tensor& t) {
    if ((dense = t.is_contiguous())) return;
    v[1] = t.size(1) > 1 ? t.stride(1) : t.size(2);
    v[0] = t.size(0) > 1 ? t.stride(0) : t.size(1) * v[1];
  }
  const int64_t* get() const { return dense ? nullptr : v; }
};

// What the calls over packed prompts share: q, k, v and the sequences' offsets.
struct Packed {
  int dev, T, Hq, Hk, d, n;
  const Tensor &q, &k, &v;
  const void *q_at, *k_at, *v_at;
  const int32_t* offsets;
  PackedSteps qs, ks, vs;
  Packed(PyObject* qo, PyObject* ko, PyObject* vo, PyObject* oo)
      : q(rows3(qo, "q")), k(rows3(ko, "k")), v(rows3(vo, "v")), qs(q), ks(k), vs(v) {
    dev = device_of(q, "q");
    T = to_int(q.size(0), "q");
    Hq = to_int(q.size(1), "q");
    d = to_int(q.size(2), "q");
    Hk = to_int(k.size(1), "k");
    q_at = operand(q, "q", at::kBFloat16, dev, q.sizes());
    k_at = operand(k, "k", at::kBFloat16, dev, {T, Hk, d});
    v_at = operand(v, "v", at::kBFloat16, dev, {T, Hk, d});
    const Tensor& o = needed(oo, "seq_offsets");
    TORCH_CHECK_VALUE(o.dim() == 1 && o.numel() >= 2,
                      "seq_offsets must have one dimension and an entry more than sequences");
    offsets = static_cast<const int32_t*>(dense(o, "seq_offsets", at::kInt, dev, o.sizes()));
    n = to_int(o.numel() - 1, "seq_offsets");
  }
  // `given`, or a new workspace of `need` bytes (-1: refused sizes).
  Tensor workspace(PyObject* o, int64_t need, const char* fn) const {
    const Tensor* const t = given(o, "workspace");
    if (t) {
      dense(*t, "workspace", at::kByte, dev, t->sizes());
      return *t;
    }
    if (need < 0) check(fn, CP_ERR_SHAPE);
    return at::empty({need}, q.options().dtype(at::kByte));
  }
};

// An output [T, H, d]: the caller's, or a new contiguous one, of zeros (the call leaves
// rows of no sequence as they are).
Tensor packed_output(PyObject* o, const char* name, const Tensor& like) {
  const Tensor* const t = given(o, name);
  return t ? *t : at::zeros(like.sizes(), like.options());
}

// (q, k, v, seq_offsets, causal, out, lse, workspace, stream) -> (out, lse)
PyObject* packed_attn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 9);
  const Packed x(a[0], a[1], a[2], a[3]);
  const Home home(a[8], x.dev);
  const bool causal = to_bool(a[4]);
  const Tensor out = packed_output(a[5], "out", x.q);
  void* const out_at = dense(out, "out", at::kBFloat16, x.dev, x.q.sizes());
  const Tensor* const lse_given = given(a[6], "lse");
  const Tensor lse =
      lse_given ? *lse_given : at::zeros({x.Hq, x.T}, x.q.options().dtype(at::kFloat));
  float* const lse_at = static_cast<float*>(dense(lse, "lse", at::kFloat, x.dev, {x.Hq, x.T}));
  if (x.T == 0) return tuple_of({&out, &lse});  // no rows
  const Tensor ws = x.workspace(
      a[7], a[7] == Py_None ? cp_packed_attn_fwd_workspace_bytes(x.T, x.n, x.Hq, x.Hk, x.d) : 0,
      "cp_packed_attn_fwd_workspace_bytes");
  run("cp_packed_attn_fwd", x.dev, [&] {
    return cp_packed_attn_fwd(x.q_at, x.qs.get(), x.k_at, x.ks.get(), x.v_at, x.vs.get(),
                              x.offsets, out_at, lse_at, x.T, x.n, x.Hq, x.Hk, x.d, causal,
                              ws.data_ptr(), ws.numel(), home.get());
  });
  home.hand_over(out, a[5] == Py_None);
  home.hand_over(lse, a[6] == Py_None);
  return tuple_of({&out, &lse});
  END_HANDLE_TH_ERRORS
}

// (q, k, v, out, lse, dout, seq_offsets, causal, dq, dk, dv, workspace, stream) -> (dq, dk, dv)
PyObject* packed_attn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 13);
  const Packed x(a[0], a[1], a[2], a[6]);
  const Home home(a[12], x.dev);
  const void* const out_at = dense(needed(a[3], "out"), "out", at::kBFloat16, x.dev, x.q.sizes());
  const float* const lse_at = static_cast<const float*>(
      dense(needed(a[4], "lse"), "lse", at::kFloat, x.dev, {x.Hq, x.T}));
  const void* const dout_at =
      dense(needed(a[5], "dout"), "dout", at::kBFloat16, x.dev, x.q.sizes());
  const bool causal = to_bool(a[7]);
  const Tensor dq = packed_output(a[8], "dq", x.q), dk = packed_output(a[9], "dk", x.k),
               dv = packed_output(a[10], "dv", x.v);
  void* const dq_at = operand(dq, "dq", at::kBFloat16, x.dev, x.q.sizes());
  void* const dk_at = operand(dk, "dk", at::kBFloat16, x.dev, x.k.sizes());
  void* const dv_at = operand(dv, "dv", at::kBFloat16, x.dev, x.v.sizes());
  if (x.T == 0) return tuple_of({&dq, &dk, &dv});  // no rows
  const Tensor ws = x.workspace(
      a[11], a[11] == Py_None ? cp_packed_attn_bwd_workspace_bytes(x.T, x.n, x.Hq, x.Hk, x.d) : 0,
      "cp_packed_attn_bwd_workspace_bytes");
  const PackedSteps dqs(dq), dks(dk), dvs(dv);
  run("cp_packed_attn_bwd", x.dev, [&] {
    return cp_packed_attn_bwd(x.q_at, x.qs.get(), x.k_at, x.ks.get(), x.v_at, x.vs.get(), out_at,
                              lse_at, dout_at, x.offsets, dq_at, dqs.get(), dk_at, dks.get(),
                              dv_at, dvs.get(), x.T, x.n, x.Hq, x.Hk, x.d, causal, ws.data_ptr(),
                              ws.numel(), home.get());
  });
  home.hand_over(dq, a[8] == Py_None);
  home.hand_over(dk, a[9] == Py_None);
  home.hand_over(dv, a[10] == Py_None);
  return tuple_of({&dq, &dk, &dv});
  END_HANDLE_TH_ERRORS
}

// The exception class that a refused call raises.
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(qk_norm_rope), METH_FASTCALL, nullptr},
    {"qk_norm_rope_bwd", reinterpret_cast<PyCFunction>(qk_norm_rope_bwd), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(paged_append), METH_FASTCALL, nullptr},
    {"paged_attn_decode", reinterpret_cast<PyCFunction>(paged_attn_decode), METH_FASTCALL,
     nullptr},
    {"packed_attn_fwd", reinterpret_cast<PyCFunction>(packed_attn_fwd), METH_FASTCALL, nullptr},
    {"packed_attn_bwd", reinterpret_cast<PyCFunction>(packed_attn_bwd), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "cpring_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_cpring_torch(void) { return PyModule_Create(&g_module); }
