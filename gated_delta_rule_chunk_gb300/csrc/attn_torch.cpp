// The attention calls' marshalling (tensor checks, output allocation, descriptor), compiled:
// at a decode step it runs once per layer and call, and in Python it took 11 us of host time
// for a 3 us kernel. binding.py hands over its arguments in order; everything else happens
// behind the C ABI, whose entry points come in as addresses (init), so that this module does
// not depend on which build of libgdn is loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/Event.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/gdn_attn.h"

namespace {

decltype(&gdn_attn_front) f_front;
decltype(&gdn_attn_prefill) f_prefill;
decltype(&gdn_attn_decode) f_decode;
decltype(&gdn_attn_workspace_size) f_workspace;
decltype(&gdn_attn_check_desc) f_check;
decltype(&gdn_attn_front_axes) f_front_axes;
decltype(&gdn_attn_append8) f_append8;
decltype(&gdn_attn_decode_cache) f_decode_cache;
decltype(&gdn_attn_decode_cache_workspace_size) f_decode_cache_workspace;
decltype(&gdn_attn_prefill_weights) f_weights;
decltype(&gdn_attn_prefill_weights_workspace_size) f_weights_workspace;
decltype(&gdn_attn_evict) f_evict;
PyObject* gdn_error;  // binding.GdnError

[[noreturn]] void fail(int status, const char* what) {
  PyObject* e = PyObject_CallFunction(gdn_error, "is", status, what);
  if (e) {
    PyErr_SetObject(gdn_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

template <typename... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw python_error();
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return &THPVariable_Unpack(o);
}

const at::Tensor& needed(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse(PyExc_TypeError, "%s must be a tensor", name);
  if (dims && t->dim() != dims) refuse(PyExc_ValueError, "%s must have %d dimensions", name, (int)dims);
  return *t;
}

int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

double real(PyObject* o) {
  const double v = o == Py_None ? 0.0 : PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

int32_t dtype_code(at::ScalarType t) {
  if (t == at::kFloat) return GDN_F32;
  if (t == at::kBFloat16) return GDN_BF16;
  refuse(PyExc_TypeError, "unsupported dtype %s", c10::toString(t));
}

// The dtype given, else `otherwise`.
at::ScalarType dtype_or(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "out_dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// Address of a contiguous CUDA tensor of this dtype and (where given) shape; null for none.
void* address(const at::Tensor* t, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
  if (!t) return nullptr;
  if (!t->is_cuda() || !t->is_contiguous())
    refuse(PyExc_ValueError, "%s must be a contiguous CUDA tensor", name);
  if (t->scalar_type() != dtype)
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(dtype),
           c10::toString(t->scalar_type()));
  if (!shape.empty() && t->sizes() != shape) {
    PyErr_Format(PyExc_ValueError, "%s has the wrong shape", name);
    throw python_error();
  }
  return t->data_ptr();
}

struct Named {
  PyObject* o;
  const char* name;
};
// Refuses tensors on another device than x: nothing below this would see that. (One that is on no
// CUDA device has its own message in `address`.)
void same_device(const at::Tensor& x, const char* x_name, std::initializer_list<Named> others) {
  const c10::Device on = x.device();
  for (const Named& n : others) {
    const at::Tensor* t = tensor(n.o, n.name);
    if (t && x.is_cuda() && t->is_cuda() && t->device() != on)
      refuse(PyExc_ValueError, "%s is on %s, %s on %s", n.name, t->device().str().c_str(), x_name,
             on.str().c_str());
  }
}

int64_t num_seqs(const at::Tensor* cu) {
  if (!cu) return 1;
  if (cu->dim() != 1 || cu->size(0) < 2)
    refuse(PyExc_ValueError, "cu_seqlens must have shape [N + 1] with N >= 1");
  return cu->size(0) - 1;
}

// Sizes beyond what the descriptor holds are refused here.
int32_t i32(int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "a size does not fit in 32 bits");
  return (int32_t)v;
}

// Whether a stream is being captured; -1 where that cannot be asked.
int captured(cudaStream_t s) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &status) == cudaSuccess) return status != cudaStreamCaptureStatusNone;
  (void)cudaGetLastError();
  return -1;
}

// Makes the tensor's device current while the call runs, and finds the call's stream. What is
// allocated comes from the current stream's memory, which that stream's queued work may still be
// using. Where the call runs in another one, that stream first waits for the current one as it
// stands (order; a call that allocates nothing does not wait), and the memory does not go to new
// work, when it is given back, before that stream is done with it (a workspace is given back when
// the call returns). Neither can be had between a captured stream and one that is not.
struct Place {
  c10::cuda::CUDAGuard device;
  c10::cuda::CUDAStream current, on;
  cudaStream_t stream;
  bool other;
  mutable bool allocated = false;
  Place(PyObject* o, const at::Tensor& t)
      : device(t.device()), current(c10::cuda::getCurrentCUDAStream(t.device().index())), on(current),
        stream(on.stream()), other(false) {
    if (o == Py_None) return;
    stream = reinterpret_cast<cudaStream_t>((uintptr_t)number(o));
    other = stream != on.stream();
    if (other) on = c10::cuda::getStreamFromExternal(stream, t.device().index());
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) const {
    if (other && !allocated) {
      const int a = captured(current.stream()), b = captured(stream);
      if (a != b || a < 0)
        refuse(PyExc_ValueError, "one of the call's stream and the current stream is being captured "
                                 "and the other is not: outputs and workspace must be given");
    }
    allocated = true;
    at::Tensor t = at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
    if (other) t.record_stream(on.unwrap());
    return t;
  }
  void order() const {
    if (!other || !allocated) return;
    c10::Event e(c10::DeviceType::CUDA);
    e.record(current.unwrap());
    e.block(on.unwrap());
  }
};

at::Tensor made(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype,
                const at::Tensor& like, const Place& place) {
  const at::Tensor* t = tensor(o, name);
  return t ? *t : place.make(shape, dtype, like);
}

void argc(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "%d arguments, expected %d", (int)n, (int)want);
}

constexpr at::ScalarType kI32 = at::kInt, kF32 = at::kFloat;

PyObject* front(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 23);
  const at::Tensor& x = needed(a[0], "x", 2);
  const int64_t H = number(a[1]), Hk = number(a[2]), D = number(a[3]), T = x.size(0);
  const at::Tensor *rope = tensor(a[7], "rope"), *cu = tensor(a[9], "cu_seqlens"),
                   *kv = tensor(a[10], "kv_lens"), *table = tensor(a[11], "page_table"),
                   *kc = tensor(a[12], "k_cache"), *vc = tensor(a[13], "v_cache"),
                   *status = tensor(a[19], "status"), *q_in = tensor(a[16], "q"),
                   *pos = tensor(a[21], "positions"), *axes = tensor(a[22], "rope_axes");
  same_device(x, "x", {{a[4], "q_weight"}, {a[5], "k_weight"}, {a[7], "rope"}, {a[9], "cu_seqlens"},
                       {a[10], "kv_lens"}, {a[11], "page_table"}, {a[12], "k_cache"},
                       {a[13], "v_cache"}, {a[16], "q"}, {a[17], "k"}, {a[18], "v"}, {a[19], "status"},
                       {a[21], "positions"}, {a[22], "rope_axes"}});
  const bool interleaved = truth(a[8]), dense = truth(a[14]);
  const int64_t N = num_seqs(cu);
  const at::ScalarType out =
      dtype_or(a[15], kc ? kc->scalar_type() : q_in ? q_in->scalar_type() : x.scalar_type());
  gdn_attn_desc d{};
  d.in_dtype = dtype_code(x.scalar_type());
  d.out_dtype = dtype_code(out);
  if (kc && (kc->dim() != 4 || !table || table->dim() != 2))
    refuse(PyExc_ValueError, "the cache needs k_cache, v_cache [n_pages, Hk, page_size, D] and "
                             "page_table [N, max_pages]");
  if (pos && (pos->dim() != 2 || !rope))
    refuse(PyExc_ValueError, "positions must have shape [n_axes, T], and need rope");
  if (axes && !pos) refuse(PyExc_ValueError, "rope_axes needs positions");
  if (rope && rope->dim() != 2) refuse(PyExc_ValueError, "rope must have shape [max_pos, rot]");
  const int64_t pages = kc ? kc->size(0) : 0, page = kc ? kc->size(2) : 0;
  const int64_t cols = table && table->dim() == 2 ? table->size(1) : 0;
  d.T = i32(T); d.N = i32(N); d.H = i32(H); d.Hk = i32(Hk); d.D = i32(D);
  d.page_size = i32(page); d.n_pages = i32(pages); d.max_pages = i32(cols);
  d.rot_dim = rope ? i32(rope->size(1)) : 0; d.max_pos = rope ? i32(rope->size(0)) : 0;
  d.flags = interleaved ? GDN_ATTN_ROPE_INTERLEAVED : 0;
  d.norm_eps = (float)real(a[6]);
  d.status = static_cast<int32_t*>(address(status, "status", kI32, {}));
  const void* px = address(&x, "x", x.scalar_type(), {T, (H + 2 * Hk) * D});
  const at::Tensor *qw = tensor(a[4], "q_weight"), *kw = tensor(a[5], "k_weight");
  const float *pqw = static_cast<float*>(address(qw, "q_weight", kF32, {D})),
              *pkw = static_cast<float*>(address(kw, "k_weight", kF32, {D})),
              *prope = static_cast<float*>(address(rope, "rope", kF32, {}));
  const int32_t *pcu = static_cast<int32_t*>(address(cu, "cu_seqlens", kI32, {})),
                *pkv = static_cast<int32_t*>(address(kv, "kv_lens", kI32, {N})),
                *ptable = static_cast<int32_t*>(address(table, "page_table", kI32, {N, cols}));
  const int64_t n_axes = pos ? pos->size(0) : 0;
  const int32_t* ppos = static_cast<int32_t*>(address(pos, "positions", kI32, {n_axes, T}));
  const uint8_t* paxes =
      static_cast<uint8_t*>(address(axes, "rope_axes", at::kByte, {d.rot_dim / 2}));
  void *pkc = address(kc, "k_cache", out, {pages, Hk, page, D}),
       *pvc = address(vc, "v_cache", out, {pages, Hk, page, D});
  const Place place(a[20], x);
  at::Tensor q = made(a[16], "q", {T, H, D}, out, x, place), k, v;
  if (dense) {
    k = made(a[17], "k", {T, Hk, D}, out, x, place);
    v = made(a[18], "v", {T, Hk, D}, out, x, place);
  }
  place.order();
  void *pq = address(&q, "q", out, {T, H, D}),
       *pk = address(dense ? &k : nullptr, "k", out, {T, Hk, D}),
       *pv = address(dense ? &v : nullptr, "v", out, {T, Hk, D});
  const int rc =
      pos ? f_front_axes(&d, px, pqw, pkw, prope, pcu, pkv, ppos, i32(n_axes), paxes, ptable, pq, pk, pv,
                         pkc, pvc, place.stream)
          : f_front(&d, px, pqw, pkw, prope, pcu, pkv, ptable, pq, pk, pv, pkc, pvc, place.stream);
  if (rc != GDN_OK) fail(rc, "gdn_attn_front");
  PyObject* r = PyTuple_New(3);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(q));
  PyTuple_SET_ITEM(r, 1, dense ? THPVariable_Wrap(k) : Py_NewRef(Py_None));
  PyTuple_SET_ITEM(r, 2, dense ? THPVariable_Wrap(v) : Py_NewRef(Py_None));
  return r;
  END_HANDLE_TH_ERRORS
}

PyObject* with_lse(const at::Tensor& out, const at::Tensor* lse) {
  if (!lse) return THPVariable_Wrap(out);
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(*lse));
  return r;
}

PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 11);
  const at::Tensor &q = needed(a[0], "q", 3), &k = needed(a[1], "k", 3), &v = needed(a[2], "v", 3);
  const at::Tensor *cu = tensor(a[3], "cu_seqlens"), *status = tensor(a[9], "status"),
                   *out_in = tensor(a[6], "out");
  same_device(q, "q", {{a[1], "k"}, {a[2], "v"}, {a[3], "cu_seqlens"}, {a[6], "out"}, {a[8], "lse"},
                       {a[9], "status"}});
  const bool return_lse = truth(a[7]), want_lse = return_lse || a[8] != Py_None;
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2), Hk = k.size(1);
  const at::ScalarType t = q.scalar_type(),
                       to = dtype_or(a[5], out_in ? out_in->scalar_type() : t);
  gdn_attn_desc d{};
  d.T = i32(T); d.N = i32(num_seqs(cu)); d.H = i32(H); d.Hk = i32(Hk); d.D = i32(D);
  d.in_dtype = dtype_code(t);
  d.out_dtype = dtype_code(to);
  d.status = static_cast<int32_t*>(address(status, "status", kI32, {}));
  const void* pq = address(&q, "q", t, {});
  const Place place(a[10], q);
  at::Tensor out = made(a[6], "out", {T, H, D}, to, q, place), lse;
  if (want_lse) lse = made(a[8], "lse", {T, H}, kF32, q, place);
  place.order();
  const int rc = f_prefill(&d, pq, address(&k, "k", t, {T, Hk, D}), address(&v, "v", t, {T, Hk, D}),
                           static_cast<int32_t*>(address(cu, "cu_seqlens", kI32, {})),
                           (float)real(a[4]), address(&out, "out", to, {T, H, D}),
                           static_cast<float*>(address(want_lse ? &lse : nullptr, "lse", kF32, {T, H})),
                           place.stream);
  if (rc != GDN_OK) fail(rc, "gdn_attn_prefill");
  return with_lse(out, return_lse ? &lse : nullptr);
  END_HANDLE_TH_ERRORS
}

PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 17);
  const at::Tensor &q = needed(a[0], "q", 0), &kc = needed(a[1], "k_cache", 4),
                   &vc = needed(a[2], "v_cache", 4), &table = needed(a[3], "page_table", 2),
                   &kv = needed(a[4], "kv_lens", 1);
  if (q.dim() != 3 && q.dim() != 4)
    refuse(PyExc_ValueError, "q must have shape [N, H, D] or [N, n_q, H, D]");
  same_device(q, "q", {{a[1], "k_cache"}, {a[2], "v_cache"}, {a[3], "page_table"}, {a[4], "kv_lens"},
                       {a[8], "out"}, {a[10], "lse"}, {a[11], "workspace"}, {a[12], "status"},
                       {a[14], "k_scale"}, {a[15], "v_scale"}, {a[16], "weights"}});
  const at::Tensor *status = tensor(a[12], "status"), *out_in = tensor(a[8], "out"),
                   *ks = tensor(a[14], "k_scale"), *vs = tensor(a[15], "v_scale"),
                   *weights = tensor(a[16], "weights");
  const bool return_lse = truth(a[9]), want_lse = return_lse || a[10] != Py_None;
  const int64_t N = q.size(0), nq = q.dim() == 3 ? 1 : q.size(1), H = q.size(-2), D = q.size(-1);
  const int64_t pages = kc.size(0), Hk = kc.size(1), page = kc.size(2), cols = table.size(1);
  const at::ScalarType t = q.scalar_type(),
                       to = dtype_or(a[7], out_in ? out_in->scalar_type() : t);
  gdn_attn_desc d{};
  d.T = i32(N * nq); d.N = i32(N); d.H = i32(H); d.Hk = i32(Hk); d.D = i32(D);
  d.page_size = i32(page); d.n_pages = i32(pages); d.max_pages = i32(cols);
  d.in_dtype = dtype_code(t);
  d.out_dtype = dtype_code(to);
  d.status = static_cast<int32_t*>(address(status, "status", kI32, {}));
  const void* pq = address(&q, "q", t, {});
  if (!ks != !vs) refuse(PyExc_ValueError, "k_scale and v_scale come together");
  const at::ScalarType tc = ks || vs ? at::kFloat8_e4m3fn : t;
  const void *pk = address(&kc, "k_cache", tc, {pages, Hk, page, D}),
             *pv = address(&vc, "v_cache", tc, {pages, Hk, page, D});
  const int32_t *ptable = static_cast<int32_t*>(address(&table, "page_table", kI32, {N, cols})),
                *pkv = static_cast<int32_t*>(address(&kv, "kv_lens", kI32, {N}));
  const float *pks = static_cast<float*>(address(ks, "k_scale", kF32, {pages, Hk, page / 16})),
              *pvs = static_cast<float*>(address(vs, "v_scale", kF32, {pages, Hk, page / 16}));
  float* pw = static_cast<float*>(address(weights, "weights", kF32, {pages, Hk, page}));
  const int32_t shared = i32(number(a[5]));
  const float scale = (float)real(a[6]);
  // (before the workspace is allocated, which holds the scores of all keys)
  if (weights && shared > 0) fail(GDN_ERR_UNSUPPORTED, "gdn_attn_decode");
  const Place place(a[13], q);
  at::Tensor out = made(a[8], "out", q.sizes(), to, q, place), lse, work;
  const at::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
  if (want_lse) lse = made(a[10], "lse", rows, kF32, q, place);
  if (const at::Tensor* w = tensor(a[11], "workspace")) {
    work = *w;
  } else {
    const size_t bytes = ks || vs || weights ? f_decode_cache_workspace(&d, weights != nullptr)
                                             : f_workspace(&d);
    if (bytes == 0) fail(f_check(&d), "gdn_attn_decode");
    work = place.make({(int64_t)bytes}, at::kByte, q);
  }
  d.workspace = address(&work, "workspace", work.scalar_type(), {});
  d.workspace_bytes = work.nbytes();
  place.order();
  void* po = address(&out, "out", to, q.sizes());
  float* pl = static_cast<float*>(address(want_lse ? &lse : nullptr, "lse", kF32, rows));
  const int rc = ks || vs || weights
                     ? f_decode_cache(&d, pq, pk, pv, pks, pvs, ptable, pkv, shared, scale, po, pl, pw,
                                      place.stream)
                     : f_decode(&d, pq, pk, pv, ptable, pkv, shared, scale, po, pl, place.stream);
  if (rc != GDN_OK) fail(rc, "gdn_attn_decode");
  return with_lse(out, return_lse ? &lse : nullptr);
  END_HANDLE_TH_ERRORS
}

// The sizes of a cache and its page table.
void cache_sizes(gdn_attn_desc& d, const at::Tensor& cache, const at::Tensor& table) {
  d.n_pages = i32(cache.size(0)); d.Hk = i32(cache.size(1)); d.page_size = i32(cache.size(2));
  d.max_pages = i32(table.size(1));
}

PyObject* append8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 11);
  const at::Tensor &k = needed(a[0], "k", 3), &v = needed(a[1], "v", 3),
                   &kc = needed(a[2], "k_cache", 4), &vc = needed(a[3], "v_cache", 4),
                   &ks = needed(a[4], "k_scale", 3), &vs = needed(a[5], "v_scale", 3),
                   &table = needed(a[6], "page_table", 2);
  const at::Tensor *kv = tensor(a[7], "kv_lens"), *cu = tensor(a[8], "cu_seqlens"),
                   *status = tensor(a[9], "status");
  same_device(k, "k", {{a[1], "v"}, {a[2], "k_cache"}, {a[3], "v_cache"}, {a[4], "k_scale"},
                       {a[5], "v_scale"}, {a[6], "page_table"}, {a[7], "kv_lens"},
                       {a[8], "cu_seqlens"}, {a[9], "status"}});
  const int64_t T = k.size(0), Hk = k.size(1), D = k.size(2), N = num_seqs(cu);
  const int64_t pages = kc.size(0), page = kc.size(2);
  const at::ScalarType t = k.scalar_type();
  gdn_attn_desc d{};
  cache_sizes(d, kc, table);
  d.T = i32(T); d.N = i32(N); d.H = d.Hk = i32(Hk); d.D = i32(D);
  d.in_dtype = d.out_dtype = dtype_code(t);
  d.status = static_cast<int32_t*>(address(status, "status", kI32, {}));
  const void* pk = address(&k, "k", t, {});
  const void* pv = address(&v, "v", t, {T, Hk, D});
  const int32_t *pcu = static_cast<int32_t*>(address(cu, "cu_seqlens", kI32, {})),
                *pkv = static_cast<int32_t*>(address(kv, "kv_lens", kI32, {N})),
                *ptable = static_cast<int32_t*>(address(&table, "page_table", kI32, {N, table.size(1)}));
  void *pkc = address(&kc, "k_cache", at::kFloat8_e4m3fn, {pages, Hk, page, D}),
       *pvc = address(&vc, "v_cache", at::kFloat8_e4m3fn, {pages, Hk, page, D});
  float *pks = static_cast<float*>(address(&ks, "k_scale", kF32, {pages, Hk, page / 16})),
        *pvs = static_cast<float*>(address(&vs, "v_scale", kF32, {pages, Hk, page / 16}));
  const Place place(a[10], k);
  const int rc = f_append8(&d, pk, pv, pcu, pkv, ptable, pkc, pvc, pks, pvs, place.stream);
  if (rc != GDN_OK) fail(rc, "gdn_attn_append8");
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* prefill_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 11);
  const at::Tensor &q = needed(a[0], "q", 3), &k = needed(a[1], "k", 3), &lse = needed(a[2], "lse", 2),
                   &weights = needed(a[3], "weights", 3), &table = needed(a[4], "page_table", 2);
  const at::Tensor *cu = tensor(a[5], "cu_seqlens"), *status = tensor(a[9], "status");
  same_device(q, "q", {{a[1], "k"}, {a[2], "lse"}, {a[3], "weights"}, {a[4], "page_table"},
                       {a[5], "cu_seqlens"}, {a[8], "workspace"}, {a[9], "status"}});
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2), Hk = k.size(1), N = num_seqs(cu);
  const at::ScalarType t = q.scalar_type();
  gdn_attn_desc d{};
  cache_sizes(d, weights, table);
  d.T = i32(T); d.N = i32(N); d.H = i32(H); d.Hk = i32(Hk); d.D = i32(D);
  d.in_dtype = d.out_dtype = dtype_code(t);
  d.status = static_cast<int32_t*>(address(status, "status", kI32, {}));
  const void* pq = address(&q, "q", t, {});
  const void* pk = address(&k, "k", t, {T, Hk, D});
  const float* pl = static_cast<float*>(address(&lse, "lse", kF32, {T, H}));
  const int32_t *pcu = static_cast<int32_t*>(address(cu, "cu_seqlens", kI32, {})),
                *ptable = static_cast<int32_t*>(address(&table, "page_table", kI32, {N, table.size(1)}));
  float* pw = static_cast<float*>(
      address(&weights, "weights", kF32, {weights.size(0), Hk, weights.size(2)}));
  const Place place(a[10], q);
  at::Tensor work;
  if (const at::Tensor* w = tensor(a[8], "workspace")) {
    work = *w;
  } else {
    const size_t bytes = f_weights_workspace(&d);
    if (bytes == 0) fail(f_check(&d), "gdn_attn_prefill_weights");
    work = place.make({(int64_t)bytes}, at::kByte, q);
  }
  d.workspace = address(&work, "workspace", work.scalar_type(), {});
  d.workspace_bytes = work.nbytes();
  place.order();
  const int rc = f_weights(&d, pq, pk, pl, pcu, ptable, i32(number(a[6])), (float)real(a[7]), pw,
                           place.stream);
  if (rc != GDN_OK) fail(rc, "gdn_attn_prefill_weights");
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 14);
  const at::Tensor &kc = needed(a[0], "k_cache", 4), &vc = needed(a[1], "v_cache", 4),
                   &weights = needed(a[2], "weights", 3), &table = needed(a[3], "page_table", 2),
                   &kv = needed(a[4], "kv_lens", 1), &fresh = needed(a[5], "new_table", 2);
  const at::Tensor *ks = tensor(a[8], "k_scale"), *vs = tensor(a[9], "v_scale"),
                   *status = tensor(a[12], "status");
  same_device(kc, "k_cache", {{a[1], "v_cache"}, {a[2], "weights"}, {a[3], "page_table"},
                              {a[4], "kv_lens"}, {a[5], "new_table"}, {a[8], "k_scale"},
                              {a[9], "v_scale"}, {a[10], "new_lens"}, {a[11], "kept"},
                              {a[12], "status"}});
  const int64_t pages = kc.size(0), Hk = kc.size(1), page = kc.size(2), D = kc.size(3), N = kv.size(0);
  const int64_t keep = number(a[6]);
  if (keep < 1) refuse(PyExc_ValueError, "keep must be at least 1");
  gdn_attn_desc d{};
  cache_sizes(d, kc, table);
  d.N = i32(N); d.H = d.Hk; d.D = i32(D);
  d.in_dtype = d.out_dtype = GDN_BF16;
  d.status = static_cast<int32_t*>(address(status, "status", kI32, {}));
  if (!ks != !vs) refuse(PyExc_ValueError, "k_scale and v_scale come together");
  const at::ScalarType tc = ks || vs ? at::kFloat8_e4m3fn : at::kBFloat16;
  void* pk = address(&kc, "k_cache", tc, {});
  void* pv = address(&vc, "v_cache", tc, {pages, Hk, page, D});
  float *pks = static_cast<float*>(address(ks, "k_scale", kF32, {pages, Hk, page / 16})),
        *pvs = static_cast<float*>(address(vs, "v_scale", kF32, {pages, Hk, page / 16})),
        *pw = static_cast<float*>(address(&weights, "weights", kF32, {pages, Hk, page}));
  const int32_t *ptable = static_cast<int32_t*>(address(&table, "page_table", kI32, {N, table.size(1)})),
                *pkv = static_cast<int32_t*>(address(&kv, "kv_lens", kI32, {N})),
                *pnew = static_cast<int32_t*>(address(&fresh, "new_table", kI32, {N, fresh.size(1)}));
  const int32_t keep32 = i32(keep), recent = i32(number(a[7])), new_max = i32(fresh.size(1));
  // (before `kept` is allocated, whose size goes by `keep`)
  int rc = f_check(&d);
  if (rc == GDN_OK && (recent < 0 || recent > keep || keep > (int64_t)new_max * page)) rc = GDN_ERR_BAD_SHAPE;
  if (rc != GDN_OK) fail(rc, "gdn_attn_evict");
  address(tensor(a[10], "new_lens"), "new_lens", kI32, {N});
  address(tensor(a[11], "kept"), "kept", kI32, {N, Hk, keep});
  const Place place(a[13], kc);
  at::Tensor lens = made(a[10], "new_lens", {N}, kI32, kc, place),
             kept = made(a[11], "kept", {N, Hk, keep}, kI32, kc, place);
  place.order();
  rc = f_evict(&d, pk, pv, pks, pvs, pw, ptable, pkv, pnew, new_max, keep32, recent,
               static_cast<int32_t*>(lens.data_ptr()), static_cast<int32_t*>(kept.data_ptr()), place.stream);
  if (rc != GDN_OK) fail(rc, "gdn_attn_evict");
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(lens));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(kept));
  return r;
  END_HANDLE_TH_ERRORS
}

// init(GdnError, {entry point: address})
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 13);
  Py_XSETREF(gdn_error, Py_NewRef(a[0]));
  f_front = reinterpret_cast<decltype(f_front)>((uintptr_t)number(a[1]));
  f_prefill = reinterpret_cast<decltype(f_prefill)>((uintptr_t)number(a[2]));
  f_decode = reinterpret_cast<decltype(f_decode)>((uintptr_t)number(a[3]));
  f_workspace = reinterpret_cast<decltype(f_workspace)>((uintptr_t)number(a[4]));
  f_check = reinterpret_cast<decltype(f_check)>((uintptr_t)number(a[5]));
  f_front_axes = reinterpret_cast<decltype(f_front_axes)>((uintptr_t)number(a[6]));
  f_append8 = reinterpret_cast<decltype(f_append8)>((uintptr_t)number(a[7]));
  f_decode_cache = reinterpret_cast<decltype(f_decode_cache)>((uintptr_t)number(a[8]));
  f_decode_cache_workspace =
      reinterpret_cast<decltype(f_decode_cache_workspace)>((uintptr_t)number(a[9]));
  f_weights = reinterpret_cast<decltype(f_weights)>((uintptr_t)number(a[10]));
  f_weights_workspace = reinterpret_cast<decltype(f_weights_workspace)>((uintptr_t)number(a[11]));
  f_evict = reinterpret_cast<decltype(f_evict)>((uintptr_t)number(a[12]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<init>("init"), method<front>("front"), method<prefill>("prefill"),
                         method<decode>("decode"), method<append8>("append8"),
                         method<prefill_weights>("prefill_weights"), method<evict>("evict"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_attn_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__attn_torch() { return PyModule_Create(&module_def); }
