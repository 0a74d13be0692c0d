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
  argc(n, 21);
  const at::Tensor& x = needed(a[0], "x", 2);
  const int64_t H = number(a[1]), Hk = number(a[2]), D = number(a[3]), T = x.size(0);
  const at::Tensor *rope = tensor(a[7], "rope"), *cu = tensor(a[9], "cu_seqlens"),
                   *kv = tensor(a[10], "kv_lens"), *table = tensor(a[11], "page_table"),
                   *kc = tensor(a[12], "k_cache"), *vc = tensor(a[13], "v_cache"),
                   *status = tensor(a[19], "status"), *q_in = tensor(a[16], "q");
  same_device(x, "x", {{a[4], "q_weight"}, {a[5], "k_weight"}, {a[7], "rope"}, {a[9], "cu_seqlens"},
                       {a[10], "kv_lens"}, {a[11], "page_table"}, {a[12], "k_cache"},
                       {a[13], "v_cache"}, {a[16], "q"}, {a[17], "k"}, {a[18], "v"}, {a[19], "status"}});
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
  const Place place(a[20], x);
  at::Tensor q = made(a[16], "q", {T, H, D}, out, x, place), k, v;
  if (dense) {
    k = made(a[17], "k", {T, Hk, D}, out, x, place);
    v = made(a[18], "v", {T, Hk, D}, out, x, place);
  }
  place.order();
  const int rc = f_front(
      &d, px, static_cast<float*>(address(qw, "q_weight", kF32, {D})),
      static_cast<float*>(address(kw, "k_weight", kF32, {D})),
      static_cast<float*>(address(rope, "rope", kF32, {})),
      static_cast<int32_t*>(address(cu, "cu_seqlens", kI32, {})),
      static_cast<int32_t*>(address(kv, "kv_lens", kI32, {N})),
      static_cast<int32_t*>(address(table, "page_table", kI32, {N, cols})),
      address(&q, "q", out, {T, H, D}), address(dense ? &k : nullptr, "k", out, {T, Hk, D}),
      address(dense ? &v : nullptr, "v", out, {T, Hk, D}),
      address(kc, "k_cache", out, {pages, Hk, page, D}),
      address(vc, "v_cache", out, {pages, Hk, page, D}), place.stream);
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
  argc(n, 14);
  const at::Tensor &q = needed(a[0], "q", 0), &kc = needed(a[1], "k_cache", 4),
                   &vc = needed(a[2], "v_cache", 4), &table = needed(a[3], "page_table", 2),
                   &kv = needed(a[4], "kv_lens", 1);
  if (q.dim() != 3 && q.dim() != 4)
    refuse(PyExc_ValueError, "q must have shape [N, H, D] or [N, n_q, H, D]");
  same_device(q, "q", {{a[1], "k_cache"}, {a[2], "v_cache"}, {a[3], "page_table"}, {a[4], "kv_lens"},
                       {a[8], "out"}, {a[10], "lse"}, {a[11], "workspace"}, {a[12], "status"}});
  const at::Tensor *status = tensor(a[12], "status"), *out_in = tensor(a[8], "out");
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
  const Place place(a[13], q);
  at::Tensor out = made(a[8], "out", q.sizes(), to, q, place), lse, work;
  const at::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
  if (want_lse) lse = made(a[10], "lse", rows, kF32, q, place);
  if (const at::Tensor* w = tensor(a[11], "workspace")) {
    work = *w;
  } else {
    const size_t bytes = f_workspace(&d);
    if (bytes == 0) fail(f_check(&d), "gdn_attn_decode");
    work = place.make({(int64_t)bytes}, at::kByte, q);
  }
  d.workspace = address(&work, "workspace", work.scalar_type(), {});
  d.workspace_bytes = work.nbytes();
  place.order();
  const int rc = f_decode(&d, pq, address(&kc, "k_cache", t, {pages, Hk, page, D}),
                          address(&vc, "v_cache", t, {pages, Hk, page, D}),
                          static_cast<int32_t*>(address(&table, "page_table", kI32, {N, cols})),
                          static_cast<int32_t*>(address(&kv, "kv_lens", kI32, {N})),
                          i32(number(a[5])), (float)real(a[6]), address(&out, "out", to, q.sizes()),
                          static_cast<float*>(address(want_lse ? &lse : nullptr, "lse", kF32, rows)),
                          place.stream);
  if (rc != GDN_OK) fail(rc, "gdn_attn_decode");
  return with_lse(out, return_lse ? &lse : nullptr);
  END_HANDLE_TH_ERRORS
}

// init(GdnError, {entry point: address})
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 6);
  Py_XSETREF(gdn_error, Py_NewRef(a[0]));
  f_front = reinterpret_cast<decltype(f_front)>((uintptr_t)number(a[1]));
  f_prefill = reinterpret_cast<decltype(f_prefill)>((uintptr_t)number(a[2]));
  f_decode = reinterpret_cast<decltype(f_decode)>((uintptr_t)number(a[3]));
  f_workspace = reinterpret_cast<decltype(f_workspace)>((uintptr_t)number(a[4]));
  f_check = reinterpret_cast<decltype(f_check)>((uintptr_t)number(a[5]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<init>("init"), method<front>("front"), method<prefill>("prefill"),
                         method<decode>("decode"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_attn_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__attn_torch() { return PyModule_Create(&module_def); }
