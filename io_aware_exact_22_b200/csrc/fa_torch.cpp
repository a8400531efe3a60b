// fa_torch.cpp - the calls of fa.py that are as short on the device as Python's marshalling is on the
// host (norm + rotation, paged cache), taken straight from torch tensors: checks, outputs that are
// not given, current device and stream, then the C function.  A CPython module without a link to
// libfa.so: fa.py hands it the addresses of the library that it loaded.  Every function returns
// its outputs, or the C status as an int when it is not FA_OK; bad tensors raise ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <vector>

#include "fa.h"

namespace {

decltype(&::fa_qk_norm_rope) c_norm_rope;
decltype(&::fa_qk_norm_rope_bwd) c_norm_rope_bwd;
decltype(&::fa_qk_norm_rope_bwd_workspace_bytes) c_norm_rope_bwd_bytes;
decltype(&::fa_paged_plan) c_plan;
decltype(&::fa_paged_append) c_append;
decltype(&::fa_paged_decode) c_decode;
decltype(&::fa_paged_decode_workspace_bytes) c_decode_bytes;

using at::Tensor;

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, not ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
int i32(int64_t n, const char* what) {
  TORCH_CHECK_VALUE(n >= INT_MIN && n <= INT_MAX, what, " does not fit 32 bits");
  return static_cast<int>(n);
}
int integer(PyObject* o, const char* what) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw python_error();
  return i32(n, what);
}
float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x != 0;
}
bool on(const Tensor& t, int index) { return t.is_cuda() && t.get_device() == index && t.layout() == at::kStrided; }

// A bf16 tensor of `dims` dimensions on CUDA device `index` (-1: any), the last one contiguous.
const Tensor& rows(PyObject* o, const char* name, int dims, int index) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16 && t.dim() == dims && t.is_cuda() && t.layout() == at::kStrided &&
                        (index < 0 || t.get_device() == index) && (t.size(-1) <= 1 || t.stride(-1) == 1),
                    name, " must be a bf16 tensor of ", dims, " dimensions, the last one contiguous, on one CUDA device");
  return t;
}

// Address of a contiguous tensor of that type and number of elements on CUDA device `index`.
void* vec(PyObject* o, const char* name, at::ScalarType type, int index, int64_t numel) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.scalar_type() == type && on(t, index) && t.is_contiguous() && t.numel() == numel, name,
                    " must be a contiguous ", type, " tensor of ", numel, " elements on CUDA device ", index);
  return t.data_ptr();
}
void* vec_or_null(PyObject* o, const char* name, at::ScalarType type, int index, int64_t numel) {
  return o == Py_None ? nullptr : vec(o, name, type, index, numel);
}

// A new contiguous tensor, by torch's dispatcher: its modes (a fill of uninitialised memory, say) see it.
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::empty(shape, at::device(at::Device(at::kCUDA, static_cast<at::DeviceIndex>(index))).dtype(type));
}

// An output: the caller's contiguous tensor, checked, or a new one.
Tensor output(PyObject* o, const char* name, at::ScalarType type, int index, at::IntArrayRef shape) {
  if (o == Py_None) return fresh(shape, type, index);
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.scalar_type() == type && on(t, index) && t.sizes() == shape && t.is_contiguous(), name,
                    " must be a contiguous ", type, " tensor ", shape, " on CUDA device ", index);
  return t;
}

// The caller's workspace, checked, or one from torch's allocator that goes back to it when the call
// returns (it is handed out again in the order of the current stream).  The device is current.
class Workspace {
 public:
  Workspace(PyObject* o, size_t bytes, int index) : bytes_(std::max<size_t>(bytes, 256)) {
    if (o == Py_None) {
      at_ = own_ = c10::cuda::CUDACachingAllocator::raw_alloc(bytes_);
      return;
    }
    const Tensor& t = tensor(o, "workspace");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kByte && on(t, index) && t.is_contiguous() && (size_t)t.numel() >= bytes,
                      "workspace must be a contiguous uint8 tensor of at least ", bytes, " bytes on CUDA device ", index);
    at_ = t.data_ptr(), bytes_ = t.numel();
  }
  ~Workspace() {
    if (own_) c10::cuda::CUDACachingAllocator::raw_delete(own_);
  }
  Workspace(const Workspace&) = delete;
  Workspace& operator=(const Workspace&) = delete;
  void* at() const { return at_; }
  size_t bytes() const { return bytes_; }

 private:
  void *at_ = nullptr, *own_ = nullptr;
  size_t bytes_;
};

// An output's elements lie at addresses of their own: each stride is past all that the smaller ones reach.
void distinct(const Tensor& t, const char* name) {
  if (t.is_contiguous()) return;
  std::vector<std::pair<int64_t, int64_t>> dims;
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1) dims.emplace_back(t.stride(i), t.size(i));
  std::sort(dims.begin(), dims.end());
  int64_t reach = 0;
  for (const auto& [stride, size] : dims) {
    TORCH_CHECK_VALUE(stride > reach, name, " must not overlap itself");
    reach += stride * (size - 1);
  }
}

struct Rope {
  const float* table = nullptr;
  int rows = 0, rot = 0;
};
Rope rope_of(PyObject* o, int index) {
  Rope r;
  if (o == Py_None) return r;
  const Tensor& t = tensor(o, "rope");
  TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && on(t, index) && t.dim() == 3 && t.size(1) == 2 && t.is_contiguous(),
                    "rope must be a contiguous fp32 table [rows, 2, rot/2] on CUDA device ", index);
  r.table = static_cast<const float*>(t.data_ptr());
  r.rows = i32(t.size(0), "rope's rows"), r.rot = i32(2 * t.size(2), "rope's columns");
  return r;
}

struct Positions {
  const int* at = nullptr;
  long long stride = 0;
};
Positions positions_of(PyObject* o, int64_t B, int64_t N, int index) {
  Positions p;
  if (o == Py_None) return p;
  const Tensor& t = tensor(o, "positions");
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && on(t, index) &&
                        ((t.dim() == 1 && t.size(0) == N) || (t.dim() == 2 && t.size(0) == B && t.size(1) == N)) &&
                        (N <= 1 || t.stride(-1) == 1),
                    "positions must be an int32 tensor [N] or [B,N], contiguous along N, on CUDA device ", index);
  p.at = static_cast<const int*>(t.data_ptr());
  if (t.dim() == 2) p.stride = t.stride(0);
  return p;
}

struct Table {
  int* at;
  long long stride;
  int rows, cols;
};
Table table_of(PyObject* o, int index) {
  const Tensor& t = tensor(o, "block_table");
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && on(t, index) && t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1),
                    "block_table must be an int32 tensor [rows, cols], its rows contiguous, on CUDA device ", index);
  return {static_cast<int*>(t.data_ptr()), t.size(0) > 1 ? t.stride(0) : t.size(1), i32(t.size(0), "block_table"),
          i32(t.size(1), "block_table")};
}

// The two pools of a cache.
struct Cache {
  const Tensor &k, &v;
  bool fp8;
  int pages, page_size, Hk, d;
  Cache(PyObject* ko, PyObject* vo, int index) : k(tensor(ko, "k_cache")), v(tensor(vo, "v_cache")) {
    const auto type = k.scalar_type();
    TORCH_CHECK_VALUE(k.dim() == 4 && v.scalar_type() == type && on(k, index) && on(v, index) && v.sizes() == k.sizes() &&
                          (type == at::kBFloat16 || type == at::kFloat8_e4m3fn || type == at::kByte) && k.stride(3) == 1,
                      "k_cache, v_cache must be bf16 or E4M3 tensors [pages, page_size, Hk, d] of one shape, the last "
                      "dimension contiguous, on CUDA device ", index);
    for (int64_t i = 0; i < 4; ++i)  // (of one element, the stride is not looked at)
      TORCH_CHECK_VALUE(k.size(i) <= 1 || v.stride(i) == k.stride(i), "k_cache and v_cache must have the same strides");
    fp8 = type != at::kBFloat16;
    pages = i32(k.size(0), "pages"), page_size = i32(k.size(1), "page_size"), Hk = i32(k.size(2), "heads");
    d = i32(k.size(3), "d");
  }
  const float* descale(PyObject* o, const char* name, int index) const {
    if (o == Py_None) return nullptr;
    TORCH_CHECK_VALUE(fp8, name, " belongs to an E4M3 cache");
    return static_cast<const float*>(vec(o, name, at::kFloat, index, Hk));
  }
};

// Runs `call(stream)` on the device's current stream, without the interpreter's lock.
template <typename F>
fa_status_t launch(int index, F call) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
  fa_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = call(stream);
  Py_END_ALLOW_THREADS;
  return st;
}

template <typename... T>
PyObject* tensors(const T&... t) {
  PyObject* items[] = {THPVariable_Wrap(t)...};
  PyObject* r = PyTuple_New(sizeof...(T));
  bool ok = r != nullptr;
  for (PyObject* x : items) ok = ok && x;
  for (size_t i = 0; i < sizeof...(T); ++i) {
    if (ok) PyTuple_SET_ITEM(r, i, items[i]);
    else Py_XDECREF(items[i]);
  }
  if (!ok) Py_CLEAR(r);
  return r;
}

void count(Py_ssize_t have, Py_ssize_t want) {
  TORCH_CHECK_TYPE(have == want, "expected ", want, " arguments, got ", have);
}

struct Qk {
  const Tensor &q, &k;
  int index;
  int B, N, Hq, Hk, d;
  Qk(PyObject* qo, PyObject* ko) : q(rows(qo, "q", 4, -1)), k(rows(ko, "k", 4, q.get_device())), index(q.get_device()) {
    TORCH_CHECK_VALUE(k.size(0) == q.size(0) && k.size(1) == q.size(1) && k.size(3) == q.size(3),
                      "q [B,N,Hq,d] and k [B,N,Hk,d] must agree in B, N and d");
    B = i32(q.size(0), "B"), N = i32(q.size(1), "N"), Hq = i32(q.size(2), "Hq"), Hk = i32(k.size(2), "Hk");
    d = i32(q.size(3), "d");
  }
};

// q, k, wq, wk, rope, positions, eps, interleaved, q_out, k_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Qk x(a[0], a[1]);
  const void* wq = vec_or_null(a[2], "wq", at::kBFloat16, x.index, x.d);
  const void* wk = vec_or_null(a[3], "wk", at::kBFloat16, x.index, x.d);
  const Rope r = rope_of(a[4], x.index);
  const Positions p = positions_of(a[5], x.B, x.N, x.index);
  const float eps = number(a[6]);
  const int inter = truth(a[7]);
  const Tensor qo = output(a[8], "q_out", at::kBFloat16, x.index, {x.B, x.Hq, x.N, x.d});
  const Tensor ko = output(a[9], "k_out", at::kBFloat16, x.index, {x.B, x.Hk, x.N, x.d});
  const fa_status_t st = launch(x.index, [&](void* stream) {
    return c_norm_rope(x.q.data_ptr(), x.k.data_ptr(), wq, wk, r.table, r.rows, r.rot, inter, p.at, p.stride, qo.data_ptr(),
                       ko.data_ptr(), x.B, x.N, x.Hq, x.Hk, x.d, x.q.stride(0), x.q.stride(1), x.q.stride(2),
                       x.k.stride(0), x.k.stride(1), x.k.stride(2), eps, stream);
  });
  return st ? PyLong_FromLong(st) : tensors(qo, ko);
  END_HANDLE_TH_ERRORS
}

// gq, gk, q, k, wq, wk, rope, positions, eps, interleaved, dq, dk, workspace
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Qk x(a[2], a[3]);
  const Tensor &gq = tensor(a[0], "gq"), &gk = tensor(a[1], "gk");
  TORCH_CHECK_VALUE(gq.sizes() == at::IntArrayRef({x.B, x.Hq, x.N, x.d}) && gk.sizes() == at::IntArrayRef({x.B, x.Hk, x.N, x.d}),
                    "gq and gk must be [B,Hq,N,d] and [B,Hk,N,d]");
  const void* gqp = vec(a[0], "gq", at::kBFloat16, x.index, gq.numel());
  const void* gkp = vec(a[1], "gk", at::kBFloat16, x.index, gk.numel());
  const void* wq = vec_or_null(a[4], "wq", at::kBFloat16, x.index, x.d);
  const void* wk = vec_or_null(a[5], "wk", at::kBFloat16, x.index, x.d);
  const Rope r = rope_of(a[6], x.index);
  const Positions p = positions_of(a[7], x.B, x.N, x.index);
  const float eps = number(a[8]);
  const int inter = truth(a[9]);
  auto gradient = [&](PyObject* o, const char* name, const Tensor& like) {
    if (o == Py_None) return fresh(like.sizes(), at::kBFloat16, x.index);
    const Tensor& t = rows(o, name, 4, x.index);
    TORCH_CHECK_VALUE(t.sizes() == like.sizes(), name, " must have the shape ", like.sizes());
    distinct(t, name);
    return t;
  };
  const Tensor dq = gradient(a[10], "dq", x.q), dk = gradient(a[11], "dk", x.k);
  const Tensor dwq = fresh({x.d}, at::kFloat, x.index), dwk = fresh({x.d}, at::kFloat, x.index);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(x.index));
  const Workspace ws(a[12], c_norm_rope_bwd_bytes(x.B, x.N, x.Hq, x.Hk, x.d), x.index);
  const fa_status_t st = launch(x.index, [&](void* stream) {
    return c_norm_rope_bwd(gqp, gkp, x.q.data_ptr(), x.k.data_ptr(), wq, wk, r.table, r.rows, r.rot, inter, p.at, p.stride,
                           dq.data_ptr(), dk.data_ptr(), static_cast<float*>(dwq.data_ptr()),
                           static_cast<float*>(dwk.data_ptr()), ws.at(), ws.bytes(), x.B, x.N, x.Hq, x.Hk, x.d,
                           x.q.stride(0), x.q.stride(1), x.q.stride(2), x.k.stride(0), x.k.stride(1), x.k.stride(2),
                           dq.stride(0), dq.stride(1), dq.stride(2), dk.stride(0), dk.stride(1), dk.stride(2), eps, stream);
  });
  return st ? PyLong_FromLong(st) : tensors(dq, dk, dwq, dwk);
  END_HANDLE_TH_ERRORS
}

// cached, new_tokens, block_table, free_pages, free_count, page_size, lens, cu_tokens, slots, positions,
// token_req, free_count_out, status
PyObject* paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Tensor& c = tensor(a[0], "cached");
  TORCH_CHECK_VALUE(c.is_cuda(), "cached must be a CUDA tensor");
  const int index = c.get_device();
  const int R = i32(c.numel(), "requests"), most = i32(tensor(a[8], "slots").numel(), "slots");
  const int pool = i32(tensor(a[3], "free_pages").numel(), "free_pages"), page_size = integer(a[5], "page_size");
  const Table t = table_of(a[2], index);
  TORCH_CHECK_VALUE(t.rows == R, "block_table must have a row for each request");
  auto ints = [&](int i, const char* name, int64_t numel) { return static_cast<int*>(vec(a[i], name, at::kInt, index, numel)); };
  const int *cached = ints(0, "cached", R), *fresh = ints(1, "new_tokens", R), *free_count = ints(4, "free_count", 1);
  int *free_pages = ints(3, "free_pages", pool), *lens = ints(6, "lens", R), *cu = ints(7, "cu_tokens", (int64_t)R + 1);
  long long* slots = static_cast<long long*>(vec(a[8], "slots", at::kLong, index, most));
  int *positions = ints(9, "positions", most), *req = ints(10, "token_req", most);
  int *count_out = ints(11, "free_count_out", 1), *status = ints(12, "status", 1);
  const fa_status_t st = launch(index, [&](void* stream) {
    return c_plan(cached, fresh, t.at, t.stride, t.cols, free_pages, pool, free_count, page_size, R, most, lens, cu, slots,
                  positions, req, count_out, status, stream);
  });
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// q, k, v, wq, wk, rope, positions, slots, k_cache, v_cache, eps, interleaved, k_descale, v_descale, q_out
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const Tensor& q = rows(a[0], "q", 3, -1);
  const int index = q.get_device(), T = i32(q.size(0), "T"), Hq = i32(q.size(1), "Hq"), d = i32(q.size(2), "d");
  const Tensor &k = rows(a[1], "k", 3, index), &v = rows(a[2], "v", 3, index);
  const Cache c(a[8], a[9], index);
  TORCH_CHECK_VALUE(k.sizes() == at::IntArrayRef({T, c.Hk, d}) && v.sizes() == k.sizes() && c.d == d,
                    "k and v must be [T,Hk,d] with the cache's Hk and q's T and d");
  distinct(c.k, "k_cache");
  distinct(c.v, "v_cache");
  TORCH_CHECK_VALUE(c.k.numel() == 0 || c.k.data_ptr() != c.v.data_ptr(), "k_cache and v_cache must not be one tensor");
  const void* wq = vec_or_null(a[3], "wq", at::kBFloat16, index, d);
  const void* wk = vec_or_null(a[4], "wk", at::kBFloat16, index, d);
  const Rope r = rope_of(a[5], index);
  TORCH_CHECK_VALUE(r.rot == 0 || a[6] != Py_None, "positions are needed for the rotation");
  const int* positions = static_cast<const int*>(vec_or_null(a[6], "positions", at::kInt, index, T));
  const long long* slots = static_cast<const long long*>(vec(a[7], "slots", at::kLong, index, T));
  const float eps = number(a[10]);
  const int inter = truth(a[11]);
  const float *kd = c.descale(a[12], "k_descale", index), *vd = c.descale(a[13], "v_descale", index);
  const Tensor qo = output(a[14], "q_out", at::kBFloat16, index, {T, Hq, d});
  const fa_status_t st = launch(index, [&](void* stream) {
    return c_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), wq, wk, r.table, r.rows, r.rot, inter, positions, slots,
                    qo.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.fp8, kd, vd, c.pages, c.page_size, T, Hq, c.Hk, d,
                    q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1), c.k.stride(0),
                    c.k.stride(1), c.k.stride(2), eps, stream);
  });
  return st ? PyLong_FromLong(st) : THPVariable_Wrap(qo);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, lens, scale, req, k_descale, v_descale, out, lse, workspace
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Tensor& q = rows(a[0], "q", 3, -1);
  const int index = q.get_device(), T = i32(q.size(0), "T"), Hq = i32(q.size(1), "Hq"), d = i32(q.size(2), "d");
  const Cache c(a[1], a[2], index);
  TORCH_CHECK_VALUE(c.d == d && c.Hk > 0 && Hq % c.Hk == 0, "q's heads must be a multiple of the cache's, with its d");
  const Table t = table_of(a[3], index);
  const int* lens = static_cast<const int*>(vec(a[4], "lens", at::kInt, index, T));
  const float scale = a[5] == Py_None ? static_cast<float>(1.0 / std::sqrt(std::max(d, 1))) : number(a[5]);
  const int* req = static_cast<const int*>(vec_or_null(a[6], "req", at::kInt, index, T));
  const float *kd = c.descale(a[7], "k_descale", index), *vd = c.descale(a[8], "v_descale", index);
  const Tensor out = output(a[9], "out", at::kBFloat16, index, {T, Hq, d});
  const Tensor lse = output(a[10], "lse", at::kFloat, index, {T, Hq});
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  const Workspace ws(a[11], c_decode_bytes(T, Hq, c.Hk, d), index);
  const fa_status_t st = launch(index, [&](void* stream) {
    return c_decode(q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.fp8, kd, vd, t.at, t.stride, t.rows, t.cols, lens, req,
                    out.data_ptr(), static_cast<float*>(lse.data_ptr()), ws.at(), ws.bytes(), c.pages, c.page_size, T,
                    Hq, c.Hk, d, q.stride(0), q.stride(1), c.k.stride(0), c.k.stride(1), c.k.stride(2), scale, stream);
  });
  return st ? PyLong_FromLong(st) : tensors(out, lse);
  END_HANDLE_TH_ERRORS
}

// The addresses of the library's functions, by name.
PyObject* bind(PyObject*, PyObject* names) {
  HANDLE_TH_ERRORS
  auto get = [&](const char* name, auto& f) {
    PyObject* o = PyDict_GetItemString(names, name);  // borrowed
    TORCH_CHECK_VALUE(o, "no address of ", name);
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(p, "no address of ", name);
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p);
  };
  TORCH_CHECK_TYPE(PyDict_Check(names), "bind takes a dict");
  get("fa_qk_norm_rope", c_norm_rope);
  get("fa_qk_norm_rope_bwd", c_norm_rope_bwd);
  get("fa_qk_norm_rope_bwd_workspace_bytes", c_norm_rope_bwd_bytes);
  get("fa_paged_plan", c_plan);
  get("fa_paged_append", c_append);
  get("fa_paged_decode", c_decode);
  get("fa_paged_decode_workspace_bytes", c_decode_bytes);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FA_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_FAST(qk_norm_rope), FA_FAST(qk_norm_rope_backward), FA_FAST(paged_plan), FA_FAST(paged_append),
                         FA_FAST(paged_decode), {"bind", bind, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
