// paged_binding.cpp -- the paged-cache calls on torch tensors: checks, outputs
// and workspaces from torch's allocator, torch's current stream, and the C ABI
// of include/fa2.h.  A Python extension module because a serving step makes
// these calls once per layer on small tensors: marshalled in Python they took
// 22 us (forward) and 20 us (plan) of host time on a GB300's CPU, most of it
// outside the two launches.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <exception>

#include "../../include/fa2.h"

namespace {

// Python's error is set; the caller returns NULL.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, const char* name = "", long long a = 0, long long b = 0) {
  PyErr_Format(type, fmt, name, a, b);
  throw Raised();
}

// A tensor argument; NULL for None where that is allowed.
const at::Tensor* tensor(PyObject* x, const char* name, bool optional = false) {
  if (optional && x == Py_None) return nullptr;
  if (!THPVariable_Check(x)) raise(PyExc_TypeError, "%s must be a torch tensor", name);
  return &THPVariable_Unpack(x);
}

int integer(PyObject* x, const char* name) {
  const long long v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT_MIN || v > INT_MAX) raise(PyExc_ValueError, "%s is out of range: %lld", name, v);
  return (int)v;
}

int size(int64_t n, const char* name) {
  if (n > INT_MAX) raise(PyExc_ValueError, "%s has %lld elements in a dimension, more than the calls take", name, n);
  return (int)n;
}

// Contiguous int32 [n] on `like`'s device.
int* int32_1d(const at::Tensor& t, const char* name, const at::Device& dev, int64_t n) {
  if (t.scalar_type() != at::kInt || t.device() != dev || t.dim() != 1 || (t.numel() > 1 && t.stride(0) != 1))
    raise(PyExc_ValueError, "%s must be a contiguous int32 tensor [n] on the call's CUDA device", name);
  if (t.numel() != n) raise(PyExc_ValueError, "%s must have %lld elements, has %lld", name, n, t.numel());
  return t.data_ptr<int>();
}

void check_table(const at::Tensor& t, const at::Device& dev, int64_t rows) {
  if (t.scalar_type() != at::kInt || t.device() != dev || t.dim() != 2 || t.size(0) != rows)
    raise(PyExc_ValueError, "%s must be an int32 tensor [%lld, max_pages] on the call's CUDA device", "block_table", rows);
  if (t.stride(1) != 1 && t.size(1) > 1)
    raise(PyExc_ValueError, "%s must have a contiguous last dimension", "block_table");
}

int dtype_code(at::ScalarType t) { return t == at::kHalf ? FA2_FP16 : t == at::kBFloat16 ? FA2_BF16 : -1; }

// k_cache, v_cache [num_pages, H_kv, page_size, d].
fa2_paged_cache cache(const at::Tensor& k, const at::Tensor& v) {
  if (k.dim() != 4 || v.sizes() != k.sizes())
    raise(PyExc_ValueError, "%s must share one [num_pages, H_kv, page_size, d] shape", "k_cache and v_cache");
  if (!k.is_cuda() || v.device() != k.device())
    raise(PyExc_ValueError, "%s must be CUDA tensors on one device", "k_cache and v_cache");
  fa2_paged_cache c;
  c.dtype = dtype_code(k.scalar_type());
  if (c.dtype < 0 || v.scalar_type() != k.scalar_type())
    raise(PyExc_TypeError, "%s must share one dtype, float16 or bfloat16", "k_cache and v_cache");
  if (k.stride(3) != 1 || v.stride(3) != 1)
    raise(PyExc_ValueError, "%s must have a contiguous last dimension", "k_cache and v_cache");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  for (int i = 0; i < 3; ++i) {
    c.k_strides[i] = k.stride(i);
    c.v_strides[i] = v.stride(i);
  }
  c.num_pages = size(k.size(0), "k_cache");
  c.heads = size(k.size(1), "k_cache");
  c.page_size = size(k.size(2), "k_cache");
  c.head_dim = size(k.size(3), "k_cache");
  return c;
}

// The same of 8-bit rows: codes [num_pages, H_kv, page_size, d], exponents [num_pages, H_kv, page_size].
fa2_paged_cache_fp8 cache_fp8(const at::Tensor& k, const at::Tensor& v, const at::Tensor& ke, const at::Tensor& ve) {
  if (k.dim() != 4 || v.sizes() != k.sizes())
    raise(PyExc_ValueError, "%s must share one [num_pages, H_kv, page_size, d] shape", "k_cache and v_cache");
  if (ke.dim() != 3 || ve.sizes() != ke.sizes() || ke.sizes() != k.sizes().slice(0, 3))
    raise(PyExc_ValueError, "%s must be [num_pages, H_kv, page_size], as the caches", "k_exps and v_exps");
  if (!k.is_cuda() || v.device() != k.device() || ke.device() != k.device() || ve.device() != k.device())
    raise(PyExc_ValueError, "%s must be CUDA tensors on one device", "the caches and their exponents");
  if (k.scalar_type() != at::kFloat8_e4m3fn || v.scalar_type() != at::kFloat8_e4m3fn)
    raise(PyExc_TypeError, "%s must be float8_e4m3fn", "k_cache and v_cache");
  if (ke.scalar_type() != at::kByte || ve.scalar_type() != at::kByte)
    raise(PyExc_TypeError, "%s must be uint8", "k_exps and v_exps");
  if (k.stride(3) != 1 || v.stride(3) != 1 || (ke.size(2) > 1 && (ke.stride(2) != 1 || ve.stride(2) != 1)))
    raise(PyExc_ValueError, "%s must have a contiguous last dimension", "the caches and their exponents");
  fa2_paged_cache_fp8 c;
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.k_exps = ke.data_ptr();
  c.v_exps = ve.data_ptr();
  for (int i = 0; i < 3; ++i) {
    c.k_strides[i] = k.stride(i);
    c.v_strides[i] = v.stride(i);
  }
  for (int i = 0; i < 2; ++i) {
    c.k_exp_strides[i] = ke.stride(i);
    c.v_exp_strides[i] = ve.stride(i);
  }
  c.num_pages = size(k.size(0), "k_cache");
  c.heads = size(k.size(1), "k_cache");
  c.page_size = size(k.size(2), "k_cache");
  c.head_dim = size(k.size(3), "k_cache");
  return c;
}

// An uninitialised contiguous tensor, past the dispatcher (host time of a plan,
// four outputs, 7.7 -> 6.5 us; of a forward, two and a workspace, 9.6 -> 8.3).
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, const at::Device& dev) {
  return at::Tensor(at::detail::empty_cuda(sizes, dtype, dev, std::nullopt));
}

// Torch is told that a caller's tensor was written in place, so that a backward
// pass that kept it says so.  (Inference tensors keep no such count.)
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void* current_stream(const at::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// Fills what follows a forward's cache in its parameters (fa2_paged_params or fa2_paged_fp8_params).
template <class P>
void fill(P& p, const at::Tensor& q, const at::Tensor& k, const at::Tensor& table, const at::Tensor& cu,
          const at::Tensor& lens, PyObject* max_q) {
  const at::Device dev = k.device();
  if (q.dim() != 3 || q.size(2) != k.size(3))
    raise(PyExc_ValueError, "%s must be [total_q, H, d] with the cache's head dim", "q");
  if (q.device() != dev || q.stride(2) != 1)
    raise(PyExc_ValueError, "%s must be on the cache's device with a contiguous last dimension", "q");
  p.batch = size(lens.numel(), "seqlens_k");
  p.seqlens_k = int32_1d(lens, "seqlens_k", dev, p.batch);
  p.cu_seqlens_q = int32_1d(cu, "cu_seqlens_q", dev, (int64_t)p.batch + 1);
  check_table(table, dev, p.batch);
  p.block_table = table.data_ptr<int>();
  p.table_stride = table.stride(0);
  p.max_pages = size(table.size(1), "block_table");
  p.q = q.data_ptr();
  p.q_strides[0] = q.stride(0);
  p.q_strides[1] = q.stride(1);
  p.total_q = size(q.size(0), "q");
  p.heads = size(q.size(1), "q");
  p.max_seqlen_q = max_q == Py_None ? p.total_q : integer(max_q, "max_seqlen_q");
}

// The inputs of a paged forward's parameters.
fa2_paged_params forward_params(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& table,
                                const at::Tensor& cu, const at::Tensor& lens, PyObject* max_q) {
  fa2_paged_params p;
  std::memset(&p, 0, sizeof(p));
  p.cache = cache(k, v);
  if (q.scalar_type() != k.scalar_type()) raise(PyExc_TypeError, "%s and the cache must share one dtype", "q");
  fill(p, q, k, table, cu, lens, max_q);
  return p;
}

// The same on 8-bit rows; a: q, k_cache, v_cache, k_exps, v_exps, block_table, cu_seqlens_q, seqlens_k.
fa2_paged_fp8_params forward_params_fp8(PyObject* const* a, PyObject* max_q) {
  const at::Tensor &q = *tensor(a[0], "q"), &k = *tensor(a[1], "k_cache");
  fa2_paged_fp8_params p;
  std::memset(&p, 0, sizeof(p));
  p.cache = cache_fp8(k, *tensor(a[2], "v_cache"), *tensor(a[3], "k_exps"), *tensor(a[4], "v_exps"));
  p.dtype = dtype_code(q.scalar_type());
  if (p.dtype < 0) raise(PyExc_TypeError, "%s must be float16 or bfloat16", "q");
  fill(p, q, k, *tensor(a[5], "block_table"), *tensor(a[6], "cu_seqlens_q"), *tensor(a[7], "seqlens_k"), max_q);
  return p;
}

// A forward's scale: a number, or None for 1 / sqrt(d).
float scale_of(PyObject* x, int d) {
  if (x == Py_None) return (float)(1.0 / std::sqrt((double)d));
  const double s = PyFloat_AsDouble(x);
  if (s == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)s;
}

// Checks a forward's o, lse and workspace arguments (a[0] .. a[2], each may be None), makes what is missing
// (`need` bytes of workspace), runs `call(workspace, bytes, stream)`: (o, lse), or a nonzero fa2_status.
template <class P, class F>
PyObject* outputs(P& p, const at::Tensor& q, PyObject* const* a, size_t need, F&& call) {
  const at::Tensor *o_in = tensor(a[0], "o", true), *lse_in = tensor(a[1], "lse", true),
                   *ws_in = tensor(a[2], "workspace", true);
  const at::Device dev = q.device();
  if (o_in && (o_in->sizes() != q.sizes() || o_in->scalar_type() != q.scalar_type() || o_in->device() != dev ||
               o_in->stride(2) != 1))
    raise(PyExc_ValueError, "%s must have q's shape, dtype and device with a contiguous last dimension", "o");
  if (lse_in && (lse_in->dim() != 2 || lse_in->size(0) != q.size(1) || lse_in->size(1) != q.size(0) ||
                 lse_in->scalar_type() != at::kFloat || lse_in->device() != dev ||
                 (lse_in->stride(1) != 1 && lse_in->size(1) > 1)))
    raise(PyExc_ValueError, "%s must be float32 [H, total_q] on q's device with a contiguous last dimension", "lse");
  if (ws_in && (ws_in->device() != dev || !ws_in->is_contiguous()))
    raise(PyExc_ValueError, "%s must be a contiguous tensor on q's device", "workspace");
  const at::Tensor o = o_in ? *o_in : empty(q.sizes(), q.scalar_type(), dev);
  const at::Tensor lse = lse_in ? *lse_in : empty({q.size(1), q.size(0)}, at::kFloat, dev);
  // a workspace made here is a block of the current stream, given back once the kernels are queued: its next
  // user on that stream follows them
  const at::Tensor ws = ws_in ? *ws_in : empty({(int64_t)(need ? need : 256)}, at::kByte, dev);
  p.o = o.data_ptr();
  p.o_strides[0] = o.stride(0);
  p.o_strides[1] = o.stride(1);
  p.lse = lse.data_ptr<float>();
  p.lse_stride = lse.stride(0);
  const int rc = call(ws.data_ptr(), ws.nbytes(), current_stream(dev));
  if (rc) return PyLong_FromLong(rc);
  if (o_in) written(o);
  if (lse_in) written(lse);
  if (ws_in) written(ws);
  PyObject* out_o = o_in ? Py_NewRef(a[0]) : THPVariable_Wrap(o);
  PyObject* out_l = lse_in ? Py_NewRef(a[1]) : THPVariable_Wrap(lse);
  return Py_BuildValue("(NN)", out_o, out_l);
}

// Runs `f` with C++ exceptions turned into Python's, torch's into their own
// types (an allocation that fails: torch.OutOfMemoryError).
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

bool arguments(Py_ssize_t n, Py_ssize_t want, const char* name) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
  return false;
}

// forward(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, o, lse, workspace, scale, window_left,
//         window_right, prefix_len, max_seqlen_q, sink_len): (o, lse), or a nonzero fa2_status
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 15, "forward")) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &q = *tensor(a[0], "q"), &k = *tensor(a[1], "k_cache"), &v = *tensor(a[2], "v_cache");
    const at::Tensor &table = *tensor(a[3], "block_table"), &cu = *tensor(a[4], "cu_seqlens_q"),
                     &lens = *tensor(a[5], "seqlens_k");
    fa2_paged_params p = forward_params(q, k, v, table, cu, lens, a[13]);
    p.scale = scale_of(a[9], p.cache.head_dim);
    p.window_left = integer(a[10], "window_left");
    p.window_right = integer(a[11], "window_right");
    p.prefix_len = integer(a[12], "prefix_len");
    p.sink_len = integer(a[14], "sink_len");
    const c10::cuda::CUDAGuard guard(q.device());
    return outputs(p, q, a + 6, a[8] == Py_None ? fa2_paged_fwd_workspace_bytes(&p) : 0,
                   [&](void* ws, size_t bytes, void* stream) { return fa2_paged_fwd(&p, ws, bytes, stream); });
  });
}

// The same with groups: a: q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, cu_groups, shared_lens.
fa2_paged_shared_params forward_params_shared(PyObject* const* a, PyObject* max_q) {
  const at::Tensor &q = *tensor(a[0], "q"), &k = *tensor(a[1], "k_cache");
  const at::Tensor &groups = *tensor(a[6], "cu_groups"), &shared = *tensor(a[7], "shared_lens");
  fa2_paged_shared_params p;
  std::memset(&p, 0, sizeof(p));
  p.fwd = forward_params(q, k, *tensor(a[2], "v_cache"), *tensor(a[3], "block_table"), *tensor(a[4], "cu_seqlens_q"),
                         *tensor(a[5], "seqlens_k"), max_q);
  p.num_groups = size(shared.numel(), "shared_lens");
  p.shared_lens = int32_1d(shared, "shared_lens", k.device(), p.num_groups);
  p.cu_groups = int32_1d(groups, "cu_groups", k.device(), (int64_t)p.num_groups + 1);
  p.fwd.window_left = -1;
  return p;
}

// forward_shared(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, cu_groups, shared_lens, o, lse, workspace,
//                scale, window_right, max_seqlen_q): (o, lse), or a nonzero fa2_status
PyObject* forward_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 14, "forward_shared")) return nullptr;
  return guarded([&]() -> PyObject* {
    fa2_paged_shared_params p = forward_params_shared(a, a[13]);
    const at::Tensor& q = *tensor(a[0], "q");
    p.fwd.scale = scale_of(a[11], p.fwd.cache.head_dim);
    p.fwd.window_right = integer(a[12], "window_right");
    const c10::cuda::CUDAGuard guard(q.device());
    return outputs(p.fwd, q, a + 8, a[10] == Py_None ? fa2_paged_fwd_shared_workspace_bytes(&p) : 0,
                   [&](void* ws, size_t bytes, void* stream) { return fa2_paged_fwd_shared(&p, ws, bytes, stream); });
  });
}

// workspace_bytes_shared(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, cu_groups, shared_lens, max_seqlen_q)
PyObject* workspace_bytes_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 9, "workspace_bytes_shared")) return nullptr;
  return guarded([&]() -> PyObject* {
    const fa2_paged_shared_params p = forward_params_shared(a, a[8]);
    return PyLong_FromSize_t(fa2_paged_fwd_shared_workspace_bytes(&p));
  });
}

// forward_fp8(q, k_cache, v_cache, k_exps, v_exps, block_table, cu_seqlens_q, seqlens_k, o, lse, workspace, scale,
//             window_left, window_right, prefix_len, max_seqlen_q, sink_len): (o, lse), or a nonzero fa2_status
PyObject* forward_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 17, "forward_fp8")) return nullptr;
  return guarded([&]() -> PyObject* {
    fa2_paged_fp8_params p = forward_params_fp8(a, a[15]);
    const at::Tensor& q = *tensor(a[0], "q");
    p.scale = scale_of(a[11], p.cache.head_dim);
    p.window_left = integer(a[12], "window_left");
    p.window_right = integer(a[13], "window_right");
    p.prefix_len = integer(a[14], "prefix_len");
    p.sink_len = integer(a[16], "sink_len");
    const c10::cuda::CUDAGuard guard(q.device());
    return outputs(p, q, a + 8, a[10] == Py_None ? fa2_paged_fwd_fp8_workspace_bytes(&p) : 0,
                   [&](void* ws, size_t bytes, void* stream) { return fa2_paged_fwd_fp8(&p, ws, bytes, stream); });
  });
}

// workspace_bytes_fp8(q, k_cache, v_cache, k_exps, v_exps, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q)
PyObject* workspace_bytes_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 9, "workspace_bytes_fp8")) return nullptr;
  return guarded([&]() -> PyObject* {
    const fa2_paged_fp8_params p = forward_params_fp8(a, a[8]);
    return PyLong_FromSize_t(fa2_paged_fwd_fp8_workspace_bytes(&p));
  });
}

// workspace_bytes(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q)
PyObject* workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 7, "workspace_bytes")) return nullptr;
  return guarded([&]() -> PyObject* {
    const fa2_paged_params p =
        forward_params(*tensor(a[0], "q"), *tensor(a[1], "k_cache"), *tensor(a[2], "v_cache"),
                       *tensor(a[3], "block_table"), *tensor(a[4], "cu_seqlens_q"), *tensor(a[5], "seqlens_k"), a[6]);
    return PyLong_FromSize_t(fa2_paged_fwd_workspace_bytes(&p));
  });
}

// append(k, v, slots, k_cache, v_cache): fa2_status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 5, "append")) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &k = *tensor(a[0], "k"), &v = *tensor(a[1], "v"), &slots = *tensor(a[2], "slots");
    const at::Tensor &kc = *tensor(a[3], "k_cache"), &vc = *tensor(a[4], "v_cache");
    fa2_paged_append_params p;
    std::memset(&p, 0, sizeof(p));
    p.cache = cache(kc, vc);
    const at::Device dev = kc.device();
    if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(1) != kc.size(1) || k.size(2) != kc.size(3))
      raise(PyExc_ValueError, "%s must be [total, H_kv, d] with the cache's heads and head dim", "k and v");
    if (k.device() != dev || v.device() != dev || k.stride(2) != 1 || v.stride(2) != 1)
      raise(PyExc_ValueError, "%s must be on the cache's device with a contiguous last dimension", "k and v");
    if (k.scalar_type() != kc.scalar_type() || v.scalar_type() != kc.scalar_type())
      raise(PyExc_TypeError, "%s and the cache must share one dtype", "k, v");
    p.total = size(k.size(0), "k");
    p.slots = int32_1d(slots, "slots", dev, p.total);
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    for (int i = 0; i < 2; ++i) {
      p.k_strides[i] = k.stride(i);
      p.v_strides[i] = v.stride(i);
    }
    const c10::cuda::CUDAGuard guard(dev);
    const int rc = fa2_paged_append(&p, current_stream(dev));
    if (rc == FA2_OK) {
      written(kc);
      written(vc);
    }
    return PyLong_FromLong(rc);
  });
}

// Fills the parameters of fa2_paged_append_fp8 or fa2_paged_read_fp8.
template <class P>
P rows_fp8(const at::Tensor& k, const at::Tensor& v, const at::Tensor& slots, const at::Tensor& kc, const at::Tensor& vc,
           const at::Tensor& ke, const at::Tensor& ve) {
  P p;
  std::memset(&p, 0, sizeof(p));
  p.cache = cache_fp8(kc, vc, ke, ve);
  const at::Device dev = kc.device();
  if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(1) != kc.size(1) || k.size(2) != kc.size(3))
    raise(PyExc_ValueError, "%s must be [total, H_kv, d] with the cache's heads and head dim", "k and v");
  if (k.device() != dev || v.device() != dev || k.stride(2) != 1 || v.stride(2) != 1)
    raise(PyExc_ValueError, "%s must be on the cache's device with a contiguous last dimension", "k and v");
  p.dtype = dtype_code(k.scalar_type());
  if (p.dtype < 0 || v.scalar_type() != k.scalar_type())
    raise(PyExc_TypeError, "%s must share one dtype, float16 or bfloat16", "k and v");
  p.total = size(k.size(0), "k");
  p.slots = int32_1d(slots, "slots", dev, p.total);
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  for (int i = 0; i < 2; ++i) {
    p.k_strides[i] = k.stride(i);
    p.v_strides[i] = v.stride(i);
  }
  return p;
}

// append_fp8(k, v, slots, k_cache, v_cache, k_exps, v_exps): fa2_status
PyObject* append_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 7, "append_fp8")) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &kc = *tensor(a[3], "k_cache"), &vc = *tensor(a[4], "v_cache"), &ke = *tensor(a[5], "k_exps"),
                     &ve = *tensor(a[6], "v_exps");
    const auto p = rows_fp8<fa2_paged_append_fp8_params>(*tensor(a[0], "k"), *tensor(a[1], "v"), *tensor(a[2], "slots"), kc,
                                                         vc, ke, ve);
    const c10::cuda::CUDAGuard guard(kc.device());
    const int rc = fa2_paged_append_fp8(&p, current_stream(kc.device()));
    if (rc == FA2_OK)
      for (const at::Tensor* t : {&kc, &vc, &ke, &ve}) written(*t);
    return PyLong_FromLong(rc);
  });
}

// read_fp8(slots, k_cache, v_cache, k_exps, v_exps, k, v, bf16): (k, v), or a nonzero fa2_status; k and v, or None
// for new ones, in bfloat16 or float16 as `bf16` says
PyObject* read_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 8, "read_fp8")) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &slots = *tensor(a[0], "slots"), &kc = *tensor(a[1], "k_cache"), &vc = *tensor(a[2], "v_cache"),
                     &ke = *tensor(a[3], "k_exps"), &ve = *tensor(a[4], "v_exps");
    const at::Tensor* in[2] = {tensor(a[5], "k", true), tensor(a[6], "v", true)};
    if (!kc.is_cuda() || kc.dim() != 4)
      raise(PyExc_ValueError, "%s must be a CUDA tensor [num_pages, H_kv, page_size, d]", "k_cache");
    const c10::cuda::CUDAGuard guard(kc.device());
    const at::ScalarType type = PyObject_IsTrue(a[7]) ? at::kBFloat16 : at::kHalf;
    at::Tensor out[2];
    for (int i = 0; i < 2; ++i)
      out[i] = in[i] ? *in[i] : empty({slots.numel(), kc.size(1), kc.size(3)}, type, kc.device());
    const auto p = rows_fp8<fa2_paged_read_fp8_params>(out[0], out[1], slots, kc, vc, ke, ve);
    const int rc = fa2_paged_read_fp8(&p, current_stream(kc.device()));
    if (rc) return PyLong_FromLong(rc);
    PyObject* result[2];
    for (int i = 0; i < 2; ++i) {
      if (in[i]) written(out[i]);
      result[i] = in[i] ? Py_NewRef(a[5 + i]) : THPVariable_Wrap(out[i]);
    }
    return Py_BuildValue("(NN)", result[0], result[1]);
  });
}

// plan(context_lens, query_lens, block_table, free_pages, free_count, num_pages, page_size, total_q, cu_seqlens_q,
//      seqlens_k, slots, free_left): (cu_seqlens_q, seqlens_k, slots, free_left), or a nonzero fa2_status
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 12, "plan")) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &ctx = *tensor(a[0], "context_lens"), &query = *tensor(a[1], "query_lens"),
                     &table = *tensor(a[2], "block_table"), &free = *tensor(a[3], "free_pages"),
                     &count = *tensor(a[4], "free_count");
    if (!ctx.is_cuda() || ctx.dim() != 1)
      raise(PyExc_ValueError, "%s must be an int32 CUDA tensor [B]", "context_lens");
    const at::Device dev = ctx.device();
    fa2_paged_plan_params p;
    std::memset(&p, 0, sizeof(p));
    p.batch = size(ctx.numel(), "context_lens");
    p.context_lens = int32_1d(ctx, "context_lens", dev, p.batch);
    p.query_lens = int32_1d(query, "query_lens", dev, p.batch);
    check_table(table, dev, p.batch);
    p.block_table = table.data_ptr<int>();
    p.table_stride = table.stride(0);
    p.max_pages = size(table.size(1), "block_table");
    p.num_free = size(free.numel(), "free_pages");
    p.free_pages = int32_1d(free, "free_pages", dev, p.num_free);
    p.free_count = int32_1d(count, "free_count", dev, 1);
    p.num_pages = integer(a[5], "num_pages");
    p.page_size = integer(a[6], "page_size");
    p.total_q = integer(a[7], "total_q");
    if (p.total_q < 1) raise(PyExc_ValueError, "%s must be at least 1", "total_q");
    const c10::cuda::CUDAGuard guard(dev);
    const char* names[4] = {"cu_seqlens_q", "seqlens_k", "slots", "free_left"};
    const int64_t sizes[4] = {(int64_t)p.batch + 1, p.batch, p.total_q, 1};
    at::Tensor out[4];
    int* at_out[4];
    for (int i = 0; i < 4; ++i) {
      const at::Tensor* given = tensor(a[8 + i], names[i], true);
      out[i] = given ? *given : empty({sizes[i]}, at::kInt, dev);
      at_out[i] = int32_1d(out[i], names[i], dev, sizes[i]);
    }
    p.cu_seqlens_q = at_out[0];
    p.seqlens_k = at_out[1];
    p.slots = at_out[2];
    p.free_left = at_out[3];
    const int rc = fa2_paged_plan(&p, current_stream(dev));
    if (rc) return PyLong_FromLong(rc);
    written(table);
    for (int i = 0; i < 4; ++i)
      if (a[8 + i] != Py_None) written(out[i]);
    PyObject* tuple = PyTuple_New(4);
    if (!tuple) return nullptr;
    for (int i = 0; i < 4; ++i)
      PyTuple_SET_ITEM(tuple, i, a[8 + i] != Py_None ? Py_NewRef(a[8 + i]) : THPVariable_Wrap(out[i]));
    return tuple;
  });
}

PyMethodDef methods[] = {
    {"forward", (PyCFunction)(void (*)(void))forward, METH_FASTCALL, nullptr},
    {"workspace_bytes", (PyCFunction)(void (*)(void))workspace_bytes, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"forward_shared", (PyCFunction)(void (*)(void))forward_shared, METH_FASTCALL, nullptr},
    {"workspace_bytes_shared", (PyCFunction)(void (*)(void))workspace_bytes_shared, METH_FASTCALL, nullptr},
    {"forward_fp8", (PyCFunction)(void (*)(void))forward_fp8, METH_FASTCALL, nullptr},
    {"workspace_bytes_fp8", (PyCFunction)(void (*)(void))workspace_bytes_fp8, METH_FASTCALL, nullptr},
    {"append_fp8", (PyCFunction)(void (*)(void))append_fp8, METH_FASTCALL, nullptr},
    {"read_fp8", (PyCFunction)(void (*)(void))read_fp8, METH_FASTCALL, nullptr},
    {"plan", (PyCFunction)(void (*)(void))plan, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
