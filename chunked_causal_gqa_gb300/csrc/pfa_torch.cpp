// pfa_torch.cpp -- the Python side of the operators around the 8-bit cache: a
// CPython module that checks torch tensors, allocates outputs and workspaces from
// torch's allocator and calls the C entry points of libpfa.so.
//
// A decode step's kernels take a few microseconds each.  The same checks written
// in Python, with a ctypes call, took 20 us for qk_norm_rope and 23 us for
// decode_attention_q8 on the host of a GB300 (Grace), several times the kernels.
//
// Everything runs on the current stream of the tensors' device; the Python
// functions switch streams before they come here.  Refusals by these checks raise
// ValueError, those of the library PfaError; C++ exceptions (torch's, out of
// memory) become Python's.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "../../include/pfa.h"

namespace {

PyObject* g_error = nullptr;  // PfaError

struct Refused {
  const char* why;
};
[[noreturn]] void refuse(const char* why) { throw Refused{why}; }

// A Python exception is set already.
struct Raised {};

const at::Tensor& tensor(PyObject* o, const char* why = "expected a torch.Tensor") {
  if (!THPVariable_Check(o)) refuse(why);
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int narrow(int64_t v) {
  if (v != (int)v) refuse("a size or window is out of range");
  return (int)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

int dtype_of(const at::Tensor& t, const char* why) {
  if (t.scalar_type() == at::kFloat) return PFA_F32;
  if (t.scalar_type() == at::kBFloat16) return PFA_BF16;
  refuse(why);
}

// What a call needs of the device: made current, with torch's current stream.
struct On {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit On(const at::Tensor& t) : guard(t.device()) {
    stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  }
};
void need_cuda(const at::Tensor& t) {
  if (!t.is_cuda()) refuse("all tensors must be CUDA tensors on one device");
}

// Runs a library call without the interpreter's lock and raises what it refuses.
template <typename F>
void call(const char* name, F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  if (rc == PFA_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", rc, name)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

struct Span {
  int64_t B, T, start;
  const int64_t* lengths;
};
Span span(const at::Tensor& t, PyObject* lengths, PyObject* start_pos) {
  if ((lengths == Py_None) == (start_pos == Py_None))
    refuse("pass either lengths (a batch) or start_pos (one sequence)");
  if (lengths == Py_None) {
    if (t.dim() != 3) refuse("with start_pos the tensors are [T, heads, D] of one sequence");
    return Span{1, t.size(0), integer(start_pos), nullptr};
  }
  if (t.dim() != 4) refuse("with lengths the tensors are [B, T, heads, D]");
  const char* why = "lengths must be a contiguous int64 tensor [B]";
  const at::Tensor& n = tensor(lengths, why);
  if (n.scalar_type() != at::kLong || n.dim() != 1 || n.size(0) != t.size(0) || !n.is_contiguous())
    refuse(why);
  return Span{t.size(0), t.size(1), 0, static_cast<const int64_t*>(n.data_ptr())};
}

// Elements from one token's row to the next of a [(B,) T, heads, D] tensor.
int64_t row_of(const at::Tensor& t, bool dense_heads = true) {
  const int64_t n = t.dim(), heads = t.size(n - 2), D = t.size(n - 1), T = t.size(n - 3);
  if (t.stride(n - 1) != 1 || (dense_heads && heads > 1 && t.stride(n - 2) != D))
    refuse("heads and elements must be dense (strides (row, D, 1))");
  if (T > 1) {
    if (n == 4 && t.size(0) > 1 && t.stride(0) != T * t.stride(1))
      refuse("a batch's sequences must follow one another (stride T * row)");
    return t.stride(n - 3);
  }
  return n == 4 && t.size(0) > 1 ? t.stride(0) : heads * D;
}

struct Cache {
  void *k, *v;
  float *ks, *vs;
  int64_t batch, cap;  // batch 0: no batch dimension
  int heads, D, block;
  const at::Tensor* first;
};
Cache cache_of(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse("cache must be a Q8Cache");
  const at::Tensor& k = tensor(PyTuple_GET_ITEM(o, 0));
  const at::Tensor& v = tensor(PyTuple_GET_ITEM(o, 1));
  const at::Tensor& ks = tensor(PyTuple_GET_ITEM(o, 2));
  const at::Tensor& vs = tensor(PyTuple_GET_ITEM(o, 3));
  const int64_t n = k.dim();
  if ((n != 3 && n != 4) || v.sizes() != k.sizes())
    refuse("cache.k and cache.v must be [(B,) Hkv, max_seq_len, D] of one shape");
  if (k.scalar_type() != at::kFloat8_e4m3fn || v.scalar_type() != at::kFloat8_e4m3fn)
    refuse("cache.k and cache.v must be float8_e4m3fn");
  if (ks.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat)
    refuse("cache.k_scale and cache.v_scale must be float32");
  const int64_t cap = k.size(n - 2), blocks = ks.dim() == n - 1 ? ks.size(n - 2) : 0;
  const int64_t block = blocks > 0 && cap % blocks == 0 ? cap / blocks : 0;
  if (ks.sizes().slice(0, ks.dim() - (ks.dim() > 0)) != k.sizes().slice(0, n - 2) ||
      vs.sizes() != ks.sizes() || (block != 16 && block != 32 && block != 64 && block != 128))
    refuse("scales must be [(B,) Hkv, max_seq_len / block], block 16, 32, 64 or 128");
  if (!k.is_contiguous() || !v.is_contiguous() || !ks.is_contiguous() || !vs.is_contiguous())
    refuse("the cache's tensors must be contiguous");
  return Cache{k.data_ptr(), v.data_ptr(), static_cast<float*>(ks.data_ptr()),
               static_cast<float*>(vs.data_ptr()), n == 4 ? k.size(0) : 0, cap,
               narrow(k.size(n - 3)), narrow(k.size(n - 1)), (int)block, &k};
}

// The workspace argument of an attention call: "auto" (None here: need bytes from
// torch's allocator), False for none, or a tensor.
struct Workspace {
  at::Tensor held;
  void* p = nullptr;
  size_t n = 0;
  Workspace(PyObject* o, size_t need, const at::Tensor& like) {
    if (o == Py_False) return;
    if (o == Py_None) {
      if (need == 0) return;
      held = empty({(int64_t)need}, at::kByte, like);
    } else {
      const char* why = "workspace must be a contiguous uint8 tensor on the output's device";
      held = tensor(o, why);
      if (held.scalar_type() != at::kByte || !held.is_contiguous() ||
          held.device() != like.device())
        refuse(why);
    }
    p = held.data_ptr();
    n = (size_t)held.numel();
  }
};

float scale_of(PyObject* o, int D) {
  return o == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)number(o);
}

// (q, k, q_weight, k_weight, inv_freq, start_pos, lengths, eps, weight_offset,
//  interleaved, q_out, k_out) -> (q_out, k_out)
PyObject* norm_rope(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]);
  const int64_t n = q.dim();
  if ((n != 3 && n != 4) || k.dim() != n || k.size(n - 1) != q.size(n - 1) ||
      q.sizes().slice(0, n - 2) != k.sizes().slice(0, n - 2))
    refuse("q must be [(B,) T, H, D] and k [(B,) T, Hkv, D]");
  const char* types = "q and k must both be float32 or both bfloat16";
  const int dt = dtype_of(q, types);
  if (k.scalar_type() != q.scalar_type()) refuse(types);
  const int H = narrow(q.size(n - 2)), Hkv = narrow(k.size(n - 2)), D = narrow(q.size(n - 1));
  const Span s = span(q, a[6], a[5]);
  const void* w[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i)
    if (a[2 + i] != Py_None) {
      const at::Tensor& t = tensor(a[2 + i]);
      if (t.dim() != 1 || t.size(0) != D || t.scalar_type() != q.scalar_type() ||
          !t.is_contiguous())
        refuse("weights must be contiguous [D] tensors of q's dtype");
      w[i] = t.data_ptr();
    }
  int rot = 0;
  const double* freq = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor(a[4]);
    if (t.scalar_type() != at::kDouble || t.dim() != 1 || !t.is_contiguous())
      refuse("inv_freq must be a contiguous float64 tensor [rot_dim / 2]");
    rot = narrow(2 * t.size(0));
    freq = static_cast<const double*>(t.data_ptr());
  }
  const int64_t q_row = row_of(q), k_row = row_of(k);
  const bool new_q = a[10] == Py_None, new_k = a[11] == Py_None;
  if (!new_q && (tensor(a[10]).sizes() != q.sizes() || tensor(a[10]).scalar_type() != q.scalar_type()))
    refuse("q_out must match q in shape and dtype");
  if (!new_k && (tensor(a[11]).sizes() != k.sizes() || tensor(a[11]).scalar_type() != k.scalar_type()))
    refuse("k_out must match k in shape and dtype");
  const float eps = (float)number(a[7]), offset = (float)number(a[8]);
  const int pairs = truth(a[9]) ? 1 : 0;
  need_cuda(q);
  const On on(q);
  const at::Tensor qo = new_q ? empty(q.sizes(), q.scalar_type(), q) : tensor(a[10]);
  const at::Tensor ko = new_k ? empty(k.sizes(), q.scalar_type(), q) : tensor(a[11]);
  const int64_t qo_row = row_of(qo), ko_row = row_of(ko, false);
  const int64_t ko_head = Hkv > 1 ? ko.stride(n - 2) : D;
  call("pfa_qk_norm_rope", [&] {
    return pfa_qk_norm_rope(q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr(), s.B, s.T,
                            s.start, s.lengths, H, Hkv, D, w[0], w[1], eps, offset,
                            rot ? freq : nullptr, rot, pairs, dt, q_row, k_row, qo_row, ko_row,
                            ko_head, on.stream);
  });
  PyObject* out = PyTuple_New(2);
  if (!out) throw Raised{};
  PyTuple_SET_ITEM(out, 0, new_q ? THPVariable_Wrap(qo) : Py_NewRef(a[10]));
  PyTuple_SET_ITEM(out, 1, new_k ? THPVariable_Wrap(ko) : Py_NewRef(a[11]));
  return out;
}

// (k, v, cache, start_pos, lengths) -> None
PyObject* cache_write(PyObject* const* a) {
  const Cache c = cache_of(a[2]);
  const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
  const int64_t n = k.dim();
  if (n != (c.batch || c.first->dim() == 4 ? 4 : 3) || v.sizes() != k.sizes() ||
      k.size(n - 1) != c.D || k.size(n - 2) != c.heads || (n == 4 && k.size(0) != c.batch))
    refuse("k and v must be [(B,) T, Hkv, D] for the cache's heads and batch");
  const char* types = "k and v must both be float32 or both bfloat16";
  const int dt = dtype_of(k, types);
  if (v.scalar_type() != k.scalar_type()) refuse(types);
  const Span s = span(k, a[4], a[3]);
  const int64_t k_row = row_of(k), v_row = row_of(v);
  need_cuda(k);
  const On on(k);
  call("pfa_cache_write_q8", [&] {
    return pfa_cache_write_q8(k.data_ptr(), v.data_ptr(), c.k, c.v, c.ks, c.vs, s.B, s.T, s.start,
                              s.lengths, c.heads, c.D, c.cap, c.block, dt, k_row, v_row, on.stream);
  });
  Py_RETURN_NONE;
}

// (cache, start, stop or None, bf16, k_out, v_out) -> (k, v)
PyObject* cache_read(PyObject* const* a) {
  const Cache c = cache_of(a[0]);
  const int64_t start = integer(a[1]), stop = a[2] == Py_None ? c.cap : integer(a[2]);
  if (start < 0 || start > stop || stop > c.cap) refuse("the rows are not in the cache");
  const at::ScalarType type = truth(a[3]) ? at::kBFloat16 : at::kFloat;
  const int64_t rows = stop - start;
  const bool batched = c.first->dim() == 4;
  const int64_t shape[4] = {c.batch, c.heads, rows, c.D};
  const at::IntArrayRef want(shape + (batched ? 0 : 1), batched ? 4 : 3);
  for (int i = 4; i < 6; ++i)
    if (a[i] != Py_None) {
      const at::Tensor& t = tensor(a[i]);
      if (t.sizes() != want || t.scalar_type() != type || !t.is_contiguous())
        refuse("k_out and v_out must be contiguous [(B,) Hkv, rows, D] of dtype");
    }
  need_cuda(*c.first);
  const On on(*c.first);
  const at::Tensor k = a[4] == Py_None ? empty(want, type, *c.first) : tensor(a[4]);
  const at::Tensor v = a[5] == Py_None ? empty(want, type, *c.first) : tensor(a[5]);
  call("pfa_cache_read_q8", [&] {
    return pfa_cache_read_q8(c.k, c.v, c.ks, c.vs, k.data_ptr(), v.data_ptr(),
                             batched ? c.batch * c.heads : c.heads, start, rows, c.D, c.cap,
                             c.block, type == at::kFloat ? PFA_F32 : PFA_BF16, rows * c.D,
                             on.stream);
  });
  PyObject* out = PyTuple_New(2);
  if (!out) throw Raised{};
  PyTuple_SET_ITEM(out, 0, a[4] == Py_None ? THPVariable_Wrap(k) : Py_NewRef(a[4]));
  PyTuple_SET_ITEM(out, 1, a[5] == Py_None ? THPVariable_Wrap(v) : Py_NewRef(a[5]));
  return out;
}

// (q, cache, lengths, out, window, scale, workspace) -> out
PyObject* decode(PyObject* const* a) {
  const Cache c = cache_of(a[1]);
  const at::Tensor& q = tensor(a[0]);
  if (q.dim() != 4 || c.first->dim() != 4 || q.size(0) != c.batch || q.size(3) != c.D)
    refuse("q must be [B, T, H, D] for the cache's batch and head_dim");
  const int dt = dtype_of(q, "q must be float32 or bfloat16");
  const int H = narrow(q.size(2)), window = narrow(integer(a[4]));
  const Span s = span(q, a[2], Py_None);
  const bool fresh = a[3] == Py_None;
  if (!fresh && (tensor(a[3]).sizes() != q.sizes() || tensor(a[3]).scalar_type() != q.scalar_type()))
    refuse("out must match q in shape and dtype");
  const int64_t q_row = row_of(q);
  const float scale = scale_of(a[5], c.D);
  need_cuda(q);
  const On on(q);
  const at::Tensor out = fresh ? empty(q.sizes(), q.scalar_type(), q) : tensor(a[3]);
  const int64_t out_row = row_of(out);
  size_t need = 0;
  if (a[6] == Py_None)
    call("pfa_decode_workspace_bytes_q8", [&] {
      return pfa_decode_workspace_bytes_q8(s.B, s.T, H, c.heads, c.D, dt, &need);
    });
  const Workspace ws(a[6], need, q);
  call("pfa_decode_attention_q8", [&] {
    return pfa_decode_attention_q8(q.data_ptr(), c.k, c.v, c.ks, c.vs, out.data_ptr(), s.B, s.T,
                                   s.lengths, H, c.heads, c.D, window, scale, dt, q_row, out_row,
                                   c.cap, c.block, ws.p, ws.n, on.stream);
  });
  return fresh ? THPVariable_Wrap(out) : Py_NewRef(a[3]);
}

// (q, cache, out, start_pos, window, scale, workspace) -> out
PyObject* prefill(PyObject* const* a) {
  const Cache c = cache_of(a[1]);
  const at::Tensor& q = tensor(a[0]);
  if (q.dim() != 3 || c.first->dim() != 3 || q.size(2) != c.D)
    refuse("q must be [T, H, D] for one sequence's cache (Q8Cache.slot)");
  const int dt = dtype_of(q, "q must be float32 or bfloat16");
  const int64_t T = q.size(0), start = integer(a[3]);
  const int H = narrow(q.size(1)), window = narrow(integer(a[4]));
  const int64_t row = row_of(q);
  const bool fresh = a[2] == Py_None;
  if (!fresh) {
    const at::Tensor& o = tensor(a[2]);
    if (o.sizes() != q.sizes() || o.scalar_type() != q.scalar_type() ||
        (T > 1 ? o.strides() != q.strides() : row_of(o) != row))
      refuse("out must match q in shape, strides and dtype");
  }
  const float scale = scale_of(a[5], c.D);
  need_cuda(q);
  const On on(q);
  const at::Tensor out =
      fresh ? at::Tensor(at::detail::empty_strided_cuda(q.sizes(), q.strides(), q.scalar_type(),
                                                        q.device()))
            : tensor(a[2]);
  size_t need = 0;
  if (a[6] == Py_None)
    call("pfa_prefill_workspace_bytes_q8", [&] {
      return pfa_prefill_workspace_bytes_q8(T, start, H, c.heads, c.D, window, dt, &need);
    });
  const Workspace ws(a[6], need, q);
  call("pfa_prefill_attention_q8", [&] {
    return pfa_prefill_attention_q8(q.data_ptr(), c.k, c.v, c.ks, c.vs, out.data_ptr(), T, start, H,
                                    c.heads, c.D, window, scale, dt, row, c.cap, c.block, ws.p,
                                    ws.n, on.stream);
  });
  return fresh ? THPVariable_Wrap(out) : Py_NewRef(a[2]);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.why);
    return nullptr;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)),
                     METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<norm_rope, 12>("qk_norm_rope"), method<cache_write, 5>("cache_write"),
                           method<cache_read, 6>("cache_read"), method<decode, 7>("decode"),
                           method<prefill, 7>("prefill"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pfa_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pfa_torch(void) {
  PyObject* b = PyImport_ImportModule("chunked_causal_gqa_gb300._binding");
  if (!b) return nullptr;
  g_error = PyObject_GetAttrString(b, "PfaError");
  Py_DECREF(b);
  return g_error ? PyModule_Create(&g_module) : nullptr;
}
