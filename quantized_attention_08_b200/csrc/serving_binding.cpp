// serving_binding.cpp -- the Python side of the serving entry points: argument
// checks, outputs and marshalling, and nothing of the computation.
//
// A decode step's kernels take two to ten microseconds; checking and passing
// seventeen arguments through ctypes takes as long again as all of them, so these
// four calls unpack torch's tensors here (host time a call: slot maps 14.7 us
// through ctypes, 6.1 here; rope 15.9, 5.9; append 10.3, 4.5; decode 16.0, 5.9).
// The library stays the C ABI of include/sage.h: its functions are handed over
// as addresses by the package, which has loaded it.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cmath>
#include <sstream>
#include <string>

#include "sage.h"

namespace {

decltype(&sage_kv_slots) f_slots;
decltype(&sage_rope_axes) f_rope;
decltype(&sage_kv_append) f_append;
decltype(&sage_attn_decode_paged) f_decode;
decltype(&sage_attn_decode_workspace_bytes) f_workspace;

// ------------------------------------------------------------------ checks
std::string show(at::IntArrayRef s) {
  std::ostringstream o;
  o << s;
  return o.str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    TORCH_CHECK_TYPE(false, name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

void check_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    TORCH_CHECK_TYPE(false, name, " must be ", type, ", got ", t.scalar_type());
  if (t.layout() != at::kStrided) TORCH_CHECK_TYPE(false, name, " must be a strided tensor");
}

void check_device(const at::Tensor& t, at::Device dev, const char* name) {
  if (t.device() != dev)
    TORCH_CHECK_VALUE(false, name, " must be on ", dev.str(), ", got ", t.device().str());
}

// A tensor with any strides but a dense last axis.
void check_strided(const at::Tensor& t, at::ScalarType type, const char* name, at::Device dev) {
  check_type(t, type, name);
  check_device(t, dev, name);
  if (t.dim() == 0 || (t.stride(-1) != 1 && t.size(-1) > 1))
    TORCH_CHECK_VALUE(false, name, " must be dense along its last axis");
}

// A contiguous tensor of a given shape; its address.
void* dense(const at::Tensor& t, at::ScalarType type, const char* name, at::Device dev, at::IntArrayRef shape) {
  check_type(t, type, name);
  check_device(t, dev, name);
  if (t.sizes() != shape)
    TORCH_CHECK_VALUE(false, name, " must have shape ", show(shape), ", got ", show(t.sizes()));
  if (!t.is_contiguous()) TORCH_CHECK_VALUE(false, name, " must be contiguous");
  return t.data_ptr();
}
void* dense(PyObject* o, at::ScalarType type, const char* name, at::Device dev, at::IntArrayRef shape) {
  return dense(tensor(o, name), type, name, dev, shape);
}

int c_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT32_MIN || v > INT32_MAX)
    TORCH_CHECK_VALUE(false, name, " must fit 32 bits, got ", v);
  return static_cast<int>(v);
}
int c_int(int64_t v, const char* name) {
  if (v > INT32_MAX) TORCH_CHECK_VALUE(false, name, " must be below 2^31, got ", v);
  return static_cast<int>(v);
}

bool truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw python_error();
  return t != 0;
}

sage_dtype_t model_type(at::ScalarType t, const char* name) {
  if (t == at::kHalf) return SAGE_F16;
  if (t == at::kBFloat16) return SAGE_BF16;
  TORCH_CHECK_TYPE(false, name, " must be Half or BFloat16, got ", t);
}

// Makes the tensors' device current for the call, and gives its current stream.
struct Launch {
  explicit Launch(at::Device dev) {
    if (!dev.is_cuda()) TORCH_CHECK_TYPE(false, "the serving calls take CUDA tensors, got ", dev.str());
    guard.reset_device(dev);
    stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  }
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
};

// The library's call with the interpreter free for other threads: a launch waits
// where the stream's queue is full.
template <typename F>
int free_call(F f) {
  PyThreadState* const state = PyEval_SaveThread();
  const int s = f();  // C functions: nothing is thrown
  PyEval_RestoreThread(state);
  return s;
}

PyObject* status(int s) { return PyLong_FromLong(s); }

// -------------------------------------------------------------------- calls
// Each returns the status of the C call as an int if it is not SAGE_OK.

// Entries [first, first + n) of a dense tensor without a gradient.  (Six dispatched
// as_strided calls took 1.6 us where this takes next to nothing: the call 7.8 us, 6.1.)
at::Tensor part(const at::Tensor& whole, int64_t first, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(whole.storage()),
                                                          whole.key_set(), whole.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(first);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// (ctx_lens, new_lens, free_pages, free_used, block_table, page_size, T, out)
PyObject* kv_slots(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const at::Tensor& ctx = tensor(a[0], "ctx_lens");
  const at::Device dev = ctx.device();
  const at::Tensor& free = tensor(a[2], "free_pages");
  const at::Tensor& table = tensor(a[4], "block_table");
  const int64_t B = ctx.numel(), F = free.numel();
  const int page_size = c_int(a[5], "page_size"), T = c_int(a[6], "T");
  if (table.dim() != 2) TORCH_CHECK_VALUE(false, "block_table must be [B, max_pages]");
  const int64_t width = table.size(1);
  auto i32 = [](void* p) { return static_cast<int32_t*>(p); };
  int32_t* const ctx_p = i32(dense(ctx, at::kInt, "ctx_lens", dev, {B}));
  int32_t* const new_p = i32(dense(a[1], at::kInt, "new_lens", dev, {B}));
  int32_t* const free_p = i32(dense(free, at::kInt, "free_pages", dev, {F}));
  int32_t* const used_p = i32(dense(a[3], at::kInt, "free_used", dev, {1}));
  int32_t* const table_p = i32(dense(table, at::kInt, "block_table", dev, {B, width}));
  if (T < 0) TORCH_CHECK_VALUE(false, "T must not be negative");
  const int64_t sizes[6] = {B, B + 1, T, T, T, 1};
  int32_t* p[6];
  const Launch launch(dev);
  PyObject* out;
  if (a[7] == Py_None) {
    // two allocations: what a request keeps from step to step, and the step's tokens
    const at::Tensor whole[2] = {at::empty({2 * B + 2}, ctx.options()),
                                 at::empty({3 * static_cast<int64_t>(T)}, ctx.options())};
    THPObjectPtr tuple(PyTuple_New(6));
    if (!tuple) throw python_error();
    int64_t used[2] = {0, 0};
    for (int i = 0; i < 6; ++i) {
      const int w = i >= 2 && i < 5;
      p[i] = whole[w].data_ptr<int32_t>() + used[w];
      PyTuple_SET_ITEM(tuple.get(), i, THPVariable_Wrap(part(whole[w], used[w], sizes[i])));
      used[w] += sizes[i];
    }
    out = tuple.release();
  } else {
    static const char* const names[6] = {"seq_lens", "cu_seqlens", "slot_map", "positions", "seq_ids", "free_used"};
    THPObjectPtr seq(PySequence_Fast(a[7], "out must be six tensors"));
    if (!seq) throw python_error();
    if (PySequence_Fast_GET_SIZE(seq.get()) != 6) TORCH_CHECK_VALUE(false, "out must be six tensors");
    for (int i = 0; i < 6; ++i)
      p[i] = i32(dense(PySequence_Fast_GET_ITEM(seq.get(), i), at::kInt, names[i], dev, {sizes[i]}));
    Py_INCREF(a[7]);
    out = a[7];
  }
  THPObjectPtr held(out);
  const int b = c_int(B, "B"), pages = c_int(F, "the number of free pages"), w = c_int(width, "max_pages");
  const int s = free_call([&] {
    return f_slots(ctx_p, new_p, b, free_p, pages, used_p, table_p, w, page_size, p[0], p[1], p[2], p[3], p[4], T, p[5],
                   launch.stream);
  });
  return s != SAGE_OK ? status(s) : held.release();
  END_HANDLE_TH_ERRORS
}

// (q, k, positions, inv_freq, sections, interleaved, q_out, k_out)
PyObject* rope_axes(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const at::Tensor& q = tensor(a[0], "q");
  const at::Device dev = q.device();
  const at::ScalarType type = q.scalar_type();
  const sage_dtype_t code = model_type(type, "q");
  const int64_t nd = q.dim();
  if (nd != 3 && nd != 4) TORCH_CHECK_VALUE(false, "q must be [B, H, N, d] or [H, N, d]");
  const int64_t B = nd == 4 ? q.size(0) : 1, H = q.size(-3), N = q.size(-2), d = q.size(-1);
  const bool has_k = a[1] != Py_None;
  if (!has_k && a[7] != Py_None) TORCH_CHECK_VALUE(false, "k_out without k");

  at::Tensor t[4];  // q, q_out, k, k_out
  static const char* const names[4] = {"q", "q_out", "k", "k_out"};
  t[0] = q;
  if (has_k) {
    t[2] = tensor(a[1], "k");
    if (t[2].dim() != nd || t[2].size(-1) != d || t[2].size(-2) != N || (nd == 4 && t[2].size(0) != B))
      TORCH_CHECK_VALUE(false, "q and k must have the same batch, tokens and channels");
  }
  for (int i = 0; i < (has_k ? 4 : 2); i += 2) {
    check_strided(t[i], type, names[i], dev);
    PyObject* given = a[6 + i / 2];
    t[i + 1] = given == Py_None ? at::empty_like(t[i]) : tensor(given, names[i + 1]);
    check_strided(t[i + 1], type, names[i + 1], dev);
    if (t[i + 1].sizes() != t[i].sizes())
      TORCH_CHECK_VALUE(false, names[i + 1], " does not have the shape of its input");
  }
  int64_t strides[4][3] = {};
  void* p[4] = {};
  for (int i = 0; i < (has_k ? 4 : 2); ++i) {
    p[i] = t[i].data_ptr();
    for (int j = 0; j < 3; ++j) strides[i][j] = j == 0 && nd == 3 ? 0 : t[i].stride(j - 4);
  }

  THPObjectPtr seq(PySequence_Fast(a[4], "sections must be a sequence of ints"));
  if (!seq) throw python_error();
  const Py_ssize_t A = PySequence_Fast_GET_SIZE(seq.get());
  int sections[8];
  int64_t R = 0;
  if (A < 1 || A > 8) TORCH_CHECK_VALUE(false, "sections must have 1 to 4 axes, got ", A);
  for (Py_ssize_t i = 0; i < A; ++i) R += sections[i] = c_int(PySequence_Fast_GET_ITEM(seq.get(), i), "a section");
  const at::Tensor& pos = tensor(a[2], "positions");
  check_strided(pos, at::kInt, "positions", dev);
  int64_t pos_strides[2] = {pos.stride(0), 0};
  if (pos.dim() == 3 && pos.size(0) == A && pos.size(1) == B && pos.size(2) == N)
    pos_strides[1] = pos.stride(1);
  else if (pos.dim() != 2 || pos.size(0) != A || pos.size(1) != N)
    TORCH_CHECK_VALUE(false, "positions must be [", A, ", ", N, "] or [", A, ", ", B, ", ", N, "], got ",
                      show(pos.sizes()));
  const void* inv = dense(a[3], at::kFloat, "inv_freq", dev, {R});
  const int interleaved = truth(a[5]);
  const Launch launch(dev);
  const int b = c_int(B, "B"), h = c_int(H, "H"), hk = has_k ? c_int(t[2].size(-3), "H_kv") : 0, n = c_int(N, "N"),
            ch = c_int(d, "d");
  const int32_t* const pos_p = static_cast<const int32_t*>(pos.data_ptr());
  const int s = free_call([&] {
    return f_rope(p[0], strides[0], p[1], strides[1], p[2], strides[2], p[3], strides[3], pos_p, pos_strides,
                  static_cast<const float*>(inv), sections, static_cast<int>(A), b, h, hk, n, ch, interleaved, code,
                  launch.stream);
  });
  if (s != SAGE_OK) return status(s);
  THPObjectPtr out(PyTuple_New(2));
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out.get(), 0, THPVariable_Wrap(t[1]));
  if (has_k) {
    PyTuple_SET_ITEM(out.get(), 1, THPVariable_Wrap(t[3]));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(out.get(), 1, Py_None);
  }
  return out.release();
  END_HANDLE_TH_ERRORS
}

const sage_kv_cache_t* cache_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw python_error();
  return static_cast<const sage_kv_cache_t*>(p);
}
at::ScalarType type_of(const sage_kv_cache_t* c) { return c->dtype == SAGE_F16 ? at::kHalf : at::kBFloat16; }

// (k, v, slot_map, cache, device number, mean_k, seq_ids)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const sage_kv_cache_t* c = cache_of(a[3]);
  const at::Device dev(at::kCUDA, static_cast<c10::DeviceIndex>(c_int(a[4], "device")));
  const at::Tensor& k = tensor(a[0], "k");
  const at::Tensor& v = tensor(a[1], "v");
  check_strided(k, type_of(c), "k", dev);
  check_strided(v, type_of(c), "v", dev);
  if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(0) != c->H_kv || k.size(2) != c->d)
    TORCH_CHECK_VALUE(false, "k and v must both be [", c->H_kv, ", T, ", c->d, "]");
  const int64_t T = k.size(1);
  const void *mean = nullptr, *ids = nullptr;
  int64_t B = 0;
  if (a[5] != Py_None) {
    if (a[6] == Py_None) TORCH_CHECK_VALUE(false, "mean_k needs seq_ids");
    const at::Tensor& m = tensor(a[5], "mean_k");
    B = m.dim() == 3 ? m.size(0) : 0;
    mean = dense(m, at::kFloat, "mean_k", dev, {B, c->H_kv, c->d});
    ids = dense(a[6], at::kInt, "seq_ids", dev, {T});
  }
  const int64_t ks[2] = {k.stride(0), k.stride(1)}, vs[2] = {v.stride(0), v.stride(1)};
  const void* slots = dense(a[2], at::kInt, "slot_map", dev, {T});
  const Launch launch(dev);
  // no request has a mean: no token has one (an empty tensor's address is null,
  // which the library takes for keys that are not smoothed)
  if (a[5] != Py_None && B == 0) return status(SAGE_OK);
  const void *k_p = k.data_ptr(), *v_p = v.data_ptr();
  const int n = c_int(T, "T"), b = c_int(B, "B");
  return status(free_call([&] {
    return f_append(k_p, ks, v_p, vs, n, static_cast<const int32_t*>(slots), static_cast<const float*>(mean),
                    static_cast<const int32_t*>(ids), b, c, launch.stream);
  }));
  END_HANDLE_TH_ERRORS
}

// (q, cache, device number, block_table, seq_lens, max_len, causal, sm_scale, o, return_lse, workspace)
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const sage_kv_cache_t* c = cache_of(a[1]);
  const at::Device dev(at::kCUDA, static_cast<c10::DeviceIndex>(c_int(a[2], "device")));
  const at::Tensor& q = tensor(a[0], "q");
  check_strided(q, type_of(c), "q", dev);
  const int64_t nd = q.dim();
  if ((nd != 3 && nd != 4) || q.size(-1) != c->d)
    TORCH_CHECK_VALUE(false, "q must be [B, H, n_q, ", c->d, "] or [B, H, ", c->d, "]");
  const int B = c_int(q.size(0), "B"), H = c_int(q.size(1), "H"), n_q = nd == 4 ? c_int(q.size(2), "n_q") : 1;
  const int64_t qs[3] = {q.stride(0), q.stride(1), nd == 4 ? q.stride(2) : 0};
  const at::Tensor& table = tensor(a[3], "block_table");
  if (table.dim() != 2) TORCH_CHECK_VALUE(false, "block_table must be [B, max_pages]");
  const void* table_p = dense(table, at::kInt, "block_table", dev, {B, table.size(1)});
  const void* lens = dense(a[4], at::kInt, "seq_lens", dev, {B});
  const int max_len = c_int(a[5], "max_len");
  const int causal = truth(a[6]);
  double scale = 1.0 / std::sqrt(static_cast<double>(c->d));
  if (a[7] != Py_None) {
    scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  }
  const Launch launch(dev);
  at::Tensor o, lse, ws;
  if (a[8] == Py_None) {
    o = at::empty(q.sizes(), q.options());
  } else {
    o = tensor(a[8], "o");
    dense(o, q.scalar_type(), "o", dev, q.sizes());
  }
  const bool want_lse = truth(a[9]);
  if (want_lse) lse = at::empty(q.sizes().slice(0, nd - 1), q.options().dtype(at::kFloat));
  void* ws_p = nullptr;
  size_t ws_bytes = 0;
  if (a[10] == Py_None) {
    ws_bytes = f_workspace(B, H, c->H_kv, n_q, c->d, max_len, c->format);
    if (ws_bytes > 0) {
      ws = at::empty({static_cast<int64_t>(ws_bytes)}, q.options().dtype(at::kByte));
      ws_p = ws.data_ptr();
    }
  } else {
    ws = tensor(a[10], "workspace");
    check_device(ws, dev, "workspace");
    if (!ws.is_contiguous()) TORCH_CHECK_VALUE(false, "workspace must be contiguous");
    ws_p = ws.data_ptr();
    ws_bytes = ws.nbytes();
  }
  const int width = c_int(table.size(1), "max_pages");
  const void* const q_p = q.data_ptr();
  void* const o_p = o.data_ptr();
  float* const lse_p = want_lse ? lse.data_ptr<float>() : nullptr;
  const int s = free_call([&] {
    return f_decode(q_p, qs, c, static_cast<const int32_t*>(table_p), width, static_cast<const int32_t*>(lens), B, H,
                    n_q, max_len, causal, static_cast<float>(scale), o_p, lse_p, ws_p, ws_bytes, launch.stream);
  });
  if (s != SAGE_OK) return status(s);
  THPObjectPtr out(THPVariable_Wrap(o));
  if (!out || !want_lse) return out.release();
  THPObjectPtr second(THPVariable_Wrap(lse));
  return second ? PyTuple_Pack(2, out.get(), second.get()) : nullptr;
  END_HANDLE_TH_ERRORS
}

// (addresses of the five library functions)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  f_slots = reinterpret_cast<decltype(f_slots)>(p[0]);
  f_rope = reinterpret_cast<decltype(f_rope)>(p[1]);
  f_append = reinterpret_cast<decltype(f_append)>(p[2]);
  f_decode = reinterpret_cast<decltype(f_decode)>(p[3]);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(p[4]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, got %zd", N, n);
    return nullptr;
  }
  if (f_slots == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  return F(self, a, n);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction as_method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"bind", as_method<bind>(), METH_FASTCALL, nullptr},
    {"kv_slots", as_method<counted<kv_slots, 8>>(), METH_FASTCALL, nullptr},
    {"rope_axes", as_method<counted<rope_axes, 8>>(), METH_FASTCALL, nullptr},
    {"kv_append", as_method<counted<kv_append, 7>>(), METH_FASTCALL, nullptr},
    {"attn_decode", as_method<counted<attn_decode, 11>>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
