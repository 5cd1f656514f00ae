// Calls of the decode step's operators on torch tensors, for the Python
// binding (__init__.py documents them): checks of the tensors, outputs and
// workspaces where none are given, the device and the current stream, and the C
// entry point, whose address the binding sets.  A decode step makes many such
// calls of a few microseconds each; from Python the checks alone take as long.
//
// Every function takes the binding's arguments by position, raises ValueError
// for tensors that do not fit, and returns the call's outputs, or the status as
// an int where the entry point refuses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <optional>
#include <stdexcept>
#include <string>

#include "mattn.h"

namespace {

struct Functions {
  decltype(&mattn_qk_rope) qk_rope;
  decltype(&mattn_decode_shared) decode_shared;
  decltype(&mattn_decode_shared_workspace) decode_shared_workspace;
  decltype(&mattn_block_means) block_means;
  decltype(&mattn_decode_select) decode_select;
  decltype(&mattn_decode_select_workspace) decode_select_workspace;
  decltype(&mattn_decode_blocks) decode_blocks;
  decltype(&mattn_decode_blocks_workspace) decode_blocks_workspace;
} g_fn = {};

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Refused {
  int rc;
};

void need(bool ok, const char* what) {
  if (!ok) throw Bad(what);
}

// The arguments of one call, by position.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) throw Bad("too few arguments");
    return a[i++];
  }
  const at::Tensor& tensor(const char* name) {
    PyObject* o = next();
    if (!THPVariable_Check(o)) throw Bad(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  const at::Tensor* optional(const char* name) {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Bad(std::string(name) + " must be a tensor or None");
    return &THPVariable_Unpack(o);
  }
  int64_t integer(const char* name) {
    PyObject* o = next();
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Bad(std::string(name) + " must be an integer");
    }
    return v;
  }
  int small(const char* name) {
    const int64_t v = integer(name);
    if (v != (int)v) throw Bad(std::string(name) + " is out of range");
    return (int)v;
  }
  bool truth(const char* name) {
    const int v = PyObject_IsTrue(next());
    if (v < 0) {
      PyErr_Clear();
      throw Bad(std::string(name) + " must be true or false");
    }
    return v == 1;
  }
  float scale() {  // None: 0, the default
    PyObject* o = next();
    if (o == Py_None) return 0.f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Bad("scale must be a number");
    }
    return (float)v;
  }
};

// A contiguous tensor of type `t` on q's device.
void fits(const at::Tensor* x, const at::Tensor& q, at::ScalarType t, const char* name) {
  if (!x) return;
  if (x->scalar_type() != t || x->device() != q.device() || !x->is_contiguous())
    throw Bad(std::string(name) + " must be a contiguous " + c10::toString(t) + " tensor on " + q.device().str());
}

bool shape(const at::Tensor& x, std::initializer_list<int64_t> s) { return x.sizes() == at::IntArrayRef(s); }

int type_code(const at::Tensor& q) {
  if (q.scalar_type() == at::kBFloat16) return MATTN_BF16;
  if (q.scalar_type() == at::kFloat) return MATTN_F32;
  throw Bad("unsupported type (bf16 or fp32)");
}

int size32(int64_t n) {
  if (n != (int)n) throw Bad("a size is out of range");
  return (int)n;
}

template <class T>
T* ptr(const at::Tensor* x) {
  return x ? static_cast<T*>(x->data_ptr()) : nullptr;
}

at::Tensor empty(std::initializer_list<int64_t> s, const at::Tensor& like, at::ScalarType t) {
  return at::empty(at::IntArrayRef(s), like.options().dtype(t));
}

// The call's device made current, and its current stream.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit On(const at::Tensor& q) {
    guard.set_device(q.device());
    stream = c10::cuda::getCurrentCUDAStream(q.get_device()).stream();
  }
};

void done(int rc) {
  if (rc) throw Refused{rc};
}

// The caller's workspace, or one of the bytes that `size` reports.
struct Workspace {
  at::Tensor own;
  void* p;
  size_t bytes;
  template <class Size>
  Workspace(const at::Tensor* given, const at::Tensor& q, Size size) {
    if (given) {
      need(given->device() == q.device() && given->is_contiguous(),
           "the workspace must be a contiguous tensor on the inputs' device");
      p = given->data_ptr();
      bytes = given->nbytes();
    } else {
      size_t n = 0;
      done(size(&n));
      own = empty({(int64_t)(n ? n : 16)}, q, at::kByte);
      p = own.data_ptr();
      bytes = n;
    }
  }
};

PyObject* give(const at::Tensor* x) {
  if (!x) Py_RETURN_NONE;
  return THPVariable_Wrap(*x);
}

PyObject* pair(const at::Tensor& a, const at::Tensor* b) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, give(b));
  return t;
}

struct Decode {
  int B, H, H_kv, L, d;
};

// Sizes of a decode call on the cache k [B, H_kv, L, d].
Decode decode_sizes(const at::Tensor& q, const at::Tensor& k, const at::Tensor* lens, const at::Tensor* sink) {
  need(q.is_cuda() && q.dim() == 3, "q must be a CUDA tensor [B, H, d]");
  need(k.dim() == 4 && k.size(0) == q.size(0) && k.size(3) == q.size(2), "the cache must be [B, H_kv, L, d]");
  const Decode s{size32(q.size(0)), size32(q.size(1)), size32(k.size(1)), size32(k.size(2)), size32(q.size(2))};
  need(!lens || shape(*lens, {s.B}), "seq_lens must be [B]");
  need(!sink || shape(*sink, {s.H}), "sink must be [H]");
  fits(&q, q, q.scalar_type(), "q");
  fits(lens, q, at::kInt, "seq_lens");
  fits(sink, q, at::kFloat, "sink");
  return s;
}

// out [B, H, d] and lse [B, H] (wanted or given), made where they are missing.
struct Outputs {
  at::Tensor out, lse;
  bool has_lse;
  Outputs(const at::Tensor& q, const at::Tensor* o, const at::Tensor* l, bool want) {
    need(!o || o->sizes() == q.sizes(), "out must be [B, H, d]");
    need(!l || shape(*l, {q.size(0), q.size(1)}), "lse must be [B, H]");
    fits(o, q, q.scalar_type(), "out");
    fits(l, q, at::kFloat, "lse");
    out = o ? *o : empty({q.size(0), q.size(1), q.size(2)}, q, q.scalar_type());
    has_lse = l || want;
    if (has_lse) lse = l ? *l : empty({q.size(0), q.size(1)}, q, at::kFloat);
  }
  float* lse_ptr() const { return has_lse ? static_cast<float*>(lse.data_ptr()) : nullptr; }
  PyObject* result() const { return pair(out, has_lse ? &lse : nullptr); }
};

PyObject* qk_rope(Args a) {
  // q, k, v, the descriptor's bytes before its pointers, the plan's tensors, then the rest
  const at::Tensor& q = a.tensor("q");
  const at::Tensor& k = a.tensor("k");
  const at::Tensor* v = a.optional("v");
  PyObject* head = a.next();
  const at::Tensor& inv_freq = a.tensor("inv_freq");
  const at::Tensor *q_weight = a.optional("q_weight"), *k_weight = a.optional("k_weight");
  const at::Tensor *q_out = a.optional("q_out"), *k_out = a.optional("k_out"), *v_out = a.optional("v_out");
  const at::Tensor *positions = a.optional("positions"), *starts = a.optional("starts"), *lens = a.optional("lens");
  need(q.is_cuda() && q.dim() == 4 && k.dim() == 4, "q and k must be CUDA tensors [B, N, heads, d]");
  const int64_t B = q.size(0), N = q.size(1), H = q.size(2), d = q.size(3), H_kv = k.size(2);
  mattn_rope_desc desc = {};
  constexpr size_t kHead = offsetof(mattn_rope_desc, inv_freq);
  need(PyBytes_Check(head) && PyBytes_GET_SIZE(head) == (Py_ssize_t)kHead, "bad plan");
  memcpy(&desc, PyBytes_AS_STRING(head), kHead);
  // the plan's tensors as they are now: a tensor may have got other storage since the plan was made
  need(desc.n_axes >= 1 && desc.n_axes <= 3, "bad plan");
  const int64_t axes = desc.n_axes;
  int64_t R = 0;
  for (int64_t i = 0; i < axes; ++i) R += desc.sections[i];
  fits(&inv_freq, q, at::kFloat, "inv_freq");
  fits(q_weight, q, at::kFloat, "q_weight");
  fits(k_weight, q, at::kFloat, "k_weight");
  need(shape(inv_freq, {R}), "inv_freq must be [R], R the sum of the sections");
  need((!q_weight || shape(*q_weight, {d})) && (!k_weight || shape(*k_weight, {d})), "the norm weights must be [d]");
  desc.inv_freq = static_cast<const float*>(inv_freq.data_ptr());
  desc.q_weight = ptr<const float>(q_weight);
  desc.k_weight = ptr<const float>(k_weight);
  const at::Tensor* in[3] = {&q, &k, v};
  for (int t = 0; t < 3; ++t) {
    desc.token_stride[t] = desc.batch_stride[t] = 0;
    if (!in[t]) continue;
    const at::Tensor& x = *in[t];
    need(x.scalar_type() == q.scalar_type() && x.device() == q.device() && shape(x, {B, N, t ? H_kv : H, d}),
         "q must be [B, N, H, d] and k, v [B, N, H_kv, d] of one type and device");
    need(x.stride(3) == 1 && (x.stride(2) == d || x.size(2) == 1), "the heads of a token must lie side by side");
    // (the stride of a dimension of one entry says nothing)
    if (N > 1) desc.token_stride[t] = x.stride(1);
    if (B > 1) desc.batch_stride[t] = x.stride(0);
  }
  need(!k_out || k_out->dim() == 4, "k_out must be [B, H_kv, L, d]");
  const int64_t L = k_out ? k_out->size(2) : N;
  if (!v) v_out = nullptr;
  need(!q_out || shape(*q_out, {B, H, N, d}), "q_out must be [B, H, N, d]");
  need((!k_out || shape(*k_out, {B, H_kv, L, d})) && (!v_out || shape(*v_out, {B, H_kv, L, d})),
       "k_out and v_out must be [B, H_kv, L, d]");
  // rows that no token goes to are the caller's: an output made here has none
  need(!starts || (k_out && (!v || v_out)), "starts needs the caches that its rows lie in (k_out, and v_out with v)");
  need(!v || v_out || L == N, "a cache of keys (k_out with L != N) needs one of values (v_out)");
  need(!positions || shape(*positions, {axes, B, N}), "positions must be [axes, B, N]");
  need((!starts || shape(*starts, {B})) && (!lens || shape(*lens, {B})), "starts and lens must be [B]");
  const at::ScalarType t = q.scalar_type();
  fits(q_out, q, t, "q_out");
  fits(k_out, q, t, "k_out");
  fits(v_out, q, t, "v_out");
  fits(positions, q, at::kInt, "positions");
  fits(starts, q, at::kInt, "starts");
  fits(lens, q, at::kInt, "lens");
  const int code = type_code(q);
  On on(q);
  // (padding, which the kernel leaves as it is: zeros)
  auto made = [&](int64_t heads, int64_t rows) {
    return lens ? at::zeros({B, heads, rows, d}, q.options()) : empty({B, heads, rows, d}, q, t);
  };
  const at::Tensor qo = q_out ? *q_out : made(H, N), ko = k_out ? *k_out : made(H_kv, L);
  at::Tensor vo;
  if (v) vo = v_out ? *v_out : made(H_kv, L);
  done(g_fn.qk_rope(q.data_ptr(), k.data_ptr(), v ? v->data_ptr() : nullptr, qo.data_ptr(), ko.data_ptr(),
                    v ? vo.data_ptr() : nullptr, ptr<int32_t>(positions), ptr<int32_t>(starts), ptr<int32_t>(lens),
                    size32(B), size32(H), size32(H_kv), size32(N), size32(L), size32(d), code, &desc, on.stream));
  PyObject* r = PyTuple_New(3);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(qo));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(ko));
  PyTuple_SET_ITEM(r, 2, give(v ? &vo : nullptr));
  return r;
}

PyObject* decode_shared(Args a) {
  const at::Tensor &q = a.tensor("q"), &kp = a.tensor("k_prefix"), &vp = a.tensor("v_prefix");
  const at::Tensor &k = a.tensor("k_cache"), &v = a.tensor("v_cache");
  const at::Tensor* lens = a.optional("seq_lens");
  PyObject* prefix = a.next();
  const at::Tensor* sink = a.optional("sink");
  const float scale = a.scale();
  const at::Tensor *out = a.optional("out"), *lse = a.optional("lse");
  const bool want = a.truth("want_lse");
  const at::Tensor* ws = a.optional("workspace");
  const Decode s = decode_sizes(q, k, lens, sink);
  need(kp.dim() == 3 && kp.size(0) == s.H_kv && kp.size(2) == s.d && vp.sizes() == kp.sizes() && v.sizes() == k.sizes(),
       "k_prefix, v_prefix must be [H_kv, P, d] and k_cache, v_cache [B, H_kv, L, d]");
  const at::ScalarType t = q.scalar_type();
  fits(&kp, q, t, "k_prefix");
  fits(&vp, q, t, "v_prefix");
  fits(&k, q, t, "k_cache");
  fits(&v, q, t, "v_cache");
  const int cap = size32(kp.size(1));
  int P = cap;
  if (prefix != Py_None) {
    Args one{&prefix, 1};
    P = one.small("prefix_len");
  }
  const int code = type_code(q);
  On on(q);
  Outputs o(q, out, lse, want);
  Workspace w(ws, q, [&](size_t* n) { return g_fn.decode_shared_workspace(s.B, s.H, s.H_kv, P, s.L, s.d, n); });
  done(g_fn.decode_shared(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), k.data_ptr(), v.data_ptr(), o.out.data_ptr(),
                          o.lse_ptr(), ptr<int32_t>(lens), s.B, s.H, s.H_kv, P, cap, s.L, s.d, code, ptr<float>(sink),
                          scale, w.p, w.bytes, on.stream));
  return o.result();
}

PyObject* block_means(Args a) {
  const at::Tensor& k = a.tensor("k_cache");
  const int block = a.small("block");
  const at::Tensor *lens = a.optional("seq_lens"), *first = a.optional("first");
  PyObject* max_new = a.next();
  const at::Tensor* out = a.optional("out");
  need(k.is_cuda() && k.dim() == 4, "k_cache must be a CUDA tensor [B, H_kv, L, d]");
  need(block >= 1, "block must be >= 1");
  need(out || !first, "an update of means (first) needs the means to update (out)");
  const int64_t B = k.size(0), H_kv = k.size(1), L = k.size(2), d = k.size(3), n = (L + block - 1) / block;
  need((!lens || shape(*lens, {B})) && (!first || shape(*first, {B})), "seq_lens and first must be [B]");
  need(!out || shape(*out, {B, H_kv, n, d}), "out must be [B, H_kv, ceil(L / block), d]");
  fits(&k, k, k.scalar_type(), "k_cache");
  fits(out, k, k.scalar_type(), "out");
  fits(lens, k, at::kInt, "seq_lens");
  fits(first, k, at::kInt, "first");
  int fresh = size32(L);
  if (max_new != Py_None) {
    Args one{&max_new, 1};
    fresh = one.small("max_new");
  }
  const int code = type_code(k);
  On on(k);
  // blocks past a sequence's end: zeros
  const at::Tensor o = out ? *out : at::zeros({B, H_kv, n, d}, k.options());
  done(g_fn.block_means(k.data_ptr(), o.data_ptr(), ptr<int32_t>(lens), ptr<int32_t>(first), size32(B), size32(H_kv),
                        size32(L), size32(d), code, block, fresh, on.stream));
  return THPVariable_Wrap(o);
}

PyObject* decode_select(Args a) {
  const at::Tensor &q = a.tensor("q"), &m = a.tensor("means");
  const int block = a.small("block"), top_k = a.small("top_k");
  const at::Tensor* lens = a.optional("seq_lens");
  const int keep_first = a.small("keep_first"), keep_recent = a.small("keep_recent");
  const at::Tensor *out = a.optional("out"), *ws = a.optional("workspace");
  const Decode s = decode_sizes(q, m, lens, nullptr);
  fits(&m, q, q.scalar_type(), "means");
  fits(out, q, at::kInt, "out");
  need(!out || shape(*out, {s.B, s.H_kv, top_k}), "out must be [B, H_kv, top_k]");
  const int code = type_code(q);
  On on(q);
  const at::Tensor o = out ? *out : empty({s.B, s.H_kv, top_k > 0 ? top_k : 0}, q, at::kInt);
  Workspace w(ws, q, [&](size_t* n) { return g_fn.decode_select_workspace(s.B, s.H, s.H_kv, s.L, s.d, n); });
  done(g_fn.decode_select(q.data_ptr(), m.data_ptr(), ptr<int32_t>(lens), static_cast<int32_t*>(o.data_ptr()), s.B, s.H,
                          s.H_kv, s.L, s.d, code, block, top_k, keep_first, keep_recent, w.p, w.bytes, on.stream));
  return THPVariable_Wrap(o);
}

PyObject* decode_blocks(Args a) {
  const at::Tensor &q = a.tensor("q"), &k = a.tensor("k_cache"), &v = a.tensor("v_cache"), &ids = a.tensor("block_ids");
  const int block = a.small("block");
  const at::Tensor *lens = a.optional("seq_lens"), *sink = a.optional("sink");
  const float scale = a.scale();
  const at::Tensor *out = a.optional("out"), *lse = a.optional("lse");
  const bool want = a.truth("want_lse");
  const at::Tensor* ws = a.optional("workspace");
  const Decode s = decode_sizes(q, k, lens, sink);
  need(v.sizes() == k.sizes() && ids.dim() == 3 && ids.size(0) == s.B && ids.size(1) == s.H_kv,
       "k_cache and v_cache must be [B, H_kv, L, d] and block_ids [B, H_kv, top_k]");
  fits(&k, q, q.scalar_type(), "k_cache");
  fits(&v, q, q.scalar_type(), "v_cache");
  fits(&ids, q, at::kInt, "block_ids");
  const int top_k = size32(ids.size(2)), code = type_code(q);
  On on(q);
  Outputs o(q, out, lse, want);
  Workspace w(ws, q, [&](size_t* n) { return g_fn.decode_blocks_workspace(s.B, s.H, s.H_kv, top_k, block, s.d, n); });
  done(g_fn.decode_blocks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.out.data_ptr(), o.lse_ptr(), ptr<int32_t>(lens),
                          static_cast<const int32_t*>(ids.data_ptr()), s.B, s.H, s.H_kv, s.L, s.d, code, block, top_k,
                          ptr<float>(sink), scale, w.p, w.bytes, on.stream));
  return o.result();
}

// No C++ exception leaves for Python.
template <PyObject* (*F)(Args)>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(Args{a, n});
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Refused& r) {
    return PyLong_FromLong(r.rc);
  } catch (...) {  // torch's own, as torch raises them (OutOfMemoryError among them)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// The entry points' addresses, in the order of Functions.
PyObject* set_functions(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != (Py_ssize_t)(sizeof(Functions) / sizeof(void*))) {
    PyErr_SetString(PyExc_ValueError, "wrong number of functions");
    return nullptr;
  }
  void* p[sizeof(Functions) / sizeof(void*)];
  for (Py_ssize_t i = 0; i < n; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function is missing");
      return nullptr;
    }
  }
  memcpy(&g_fn, p, sizeof(g_fn));
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {
    {"set_functions", FAST(set_functions)},
    {"qk_rope", FAST((call<qk_rope>))},
    {"decode_shared", FAST((call<decode_shared>))},
    {"block_means", FAST((call<block_means>))},
    {"decode_select", FAST((call<decode_select>))},
    {"decode_blocks", FAST((call<decode_blocks>))},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
