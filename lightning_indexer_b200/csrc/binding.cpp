// The Python binding of the calls that a decode step makes: checks of the tensors, outputs and
// workspaces, and the call of the C ABI, in native code.  The kernels of these calls take 3 to
// 7 us at decode sizes; the same marshalling in Python and ctypes took 10 to 27 us a call.
//
// Every function takes positional arguments from the wrappers in __init__.py, which hold the
// signatures and the documentation.  Sizes that the library cannot see in a pointer (rows,
// tables, pages) are checked here against one another and refused with ValueError; statuses of
// the library become DSAError.  The work is enqueued on the tensors' own device, on its
// current stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/full.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/dsa.h"

namespace {

using at::Tensor;

PyObject *g_dsa_error = nullptr, *g_oom_error = nullptr;  // DSAError, torch.OutOfMemoryError

// Thrown where a Python error is set already or is set from the message.
struct PyError {};
[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw PyError();
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const char* type_text(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    default: return "torch.uint8";
  }
}

using Shape = std::initializer_list<int64_t>;

// An uninitialised tensor on `like`'s device, without the dispatcher (half the cost).
Tensor new_tensor(Shape shape, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(at::IntArrayRef(shape), type, like.device(), std::nullopt);
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The checks of one call: all tensors on the device of the first.
struct Call {
  int dev = -1;

  void common(const Tensor& t, const char* name, at::ScalarType type, Shape shape) {
    if (t.scalar_type() != type)
      refuse(std::string(name) + " must be " + type_text(type) + ", got " + c10::toString(t.scalar_type()));
    if (!t.is_cuda() || (dev >= 0 && t.get_device() != dev))
      refuse(std::string(name) + " must be a CUDA tensor on the device of the others");
    if (t.sizes() != at::IntArrayRef(shape))
      refuse(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    dev = t.get_device();
  }
  void* dense(const Tensor& t, const char* name, at::ScalarType type, Shape shape) {
    common(t, name, type, shape);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
  template <typename T = void>
  T* arg(PyObject* o, const char* name, at::ScalarType type, Shape shape) {
    return static_cast<T*>(dense(tensor(o, name), name, type, shape));
  }
  template <typename T = void>
  T* optional(PyObject* o, const char* name, at::ScalarType type, Shape shape) {
    return o == Py_None ? nullptr : arg<T>(o, name, type, shape);
  }
  // bf16 rows whose heads are dense; the token stride may be larger
  void* rows(const Tensor& t, const char* name, Shape shape, int64_t* stride) {
    common(t, name, at::kBFloat16, shape);
    const int64_t* n = shape.begin();
    const bool heads = shape.size() == 3;
    const int64_t d = n[shape.size() - 1], H = heads ? n[1] : 1;
    if ((t.stride(-1) != 1 && d > 1) || (heads && H > 1 && t.stride(1) != d))
      refuse(std::string(name) + " must have dense heads (only the token stride may be larger)");
    *stride = n[0] > 1 ? t.stride(0) : H * d;
    return t.data_ptr();
  }
  void* rows(PyObject* o, const char* name, Shape shape, int64_t* stride) {
    return rows(tensor(o, name), name, shape, stride);
  }
  // a bf16 cache whose pages are dense; the page stride may be larger
  void* pool(PyObject* o, const char* name, Shape shape, int64_t* stride) {
    const Tensor& t = tensor(o, name);
    common(t, name, at::kBFloat16, shape);
    int64_t dense = 1;
    for (int i = (int)shape.size() - 1; i > 0; --i) {
      const int64_t n = shape.begin()[i];
      if (n > 1 && t.stride(i) != dense) refuse(std::string(name) + " must have dense pages (only the page stride may be larger)");
      dense *= n;
    }
    *stride = shape.begin()[0] > 1 ? t.stride(0) : dense;
    return t.data_ptr();
  }
};

// Runs fn(stream) with the call's device current; a status that is not DSA_OK becomes DSAError.
template <typename F>
void launch(const Call& c, const char* name, F&& fn) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
  const int st = fn(static_cast<void*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.dev)).stream()));
  if (st == DSA_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_dsa_error, "si", name, st)) {
    PyErr_SetObject(g_dsa_error, e);
    Py_DECREF(e);
  }
  throw PyError();
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <typename... Ts>
PyObject* pack(const Ts&... ts) {
  PyObject* r = PyTuple_New(sizeof...(ts));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(ts)), ...);
  return r;
}

int int32(int64_t v, const char* name) {
  if (v != (int)v) refuse(std::string(name) + " does not fit in 32 bits");
  return (int)v;
}
int as_int(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  return int32(v, name);
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError();
  return (float)v;
}
int as_flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError();
  return v;
}
void dims(const Tensor& t, const char* name, int n) {
  if (t.dim() != n) refuse(std::string(name) + " must have " + std::to_string(n) + " dims, got " + std::to_string(t.dim()));
}
// the i-th of the tensors given as `out`
const Tensor* out_tensor(PyObject* out, Py_ssize_t i, Py_ssize_t n, const char* name) {
  if (!PyTuple_Check(out) && !PyList_Check(out)) refuse("out must be a tuple");
  if (PySequence_Fast_GET_SIZE(out) != n) refuse("out must have " + std::to_string(n) + " entries");
  PyObject* o = PySequence_Fast_GET_ITEM(out, i);
  return o == Py_None ? nullptr : &tensor(o, name);
}

// inv_freq and what it says of the rotation
struct Rope {
  const double* freq = nullptr;
  int rotary = 0;
  Rope(Call& c, PyObject* o, const char* name) {
    if (o == Py_None) return;
    const Tensor& t = tensor(o, name);
    rotary = int32(2 * t.numel(), "the rotated width");
    freq = c.arg<double>(o, name, at::kDouble, {t.numel()});
  }
};

struct TokenMap {
  const int32_t *positions, *cu, *lens;
  int batch = 1;
  TokenMap(Call& c, int64_t T, PyObject* pos, PyObject* cu_o, PyObject* lens_o) {
    positions = c.optional<int32_t>(pos, "positions", at::kInt, {T});
    cu = nullptr;
    if (cu_o != Py_None) {
      batch = int32(tensor(cu_o, "cu_seqlens_q").numel() - 1, "the number of sequences");
      cu = c.arg<int32_t>(cu_o, "cu_seqlens_q", at::kInt, {batch + 1});
    }
    lens = c.optional<int32_t>(lens_o, "seqlens_k", at::kInt, {batch});
  }
};

// block_table and seqlens_k of B sequences
struct Table {
  const int32_t *table, *lens;
  int width, batch;
  Table(Call& c, PyObject* table_o, PyObject* lens_o, int64_t B) {
    const Tensor& t = tensor(table_o, "block_table");
    dims(t, "block_table", 2);
    width = int32(t.size(1), "the width of block_table");
    batch = int32(B, "the number of sequences");
    table = c.arg<int32_t>(table_o, "block_table", at::kInt, {B, t.size(1)});
    lens = c.arg<int32_t>(lens_o, "seqlens_k", at::kInt, {B});
  }
};

// k_cache, v_cache [pages, page, Hkv, d]
struct KvPool {
  void *k, *v;
  int64_t ks, vs, pages, page, Hkv;
  KvPool(Call& c, PyObject* k_o, PyObject* v_o, int64_t d) {
    const Tensor& t = tensor(k_o, "k_cache");
    dims(t, "k_cache", 4);
    pages = t.size(0), page = t.size(1), Hkv = t.size(2);
    k = c.pool(k_o, "k_cache", {pages, page, Hkv, d}, &ks);
    v = c.pool(v_o, "v_cache", {pages, page, Hkv, d}, &vs);
  }
};

void* weight(Call& c, PyObject* o, const char* name, int64_t d) { return c.optional(o, name, at::kBFloat16, {d}); }

// norm_rope(Q, K, q_weight, k_weight, inv_freq, positions, cu_seqlens_q, seqlens_k, interleaved, eps, out)
PyObject* norm_rope(PyObject* const* a) {
  Call c;
  const Tensor& Q = tensor(a[0], "Q");
  dims(Q, "Q", 3);
  const int64_t T = Q.size(0), Hq = Q.size(1), d = Q.size(2);
  int64_t qs = 0, ks = 0, qos = 0, kos = 0, Hk = 0;
  void *q = c.rows(Q, "Q", {T, Hq, d}, &qs), *k = nullptr, *ko = nullptr;
  const bool has_k = a[1] != Py_None;  // K of no tokens has a null pointer
  if (has_k) {
    const Tensor& K = tensor(a[1], "K");
    dims(K, "K", 3);
    Hk = K.size(1);
    k = c.rows(K, "K", {T, Hk, d}, &ks);
  }
  void *gq = weight(c, a[2], "q_weight", d), *gk = has_k ? weight(c, a[3], "k_weight", d) : nullptr;
  const Rope rope(c, a[4], "inv_freq");
  const TokenMap tk(c, T, a[5], a[6], a[7]);
  const int inter = as_flag(a[8]);
  const float eps = as_float(a[9]);
  Tensor Qo, Ko;
  if (a[10] != Py_None) {
    const Tensor *x = out_tensor(a[10], 0, 2, "out"), *y = out_tensor(a[10], 1, 2, "out");
    if (!x || (has_k && !y)) refuse("out must give a tensor for every input");
    Qo = *x;
    if (has_k) Ko = *y;
  } else {
    Qo = new_tensor({T, Hq, d}, at::kBFloat16, Q);
    if (has_k) Ko = new_tensor({T, Hk, d}, at::kBFloat16, Q);
  }
  void* qo = c.rows(Qo, "Q out", {T, Hq, d}, &qos);
  if (has_k) ko = c.rows(Ko, "K out", {T, Hk, d}, &kos);
  // a new tensor holds zeros in the rows of tokens outside the sequences
  const auto fn = a[10] == Py_None ? dsa_norm_rope_zeroed : dsa_norm_rope;
  if (T > 0)
    launch(c, "dsa_norm_rope", [&](void* st) {
      return fn(q, qs, k, ks, gq, gk, eps, rope.freq, rope.rotary, inter, tk.positions, tk.cu, tk.lens, tk.batch, T, (int)Hq,
                (int)Hk, (int)d, qo, qos, ko, kos, st);
    });
  return pack(Qo, Ko);
}

// norm_rope_bwd(Q, K, dQ_out, dK_out, q_weight, k_weight, inv_freq, positions, cu_seqlens_q, seqlens_k,
//               interleaved, eps, out, workspace)
PyObject* norm_rope_bwd(PyObject* const* a) {
  Call c;
  const Tensor& Q = tensor(a[0], "Q");
  dims(Q, "Q", 3);
  const int64_t T = Q.size(0), Hq = Q.size(1), d = Q.size(2);
  int64_t qs = 0, ks = 0, dqos = 0, dkos = 0, dqs = 0, dks = 0, Hk = 0;
  void *q = c.rows(Q, "Q", {T, Hq, d}, &qs), *k = nullptr, *dko = nullptr, *dk = nullptr;
  void* dqo = c.rows(a[2], "dQ_out", {T, Hq, d}, &dqos);
  const bool has_k = a[1] != Py_None;  // K of no tokens has a null pointer
  if (has_k) {
    const Tensor& K = tensor(a[1], "K");
    dims(K, "K", 3);
    Hk = K.size(1);
    k = c.rows(K, "K", {T, Hk, d}, &ks);
    dko = c.rows(a[3], "dK_out", {T, Hk, d}, &dkos);
  }
  void *gq = weight(c, a[4], "q_weight", d), *gk = has_k ? weight(c, a[5], "k_weight", d) : nullptr;
  const Rope rope(c, a[6], "inv_freq");
  const TokenMap tk(c, T, a[7], a[8], a[9]);
  const int inter = as_flag(a[10]);
  const float eps = as_float(a[11]);
  Tensor dQ, dK, dgq, dgk, ws;
  if (a[12] != Py_None) {
    const Tensor *x = out_tensor(a[12], 0, 2, "out"), *y = out_tensor(a[12], 1, 2, "out");
    if (!x || (has_k && !y)) refuse("out must give a tensor for every input");
    dQ = *x;
    if (has_k) dK = *y;
  } else {
    dQ = new_tensor({T, Hq, d}, at::kBFloat16, Q);
    if (has_k) dK = new_tensor({T, Hk, d}, at::kBFloat16, Q);
  }
  void* dq = c.rows(dQ, "dQ", {T, Hq, d}, &dqs);
  if (has_k) dk = c.rows(dK, "dK", {T, Hk, d}, &dks);
  if (T == 0) {
    const auto f32 = Q.options().dtype(at::kFloat);
    if (gq) dgq = at::zeros({d}, f32);
    if (gk) dgk = at::zeros({d}, f32);
    return pack(dQ, dK, dgq, dgk);
  }
  if (gq) dgq = new_tensor({d}, at::kFloat, Q);
  // (K of no heads has a null pointer and takes no part in the call)
  if (gk) dgk = Hk > 0 ? new_tensor({d}, at::kFloat, Q) : at::zeros({d}, Q.options().dtype(at::kFloat));
  if (a[13] != Py_None) {
    ws = tensor(a[13], "workspace");
    c.dense(ws, "workspace", at::kByte, {ws.numel()});
  } else if (gq || gk) {
    ws = new_tensor({(int64_t)dsa_norm_rope_bwd_workspace_size(T, (int)Hq, (int)Hk, (int)d)}, at::kByte, Q);
  }
  const auto fn = a[12] == Py_None ? dsa_norm_rope_bwd_zeroed : dsa_norm_rope_bwd;  // as in norm_rope
  launch(c, "dsa_norm_rope_bwd", [&](void* st) {
    return fn(q, qs, k, ks, dqo, dqos, dko, dkos, gq, gk, eps, rope.freq, rope.rotary, inter, tk.positions, tk.cu, tk.lens,
              tk.batch, T, (int)Hq, (int)Hk, (int)d, dq, dqs, dk, dks, gq ? dgq.data_ptr<float>() : nullptr,
              gk ? dgk.data_ptr<float>() : nullptr, ws.defined() ? ws.data_ptr() : nullptr,
              ws.defined() ? (size_t)ws.numel() : 0, st);
  });
  return pack(dQ, dK, dgq, dgk);
}

// cache_append(K, V, k_idx, k_cache, v_cache, k_idx_cache, block_table, cu_seqlens_q, seqlens_k, k_weight,
//              k_idx_weight, inv_freq, idx_inv_freq, positions, interleaved, idx_interleaved, eps)
PyObject* cache_append(PyObject* const* a) {
  Call c;
  const Tensor& K = tensor(a[0], "K");
  dims(K, "K", 3);
  const int64_t T = K.size(0), Hkv = K.size(1), d = K.size(2);
  int64_t ks = 0, vs = 0, is = 0, ics = 0, d_I = 0;
  void *k = c.rows(K, "K", {T, Hkv, d}, &ks), *v = c.rows(a[1], "V", {T, Hkv, d}, &vs), *i = nullptr, *ic = nullptr;
  const KvPool kv(c, a[3], a[4], d);
  if (kv.Hkv != Hkv) refuse("k_cache must have " + std::to_string(Hkv) + " heads, got " + std::to_string(kv.Hkv));
  const bool has_i = a[2] != Py_None;
  if (has_i) {
    const Tensor& I = tensor(a[2], "k_idx");
    dims(I, "k_idx", 2);
    d_I = I.size(1);
    i = c.rows(I, "k_idx", {T, d_I}, &is);
    ic = c.pool(a[5], "k_idx_cache", {kv.pages, kv.page, d_I}, &ics);
  }
  const Table tab(c, a[6], a[8], tensor(a[6], "block_table").size(0));
  const int32_t* cu = c.arg<int32_t>(a[7], "cu_seqlens_q", at::kInt, {tab.batch + 1});
  void *gk = weight(c, a[9], "k_weight", d), *gi = has_i ? weight(c, a[10], "k_idx_weight", d_I) : nullptr;
  const Rope rope(c, a[11], "inv_freq"), irope(c, has_i ? a[12] : Py_None, "idx_inv_freq");
  const int32_t* pos = c.optional<int32_t>(a[13], "positions", at::kInt, {T});
  const int inter = as_flag(a[14]), iinter = as_flag(a[15]);
  const float eps = as_float(a[16]);
  if (T > 0)
    launch(c, "dsa_cache_append", [&](void* st) {
      return dsa_cache_append(k, ks, v, vs, i, is, gk, gi, eps, rope.freq, rope.rotary, inter, irope.freq, irope.rotary,
                              iinter, pos, cu, T, (int)Hkv, (int)d, (int)d_I, kv.k, kv.ks, kv.v, kv.vs, ic, ics,
                              tab.table, tab.width, tab.lens, tab.batch, (int)kv.pages, (int)kv.page, st);
    });
  Py_RETURN_NONE;
}

int64_t score_ld(int max_seqlen_k) { return max_seqlen_k < 4 ? 4 : (max_seqlen_k + 3LL) / 4 * 4; }

// index_paged(q_idx, k_idx_cache, w, block_table, seqlens_k, max_seqlen_k, scores)
PyObject* index_paged(PyObject* const* a) {
  Call c;
  const Tensor& q = tensor(a[0], "q_idx");
  dims(q, "q_idx", 3);
  const int64_t B = q.size(0), H = q.size(1), d = q.size(2);
  void* qp = c.dense(q, "q_idx", at::kBFloat16, {B, H, d});
  const Tensor& cache = tensor(a[1], "k_idx_cache");
  dims(cache, "k_idx_cache", 3);
  int64_t ics = 0;
  void *ic = c.pool(a[1], "k_idx_cache", {cache.size(0), cache.size(1), d}, &ics), *w = c.arg(a[2], "w", at::kBFloat16, {B, H});
  const Table tab(c, a[3], a[4], B);
  const int maxk = as_int(a[5], "max_seqlen_k");
  Tensor scores;
  if (a[6] != Py_None) {
    scores = tensor(a[6], "scores");
    dims(scores, "scores", 2);
    c.dense(scores, "scores", at::kFloat, {B, scores.size(1)});
  } else {
    scores = at::full({B, score_ld(maxk)}, -INFINITY, q.options().dtype(at::kFloat));
  }
  launch(c, "dsa_index_paged", [&](void* st) {
    return dsa_index_paged(qp, ic, ics, w, tab.table, tab.width, tab.lens, tab.batch, (int)cache.size(0), (int)cache.size(1),
                           maxk, (int)H, (int)d, scores.data_ptr<float>(), scores.size(1), st);
  });
  return wrap(scores);
}

float softmax_scale(PyObject* o, int64_t d) { return o == Py_None ? (float)(1.0 / std::sqrt((double)d)) : as_float(o); }

// O and lse of a decode call, given or new
struct DecodeOut {
  Tensor indices, O, lse;
  DecodeOut(Call& c, PyObject* out, int64_t B, int64_t k, int64_t Hq, int64_t d, const Tensor& Q, bool with_indices) {
    const int n = with_indices ? 3 : 2;
    if (out != Py_None) {
      const Tensor *o = out_tensor(out, n - 2, n, "O"), *l = out_tensor(out, n - 1, n, "lse");
      if (!o) refuse("out must give O");
      O = *o;
      c.dense(O, "O", at::kBFloat16, {B, Hq, d});
      if (l) c.dense(*l, "lse", at::kFloat, {B, Hq}), lse = *l;
      if (with_indices) {
        const Tensor* i = out_tensor(out, 0, n, "indices");
        if (!i) refuse("out must give indices");
        indices = *i;
        c.dense(indices, "indices", at::kInt, {B, k});
      }
      return;
    }
    O = new_tensor({B, Hq, d}, at::kBFloat16, Q);
    lse = new_tensor({B, Hq}, at::kFloat, Q);
    if (with_indices) indices = new_tensor({B, k > 0 ? k : 0}, at::kInt, Q);
  }
  float* lse_ptr() const { return lse.defined() ? lse.data_ptr<float>() : nullptr; }
};

// sparse_attn_decode_paged(Q, k_cache, v_cache, indices, block_table, seqlens_k, scale, out)
PyObject* sparse_attn_decode_paged(PyObject* const* a) {
  Call c;
  const Tensor& Q = tensor(a[0], "Q");
  dims(Q, "Q", 3);
  const int64_t B = Q.size(0), Hq = Q.size(1), d = Q.size(2);
  void* q = c.dense(Q, "Q", at::kBFloat16, {B, Hq, d});
  const KvPool kv(c, a[1], a[2], d);
  const Tensor& idx = tensor(a[3], "indices");
  dims(idx, "indices", 2);
  const int k = int32(idx.size(1), "the number of slots");
  const int32_t* ip = c.arg<int32_t>(a[3], "indices", at::kInt, {B, idx.size(1)});
  const Table tab(c, a[4], a[5], B);
  const float scale = softmax_scale(a[6], d);
  const DecodeOut o(c, a[7], B, 0, Hq, d, Q, false);
  launch(c, "dsa_sparse_attn_decode_paged", [&](void* st) {
    return dsa_sparse_attn_decode_paged(q, kv.k, kv.ks, kv.v, kv.vs, ip, tab.table, tab.width, tab.lens, tab.batch, (int)kv.pages,
                                        (int)kv.page, (int)Hq, (int)kv.Hkv, (int)d, k, scale, o.O.data_ptr(), o.lse_ptr(), st);
  });
  return pack(o.O, o.lse);
}

Tensor workspace(Call& c, PyObject* o, size_t bytes, const Tensor& like) {
  if (o == Py_None) return new_tensor({(int64_t)bytes}, at::kByte, like);
  const Tensor& t = tensor(o, "workspace");
  c.dense(t, "workspace", at::kByte, {t.numel()});
  return t;
}

// decode_paged(q_idx, w, Q, k_cache, v_cache, k_idx_cache, block_table, seqlens_k, max_seqlen_k, k, scale, workspace, out)
PyObject* decode_paged(PyObject* const* a) {
  Call c;
  const Tensor &qi = tensor(a[0], "q_idx"), &Q = tensor(a[2], "Q");
  dims(qi, "q_idx", 3);
  dims(Q, "Q", 3);
  const int64_t B = Q.size(0), Hq = Q.size(1), d = Q.size(2), H_I = qi.size(1), d_I = qi.size(2);
  void *q = c.dense(Q, "Q", at::kBFloat16, {B, Hq, d}), *qip = c.dense(qi, "q_idx", at::kBFloat16, {B, H_I, d_I});
  void* w = c.arg(a[1], "w", at::kBFloat16, {B, H_I});
  const KvPool kv(c, a[3], a[4], d);
  int64_t ics = 0;
  void* ic = c.pool(a[5], "k_idx_cache", {kv.pages, kv.page, d_I}, &ics);
  const Table tab(c, a[6], a[7], B);
  const int maxk = as_int(a[8], "max_seqlen_k"), k = as_int(a[9], "k");
  const float scale = softmax_scale(a[10], d);
  const Tensor ws = workspace(c, a[11], dsa_decode_paged_workspace_size((int)B, maxk), Q);
  const DecodeOut o(c, a[12], B, k, Hq, d, Q, true);
  launch(c, "dsa_decode_paged", [&](void* st) {
    return dsa_decode_paged(qip, w, q, kv.k, kv.ks, kv.v, kv.vs, ic, ics, tab.table, tab.width, tab.lens, tab.batch,
                            (int)kv.pages, (int)kv.page, maxk, (int)Hq, (int)kv.Hkv, (int)d, (int)H_I, (int)d_I, k, scale,
                            o.indices.data_ptr<int32_t>(), o.O.data_ptr(), o.lse_ptr(), ws.data_ptr(), (size_t)ws.numel(), st);
  });
  return pack(o.indices, o.O, o.lse);
}

// decode_step_paged(q_idx, w, Q, K, V, k_idx, k_cache, v_cache, k_idx_cache, block_table, seqlens_k, max_seqlen_k, k,
//                   q_weight, k_weight, q_idx_weight, k_idx_weight, inv_freq, idx_inv_freq, positions, interleaved,
//                   idx_interleaved, eps, scale, workspace, out)
PyObject* decode_step_paged(PyObject* const* a) {
  Call c;
  const Tensor &qi = tensor(a[0], "q_idx"), &Q = tensor(a[2], "Q");
  dims(qi, "q_idx", 3);
  dims(Q, "Q", 3);
  const int64_t B = Q.size(0), Hq = Q.size(1), d = Q.size(2), H_I = qi.size(1), d_I = qi.size(2);
  int64_t qis = 0, qs = 0, ks = 0, vs = 0, is = 0, ics = 0;
  void *q = c.rows(Q, "Q", {B, Hq, d}, &qs), *qip = c.rows(qi, "q_idx", {B, H_I, d_I}, &qis);
  void* w = c.arg(a[1], "w", at::kBFloat16, {B, H_I});
  const KvPool kv(c, a[6], a[7], d);
  void *k = c.rows(a[3], "K", {B, kv.Hkv, d}, &ks), *v = c.rows(a[4], "V", {B, kv.Hkv, d}, &vs);
  void* i = c.rows(a[5], "k_idx", {B, d_I}, &is);
  void* ic = c.pool(a[8], "k_idx_cache", {kv.pages, kv.page, d_I}, &ics);
  const Table tab(c, a[9], a[10], B);
  const int maxk = as_int(a[11], "max_seqlen_k"), top = as_int(a[12], "k");
  void *gq = weight(c, a[13], "q_weight", d), *gk = weight(c, a[14], "k_weight", d);
  void *gqi = weight(c, a[15], "q_idx_weight", d_I), *gki = weight(c, a[16], "k_idx_weight", d_I);
  const Rope rope(c, a[17], "inv_freq"), irope(c, a[18], "idx_inv_freq");
  const int32_t* pos = c.optional<int32_t>(a[19], "positions", at::kInt, {B});
  const int inter = as_flag(a[20]), iinter = as_flag(a[21]);
  const float eps = as_float(a[22]), scale = softmax_scale(a[23], d);
  const Tensor ws = workspace(c, a[24], dsa_decode_step_paged_workspace_size((int)B, maxk, (int)Hq, (int)d, (int)H_I, (int)d_I), Q);
  const DecodeOut o(c, a[25], B, top, Hq, d, Q, true);
  launch(c, "dsa_decode_step_paged", [&](void* st) {
    return dsa_decode_step_paged(qip, qis, w, q, qs, k, ks, v, vs, i, is, gq, gk, gqi, gki, eps, rope.freq, rope.rotary, inter,
                                 irope.freq, irope.rotary, iinter, pos, kv.k, kv.ks, kv.v, kv.vs, ic, ics, tab.table,
                                 tab.width, tab.lens, tab.batch, (int)kv.pages, (int)kv.page, maxk, (int)Hq, (int)kv.Hkv,
                                 (int)d, (int)H_I, (int)d_I, top, scale, o.indices.data_ptr<int32_t>(), o.O.data_ptr(),
                                 o.lse_ptr(), ws.data_ptr(), (size_t)ws.numel(), st);
  });
  return pack(o.indices, o.O, o.lse);
}

// Python entry: N positional arguments; no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != N) {
    PyErr_Format(PyExc_TypeError, "takes %zd arguments, got %zd", N, nargs);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_oom_error, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* set_errors(PyObject*, PyObject* args) {
  PyObject *dsa, *oom;
  if (!PyArg_ParseTuple(args, "OO", &dsa, &oom)) return nullptr;
  Py_INCREF(dsa);
  Py_INCREF(oom);
  Py_XSETREF(g_dsa_error, dsa);
  Py_XSETREF(g_oom_error, oom);
  Py_RETURN_NONE;
}

#define DSA_ENTRY(f, n) {#f, (PyCFunction)(void (*)(void))(entry<f, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"set_errors", set_errors, METH_VARARGS, nullptr},
    DSA_ENTRY(norm_rope, 11),
    DSA_ENTRY(norm_rope_bwd, 14),
    DSA_ENTRY(cache_append, 17),
    DSA_ENTRY(index_paged, 7),
    DSA_ENTRY(sparse_attn_decode_paged, 8),
    DSA_ENTRY(decode_paged, 13),
    DSA_ENTRY(decode_step_paged, 26),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module_def);
  // read by the build, which makes the module anew for another torch or Python
  if (m && PyModule_AddStringConstant(m, "built_for", DSA_BINDING_STAMP) < 0) Py_CLEAR(m);
  return m;
}
