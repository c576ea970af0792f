// The Python side of the calls that a model makes once or more per layer and token: norm
// and rotation, append, chunk attention.  Through ctypes such a call took 14 to 19 us of host
// time (argument conversion, checks and allocations in Python), several times what its kernel
// runs for a decode step; here norm and rotation takes 5.7 us (14.5), append 5.1 (15.5), chunk
// attention 9.5 (19), and the backward of the norm 11 (25).  The calls' names, defaults and
// documentation stand in __init__.py, which passes every argument by position.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/ExpandUtils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <vector>

#include "../../include/fa.h"

namespace {

using at::Tensor;
using Opt = std::optional<Tensor>;

// The C ABI's entry points, from the library that __init__.py has loaded.
struct {
  decltype(&fa_norm_rope) norm_rope;
  decltype(&fa_norm_rope_backward) norm_rope_backward;
  decltype(&fa_norm_rope_backward_workspace_size) norm_rope_backward_workspace_size;
  decltype(&fa_append_paged) append_paged;
  decltype(&fa_extend_paged) extend_paged;
  decltype(&fa_extend_paged_workspace_size) extend_paged_workspace_size;
} abi;
PyObject* fa_error = nullptr;  // the exception of a status other than FA_OK

struct Failed {};  // a Python exception is set

// ---------------------------------------------------------------- arguments
Tensor tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
// The first tensor of a call: a CPU one is refused ahead of all other checks.
Tensor first_tensor(PyObject* o, const char* name) {
  Tensor t = tensor(o, name);
  TORCH_CHECK_VALUE(!t.is_cpu(), "tensors must be on a CUDA device (there is no CPU path)");
  return t;
}
Opt optional(PyObject* o, const char* name) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, name);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed{};
  return v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Failed{};
  return v;
}
// n integers of a tuple.
std::optional<std::vector<int64_t>> integers(PyObject* o, int64_t n) {
  if (o == Py_None) return std::nullopt;
  TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == n, "strides must be a tuple of ", n, " integers");
  std::vector<int64_t> v;
  for (int64_t i = 0; i < n; ++i) {
    v.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(o, i)));
    if (v.back() == -1 && PyErr_Occurred()) throw Failed{};
  }
  return v;
}
void* ptr(const Opt& t) { return t ? t->data_ptr() : nullptr; }

fa_dtype dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return FA_BF16;
    case at::kHalf: return FA_FP16;
    case at::kFloat: return FA_FP32;
    default: TORCH_CHECK_TYPE(false, "unsupported dtype ", t, ": use torch.bfloat16, torch.float16 or torch.float32");
  }
}
int size(int64_t v) {
  TORCH_CHECK_VALUE(v <= 0x7fffffff, "a size passes 2^31");
  return static_cast<int>(v);
}

// Sets the device that every tensor of the call sits on for the call's length.
struct On {
  int device;
  std::optional<c10::cuda::CUDAGuard> guard;
  explicit On(const Tensor& first) {
    TORCH_CHECK_VALUE(first.is_cuda(), "tensors must be on a CUDA device (there is no CPU path)");
    device = first.get_device();
  }
  On& with(const Opt& t) {
    TORCH_CHECK_VALUE(!t || (t->is_cuda() && t->get_device() == device), "tensors must all be on the same CUDA device");
    return *this;
  }
  void* stream() {
    if (c10::cuda::current_device() != device) guard.emplace(static_cast<c10::DeviceIndex>(device));
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  }
};
void check(fa_status st, const char* name) {
  if (st == FA_OK) return;
  PyObject* e = PyObject_CallFunction(fa_error, "is", static_cast<int>(st), name);
  if (e != nullptr) {
    PyErr_SetObject(fa_error, e);
    Py_DECREF(e);
  }
  throw Failed{};
}

// Raises the version of a tensor of the caller's that the call has written, as torch's in-place
// operations do: autograd then refuses a backward pass that saved the values from before.
void written(const Opt& t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// Lets Python's other threads run for as long as it lives: a launch waits while the device's queue
// is full, an allocation may wait for the device.  No Python object is touched meanwhile.
struct OtherThreadsRun {
  PyThreadState* state = PyEval_SaveThread();
  ~OtherThreadsRun() { PyEval_RestoreThread(state); }
};
template <class F> auto without_gil(F f) {
  const OtherThreadsRun others;
  return f();
}

Tensor new_like(const Tensor& t) { return at::empty(t.sizes(), t.options().requires_grad(false)); }
// The output for x: the given one, or a new contiguous one.
Tensor out_like(const Tensor& x, const Opt& out) { return out ? *out : new_like(x); }
void check_out(const Tensor& x, const Opt& out) {
  TORCH_CHECK_VALUE(!out || (out->sizes() == x.sizes() && out->scalar_type() == x.scalar_type()),
                    "an output must have its input's shape and dtype");
}
// A workspace's bytes are written as one run: an expanded or strided one has fewer than its elements'.
void check_workspace(const Opt& ws) {
  TORCH_CHECK_VALUE(!ws || ws->is_contiguous(), "workspace must be contiguous");
}
Tensor bytes(const Tensor& like, size_t n) {
  return at::empty({static_cast<int64_t>(n)}, at::TensorOptions(like.device()).dtype(at::kByte));
}

// ---------------------------------------------------------------- norm and rotation
struct Rows {
  int B, Hq, Hk, N, d;
  bool packed;
};
// Queries and keys, [B, H, N, d] or packed [T, H, d].
Rows rows_of(const Tensor& q, const Opt& k) {
  const auto s = q.sizes();
  TORCH_CHECK_VALUE(s.size() == 3 || s.size() == 4, "q must be [B, H, N, d] or packed [T, H, d]");
  const bool packed = s.size() == 3;
  Rows r{packed ? 1 : size(s[0]), size(s[1]), 0, size(packed ? s[0] : s[2]), size(s[packed ? 2 : 3]), packed};
  if (k) {
    const auto t = k->sizes();
    bool same = t.size() == s.size() && k->scalar_type() == q.scalar_type();
    for (size_t i = 0; same && i < s.size(); ++i) same = i == 1 || t[i] == s[i];
    TORCH_CHECK_VALUE(same, "q and k must share dtype and every size but the heads");
    r.Hk = size(t[1]);
  }
  return r;
}
// (batch, head, row) strides into st.
void strides_of(const Tensor& t, bool packed, int64_t* st) {
  const auto s = t.strides();
  TORCH_CHECK_VALUE(s.back() == 1, "the rows (last dimension) of q, k, their outputs and gradients must be contiguous");
  st[0] = packed ? 0 : s[0];
  st[1] = s[1];
  st[2] = packed ? s[0] : s[2];
}
struct Turn {
  int rot = 0, max_pos = 0;
  float eps;
  fa_dtype weight;
};
Turn turn_of(at::ScalarType dtype, const Opt& q_weight, const Opt& k_weight, const Opt& rope, PyObject* eps, int64_t d) {
  Turn t;
  if (rope) {
    TORCH_CHECK_VALUE(rope->dim() == 2 && rope->scalar_type() == at::kFloat && rope->is_contiguous(),
                      "rope must be a contiguous float32 tensor [positions, rot]: rot/2 cosines, rot/2 sines");
    const int64_t rot = rope->size(1);
    TORCH_CHECK_VALUE(rot > 0 && rot % 16 == 0 && rot <= d,
                      "rope's second dimension must be a multiple of 16 up to the head dimension");
    t.rot = size(rot);
    t.max_pos = size(rope->size(0));
  }
  if (eps == Py_None) {
    TORCH_CHECK_VALUE(!q_weight && !k_weight, "weights need eps: without it there is no norm");
    t.eps = -1.f;
    t.weight = dtype_code(dtype);
    return t;
  }
  const double e = number(eps);
  TORCH_CHECK_VALUE(e >= 0, "eps must be >= 0 (None: no norm)");
  t.eps = static_cast<float>(e);
  std::optional<at::ScalarType> type;
  for (const Opt* w : {&q_weight, &k_weight}) {
    if (!*w) continue;
    TORCH_CHECK_VALUE((*w)->dim() == 1 && (*w)->size(0) == d && (*w)->is_contiguous(),
                      "weights must be contiguous tensors of the head dimension");
    const at::ScalarType wt = (*w)->scalar_type();
    TORCH_CHECK_VALUE((wt == dtype || wt == at::kFloat) && (!type || *type == wt),
                      "weights must share one dtype: the tensors' or float32");
    type = wt;
  }
  t.weight = dtype_code(type.value_or(dtype));
  return t;
}
long long position_stride(const Opt& p, const Rows& r) {
  if (!p) return 0;
  const auto s = p->sizes();
  TORCH_CHECK_VALUE(p->scalar_type() == at::kInt && p->is_contiguous() &&
                        ((s.size() == 1 && s[0] == r.N) || (s.size() == 2 && s[0] == r.B && s[1] == r.N)),
                    "positions must be a contiguous int32 tensor [N] or [B, N] (packed: [T])");
  return s.size() == 2 ? r.N : 0;
}

PyObject* wrap(const Opt& t) {
  if (!t) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}
PyObject* tuple(std::initializer_list<Opt> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) throw Failed{};
  Py_ssize_t i = 0;
  for (const Opt& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}
void arguments(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "takes ", want, " arguments, got ", n); }

// q, k, q_weight, k_weight, rope, positions, eps, interleaved, q_out, k_out
PyObject* norm_rope(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 10);
  const Tensor q = first_tensor(a[0], "q");
  const Opt k = optional(a[1], "k"), qw = optional(a[2], "q_weight"), kw = optional(a[3], "k_weight"),
            rope = optional(a[4], "rope"), pos = optional(a[5], "positions"), qo = optional(a[8], "q_out"),
            ko = optional(a[9], "k_out");
  TORCH_CHECK_VALUE(k || (!kw && !ko), "k_weight and k_out need k");
  const Rows r = rows_of(q, k);
  const Turn t = turn_of(q.scalar_type(), qw, kw, rope, a[6], r.d);
  const long long ps = position_stride(pos, r);
  const int inter = truth(a[7]);
  const fa_dtype code = dtype_code(q.scalar_type());
  int64_t st[12] = {};
  strides_of(q, r.packed, st);
  if (k) strides_of(*k, r.packed, st + 3);
  check_out(q, qo);
  if (k) check_out(*k, ko);
  On on(q);
  on.with(k).with(qw).with(kw).with(rope).with(pos).with(qo).with(ko);
  Opt q_out, k_out;
  check(without_gil([&] {
          q_out = out_like(q, qo);
          strides_of(*q_out, r.packed, st + 6);
          if (k) {
            k_out = out_like(*k, ko);
            strides_of(*k_out, r.packed, st + 9);
          }
          return abi.norm_rope(q.data_ptr(), ptr(k), ptr(q_out), ptr(k_out), st, ptr(qw), ptr(kw),
                               static_cast<const float*>(ptr(rope)), static_cast<const int32_t*>(ptr(pos)), ps, r.B, r.Hq,
                               r.Hk, r.N, r.d, t.rot, t.max_pos, t.eps, inter, code, t.weight, on.stream());
        }),
        "fa_norm_rope");
  written(qo);
  written(ko);
  return k ? tuple({q_out, k_out}) : wrap(q_out);
}

// q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, eps, interleaved, workspace; whether
// q_weight's and k_weight's gradients are wanted; q's and k's strides, where they are None themselves
// but dq and dk are to be laid out as they were, or None
PyObject* norm_rope_backward(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 15);
  // The rotation alone needs no rows: sizes then come from the gradients.
  const bool norm = a[8] != Py_None, rows = norm || a[0] != Py_None || a[1] != Py_None;
  const Tensor q = first_tensor(a[rows ? 0 : 2], rows ? "q" : "dq_out"), gq = tensor(a[2], "dq_out");
  const Opt k = optional(a[rows ? 1 : 3], "k"), gk = optional(a[3], "dk_out"), qw = optional(a[4], "q_weight"),
            kw = optional(a[5], "k_weight"), rope = optional(a[6], "rope"), pos = optional(a[7], "positions");
  Opt ws = optional(a[10], "workspace");
  TORCH_CHECK_VALUE(k.has_value() == gk.has_value(), "k and dk_out go together");
  TORCH_CHECK_VALUE(k || !kw, "k_weight needs k");
  const Rows r = rows_of(q, k);
  TORCH_CHECK_VALUE(gq.sizes() == q.sizes() && gq.scalar_type() == q.scalar_type(), "dq_out must have q's shape and dtype");
  TORCH_CHECK_VALUE(!k || (gk->sizes() == k->sizes() && gk->scalar_type() == k->scalar_type()),
                    "dk_out must have k's shape and dtype");
  check_workspace(ws);
  const Turn t = turn_of(q.scalar_type(), qw, kw, rope, a[8], r.d);
  const long long ps = position_stride(pos, r);
  const int inter = truth(a[9]);
  const bool want_qw = qw && truth(a[11]), want_kw = kw && truth(a[12]);
  const fa_dtype code = dtype_code(q.scalar_type());
  int64_t st[18] = {};
  strides_of(q, r.packed, st);
  strides_of(gq, r.packed, st + 6);
  if (k) {
    strides_of(*k, r.packed, st + 3);
    strides_of(*gk, r.packed, st + 9);
  }
  On on(q);
  on.with(k).with(gq).with(gk).with(qw).with(kw).with(rope).with(pos).with(ws);
  // Laid out as x, dense in its strides' order; contiguous where that would part a row's elements
  // (expanded views).
  auto grad_like = [](const Tensor& x, const std::optional<std::vector<int64_t>>& strides) {
    const auto dense = at::infer_dense_strides(x.sizes(), strides ? at::IntArrayRef(*strides) : x.strides());
    return dense.back() == 1 ? at::empty_strided(x.sizes(), dense, x.options().requires_grad(false)) : new_like(x);
  };
  const auto q_strides = integers(a[13], q.dim()), k_strides = integers(a[14], q.dim());
  Opt dq, dk, dqw, dkw;
  check(without_gil([&] {
          dq = grad_like(q, q_strides);
          strides_of(*dq, r.packed, st + 12);
          if (k) {
            dk = grad_like(*k, k_strides);
            strides_of(*dk, r.packed, st + 15);
          }
          if (want_qw) dqw = new_like(*qw);
          if (want_kw) dkw = new_like(*kw);
          size_t ws_bytes = 0;
          if (want_qw || want_kw) {
            if (!ws) ws = bytes(q, abi.norm_rope_backward_workspace_size(r.d));
            ws_bytes = ws->nbytes();
          }
          return abi.norm_rope_backward(norm ? q.data_ptr() : nullptr, norm ? ptr(k) : nullptr, gq.data_ptr(), ptr(gk),
                                        ptr(dq), ptr(dk), st, ptr(qw), ptr(kw), ptr(dqw), ptr(dkw), static_cast<const float*>(ptr(rope)),
                                        static_cast<const int32_t*>(ptr(pos)), ps, r.B, r.Hq, r.Hk, r.N, r.d, t.rot,
                                        t.max_pos, t.eps, inter, code, t.weight, ptr(ws), ws_bytes, on.stream());
        }),
        "fa_norm_rope_backward");
  return tuple({dq, dk, dqw, dkw});
}

// ---------------------------------------------------------------- the paged cache
// The token stride of a packed [T, H, d] tensor whose heads are contiguous.
long long token_stride(const char* name, const Tensor& t, int64_t T, int64_t H, int64_t d, at::ScalarType dtype) {
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == T && t.size(1) == H && t.size(2) == d && t.scalar_type() == dtype, name,
                    " must be packed [", T, ", ", H, ", ", d, "] with the pools' dtype");
  TORCH_CHECK_VALUE(t.stride(2) == 1 && (t.stride(1) == d || H <= 1), name, ": the heads of a token must be contiguous");
  return t.stride(0);
}
void int32(const char* name, const Tensor& t, at::IntArrayRef shape) {
  TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == at::kInt && t.is_contiguous(), name,
                    " must be a contiguous int32 tensor of shape ", shape);
}
struct Paged {
  int num_blocks, Hkv, block_size, d, B, max_blocks;
};
Paged paged_of(const Tensor& kp, const Tensor& vp, const Tensor& table, const Tensor& lens, const Opt& cu, int64_t T) {
  TORCH_CHECK_VALUE(kp.dim() == 4 && vp.sizes() == kp.sizes() && vp.scalar_type() == kp.scalar_type(),
                    "kpool and vpool must be [num_blocks, Hkv, block_size, d] and share dtype");
  TORCH_CHECK_VALUE(kp.is_contiguous() && vp.is_contiguous(), "kpool and vpool must be contiguous");
  TORCH_CHECK_VALUE(table.dim() == 2, "block_table must be an int32 tensor of shape [B, max_blocks]");
  const int64_t B = table.size(0);
  int32("block_table", table, {B, table.size(1)});
  int32("seqlens", lens, {B});
  if (cu) int32("cu_tokens", *cu, {B + 1});
  TORCH_CHECK_VALUE(cu || T == B, "without cu_tokens there is one token for each sequence");
  return Paged{size(kp.size(0)), size(kp.size(1)), size(kp.size(2)), size(kp.size(3)), size(B), size(table.size(1))};
}

// k, v, kpool, vpool, block_table, seqlens, cu_tokens, rope, q, q_weight, k_weight, eps, interleaved, q_out
PyObject* append_paged(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 14);
  const Tensor k = first_tensor(a[0], "k"), v = tensor(a[1], "v"), kp = tensor(a[2], "kpool"), vp = tensor(a[3], "vpool"),
               table = tensor(a[4], "block_table"), lens = tensor(a[5], "seqlens");
  const Opt cu = optional(a[6], "cu_tokens"), rope = optional(a[7], "rope"), q = optional(a[8], "q"),
            qw = optional(a[9], "q_weight"), kw = optional(a[10], "k_weight"), qo = optional(a[13], "q_out");
  TORCH_CHECK_VALUE(k.dim() == 3, "k must be packed [T, Hkv, d]");
  const int T = size(k.size(0));
  const at::ScalarType dtype = kp.scalar_type();
  const Paged p = paged_of(kp, vp, table, lens, cu, T);
  const long long ks = token_stride("k", k, T, p.Hkv, p.d, dtype), vs = token_stride("v", v, T, p.Hkv, p.d, dtype);
  const Turn t = turn_of(dtype, qw, kw, rope, a[11], p.d);
  const int inter = truth(a[12]);
  const fa_dtype code = dtype_code(dtype);
  int Hq = 0;
  long long qs = 0;
  if (q) {
    TORCH_CHECK_VALUE(q->dim() == 3, "q must be packed [T, Hq, d]");
    Hq = size(q->size(1));
    qs = token_stride("q", *q, T, Hq, p.d, dtype);
    check_out(*q, qo);
    TORCH_CHECK_VALUE(!qo || qo->is_contiguous(), "q_out must be contiguous");
  } else {
    TORCH_CHECK_VALUE(!qo, "q_out needs q");
  }
  On on(k);
  on.with(v).with(kp).with(vp).with(table).with(lens).with(cu).with(rope).with(q).with(qw).with(kw).with(qo);
  Opt q_out;
  check(without_gil([&] {
          if (q) q_out = out_like(*q, qo);
          return abi.append_paged(k.data_ptr(), v.data_ptr(), ptr(q), ptr(q_out), kp.data_ptr(), vp.data_ptr(),
                                  static_cast<const int32_t*>(table.data_ptr()), static_cast<const int32_t*>(ptr(cu)),
                                  static_cast<const int32_t*>(lens.data_ptr()), qs, ks, vs, ptr(qw), ptr(kw),
                                  static_cast<const float*>(ptr(rope)), T, p.B, Hq, p.Hkv, p.num_blocks, p.block_size,
                                  p.max_blocks, p.d, t.rot, t.max_pos, t.eps, inter, code, t.weight, on.stream());
        }),
        "fa_append_paged");
  written(kp);
  written(vp);
  written(qo);
  return wrap(q_out);
}

// q, kpool, vpool, block_table, seqlens, cu_tokens, causal, window, scale (0: the default), workspace, out, lse
PyObject* extend_paged(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 12);
  const Tensor q = first_tensor(a[0], "q"), kp = tensor(a[1], "kpool"), vp = tensor(a[2], "vpool"),
               table = tensor(a[3], "block_table"), lens = tensor(a[4], "seqlens");
  const Opt cu = optional(a[5], "cu_tokens"), o = optional(a[10], "out"), l = optional(a[11], "lse");
  Opt ws = optional(a[9], "workspace");
  TORCH_CHECK_VALUE(q.dim() == 3, "q must be packed [T, Hq, d]");
  const int T = size(q.size(0)), Hq = size(q.size(1));
  const at::ScalarType dtype = kp.scalar_type();
  const Paged p = paged_of(kp, vp, table, lens, cu, T);
  const long long qs = token_stride("q", q, T, Hq, p.d, dtype);
  TORCH_CHECK_VALUE(p.Hkv >= 1 && Hq % p.Hkv == 0, "the query heads must be a multiple of the pools' heads");
  TORCH_CHECK_VALUE(!l || (l->dim() == 2 && l->size(0) == T && l->size(1) == Hq && l->scalar_type() == at::kFloat &&
                           l->is_contiguous()),
                    "lse must be a contiguous float32 tensor [T, Hq]");
  TORCH_CHECK_VALUE(!o || o->is_contiguous(), "out must be contiguous");
  check_workspace(ws);
  const int causal = truth(a[6]);
  const long long window = PyLong_AsLongLong(a[7]);
  if (window == -1 && PyErr_Occurred()) throw Failed{};
  TORCH_CHECK_VALUE(window >= 0 && window <= 0x7fffffff, "window must be >= 0 (0: none)");
  const float scale = static_cast<float>(number(a[8]));
  const fa_dtype code = dtype_code(dtype);
  check_out(q, o);
  On on(q);
  on.with(kp).with(vp).with(table).with(lens).with(cu).with(ws).with(o).with(l);
  Opt out, lse;
  check(without_gil([&] {
          out = out_like(q, o);
          lse = l ? *l : at::empty({T, Hq}, at::TensorOptions(q.device()).dtype(at::kFloat));
          if (!ws) {
            const size_t need = abi.extend_paged_workspace_size(T, Hq, p.Hkv, p.d);
            ws = bytes(q, need < 256 ? 256 : need);
          }
          return abi.extend_paged(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), static_cast<const int32_t*>(table.data_ptr()),
                                  static_cast<const int32_t*>(ptr(cu)), static_cast<const int32_t*>(lens.data_ptr()),
                                  ptr(out), static_cast<float*>(ptr(lse)), qs, T, p.B, Hq, p.Hkv, p.num_blocks, p.block_size,
                                  p.max_blocks, p.d, scale, causal, static_cast<int>(window), code, ptr(ws), ws->nbytes(),
                                  on.stream());
        }),
        "fa_extend_paged");
  written(o);
  written(l);
  return tuple({out, lse});
}

// ---------------------------------------------------------------- the module
// bind(exception class, the six entry points' addresses in the order of `abi`)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 7);
  void* at[6];
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      throw Failed{};
    }
  }
  abi = {reinterpret_cast<decltype(abi.norm_rope)>(at[0]),
         reinterpret_cast<decltype(abi.norm_rope_backward)>(at[1]),
         reinterpret_cast<decltype(abi.norm_rope_backward_workspace_size)>(at[2]),
         reinterpret_cast<decltype(abi.append_paged)>(at[3]),
         reinterpret_cast<decltype(abi.extend_paged)>(at[4]),
         reinterpret_cast<decltype(abi.extend_paged_workspace_size)>(at[5])};
  Py_INCREF(a[0]);
  fa_error = a[0];
  Py_RETURN_NONE;
}

// Exceptions become Python's: the checks' ValueError and TypeError, the allocator's out-of-memory error.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    TORCH_CHECK(F == bind || fa_error != nullptr, "the library is not bound: call through the package");
    return F(a, n);
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define FA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_METHOD(bind),         FA_METHOD(norm_rope),    FA_METHOD(norm_rope_backward),
                         FA_METHOD(append_paged), FA_METHOD(extend_paged), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  // The Python and torch that this file was compiled against, for __init__.py to compare.
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", FA_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
