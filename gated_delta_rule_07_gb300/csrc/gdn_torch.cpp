// gdn_torch.cpp -- Python's way to the calls of the softmax-attention layers, of linear attention and
// of the 8-bit checkpoints: checks torch tensors, allocates the outputs and calls the C ABI (gdn.h).
//
// A decode step's kernels take a few microseconds, and so would each look at a tensor from Python;
// here a look is a load.  Functions take positional arguments only (gdn.py has the signatures that
// users see) and return new tensors.  A refusal raises gdn.GdnError before any CUDA work, with the
// status that the C ABI gives for its kind; the C ABI's own refusals are raised the same way.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include "gdn.h"

namespace {

PyObject* g_error = nullptr;  // gdn.GdnError

struct Refusal {
  gdn_status status;
  std::string why;
};

[[noreturn]] void refuse(const std::string& why, gdn_status status = GDN_ERR_INVALID_ARGUMENT) {
  throw Refusal{status, why};
}
void check(gdn_status s, const char* where) {
  if (s != GDN_OK) refuse(where, s);
}

std::string shown(const at::Tensor& t) {
  std::ostringstream o;
  o << t.scalar_type() << " " << t.sizes() << " with strides " << t.strides() << " on " << t.device();
  return o.str();
}

// ------------------------------------------------------------------------------- arguments

// A cache as gdn.KVCache keeps it: the C ABI's description and the GPU that the buffers are on.
struct Cache {
  gdn_kv_cache desc;
  int32_t device;
};

class Args {
 public:
  Args(const char* name, PyObject* const* v, Py_ssize_t n, Py_ssize_t want) : name_(name), v_(v) {
    if (want >= 0 ? n != want : n < -want)  // (negative: so many or more)
      refuse(std::string(name) + ": wrong number of arguments");
    count_ = n;
  }
  Py_ssize_t count() const { return count_; }
  // The call's GPU is that of its cache or first tensor: all the others are to be on it.
  void on(int device, const char* what) const {
    if (device_ < 0) device_ = device;
    if (device != device_)
      refuse(at(what) + " is on cuda:" + std::to_string(device) + ", what comes before it on cuda:" +
             std::to_string(device_));
  }
  const at::Tensor& tensor(int i, const char* what) const {
    const at::Tensor* t = optional(i, what);
    if (!t) refuse(at(what) + " is to be a tensor");
    return *t;
  }
  const at::Tensor* optional(int i, const char* what) const {
    if (v_[i] == Py_None) return nullptr;
    if (!THPVariable_Check(v_[i])) refuse(at(what) + " is to be a tensor");
    const at::Tensor& t = THPVariable_Unpack(v_[i]);
    return &t;
  }
  // a contiguous GPU tensor of this dtype and shape (a negative length: any)
  const at::Tensor& packed(int i, const char* what, at::ScalarType dtype,
                           std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = tensor(i, what);
    bool ok = t.is_cuda() && t.scalar_type() == dtype && t.dim() == (int64_t)shape.size() &&
              t.is_contiguous();
    if (ok) {
      int64_t d = 0;
      for (int64_t n : shape) ok = ok && (n < 0 || t.size(d) == n), ++d;
    }
    if (!ok) {
      std::ostringstream o;
      o << at(what) << " is to be a contiguous " << dtype << " tensor [";
      for (int64_t n : shape) (n < 0 ? o << "any" : o << n) << " ";
      o << "] on the GPU, got " << shown(t);
      refuse(o.str());
    }
    on(t.get_device(), what);
    return t;
  }
  const void* packed_or_null(int i, const char* what, at::ScalarType dtype,
                             std::initializer_list<int64_t> shape) const {
    return v_[i] == Py_None ? nullptr : packed(i, what, dtype, shape).data_ptr();
  }
  // a [T, heads, D] GPU tensor whose last dimension is contiguous
  const at::Tensor& rows(int i, const char* what, at::ScalarType dtype) const {
    const at::Tensor& t = tensor(i, what);
    if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1))
      refuse(at(what) + " is to be [tokens, heads, D] with a contiguous last dimension, got " +
             shown(t));
    if (t.scalar_type() != dtype || !t.is_cuda())
      refuse(at(what) + " is not on the GPU, or has another dtype than the call: " + shown(t));
    on(t.get_device(), what);
    return t;
  }
  int io(int i, const char* what) const {
    const at::ScalarType s = tensor(i, what).scalar_type();
    if (s == at::kBFloat16) return GDN_BF16;
    if (s == at::kFloat) return GDN_F32;
    refuse(at(what) + ": dtype " + std::string(c10::toString(s)), GDN_ERR_UNSUPPORTED);
  }
  double real(int i) const {
    const double x = PyFloat_AsDouble(v_[i]);
    if (x == -1.0 && PyErr_Occurred()) throw std::exception();
    return x;
  }
  int64_t whole(int i) const {
    const int64_t x = PyLong_AsLongLong(v_[i]);
    if (x == -1 && PyErr_Occurred()) throw std::exception();
    return x;
  }
  bool none(int i) const { return v_[i] == Py_None; }
  const gdn_kv_cache* cache(int i) const {
    const Cache* c = static_cast<const Cache*>(PyLong_AsVoidPtr(v_[i]));
    on(c->device, "cache");
    return &c->desc;
  }
  const at::Tensor& workspace(int i) const {
    const at::Tensor& t = tensor(i, "workspace");
    if (!t.is_cuda() || !t.is_contiguous())
      refuse(at("workspace is to be a contiguous tensor on the GPU, got ") + shown(t));
    on(t.get_device(), "workspace");
    return t;
  }
  // the status word: an int32 tensor, or None
  int32_t* status(int i) const {
    return static_cast<int32_t*>(const_cast<void*>(packed_or_null(i, "dev_status", at::kInt, {1})));
  }
  // torch's current stream on the call's GPU, which becomes the current one until the call's end
  // (gdn.py makes the stream that a user names the current one)
  cudaStream_t stream() const {
    const auto d = static_cast<c10::DeviceIndex>(device_);
    if (d != c10::cuda::current_device()) guard_.emplace(d);
    return c10::cuda::getCurrentCUDAStream(d).stream();
  }
  std::string at(const char* what) const { return std::string(name_) + ": " + what; }

 private:
  const char* name_;
  PyObject* const* v_;
  Py_ssize_t count_ = 0;
  mutable int device_ = -1;
  mutable std::optional<c10::cuda::CUDAGuard> guard_;
};

const float* f32(const void* p) { return static_cast<const float*>(p); }
const int32_t* i32(const void* p) { return static_cast<const int32_t*>(p); }
// (torch.empty without the operator's way through the dispatcher, which costs as much again)
at::Tensor empty(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType dtype) {
  return at::Tensor(at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt));
}
PyObject* tuple_of(std::initializer_list<at::Tensor> tensors) {
  PyObject* t = PyTuple_New((Py_ssize_t)tensors.size());
  if (!t) throw std::exception();
  Py_ssize_t i = 0;
  for (const at::Tensor& x : tensors) {
    PyObject* o = THPVariable_Wrap(x);
    if (!o) {
      Py_DECREF(t);
      throw std::exception();
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// ------------------------------------------------------------------------------- the calls

struct Rope {
  gdn_qk_rope_problem p;
  const at::Tensor &q, &k;
  const int32_t* pos;
  const float *table, *qw, *kw;
};
// q, k, positions, cos_sin, q_weight, k_weight at 0 .. 5; eps, weight_offset, style at e ..
Rope rope_of(const Args& a, int e) {
  const int io = a.io(0, "q");
  const at::ScalarType dtype = io == GDN_BF16 ? at::kBFloat16 : at::kFloat;
  const at::Tensor& q = a.rows(0, "q", dtype);
  const at::Tensor& k = a.rows(1, "k", dtype);
  const int64_t T = q.size(0), D = q.size(2);
  if (k.size(0) != T || k.size(2) != D)
    refuse(a.at("q and k do not go together: ") + shown(q) + ", " + shown(k));
  const at::Tensor& table = a.packed(3, "cos_sin", at::kFloat, {-1, -1});
  const int64_t most = INT32_MAX;
  gdn_qk_rope_problem p = {T, (int32_t)std::min(q.size(1), most), (int32_t)std::min(k.size(1), most),
                           (int32_t)std::min(D, most), (int32_t)std::min(table.size(1), most),
                           (int32_t)a.whole(e + 2), io, (int32_t)std::min(table.size(0), most),
                           (float)a.real(e), (float)a.real(e + 1), q.stride(0), q.stride(1),
                           k.stride(0), k.stride(1)};
  return Rope{p, q, k, i32(a.packed(2, "positions", at::kInt, {T}).data_ptr()),
              f32(table.data_ptr()), f32(a.packed_or_null(4, "q_weight", at::kFloat, {D})),
              f32(a.packed_or_null(5, "k_weight", at::kFloat, {D}))};
}

// q, k, positions, cos_sin, q_weight, k_weight, eps, weight_offset, style, status
PyObject* qk_norm_rope(const Args& a) {
  const Rope r = rope_of(a, 6);
  at::Tensor q_out = empty(r.q.sizes(), r.q, r.q.scalar_type());
  at::Tensor k_out = empty(r.k.sizes(), r.k, r.q.scalar_type());
  check(gdn_qk_norm_rope(&r.p, r.q.data_ptr(), r.k.data_ptr(), r.pos, r.table, r.qw, r.kw,
                         q_out.data_ptr(), k_out.data_ptr(), a.status(9), a.stream()),
        "qk_norm_rope");
  return tuple_of({q_out, k_out});
}

// .., dq_out, dk_out, eps, weight_offset, style, workspace, status
PyObject* qk_norm_rope_backward(const Args& a) {
  const Rope r = rope_of(a, 8);
  const at::ScalarType dtype = r.q.scalar_type();
  const int64_t T = r.q.size(0), D = r.q.size(2);
  const at::Tensor& dqo = a.packed(6, "dq_out", dtype, {T, r.q.size(1), D});
  const at::Tensor& dko = a.packed(7, "dk_out", dtype, {T, r.k.size(1), D});
  at::Tensor dq = empty(r.q.sizes(), r.q, dtype), dk = empty(r.k.sizes(), r.k, dtype);
  at::Tensor dqw = empty({D}, r.q, at::kFloat), dkw = empty({D}, r.q, at::kFloat);
  const size_t need = gdn_qk_norm_rope_backward_workspace_size(&r.p);
  at::Tensor ws = a.none(11) ? empty({(int64_t)need}, r.q, at::kByte) : a.workspace(11);
  check(gdn_qk_norm_rope_backward(&r.p, r.q.data_ptr(), r.k.data_ptr(), r.pos, r.table, r.qw, r.kw,
                                  dqo.data_ptr(), dko.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                  dqw.data_ptr<float>(), dkw.data_ptr<float>(), ws.data_ptr(),
                                  ws.nbytes(), a.status(12), a.stream()),
        "qk_norm_rope_backward");
  return tuple_of({dq, dk, dqw, dkw});
}

// the tables of a cache call: block_table, lengths (or None), cu_seqlens (or None) at i ..
struct Tables {
  const at::Tensor& table;
  const int32_t *lens, *cu;
};
Tables tables_of(const Args& a, int i, int64_t T, gdn_kv_problem& p) {
  const at::Tensor& table = a.packed(i, "block_table", at::kInt, {-1, -1});
  const int64_t N = table.size(0), most = INT32_MAX;
  Tables t = {table, i32(a.packed_or_null(i + 1, "lengths", at::kInt, {N})),
              i32(a.packed_or_null(i + 2, "cu_seqlens", at::kInt, {N + 1}))};
  p.total_tokens = T;
  p.num_seqs = (int32_t)std::min(N, most);
  p.max_pages = (int32_t)std::min(table.size(1), most);
  return t;
}
void heads_of(const Args& a, const at::Tensor& t, const char* what, const gdn_kv_cache* c) {
  if (t.size(1) != c->hkv || t.size(2) != c->head_dim)
    refuse(a.at(what) + " does not fit a cache of " + std::to_string(c->hkv) + " heads of " +
           std::to_string(c->head_dim) + ": " + shown(t));
}

// cache, k, v, block_table, ctx_lens, cu_seqlens, status
PyObject* kv_append(const Args& a) {
  const gdn_kv_cache* c = a.cache(0);
  gdn_kv_problem p = {};
  p.io_dtype = a.io(1, "k");
  const at::ScalarType dtype = p.io_dtype == GDN_BF16 ? at::kBFloat16 : at::kFloat;
  const at::Tensor& k = a.rows(1, "k", dtype);
  const at::Tensor& v = a.rows(2, "v", dtype);
  heads_of(a, k, "k", c);
  heads_of(a, v, "v", c);
  if (v.size(0) != k.size(0)) refuse(a.at("k and v have different numbers of tokens"));
  const Tables t = tables_of(a, 3, k.size(0), p);
  p.k_token_stride = k.stride(0);
  p.k_head_stride = k.stride(1);
  p.v_token_stride = v.stride(0);
  p.v_head_stride = v.stride(1);
  check(gdn_kv_append(c, &p, k.data_ptr(), v.data_ptr(), i32(t.table.data_ptr()), t.lens, t.cu,
                      a.status(6), a.stream()),
        "kv_append");
  Py_RETURN_NONE;
}

// cache, block_table, start, cu_seqlens, tokens, io dtype, status
PyObject* kv_read(const Args& a) {
  const gdn_kv_cache* c = a.cache(0);
  gdn_kv_problem p = {};
  const int64_t T = a.whole(4);
  const Tables t = tables_of(a, 1, T, p);
  p.io_dtype = (int32_t)a.whole(5);
  const at::ScalarType dtype = p.io_dtype == GDN_BF16 ? at::kBFloat16 : at::kFloat;
  if (T < 0) refuse(a.at("tokens is negative"));
  const std::vector<int64_t> shape = {T, c->hkv, c->head_dim};
  at::Tensor k = empty(shape, t.table, dtype), v = empty(shape, t.table, dtype);
  check(gdn_kv_read(c, &p, i32(t.table.data_ptr()), t.lens, t.cu, k.data_ptr(), v.data_ptr(),
                    a.status(6), a.stream()),
        "kv_read");
  return tuple_of({k, v});
}

// cache, q, block_table, kv_lens, cu_seqlens, scale (or None), window, workspace, status
PyObject* kv_attention(const Args& a) {
  const gdn_kv_cache* c = a.cache(0);
  gdn_kv_problem p = {};
  p.io_dtype = a.io(1, "q");
  const at::Tensor& q = a.rows(1, "q", p.io_dtype == GDN_BF16 ? at::kBFloat16 : at::kFloat);
  const int64_t T = q.size(0), D = q.size(2), most = INT32_MAX;
  if (D != c->head_dim)
    refuse(a.at("q does not fit a cache of heads of ") + std::to_string(c->head_dim) + ": " +
           shown(q));
  const Tables t = tables_of(a, 2, T, p);
  p.hq = (int32_t)std::min(q.size(1), most);
  p.q_token_stride = q.stride(0);
  p.q_head_stride = q.stride(1);
  const float scale = a.none(5) ? (float)(1.0 / std::sqrt((double)D)) : (float)a.real(5);
  const int64_t window = a.whole(6);
  if (window < 0 || window > most) refuse(a.at("window is to be in [0, 2^31)"));
  at::Tensor out = empty(q.sizes(), q, q.scalar_type()), lse = empty({T, q.size(1)}, q, at::kFloat);
  at::Tensor ws = a.none(7)
      ? empty({(int64_t)gdn_kv_attention_workspace_size(c, &p)}, q, at::kByte)
      : a.workspace(7);
  check(gdn_kv_attention(c, &p, q.data_ptr(), i32(t.table.data_ptr()), t.lens, t.cu, scale,
                         (int32_t)window, out.data_ptr(), lse.data_ptr<float>(), ws.data_ptr(),
                         ws.nbytes(), a.status(8), a.stream()),
        "kv_attention");
  return tuple_of({out, lse});
}

// ------------------------------------------------ linear attention and the 8-bit checkpoints

at::ScalarType io_type(int io) { return io == GDN_BF16 ? at::kBFloat16 : at::kFloat; }
float* f32_out(const at::Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; }

void strides_of(const at::Tensor& t, int64_t& token, int64_t& head) {
  token = t.stride(0);
  head = t.stride(1);
}
// q, k [T, hk, K] and v [T, hv, V], as they go together; strides are the caller's
gdn_linear_problem linear_of(const Args& a, const at::Tensor& q, const at::Tensor& k,
                             const at::Tensor& v, int io) {
  const int64_t T = q.size(0), most = INT32_MAX;
  if (k.sizes() != q.sizes() || v.size(0) != T)
    refuse(a.at("q, k and v do not go together: ") + shown(q) + ", " + shown(k) + ", " + shown(v));
  gdn_linear_problem p = {};
  p.total_tokens = T;
  p.num_seqs = 1;
  p.hk = (int32_t)std::min(q.size(1), most);
  p.hv = (int32_t)std::min(v.size(1), most);
  p.k_dim = (int32_t)std::min(q.size(2), most);
  p.v_dim = (int32_t)std::min(v.size(2), most);
  p.io_dtype = io;
  return p;
}
// cu_seqlens (or None) at i: how many sequences
const int32_t* sequences(const Args& a, int i, gdn_linear_problem& p) {
  if (a.none(i)) return nullptr;
  const at::Tensor& cu = a.packed(i, "cu_seqlens", at::kInt, {-1});
  if (cu.size(0) < 2) refuse(a.at("cu_seqlens is to have an entry a sequence and one more"));
  p.num_seqs = (int32_t)std::min(cu.size(0) - 1, (int64_t)INT32_MAX);
  return i32(cu.data_ptr());
}
at::Tensor workspace_of(const Args& a, int i, size_t need, const at::Tensor& like) {
  return a.none(i) ? empty({(int64_t)need}, like, at::kByte) : a.workspace(i);
}

// q, k, v, log_decay, h0, cu_seqlens, workspace, status
PyObject* linear_attention(const Args& a) {
  const int io = a.io(0, "q");
  const at::Tensor& q = a.rows(0, "q", io_type(io));
  const at::Tensor& k = a.rows(1, "k", io_type(io));
  const at::Tensor& v = a.rows(2, "v", io_type(io));
  gdn_linear_problem p = linear_of(a, q, k, v, io);
  strides_of(q, p.q_token_stride, p.q_head_stride);
  strides_of(k, p.k_token_stride, p.k_head_stride);
  strides_of(v, p.v_token_stride, p.v_head_stride);
  const at::Tensor& decay = a.packed(3, "log_decay", at::kFloat, {v.size(1)});
  const int32_t* cu = sequences(a, 5, p);
  const std::vector<int64_t> states = {p.num_seqs, v.size(1), q.size(2), v.size(2)};
  const float* h0 = f32(a.packed_or_null(4, "h0", at::kFloat,
                                         {states[0], states[1], states[2], states[3]}));
  check(gdn_check_linear_problem(&p), "linear_attention");
  at::Tensor out = empty(v.sizes(), v, v.scalar_type()), last = empty(states, v, at::kFloat);
  at::Tensor ws = workspace_of(a, 6, gdn_linear_attention_workspace_size(&p), q);
  check(gdn_linear_attention(&p, q.data_ptr(), k.data_ptr(), v.data_ptr(), f32(decay.data_ptr()), h0,
                             cu, out.data_ptr(), f32_out(last), ws.data_ptr(), ws.nbytes(),
                             a.status(7), a.stream()),
        "linear_attention");
  return tuple_of({out, last});
}

// q, k, v (or their codes), q_scale, k_scale, v_scale (or None each), io dtype (of codes), log_decay,
// dout, h0, dh_final, cu_seqlens, workspace, status
PyObject* linear_attention_backward(const Args& a) {
  const bool held = !a.none(3);
  const int io = held ? (int)a.whole(6) : a.io(0, "q");
  at::ScalarType type = io_type(io);
  if (held) {
    type = a.tensor(0, "q").scalar_type();
    if (type != at::kChar && type != at::kFloat8_e4m3fn)
      refuse(a.at("the checkpoints' codes are ") + shown(a.tensor(0, "q")), GDN_ERR_UNSUPPORTED);
  }
  const at::Tensor& q = a.rows(0, "q", type);
  const at::Tensor& k = a.rows(1, "k", type);
  const at::Tensor& v = a.rows(2, "v", type);
  gdn_linear_problem p = linear_of(a, q, k, v, io);
  const int64_t T = q.size(0), hk = q.size(1), hv = v.size(1), K = q.size(2), V = v.size(2);
  gdn_linear_saved saved = {};
  if (held) {
    const char* names[] = {"q", "k", "v"};
    const float** scales[] = {&saved.q_scale, &saved.k_scale, &saved.v_scale};
    for (int i = 0; i < 3; ++i) {
      const at::Tensor& c = i == 0 ? q : i == 1 ? k : v;
      if (!c.is_contiguous()) refuse(a.at(names[i]) + "'s codes are to be contiguous: " + shown(c));
      *scales[i] = f32(a.packed(3 + i, "scale", at::kFloat, {T, i < 2 ? hk : hv}).data_ptr());
    }
    saved.q_codes = q.data_ptr();
    saved.k_codes = k.data_ptr();
    saved.v_codes = v.data_ptr();
    saved.format = type == at::kChar ? GDN_KV_INT8 : GDN_KV_E4M3;
  } else {
    strides_of(q, p.q_token_stride, p.q_head_stride);
    strides_of(k, p.k_token_stride, p.k_head_stride);
    strides_of(v, p.v_token_stride, p.v_head_stride);
  }
  const at::Tensor& decay = a.packed(7, "log_decay", at::kFloat, {hv});
  const at::Tensor& dout = a.packed(8, "dout", io_type(io), {T, hv, V});
  const int32_t* cu = sequences(a, 11, p);
  const std::vector<int64_t> states = {p.num_seqs, hv, K, V};
  const float* h0 = f32(a.packed_or_null(9, "h0", at::kFloat, {states[0], hv, K, V}));
  const float* dh = f32(a.packed_or_null(10, "dh_final", at::kFloat, {states[0], hv, K, V}));
  check(gdn_check_linear_problem(&p), "linear_attention_backward");
  at::Tensor dq = empty(q.sizes(), q, io_type(io)), dk = empty(k.sizes(), q, io_type(io));
  at::Tensor dv = empty(v.sizes(), q, io_type(io)), dh0 = empty(states, q, at::kFloat);
  at::Tensor ws =
      workspace_of(a, 12, gdn_linear_attention_backward_workspace_size(&p, held), q);
  check(gdn_linear_attention_backward(
            &p, held ? nullptr : q.data_ptr(), held ? nullptr : k.data_ptr(),
            held ? nullptr : v.data_ptr(), held ? &saved : nullptr, f32(decay.data_ptr()), h0, cu,
            dout.data_ptr(), dh, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), f32_out(dh0),
            ws.data_ptr(), ws.nbytes(), a.status(13), a.stream()),
        "linear_attention_backward");
  return tuple_of({dq, dk, dv, dh0});
}

// q, k, v, log_decay, slot, state, status
PyObject* linear_attention_decode(const Args& a) {
  const int io = a.io(0, "q");
  const at::Tensor& q = a.rows(0, "q", io_type(io));
  const at::Tensor& k = a.rows(1, "k", io_type(io));
  const at::Tensor& v = a.rows(2, "v", io_type(io));
  gdn_linear_problem p = linear_of(a, q, k, v, io);
  strides_of(q, p.q_token_stride, p.q_head_stride);
  strides_of(k, p.k_token_stride, p.k_head_stride);
  strides_of(v, p.v_token_stride, p.v_head_stride);
  const at::Tensor& decay = a.packed(3, "log_decay", at::kFloat, {v.size(1)});
  const at::Tensor& slot = a.packed(4, "slot", at::kInt, {q.size(0)});
  const at::Tensor& state = a.packed(5, "state", at::kFloat, {-1, v.size(1), q.size(2), v.size(2)});
  check(gdn_check_linear_problem(&p), "linear_attention_decode");
  at::Tensor out = empty(v.sizes(), v, v.scalar_type());
  check(gdn_linear_attention_decode(&p, (int32_t)std::min(state.size(0), (int64_t)INT32_MAX),
                                    q.data_ptr(), k.data_ptr(), v.data_ptr(), f32(decay.data_ptr()),
                                    i32(slot.data_ptr()), state.data_ptr<float>(), out.data_ptr(),
                                    a.status(6), a.stream()),
        "linear_attention_decode");
  return tuple_of({out});
}

gdn_checkpoint checkpoint_of(const at::Tensor& x, const at::Tensor& codes, const at::Tensor& scale,
                             int io) {
  const int64_t most = INT32_MAX;
  return {x.data_ptr(), codes.data_ptr(), scale.data_ptr<float>(), x.size(0), x.stride(0), x.stride(1),
          (int32_t)std::min(x.size(1), most), (int32_t)std::min(x.size(2), most), io};
}
constexpr Py_ssize_t kCheckpoints = 8;  // tensors of one C call
PyObject* tuple_of(const std::vector<at::Tensor>& tensors) {
  PyObject* t = PyTuple_New((Py_ssize_t)tensors.size());
  if (!t) throw std::exception();
  for (size_t i = 0; i < tensors.size(); ++i) {
    PyObject* o = THPVariable_Wrap(tensors[i]);
    if (!o) {
      Py_DECREF(t);
      throw std::exception();
    }
    PyTuple_SET_ITEM(t, (Py_ssize_t)i, o);
  }
  return t;
}

// status, format, tensors: (codes, scale) of each
PyObject* checkpoint_pack(const Args& a) {
  const int64_t format = a.whole(1);
  const Py_ssize_t n = a.count() - 2;
  if (n > kCheckpoints) refuse(a.at("at most 8 tensors a call"));
  std::vector<at::Tensor> made;
  gdn_checkpoint t[kCheckpoints];
  for (Py_ssize_t i = 0; i < n; ++i) {
    const int io = a.io(2 + (int)i, "tensor");
    const at::Tensor& x = a.rows(2 + (int)i, "tensor", io_type(io));
    if (x.size(1) == 0 || x.size(2) == 0) refuse(a.at("a tensor without heads: ") + shown(x));
    made.push_back(empty(x.sizes(), x, format == GDN_KV_INT8 ? at::kChar : at::kFloat8_e4m3fn));
    made.push_back(empty({x.size(0), x.size(1)}, x, at::kFloat));
    t[i] = checkpoint_of(x, made[2 * i], made[2 * i + 1], io);
  }
  check(gdn_checkpoint_pack(t, (int32_t)n, (int32_t)format, a.status(0), a.stream()),
        "checkpoint_pack");
  return tuple_of(made);
}

// then codes, scale and io dtype of each: the tensors
PyObject* checkpoint_open(const Args& a) {
  const Py_ssize_t n = a.count() / 3;
  if (a.count() % 3 || n > kCheckpoints) refuse(a.at("at most 8 checkpoints a call"));
  std::vector<at::Tensor> made;
  gdn_checkpoint t[kCheckpoints];
  const at::ScalarType type = a.tensor(0, "codes").scalar_type();
  if (type != at::kChar && type != at::kFloat8_e4m3fn)
    refuse(a.at("codes are ") + shown(a.tensor(0, "codes")), GDN_ERR_UNSUPPORTED);
  for (int i = 0; i < (int)n; ++i) {
    const at::Tensor& codes = a.packed(3 * i, "codes", type, {-1, -1, -1});
    const at::Tensor& scale =
        a.packed(3 * i + 1, "scale", at::kFloat, {codes.size(0), codes.size(1)});
    const int io = (int)a.whole(3 * i + 2);
    made.push_back(empty(codes.sizes(), codes, io_type(io)));
    t[i] = checkpoint_of(made.back(), codes, scale, io);
  }
  check(gdn_checkpoint_open(t, (int32_t)n, type == at::kChar ? GDN_KV_INT8 : GDN_KV_E4M3,
                            a.stream()),
        "checkpoint_open");
  return tuple_of(made);
}

// ------------------------------------------------------------------------------- the module

struct Call {
  PyObject* (*f)(const Args&);
  const char* name;
};
constexpr Call kCalls[] = {{kv_append, "kv_append"},
                           {kv_read, "kv_read"},
                           {kv_attention, "kv_attention"},
                           {qk_norm_rope, "qk_norm_rope"},
                           {qk_norm_rope_backward, "qk_norm_rope_backward"},
                           {linear_attention, "linear_attention"},
                           {linear_attention_backward, "linear_attention_backward"},
                           {linear_attention_decode, "linear_attention_decode"},
                           {checkpoint_pack, "checkpoint_pack"},
                           {checkpoint_open, "checkpoint_open"}};
template <PyObject* (*F)(const Args&)> constexpr const char* name_of() {
  for (const Call& c : kCalls)
    if (c.f == F) return c.name;
  return "";
}

template <PyObject* (*F)(const Args&), int N>
PyObject* entry(PyObject*, PyObject* const* v, Py_ssize_t n) {
  static constexpr const char* name = name_of<F>();
  try {
    return F(Args(name, v, n, N));
  } catch (const Refusal& r) {
    if (PyObject* e = PyObject_CallFunction(g_error, "is", (int)r.status, r.why.c_str())) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  } catch (const std::exception& e) {  // (torch's: out of memory, for one)
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(const Args&), int N> PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {
    method<qk_norm_rope, 10>("qk_norm_rope"),
    method<qk_norm_rope_backward, 13>("qk_norm_rope_backward"),
    method<kv_append, 7>("kv_append"),
    method<kv_read, 7>("kv_read"),
    method<kv_attention, 9>("kv_attention"),
    method<linear_attention, 8>("linear_attention"),
    method<linear_attention_backward, 14>("linear_attention_backward"),
    method<linear_attention_decode, 7>("linear_attention_decode"),
    method<checkpoint_pack, -3>("checkpoint_pack"),
    method<checkpoint_open, -3>("checkpoint_open"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_torch() { return PyModule_Create(&module); }
