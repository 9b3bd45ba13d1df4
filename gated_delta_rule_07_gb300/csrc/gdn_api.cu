// gdn_api.cu -- the C ABI of libgdn: host-side validation, workspace carving and the
// order of kernel launches for each entry point declared in include/gdn.h.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "gdn.h"
#include "gdn_attention.h"
#include "gdn_internal.h"
#include "gdn_linear.h"

namespace {

using gdn::Args;

constexpr size_t kAlign = 256;
constexpr size_t kStatusBytes = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The kernel family a problem runs on (the problem decides; there is no caller-side choice):
// the tcgen05 tensor-core kernels cover bf16 I/O with K = V = 128.
bool use_tensor_path(const gdn_problem* p) {
  return p->io_dtype == GDN_BF16 && p->k_dim == 128 && p->v_dim == 128;
}

// Phase 1 and phase 3 with the factors recomputed on chip (tensor-core kernels).
cudaError_t fused_summary(const gdn_problem*, const Args& a, cudaStream_t s,
                          cudaEvent_t mid = nullptr) {
  return gdn::tc5_summary(a, s, mid);
}
cudaError_t fused_emit(const gdn_problem*, const Args& a, cudaStream_t s) {
  return gdn::tc5_emit(a, s);
}

gdn_status check_problem(const gdn_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens < 0 || p->total_tokens > (int64_t)INT32_MAX || p->num_seqs < 1 ||
      p->hk < 1 || p->hv < 1 || p->k_dim < 1 || p->v_dim < 1 || p->chunk < 1 ||
      p->segments_per_seq < 1)
    return GDN_ERR_INVALID_ARGUMENT;
  if (p->hv % p->hk != 0) return GDN_ERR_INVALID_ARGUMENT;
  if (p->io_dtype != GDN_BF16 && p->io_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (p->chunk != 64) return GDN_ERR_UNSUPPORTED;
  if ((p->k_dim != 64 && p->k_dim != 128) || (p->v_dim != 64 && p->v_dim != 128))
    return GDN_ERR_UNSUPPORTED;
  if (p->hv > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y
  // grid.x of the per-segment kernels and element offsets in 64 bits
  if ((int64_t)p->num_seqs * p->segments_per_seq > (int64_t)INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

Args base_args(const gdn_problem* p) {
  Args a;
  memset(&a, 0, sizeof(a));
  a.T = p->total_tokens;
  a.N = p->num_seqs;
  a.hk = p->hk;
  a.hv = p->hv;
  a.K = p->k_dim;
  a.V = p->v_dim;
  a.P = p->segments_per_seq;
  a.bf16 = p->io_dtype == GDN_BF16;
  return a;
}

// cu_seqlens may be null only for a single sequence.
bool cu_ok(const gdn_problem* p, const int32_t* cu) { return cu != nullptr || p->num_seqs == 1; }

// The last CUDA error an entry point met on this host thread (reported by
// gdn_last_error_string).
thread_local cudaError_t t_last_error = cudaSuccess;

gdn_status to_status(cudaError_t e) {
  if (e == cudaSuccess) return GDN_OK;
  t_last_error = e;
  return GDN_ERR_CUDA;
}

#define GDN_TRY(expr)                              \
  do {                                             \
    cudaError_t _e = (expr);                       \
    if (_e != cudaSuccess) return to_status(_e);   \
  } while (0)

struct Layout {
  size_t status, M, U, h_in, w, u, gcum, wy, total;
};

// Workspace: [status word | M | U | h_in | w | u | gcum | records], each piece 256-byte
// aligned.  The summaries and incoming states exist only for P > 1; the materialised chunk
// factors only on the SIMT path (the tensor-core kernels recompute them on chip); the records
// (-w^T, fp16 K, u^T and the decay of each chunk, 49,664 bytes per chunk and value head) only
// on the tcgen05 path with P > 1, where the U summary writes them and the M summary and the
// emit kernel read them.
Layout layout(const gdn_problem* p, bool records = true) {
  Layout L;
  const size_t S = (size_t)p->num_seqs * p->segments_per_seq * p->hv;
  const size_t K = p->k_dim, V = p->v_dim, T = (size_t)p->total_tokens;
  const bool seg = p->segments_per_seq > 1;
  const bool mat = !use_tensor_path(p);
  size_t off = 0;
  L.status = off;
  off += kStatusBytes;
  L.M = off;
  off += seg ? align_up(S * K * K * 4) : 0;
  L.U = off;
  off += seg ? align_up(S * K * V * 4) : 0;
  L.h_in = off;
  off += seg ? align_up(S * K * V * 4) : 0;
  L.w = off;
  off += mat ? align_up(T * p->hv * K * 4) : 0;
  L.u = off;
  off += mat ? align_up(T * p->hv * V * 4) : 0;
  L.gcum = off;
  off += mat ? align_up(T * p->hv * 4) : 0;
  L.wy = off;  // tcgen05 path: the U summary's per-chunk records for the M summary
  off += (records && seg && !mat)
             ? align_up(gdn::tc5_records_bytes(p->total_tokens, p->num_seqs, p->hv))
             : 0;
  L.total = off;
  return L;
}

}  // namespace

extern "C" {

const char* gdn_status_string(gdn_status s) {
  switch (s) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_INVALID_ARGUMENT: return "GDN_ERR_INVALID_ARGUMENT: bad pointer, size or alignment";
    case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED: dtype/K/V/chunk outside the built set";
    case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE: workspace missing or too small";
    case GDN_ERR_CUDA: return "GDN_ERR_CUDA: a CUDA launch or runtime call failed";
    case GDN_ERR_DEVICE_TIMEOUT: return "GDN_ERR_DEVICE_TIMEOUT: a bounded device wait expired";
    case GDN_ERR_DEVICE_INPUT: return "GDN_ERR_DEVICE_INPUT: cu_seqlens inconsistent on the device";
    case GDN_ERR_DEVICE_RANGE: return "GDN_ERR_DEVICE_RANGE: a tensor-core operand exceeded the fp16 range";
  }
  return "GDN_UNKNOWN_STATUS";
}

int gdn_version(void) { return 100; }

const char* gdn_last_error_string(void) {
  return t_last_error == cudaSuccess ? "no CUDA error" : cudaGetErrorString(t_last_error);
}

gdn_status gdn_check_problem(const gdn_problem* p) { return check_problem(p); }

size_t gdn_workspace_size(const gdn_problem* p) {
  if (check_problem(p) != GDN_OK) return 0;
  return layout(p).total;
}

}  // extern "C"

size_t gdn::workspace_min_bytes(const gdn_problem* p) {
  return check_problem(p) != GDN_OK ? 0 : layout(p, false).total;
}

extern "C" {

gdn_status gdn_chunk_prepare(const gdn_problem* p, const void* k, const void* v, const float* g,
                             const float* beta, const int32_t* cu_seqlens, void* w, void* u,
                             float* gcum, int32_t* dev_status, cudaStream_t stream) {
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (p->total_tokens > 0 && (!k || !v || !g || !beta || !w || !u || !gcum))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(k) || !aligned16(v) || !aligned16(w) || !aligned16(u))
    return GDN_ERR_INVALID_ARGUMENT;
  Args a = base_args(p);
  a.k = k; a.v = v; a.g = g; a.beta = beta; a.cu = cu_seqlens;
  a.w_out = w; a.u_out = u; a.gcum_out = gcum; a.status = dev_status;
  if (a.T == 0) return GDN_OK;
  GDN_TRY(gdn::launch_validate_cu(a, stream));
  return to_status(gdn::simt_prepare(a, stream));
}

gdn_status gdn_segment_summary(const gdn_problem* p, const void* k, const void* w, const void* u,
                               const float* gcum, const int32_t* cu_seqlens, float* M, float* U,
                               int32_t* dev_status, cudaStream_t stream) {
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (!M || !U) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens > 0 && (!k || !w || !u || !gcum)) return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(k) || !aligned16(w) || !aligned16(u) || !aligned16(M) || !aligned16(U))
    return GDN_ERR_INVALID_ARGUMENT;
  Args a = base_args(p);
  a.k = k; a.w = w; a.u = u; a.gcum = gcum; a.cu = cu_seqlens;
  a.M_out = M; a.U_out = U; a.status = dev_status;
  GDN_TRY(gdn::launch_validate_cu(a, stream));
  return to_status(gdn::simt_summary(a, stream));
}

gdn_status gdn_state_prefix_scan(const gdn_problem* p, const float* M, const float* U,
                                 const float* h0, float* h_in, float* h_final,
                                 cudaStream_t stream) {
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (!M || !U || !h_in) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(M) || !aligned16(U) || !aligned16(h_in) || !aligned16(h0) || !aligned16(h_final))
    return GDN_ERR_INVALID_ARGUMENT;
  Args a = base_args(p);
  a.M = M; a.U = U; a.h0 = h0; a.h_in_out = h_in; a.h_final = h_final;
  return to_status(gdn::simt_scan(a, stream));
}

gdn_status gdn_chunk_emit(const gdn_problem* p, const void* q, const void* k, const void* w,
                          const void* u, const float* gcum, const float* h_in,
                          const int32_t* cu_seqlens, void* out, float* h_final,
                          int32_t* dev_status, cudaStream_t stream) {
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (p->total_tokens > 0 && (!q || !k || !w || !u || !gcum || !out))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(w) || !aligned16(u) || !aligned16(out) ||
      !aligned16(h_in) || !aligned16(h_final))
    return GDN_ERR_INVALID_ARGUMENT;
  Args a = base_args(p);
  a.q = q; a.k = k; a.w = w; a.u = u; a.gcum = gcum; a.h_in = h_in; a.cu = cu_seqlens;
  a.out = out; a.h_final = h_final; a.status = dev_status;
  GDN_TRY(gdn::launch_validate_cu(a, stream));
  return to_status(gdn::simt_emit(a, stream));
}

}  // extern "C"

namespace {
// gdn_forward, recording ev[0..4] (when given) before phase 1, after phase 1, after the scan,
// after phase 3, and between the two kernels of phase 1 (after phase 1's only launch on the
// paths with one).
gdn_status forward_impl(const gdn_problem* p, const void* q, const void* k, const void* v,
                        const float* g, const float* beta, const float* h0,
                        const int32_t* cu_seqlens, void* out, float* h_final, void* workspace,
                        size_t ws_bytes, cudaStream_t stream, cudaEvent_t* ev,
                        long long wait_cycles = 0, int fault = 0) {
  auto mark = [&](int i) { return ev ? cudaEventRecord(ev[i], stream) : cudaSuccess; };
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (p->total_tokens > 0 && (!q || !k || !v || !g || !beta || !out))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(h0) ||
      !aligned16(h_final))
    return GDN_ERR_INVALID_ARGUMENT;
  // The records are optional: without room for them both summaries compute their factors.
  const Layout Lr = layout(p, true), L = ws_bytes >= Lr.total ? Lr : layout(p, false);
  if (!workspace || ws_bytes < L.total || !aligned16(workspace)) return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws + L.status);
  GDN_TRY(cudaMemsetAsync(status, 0, sizeof(int32_t), stream));

  Args a = base_args(p);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h0 = h0; a.cu = cu_seqlens;
  a.out = out; a.h_final = h_final; a.status = status;
  a.wait_cycles = wait_cycles;
  a.fault = fault;
  const bool seg = p->segments_per_seq > 1;
  if (seg) {
    a.M_out = reinterpret_cast<float*>(ws + L.M);
    a.U_out = reinterpret_cast<float*>(ws + L.U);
    a.M = a.M_out;
    a.U = a.U_out;
    a.h_in_out = reinterpret_cast<float*>(ws + L.h_in);
    if (use_tensor_path(p) && L.total == Lr.total && Lr.total > Lr.wy)
      a.wy = ws + L.wy;
  }
  // With P = 1 the incoming state of the only segment is h0 itself.
  a.h_in = seg ? a.h_in_out : h0;
  GDN_TRY(gdn::launch_validate_cu(a, stream));

  GDN_TRY(mark(0));
  if (use_tensor_path(p)) {
    if (seg) {
      Args ma = a;
      ma.skip_last_summary = true;
      GDN_TRY(fused_summary(p, ma, stream, ev ? ev[4] : nullptr));
      GDN_TRY(mark(1));
      Args sa = a;
      sa.h_final = nullptr;  // the last segment's emit writes the final state
      GDN_TRY(gdn::simt_scan(sa, stream));
    } else {
      GDN_TRY(mark(1));
      GDN_TRY(mark(4));
    }
    GDN_TRY(mark(2));
    GDN_TRY(fused_emit(p, a, stream));
    return to_status(mark(3));
  }
  a.w_out = ws + L.w;
  a.u_out = ws + L.u;
  a.gcum_out = reinterpret_cast<float*>(ws + L.gcum);
  a.w = a.w_out;
  a.u = a.u_out;
  a.gcum = a.gcum_out;
  if (a.T > 0) GDN_TRY(gdn::simt_prepare(a, stream));
  if (seg) {
    GDN_TRY(gdn::simt_summary(a, stream));  // (the SIMT summary computes every segment)
    GDN_TRY(mark(4));
    GDN_TRY(mark(1));
    Args sa = a;
    sa.h_final = nullptr;
    GDN_TRY(gdn::simt_scan(sa, stream));
  } else {
    GDN_TRY(mark(1));
    GDN_TRY(mark(4));
  }
  GDN_TRY(mark(2));
  GDN_TRY(gdn::simt_emit(a, stream));
  return to_status(mark(3));
}
}  // namespace

extern "C" {

gdn_status gdn_forward(const gdn_problem* p, const void* q, const void* k, const void* v,
                       const float* g, const float* beta, const float* h0,
                       const int32_t* cu_seqlens, void* out, float* h_final, void* workspace,
                       size_t ws_bytes, cudaStream_t stream) {
  return forward_impl(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace, ws_bytes,
                      stream, nullptr);
}

gdn_status gdn_forward_with_limits(const gdn_problem* p, const void* q, const void* k,
                                   const void* v, const float* g, const float* beta,
                                   const float* h0, const int32_t* cu_seqlens, void* out,
                                   float* h_final, void* workspace, size_t ws_bytes,
                                   cudaStream_t stream, long long wait_cycles, int fault) {
  if (wait_cycles < 0 || fault < 0 || fault > 1) return GDN_ERR_INVALID_ARGUMENT;
  return forward_impl(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace, ws_bytes,
                      stream, nullptr, wait_cycles, fault);
}

gdn_status gdn_forward_timed(const gdn_problem* p, const void* q, const void* k, const void* v,
                             const float* g, const float* beta, const float* h0,
                             const int32_t* cu_seqlens, void* out, float* h_final,
                             void* workspace, size_t ws_bytes, cudaStream_t stream,
                             float* phase_ms) {
  if (!phase_ms) return GDN_ERR_INVALID_ARGUMENT;
  cudaEvent_t ev[5] = {};
  for (int i = 0; i < 5; ++i)
    if (cudaEventCreate(&ev[i]) != cudaSuccess) {
      for (int k2 = 0; k2 < i; ++k2) cudaEventDestroy(ev[k2]);
      return to_status(cudaGetLastError());
    }
  gdn_status st = forward_impl(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace,
                               ws_bytes, stream, ev);
  if (st == GDN_OK) {
    cudaError_t e = cudaEventSynchronize(ev[3]);
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = cudaEventElapsedTime(&phase_ms[i], ev[i], ev[i + 1]);
    if (e == cudaSuccess) e = cudaEventElapsedTime(&phase_ms[3], ev[0], ev[4]);
    if (e != cudaSuccess) st = to_status(e);
  }
  for (int i = 0; i < 5; ++i) cudaEventDestroy(ev[i]);
  return st;
}

gdn_status gdn_segment_summary_fused(const gdn_problem* p, const void* k, const void* v,
                                     const float* g, const float* beta,
                                     const int32_t* cu_seqlens, float* M, float* U,
                                     int skip_last, int32_t* dev_status, cudaStream_t stream) {
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (!use_tensor_path(p)) return GDN_ERR_UNSUPPORTED;
  if (!M || !U) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens > 0 && (!k || !v || !g || !beta)) return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(k) || !aligned16(v) || !aligned16(M) || !aligned16(U))
    return GDN_ERR_INVALID_ARGUMENT;
  Args a = base_args(p);
  a.k = k; a.v = v; a.g = g; a.beta = beta; a.cu = cu_seqlens;
  a.M_out = M; a.U_out = U; a.status = dev_status; a.skip_last_summary = skip_last != 0;
  GDN_TRY(gdn::launch_validate_cu(a, stream));
  return to_status(fused_summary(p, a, stream));
}

gdn_status gdn_chunk_emit_fused(const gdn_problem* p, const void* q, const void* k,
                                const void* v, const float* g, const float* beta,
                                const float* h_in, const int32_t* cu_seqlens, void* out,
                                float* h_final, int32_t* dev_status, cudaStream_t stream) {
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (!use_tensor_path(p)) return GDN_ERR_UNSUPPORTED;
  if (p->total_tokens > 0 && (!q || !k || !v || !g || !beta || !out))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(h_in) ||
      !aligned16(h_final))
    return GDN_ERR_INVALID_ARGUMENT;
  Args a = base_args(p);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h_in = h_in; a.cu = cu_seqlens;
  a.out = out; a.h_final = h_final; a.status = dev_status;
  GDN_TRY(gdn::launch_validate_cu(a, stream));
  return to_status(fused_emit(p, a, stream));
}

// ------------------------------------------------------------------ backward

// CTAs of the per-chunk gradient kernel (two per SM of a 152-SM GB300); the workspace holds one
// slice of intermediates for each.  The kernel walks all units with a grid stride, so any SM
// count computes the same result.
constexpr int kGradCtas = 304;

struct BwdLayout {
  size_t status, states, dstates, dqv, dkv, scratch, total;
};
BwdLayout bwd_layout(const gdn_problem* p) {
  BwdLayout L;
  const size_t K = p->k_dim, V = p->v_dim, T = (size_t)p->total_tokens;
  const size_t slots = (size_t)gdn::bwd_slots(p->total_tokens, p->num_seqs);
  size_t off = 0;
  L.status = off;
  off += kStatusBytes;
  L.states = off;
  off += align_up(slots * p->hv * K * V * 4);
  L.dstates = off;
  off += align_up(slots * p->hv * K * V * 4);
  L.dqv = off;
  off += align_up(T * p->hv * K * 4);
  L.dkv = off;
  off += align_up(T * p->hv * K * 4);
  L.scratch = off;
  off += align_up(gdn::bwd_scratch_floats(p->k_dim, p->v_dim, kGradCtas) * 4);
  L.total = off;
  return L;
}

gdn_status gdn_prologue(const gdn_prologue_problem* p, const void* x, const float* conv_w,
                        const void* conv_state_in, const void* a, const void* b,
                        const float* A_log, const float* dt_bias, const int32_t* cu_seqlens,
                        void* q, void* k, void* v, float* g, float* beta, void* conv_state_out,
                        int32_t* dev_status, cudaStream_t stream) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens < 0 || p->total_tokens > (int64_t)INT32_MAX || p->num_seqs < 1 ||
      p->hk < 1 || p->hv < 1 || p->k_dim < 1 || p->v_dim < 1 || p->hv % p->hk != 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (p->io_dtype != GDN_BF16 && p->io_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (p->k_dim > 128 || p->v_dim > 128 || p->k_dim % 8 || p->v_dim % 8 || p->conv_width < 1 ||
      p->conv_width > 4 ||
      (p->activation != 0 && p->activation != 1) || 2 * p->hk + p->hv > 65535)
    return GDN_ERR_UNSUPPORTED;
  if (!conv_w || !A_log || !dt_bias || (p->total_tokens > 0 &&
      (!x || !a || !b || !q || !k || !v || !g || !beta)))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens && p->num_seqs != 1) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(q) || !aligned16(k) || !aligned16(v))
    return GDN_ERR_INVALID_ARGUMENT;
  gdn::PrologueArgs pa;
  memset(&pa, 0, sizeof(pa));
  pa.T = p->total_tokens;
  pa.N = p->num_seqs;
  pa.hk = p->hk;
  pa.hv = p->hv;
  pa.K = p->k_dim;
  pa.V = p->v_dim;
  pa.W = p->conv_width;
  pa.bf16 = p->io_dtype == GDN_BF16;
  pa.silu = p->activation == 1;
  pa.x = x; pa.state_in = conv_state_in; pa.a = a; pa.b = b;
  pa.conv_w = conv_w; pa.A_log = A_log; pa.dt_bias = dt_bias; pa.cu = cu_seqlens;
  pa.q = q; pa.k = k; pa.v = v; pa.state_out = conv_state_out; pa.g = g; pa.beta = beta;
  pa.status = dev_status;
  if (cu_seqlens) {
    Args va;
    memset(&va, 0, sizeof(va));
    va.T = p->total_tokens;
    va.N = p->num_seqs;
    va.cu = cu_seqlens;
    va.status = dev_status;
    GDN_TRY(gdn::launch_validate_cu(va, stream));
  }
  return to_status(gdn::prologue(pa, stream));
}

gdn_status gdn_check_decode_problem(const gdn_decode_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  if (p->batch < 0 || p->slots < 1 || p->hk < 1 || p->hv < 1 || p->k_dim < 1 || p->v_dim < 1)
    return GDN_ERR_INVALID_ARGUMENT;
  if (p->hv % p->hk != 0) return GDN_ERR_INVALID_ARGUMENT;
  if (p->io_dtype != GDN_BF16 && p->io_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if ((p->k_dim != 64 && p->k_dim != 128) || (p->v_dim != 64 && p->v_dim != 128))
    return GDN_ERR_UNSUPPORTED;
  if (p->hv > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y
  return GDN_OK;
}

gdn_status gdn_decode_step(const gdn_decode_problem* p, const void* q, const void* k,
                           const void* v, const float* g, const float* beta,
                           const int32_t* slot, float* state, void* out, int32_t* dev_status,
                           cudaStream_t stream) {
  gdn_status st = gdn_check_decode_problem(p);
  if (st != GDN_OK) return st;
  if (p->batch == 0) return GDN_OK;
  if (!q || !k || !v || !g || !beta || !slot || !state || !out) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
      !aligned16(slot) || !aligned16(state) || !aligned16(out))
    return GDN_ERR_INVALID_ARGUMENT;
  gdn::DecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.batch = p->batch;
  a.slots = p->slots;
  a.hk = p->hk;
  a.hv = p->hv;
  a.K = p->k_dim;
  a.V = p->v_dim;
  a.bf16 = p->io_dtype == GDN_BF16;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.slot = slot;
  a.state = state;
  a.out = out;
  a.status = dev_status;
  return to_status(gdn::decode_step(a, stream));
}

size_t gdn_backward_workspace_size(const gdn_problem* p) {
  return check_problem(p) != GDN_OK ? 0 : bwd_layout(p).total;
}

gdn_status gdn_backward(const gdn_problem* p, const void* q, const void* k, const void* v,
                        const float* g, const float* beta, const float* h0,
                        const int32_t* cu_seqlens, const void* dout, const float* dh_final,
                        void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dh0,
                        void* workspace, size_t ws_bytes, cudaStream_t stream) {
  gdn_status st = check_problem(p);
  if (st != GDN_OK) return st;
  if (p->total_tokens > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv ||
                              !dg || !dbeta))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned16(h0) || !aligned16(dh_final) ||
      !aligned16(dh0))
    return GDN_ERR_INVALID_ARGUMENT;
  const BwdLayout L = bwd_layout(p);
  if (!workspace || ws_bytes < L.total || !aligned16(workspace)) return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws + L.status);
  GDN_TRY(cudaMemsetAsync(status, 0, sizeof(int32_t), stream));
  Args va = base_args(p);
  va.cu = cu_seqlens;
  va.status = status;
  GDN_TRY(gdn::launch_validate_cu(va, stream));
  gdn::BwdArgs a;
  memset(&a, 0, sizeof(a));
  a.T = p->total_tokens;
  a.nslots = gdn::bwd_slots(p->total_tokens, p->num_seqs);
  a.N = p->num_seqs;
  a.hk = p->hk;
  a.hv = p->hv;
  a.K = p->k_dim;
  a.V = p->v_dim;
  a.bf16 = p->io_dtype == GDN_BF16;
  a.q = q; a.k = k; a.v = v; a.dout = dout;
  a.g = g; a.beta = beta; a.h0 = h0; a.dh_final = dh_final; a.cu = cu_seqlens;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
  a.states = reinterpret_cast<float*>(ws + L.states);
  a.dstates = reinterpret_cast<float*>(ws + L.dstates);
  a.dqv = reinterpret_cast<float*>(ws + L.dqv);
  a.dkv = reinterpret_cast<float*>(ws + L.dkv);
  a.scratch = reinterpret_cast<float*>(ws + L.scratch);
  a.grad_ctas = kGradCtas;
  a.status = status;
  if (a.T == 0) {  // no tokens: the state passes through, dh0 = dh_final
    if (dh0) {
      const size_t bytes = (size_t)p->num_seqs * p->hv * p->k_dim * p->v_dim * 4;
      if (dh_final)
        GDN_TRY(cudaMemcpyAsync(dh0, dh_final, bytes, cudaMemcpyDeviceToDevice, stream));
      else
        GDN_TRY(cudaMemsetAsync(dh0, 0, bytes, stream));
    }
    return GDN_OK;
  }
  return to_status(gdn::backward(a, stream));
}

// ------------------------------------------------ softmax-attention layers' operators

namespace {

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// a dimension's stride; that of a single row means nothing
int64_t stride_of(int64_t stride, int64_t rows) { return rows > 1 ? stride : 0; }

// rows strided in elements: every row starts on a 16-byte boundary
bool strides_ok(int64_t token, int64_t tokens, int64_t head, int64_t heads, int io) {
  const int64_t unit = io == GDN_BF16 ? 8 : 4;
  token = stride_of(token, tokens);
  head = stride_of(head, heads);
  return token >= 0 && head >= 0 && token % unit == 0 && head % unit == 0;
}

gdn_status check_rope(const gdn_qk_rope_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens < 0 || p->total_tokens > (int64_t)INT32_MAX || p->hq < 1 || p->hkv < 1 ||
      p->max_positions < 1 || p->rotary_dim < 0 || p->rotary_dim > p->head_dim ||
      (p->style != 0 && p->style != 1) || !(p->eps >= 0.f))
    return GDN_ERR_INVALID_ARGUMENT;
  if (p->io_dtype != GDN_BF16 && p->io_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (!head_dim_ok(p->head_dim) || p->rotary_dim % 16 || p->hq > 65535 || p->hkv > 65535)
    return GDN_ERR_UNSUPPORTED;
  if (!strides_ok(p->q_token_stride, p->total_tokens, p->q_head_stride, p->hq, p->io_dtype) ||
      !strides_ok(p->k_token_stride, p->total_tokens, p->k_head_stride, p->hkv, p->io_dtype))
    return GDN_ERR_INVALID_ARGUMENT;
  return GDN_OK;
}

gdn::QkRopeArgs rope_args(const gdn_qk_rope_problem* p, const void* q, const void* k,
                          const int32_t* positions, const float* cos_sin, const float* wq,
                          const float* wk, int32_t* dev_status) {
  gdn::QkRopeArgs a;
  memset(&a, 0, sizeof(a));
  a.T = p->total_tokens;
  a.q_ts = stride_of(p->q_token_stride, p->total_tokens);
  a.q_hs = stride_of(p->q_head_stride, p->hq);
  a.k_ts = stride_of(p->k_token_stride, p->total_tokens);
  a.k_hs = stride_of(p->k_head_stride, p->hkv);
  a.hq = p->hq; a.hkv = p->hkv; a.D = p->head_dim; a.R = p->rotary_dim;
  a.max_pos = p->max_positions;
  a.bf16 = p->io_dtype == GDN_BF16;
  a.pairs = p->style == 1;
  a.eps = p->eps; a.offset = p->weight_offset;
  a.q = q; a.k = k; a.pos = positions; a.table = cos_sin; a.wq = wq; a.wk = wk;
  a.status = dev_status;
  return a;
}

gdn_status check_kv(const gdn_kv_cache* c, const gdn_kv_problem* p) {
  if (!c || !p) return GDN_ERR_INVALID_ARGUMENT;
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !aligned16(c->k_codes) ||
      !aligned16(c->v_codes) || c->num_pages < 1 || c->hkv < 1 || p->total_tokens < 0 ||
      p->total_tokens > (int64_t)INT32_MAX || p->num_seqs < 1 || p->max_pages < 1)
    return GDN_ERR_INVALID_ARGUMENT;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return GDN_ERR_UNSUPPORTED;
  if (c->format != GDN_KV_INT8 && c->format != GDN_KV_E4M3) return GDN_ERR_UNSUPPORTED;
  if (p->io_dtype != GDN_BF16 && p->io_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (!head_dim_ok(c->head_dim) || c->hkv > 65535) return GDN_ERR_UNSUPPORTED;
  // positions are 32-bit (with room for a tile past the end); slots of touched pages are grid.x
  if ((int64_t)p->max_pages * c->page_size > (int64_t)1 << 30 ||
      p->total_tokens / c->page_size + 2 * (int64_t)p->num_seqs > (int64_t)INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

bool rows_ok(const gdn_kv_problem* p, const int32_t* cu) {
  return cu != nullptr || p->num_seqs == 1 || p->total_tokens == p->num_seqs;
}

gdn::KvArgs kv_args(const gdn_kv_cache* c, const gdn_kv_problem* p, const int32_t* table,
                    const int32_t* pos0, const int32_t* cu, int32_t* dev_status) {
  gdn::KvArgs a;
  memset(&a, 0, sizeof(a));
  a.T = p->total_tokens;
  a.N = p->num_seqs; a.hq = p->hq; a.hkv = c->hkv; a.D = c->head_dim;
  a.group = p->hq / c->hkv;
  if (a.group > 1) a.group_mul = (uint32_t)((0xffffffffu / (uint32_t)a.group) + 1);
  a.page = c->page_size;
  while ((1 << a.page_shift) < a.page) ++a.page_shift;
  a.num_pages = c->num_pages; a.max_pages = p->max_pages;
  a.k_ts = stride_of(p->k_token_stride, p->total_tokens);
  a.k_hs = stride_of(p->k_head_stride, c->hkv);
  a.v_ts = stride_of(p->v_token_stride, p->total_tokens);
  a.v_hs = stride_of(p->v_head_stride, c->hkv);
  a.q_ts = stride_of(p->q_token_stride, p->total_tokens);
  a.q_hs = stride_of(p->q_head_stride, p->hq);
  a.bf16 = p->io_dtype == GDN_BF16;
  a.e4m3 = c->format == GDN_KV_E4M3;
  a.table = table; a.pos0 = pos0; a.cu = cu;
  a.k_codes = static_cast<uint8_t*>(c->k_codes);
  a.v_codes = static_cast<uint8_t*>(c->v_codes);
  a.k_scale = c->k_scale; a.v_scale = c->v_scale;
  a.status = dev_status;
  return a;
}

}  // namespace

gdn_status gdn_qk_norm_rope(const gdn_qk_rope_problem* p, const void* q, const void* k,
                            const int32_t* positions, const float* cos_sin,
                            const float* q_weight, const float* k_weight, void* q_out,
                            void* k_out, int32_t* dev_status, cudaStream_t stream) {
  const gdn_status st = check_rope(p);
  if (st != GDN_OK) return st;
  if (p->total_tokens == 0) return GDN_OK;
  if (!q || !k || !positions || !q_out || !k_out || (!cos_sin && p->rotary_dim))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(cos_sin) || !aligned16(q_weight) || !aligned16(k_weight))
    return GDN_ERR_INVALID_ARGUMENT;
  gdn::QkRopeArgs a = rope_args(p, q, k, positions, cos_sin, q_weight, k_weight, dev_status);
  a.q_out = q_out;
  a.k_out = k_out;
  return to_status(gdn::qk_rope(a, false, stream));
}

size_t gdn_qk_norm_rope_backward_workspace_size(const gdn_qk_rope_problem* p) {
  return check_rope(p) != GDN_OK ? 0 : (size_t)gdn::kRopeCtas * p->head_dim * sizeof(float);
}

gdn_status gdn_qk_norm_rope_backward(const gdn_qk_rope_problem* p, const void* q, const void* k,
                                     const int32_t* positions, const float* cos_sin,
                                     const float* q_weight, const float* k_weight,
                                     const void* dq_out, const void* dk_out, void* dq, void* dk,
                                     float* dq_weight, float* dk_weight, void* workspace,
                                     size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  const gdn_status st = check_rope(p);
  if (st != GDN_OK) return st;
  if (!dq_weight || !dk_weight) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens == 0) {  // sums over no rows
    GDN_TRY(cudaMemsetAsync(dq_weight, 0, p->head_dim * sizeof(float), stream));
    GDN_TRY(cudaMemsetAsync(dk_weight, 0, p->head_dim * sizeof(float), stream));
    return GDN_OK;
  }
  if (!q || !k || !positions || !dq_out || !dk_out || !dq || !dk || (!cos_sin && p->rotary_dim))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(dq_out) || !aligned16(dk_out) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(cos_sin) || !aligned16(q_weight) ||
      !aligned16(k_weight))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!workspace || !aligned16(workspace) ||
      ws_bytes < gdn_qk_norm_rope_backward_workspace_size(p))
    return GDN_ERR_WORKSPACE;
  gdn::QkRopeArgs a = rope_args(p, q, k, positions, cos_sin, q_weight, k_weight, dev_status);
  a.dq_out = dq_out; a.dk_out = dk_out; a.dq = dq; a.dk = dk;
  a.dwq = dq_weight; a.dwk = dk_weight;
  a.partial = static_cast<float*>(workspace);
  return to_status(gdn::qk_rope(a, true, stream));
}

gdn_status gdn_kv_append(const gdn_kv_cache* cache, const gdn_kv_problem* p, const void* k,
                         const void* v, const int32_t* block_table, const int32_t* ctx_lens,
                         const int32_t* cu_seqlens, int32_t* dev_status, cudaStream_t stream) {
  const gdn_status st = check_kv(cache, p);
  if (st != GDN_OK) return st;
  if (!strides_ok(p->k_token_stride, p->total_tokens, p->k_head_stride, cache->hkv, p->io_dtype) ||
      !strides_ok(p->v_token_stride, p->total_tokens, p->v_head_stride, cache->hkv, p->io_dtype) ||
      !rows_ok(p, cu_seqlens))
    return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens == 0) return GDN_OK;
  if (!k || !v || !block_table || !ctx_lens || !aligned16(k) || !aligned16(v))
    return GDN_ERR_INVALID_ARGUMENT;
  gdn::KvArgs a = kv_args(cache, p, block_table, ctx_lens, cu_seqlens, dev_status);
  a.k = k;
  a.v = v;
  return to_status(gdn::kv_append(a, stream));
}

gdn_status gdn_kv_read(const gdn_kv_cache* cache, const gdn_kv_problem* p,
                       const int32_t* block_table, const int32_t* start,
                       const int32_t* cu_seqlens, void* k_out, void* v_out, int32_t* dev_status,
                       cudaStream_t stream) {
  const gdn_status st = check_kv(cache, p);
  if (st != GDN_OK) return st;
  if (!rows_ok(p, cu_seqlens)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens == 0) return GDN_OK;
  if (!block_table || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return GDN_ERR_INVALID_ARGUMENT;
  gdn::KvArgs a = kv_args(cache, p, block_table, start, cu_seqlens, dev_status);
  a.k_out = k_out;
  a.v_out = v_out;
  return to_status(gdn::kv_read(a, stream));
}

static gdn_status check_kv_attention(const gdn_kv_cache* cache, const gdn_kv_problem* p) {
  const gdn_status st = check_kv(cache, p);
  if (st != GDN_OK) return st;
  if (p->hq < 1 || p->hq % cache->hkv ||
      !strides_ok(p->q_token_stride, p->total_tokens, p->q_head_stride, p->hq, p->io_dtype))
    return GDN_ERR_INVALID_ARGUMENT;
  // rows (tokens x query heads) are 32-bit
  return p->hq > 32768 || p->total_tokens * p->hq > (int64_t)INT32_MAX ? GDN_ERR_UNSUPPORTED
                                                                     : GDN_OK;
}

size_t gdn_kv_attention_workspace_size(const gdn_kv_cache* cache, const gdn_kv_problem* p) {
  if (check_kv_attention(cache, p) != GDN_OK) return 0;
  return gdn::kv_attention_workspace(kv_args(cache, p, nullptr, nullptr, nullptr, nullptr));
}

gdn_status gdn_kv_attention(const gdn_kv_cache* cache, const gdn_kv_problem* p, const void* q,
                            const int32_t* block_table, const int32_t* kv_lens,
                            const int32_t* cu_seqlens, float scale, int32_t window, void* out,
                            float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status,
                            cudaStream_t stream) {
  const gdn_status st = check_kv_attention(cache, p);
  if (st != GDN_OK) return st;
  if (!rows_ok(p, cu_seqlens) || window < 0) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens == 0) return GDN_OK;
  if (!q || !block_table || !kv_lens || !out || !aligned16(q) || !aligned16(out))
    return GDN_ERR_INVALID_ARGUMENT;
  gdn::KvArgs a = kv_args(cache, p, block_table, kv_lens, cu_seqlens, dev_status);
  const size_t need = gdn::kv_attention_workspace(a);
  if (need && (!workspace || !aligned16(workspace) || ws_bytes < need))
    return GDN_ERR_WORKSPACE;
  a.q = q; a.out = out; a.lse = lse;
  a.scale = scale;
  a.window = window;
  a.workspace = static_cast<float*>(workspace);
  return to_status(gdn::kv_attention(a, stream));
}

// ------------------------------------------------ linear attention with a decay for each head

namespace {

gdn_status check_linear(const gdn_linear_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens < 0 || p->total_tokens > (int64_t)INT32_MAX || p->num_seqs < 1 ||
      p->hk < 1 || p->hv < 1 || p->k_dim < 1 || p->v_dim < 1 || p->hv % p->hk != 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (p->io_dtype != GDN_BF16 && p->io_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if ((p->k_dim != 64 && p->k_dim != 128) || (p->v_dim != 64 && p->v_dim != 128))
    return GDN_ERR_UNSUPPORTED;
  if (p->hv > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y
  // segments (times heads) are grid.x, of at least 64 tokens each but the last of a sequence
  if ((p->total_tokens / 64 + p->num_seqs) * p->hv > (int64_t)INT32_MAX) return GDN_ERR_UNSUPPORTED;
  if (!strides_ok(p->q_token_stride, p->total_tokens, p->q_head_stride, p->hk, p->io_dtype) ||
      !strides_ok(p->k_token_stride, p->total_tokens, p->k_head_stride, p->hk, p->io_dtype) ||
      !strides_ok(p->v_token_stride, p->total_tokens, p->v_head_stride, p->hv, p->io_dtype))
    return GDN_ERR_INVALID_ARGUMENT;
  return GDN_OK;
}

// The problem of a call that is given 8-bit activations: they are opened to packed rows.
gdn_linear_problem linear_opened(const gdn_linear_problem* p) {
  gdn_linear_problem o = *p;
  o.q_token_stride = o.k_token_stride = (int64_t)p->hk * p->k_dim;
  o.v_token_stride = (int64_t)p->hv * p->v_dim;
  o.q_head_stride = o.k_head_stride = p->k_dim;
  o.v_head_stride = p->v_dim;
  return o;
}

// Whether the tensor-core kernels take a problem.  (They read rows through tensor maps, which have no
// way to say that a row is all tokens' or heads': broadcast rows go to the CUDA cores.)
bool linear_on_tc(const gdn_linear_problem* p) {
  const int64_t T = p->total_tokens;
  auto mapped = [T](int64_t ts, int64_t hs, int heads) {
    return (T == 1 || (ts > 0 && ts < (int64_t)1 << 38)) &&
           (heads == 1 || (hs > 0 && hs < (int64_t)1 << 38));
  };
  return p->io_dtype == GDN_BF16 &&
         mapped(p->q_token_stride, p->q_head_stride, p->hk) &&
         mapped(p->k_token_stride, p->k_head_stride, p->hk) &&
         mapped(p->v_token_stride, p->v_head_stride, p->hv);
}

// A segment's tokens, in whole chunks.  An SM holds one segment of one output head at a time (in the
// tensor cores' backward pass of shared heads, of all the value heads that it sums), so what counts is how
// many rounds of the part's SMs there are (a constant: a workspace's size is asked for on the host, without
// a device) and how long one takes: its tokens and some more for its start and end, 640 on the tensor
// cores, 96 on the CUDA cores.  (bf16, 65536 tokens of 32 heads: 4 segments, one round of 128 SMs,
// 599 us; 9, two rounds of 144, 552; 16, 638; 19, four rounds of 152, 562; 32, 625.)  Only the sum of the
// sequences' lengths is known here: they are taken as alike, give or take a seventh.
constexpr int kSms = 152;
int linear_segment(const gdn_linear_problem* p, bool backward) {
  const int64_t T = p->total_tokens, N = p->num_seqs, hv = p->hv;
  const bool tc = linear_on_tc(p);
  const int64_t chunk = tc ? 128 : 64, more = tc ? 640 : 96;
  const int64_t heads = backward && tc ? p->hk : hv, share = hv / heads;
  const int64_t each = N == 1 ? T : (T + N - 1) / N * 8 / 7 + 1;
  int64_t best = 0, least = INT64_MAX;
  for (int64_t k = 1; k <= 128 && (k == 1 || each > (k - 1) * chunk); ++k) {
    const int64_t length = ((each + k - 1) / k + chunk - 1) / chunk * chunk;
    const int64_t rounds = (N * k * heads + kSms - 1) / kSms, cost = rounds * share * (length + more);
    if (cost < least) {
      least = cost;
      best = length;
    }
  }
  return (int)(best < chunk ? chunk : best < (int64_t)1 << 30 ? best : (int64_t)1 << 30);
}

gdn::LinearShape linear_shape(const gdn_linear_problem* p, bool backward, const float* log_decay,
                              const int32_t* cu, int32_t* dev_status) {
  gdn::LinearShape s;
  memset(&s, 0, sizeof(s));
  s.T = p->total_tokens;
  s.N = p->num_seqs; s.hk = p->hk; s.hv = p->hv; s.K = p->k_dim; s.V = p->v_dim;
  s.seg = linear_segment(p, backward);
  s.slots = s.T / s.seg + s.N;
  s.bf16 = p->io_dtype == GDN_BF16;
  s.log_decay = log_decay; s.cu = cu; s.status = dev_status;
  return s;
}

gdn::LinearRows linear_rows(const void* x, int64_t ts, int64_t hs, int64_t T, int heads, int hv) {
  return gdn::LinearRows{x, stride_of(ts, T), stride_of(hs, heads), hv / heads};
}

// The segments' states, and behind them their rows' exponents.
size_t linear_tops_at(const gdn::LinearShape& s) {
  return align_up((size_t)s.slots * s.hv * s.K * s.V * sizeof(float));
}
size_t linear_states_bytes(const gdn::LinearShape& s) {
  return linear_tops_at(s) + align_up((size_t)s.slots * s.hv * 2 * sizeof(int)) + kAlign;
}
// (and a word for whether the table and the decays can be used: a kernel of its own looks at those of many
// sequences, else the call's first kernels do)
cudaError_t linear_look(gdn::LinearShape& s, void* states, cudaStream_t stream) {
  s.refused = reinterpret_cast<int32_t*>(static_cast<char*>(states) + linear_states_bytes(s) - kAlign);
  if (s.N <= gdn::kLinearLooked) return cudaSuccess;
  const cudaError_t e = gdn::linear_check(s, stream);
  s.looked = true;
  return e;
}
int* linear_tops(const gdn::LinearShape& s, float* states) {
  return reinterpret_cast<int*>(reinterpret_cast<char*>(states) + linear_tops_at(s));
}

cudaError_t linear_state(const gdn_linear_problem* p, const gdn::LinearState& a, cudaStream_t s) {
  return linear_on_tc(p) ? gdn::linear_state_tc(a, s) : gdn::linear_state_simt(a, s);
}
cudaError_t linear_pass(const gdn_linear_problem* p, const gdn::LinearPass& a, cudaStream_t s) {
  return linear_on_tc(p) ? gdn::linear_pass_tc(a, s) : gdn::linear_pass_simt(a, s);
}

struct LinearBwdLayout {
  size_t h, d, partial, q, k, v, total;
};
LinearBwdLayout linear_bwd_layout(const gdn::LinearShape& s, bool tc, bool saved) {
  LinearBwdLayout L;
  const size_t e = s.bf16 ? 2 : 4, keys = (size_t)s.T * s.hk * s.K, values = (size_t)s.T * s.hv * s.V;
  L.h = 0;
  L.d = L.h + linear_states_bytes(s);
  L.partial = L.d + linear_states_bytes(s);
  L.q = L.partial + (s.hv == s.hk ? 0 : align_up(keys * (tc ? 1 : s.hv / s.hk) * sizeof(float)));
  L.k = L.q + (saved ? align_up(keys * e) : 0);
  L.v = L.k + (saved ? align_up(keys * e) : 0);
  L.total = L.v + (saved ? align_up(values * e) : 0);
  return L;
}

gdn_status checkpoint_args(const gdn_checkpoint* t, int count, int format,
                           gdn::CheckpointArgs& a) {
  if (!t || count < 1) return GDN_ERR_INVALID_ARGUMENT;
  if (count > gdn::kCheckpoints || (format != GDN_KV_INT8 && format != GDN_KV_E4M3))
    return GDN_ERR_UNSUPPORTED;
  memset(&a, 0, sizeof(a));
  a.count = count;
  a.e4m3 = format == GDN_KV_E4M3;
  int64_t blocks = 0;
  for (int i = 0; i < count; ++i) {
    const gdn_checkpoint& c = t[i];
    if (c.total_tokens < 0 || c.total_tokens > (int64_t)INT32_MAX || c.heads < 1 || c.head_dim < 1)
      return GDN_ERR_INVALID_ARGUMENT;
    if ((c.io_dtype != GDN_BF16 && c.io_dtype != GDN_F32) || !head_dim_ok(c.head_dim) ||
        c.total_tokens * c.heads > (int64_t)INT32_MAX)
      return GDN_ERR_UNSUPPORTED;
    if (!strides_ok(c.token_stride, c.total_tokens, c.head_stride, c.heads, c.io_dtype))
      return GDN_ERR_INVALID_ARGUMENT;
    if (c.total_tokens > 0 && (!c.x || !c.codes || !c.scale)) return GDN_ERR_INVALID_ARGUMENT;
    // (a scale is read by itself: those of a part of the tokens may start at any of them)
    if (!aligned16(c.x) || !aligned16(c.codes) || reinterpret_cast<uintptr_t>(c.scale) % sizeof(float))
      return GDN_ERR_INVALID_ARGUMENT;
    a.t[i] = {c.x, static_cast<uint8_t*>(c.codes), c.scale, c.total_tokens * c.heads,
              stride_of(c.token_stride, c.total_tokens), stride_of(c.head_stride, c.heads),
              c.heads, c.head_dim, c.io_dtype == GDN_BF16, false};
    a.t[i].packed = (c.heads == 1 || a.t[i].hs == c.head_dim) &&
                    (c.total_tokens == 1 || a.t[i].ts == (int64_t)c.heads * c.head_dim);
    blocks += a.t[i].rows / 32 + 1;  // (a block has 32 rows at least)
  }
  return blocks > (int64_t)INT32_MAX ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

}  // namespace

gdn_status gdn_check_linear_problem(const gdn_linear_problem* p) { return check_linear(p); }

size_t gdn_linear_attention_workspace_size(const gdn_linear_problem* p) {
  if (check_linear(p) != GDN_OK) return 0;
  return linear_states_bytes(linear_shape(p, false, nullptr, nullptr, nullptr));
}

gdn_status gdn_linear_attention(const gdn_linear_problem* p, const void* q, const void* k,
                                const void* v, const float* log_decay, const float* h0,
                                const int32_t* cu_seqlens, void* out, float* h_final,
                                void* workspace, size_t ws_bytes, int32_t* dev_status,
                                cudaStream_t stream) {
  const gdn_status st = check_linear(p);
  if (st != GDN_OK) return st;
  if (!log_decay || (!cu_seqlens && p->num_seqs != 1)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens > 0 && (!q || !k || !v || !out)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(h0) ||
      !aligned16(h_final))
    return GDN_ERR_INVALID_ARGUMENT;
  gdn::LinearShape s = linear_shape(p, false, log_decay, cu_seqlens, dev_status);
  if (!workspace || !aligned16(workspace) || ws_bytes < linear_states_bytes(s))
    return GDN_ERR_WORKSPACE;
  float* states = static_cast<float*>(workspace);
  GDN_TRY(linear_look(s, states, stream));
  const int64_t T = s.T;
  const gdn::LinearRows qr = linear_rows(q, p->q_token_stride, p->q_head_stride, T, s.hk, s.hv),
                        kr = linear_rows(k, p->k_token_stride, p->k_head_stride, T, s.hk, s.hv),
                        vr = linear_rows(v, p->v_token_stride, p->v_head_stride, T, s.hv, s.hv);
  int* tops = linear_tops(s, states);  // of k, and of v
  if (T > 0) GDN_TRY(linear_state(p, {s, kr, vr, false, states, tops}, stream));
  const gdn::LinearScan scan = {s, false, states, h0, h_final};
  s.looked = true;
  GDN_TRY(gdn::linear_scan(&scan, 1, stream));
  if (T > 0)
    GDN_TRY(linear_pass(p, {s, qr, kr, vr, s.K, s.V, false, false, states, out, 1, nullptr, tops,
                            tops + 1}, stream));
  return GDN_OK;
}

size_t gdn_linear_attention_backward_workspace_size(const gdn_linear_problem* p, int saved) {
  if (check_linear(p) != GDN_OK) return 0;
  const gdn_linear_problem o = saved ? linear_opened(p) : *p;
  return linear_bwd_layout(linear_shape(&o, true, nullptr, nullptr, nullptr), linear_on_tc(&o), saved != 0).total;
}

gdn_status gdn_linear_attention_backward(const gdn_linear_problem* p, const void* q,
                                         const void* k, const void* v,
                                         const gdn_linear_saved* saved, const float* log_decay,
                                         const float* h0, const int32_t* cu_seqlens,
                                         const void* dout, const float* dh_final, void* dq,
                                         void* dk, void* dv, float* dh0, void* workspace,
                                         size_t ws_bytes, int32_t* dev_status,
                                         cudaStream_t stream) {
  const gdn_status st = check_linear(p);
  if (st != GDN_OK) return st;
  if (!log_decay || (!cu_seqlens && p->num_seqs != 1)) return GDN_ERR_INVALID_ARGUMENT;
  if (saved && (q || k || v)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens > 0 && (!dout || !dq || !dk || !dv || (!saved && (!q || !k || !v))))
    return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned16(h0) || !aligned16(dh_final) ||
      !aligned16(dh0))
    return GDN_ERR_INVALID_ARGUMENT;
  const gdn_linear_problem opened = linear_opened(p);
  if (saved) p = &opened;
  gdn::LinearShape s = linear_shape(p, true, log_decay, cu_seqlens, dev_status);
  const LinearBwdLayout L = linear_bwd_layout(s, linear_on_tc(p), saved != nullptr);
  if (!workspace || !aligned16(workspace) || ws_bytes < L.total) return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  float* h = reinterpret_cast<float*>(ws + L.h);
  float* d = reinterpret_cast<float*>(ws + L.d);
  const int64_t T = s.T;
  const int share = s.hv / s.hk;
  if (saved) {
    q = ws + L.q;
    k = ws + L.k;
    v = ws + L.v;
    auto held = [&](const void* to, const void* codes, const float* scale, int heads, int d) {
      return gdn_checkpoint{const_cast<void*>(to), const_cast<void*>(codes),
                            const_cast<float*>(scale), T, (int64_t)heads * d, d, heads, d,
                            p->io_dtype};
    };
    const gdn_checkpoint t[3] = {held(q, saved->q_codes, saved->q_scale, s.hk, s.K),
                                 held(k, saved->k_codes, saved->k_scale, s.hk, s.K),
                                 held(v, saved->v_codes, saved->v_scale, s.hv, s.V)};
    gdn::CheckpointArgs ca;
    const gdn_status cs = checkpoint_args(t, 3, saved->format, ca);
    if (cs != GDN_OK) return cs;
    GDN_TRY(gdn::checkpoint_open(ca, stream));
  }
  GDN_TRY(linear_look(s, h, stream));
  const gdn::LinearRows qr = linear_rows(q, p->q_token_stride, p->q_head_stride, T, s.hk, s.hv),
                        kr = linear_rows(k, p->k_token_stride, p->k_head_stride, T, s.hk, s.hv),
                        vr = linear_rows(v, p->v_token_stride, p->v_head_stride, T, s.hv, s.hv);
  const gdn::LinearRows gr =
      linear_rows(dout, (int64_t)s.hv * s.V, s.V, T, s.hv, s.hv);
  if (T > 0) {
    GDN_TRY(linear_state(p, {s, kr, vr, false, h, linear_tops(s, h)}, stream));
    GDN_TRY(linear_state(p, {s, qr, gr, true, d, linear_tops(s, d)}, stream));
  }
  const gdn::LinearScan scans[2] = {{s, true, d, dh_final, dh0}, {s, false, h, h0, nullptr}};
  s.looked = true;
  GDN_TRY(gdn::linear_scan(scans, T > 0 ? 2 : 1, stream));
  if (T > 0) {
    float* partial = reinterpret_cast<float*>(ws + L.partial);
    const int *tk = linear_tops(s, h), *tv = tk + 1, *tq = linear_tops(s, d), *tg = tq + 1;
    GDN_TRY(linear_pass(p, {s, gr, vr, kr, s.V, s.K, false, true, h, dq, share, partial, tv, tk},
                        stream));
    GDN_TRY(linear_pass(p, {s, vr, gr, qr, s.V, s.K, true, true, d, dk, share, partial, tg, tq},
                        stream));
    GDN_TRY(linear_pass(p, {s, kr, qr, gr, s.K, s.V, true, false, d, dv, 1, nullptr, tq, tg},
                        stream));
  }
  return GDN_OK;
}

gdn_status gdn_linear_attention_decode(const gdn_linear_problem* p, int32_t slots, const void* q,
                                       const void* k, const void* v, const float* log_decay,
                                       const int32_t* slot, float* state, void* out,
                                       int32_t* dev_status, cudaStream_t stream) {
  const gdn_status st = check_linear(p);
  if (st != GDN_OK) return st;
  if (slots < 1) return GDN_ERR_INVALID_ARGUMENT;
  if (p->total_tokens == 0) return GDN_OK;
  if (!q || !k || !v || !log_decay || !slot || !state || !out) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state) || !aligned16(out))
    return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->total_tokens;
  const gdn::LinearDecode a = {
      (int)B, slots, p->hk, p->hv, p->k_dim, p->v_dim, p->io_dtype == GDN_BF16,
      linear_rows(q, p->q_token_stride, p->q_head_stride, B, p->hk, p->hv),
      linear_rows(k, p->k_token_stride, p->k_head_stride, B, p->hk, p->hv),
      linear_rows(v, p->v_token_stride, p->v_head_stride, B, p->hv, p->hv), log_decay, slot, state,
      out, dev_status};
  return to_status(gdn::linear_decode(a, stream));
}

gdn_status gdn_checkpoint_pack(const gdn_checkpoint* tensors, int32_t count, int32_t format,
                               int32_t* dev_status, cudaStream_t stream) {
  gdn::CheckpointArgs a;
  const gdn_status st = checkpoint_args(tensors, count, format, a);
  if (st != GDN_OK) return st;
  a.status = dev_status;
  return to_status(gdn::checkpoint_pack(a, stream));
}

gdn_status gdn_checkpoint_open(const gdn_checkpoint* tensors, int32_t count, int32_t format,
                               cudaStream_t stream) {
  gdn::CheckpointArgs a;
  const gdn_status st = checkpoint_args(tensors, count, format, a);
  return st != GDN_OK ? st : to_status(gdn::checkpoint_open(a, stream));
}

gdn_status gdn_device_status(const void* status_word, int reset, cudaStream_t stream) {
  if (!status_word) return GDN_ERR_INVALID_ARGUMENT;
  int32_t host = 0;
  int32_t* dev = const_cast<int32_t*>(static_cast<const int32_t*>(status_word));
  GDN_TRY(cudaMemcpyAsync(&host, dev, sizeof(int32_t), cudaMemcpyDeviceToHost, stream));
  if (reset) GDN_TRY(cudaMemsetAsync(dev, 0, sizeof(int32_t), stream));
  GDN_TRY(cudaStreamSynchronize(stream));
  return static_cast<gdn_status>(host);
}

}  // extern "C"
