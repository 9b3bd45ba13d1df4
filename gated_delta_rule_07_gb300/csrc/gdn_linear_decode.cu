// gdn_linear_decode.cu -- one token of linear attention with a decay for each head over a pool of
// per-slot states: per row b and value head, with h = state[slot[b]] and a = exp(log_decay),
//     h <- a h + k v^T,     o = h^T q.
//
// The step reads and writes each K x V fp32 state once (128 KiB a row and head at K = V = 128) and does
// four operations an element: it is bound by HBM.  (256 requests of 32 heads of 128, 1.08 GB:
// 159.5 us, the measured copy's rate; five fp32 requests of 6 heads: 2.7 us.)  One block of 256 threads
// a (row, value head): a
// thread holds K V / 1024 rows of four columns, so that a warp's accesses are whole 512- or 256-byte
// runs; the new state is stored before the sums of o are joined, which only need it in registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_common.cuh"
#include "gdn_elements.cuh"
#include "gdn_linear.h"
#include "gdn_stream_order.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename IO>
__device__ __forceinline__ const IO* row_of(const LinearRows& r, int row, int head) {
  return static_cast<const IO*>(r.p) + (int64_t)row * r.ts + (int64_t)(head / r.share) * r.hs;
}

template <int K, int V, typename IO>
__global__ void __launch_bounds__(kThreads) linear_decode_kernel(LinearDecode a) {
  constexpr int CG = V / 4;             // column groups of 4
  constexpr int RG = kThreads / CG;     // row groups
  constexpr int RPT = K / RG;           // state rows a thread, 4 to 16
  __shared__ __align__(16) float part[RG][V];
  stream_order();
  const int b = blockIdx.x, j = blockIdx.y;
  const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
  const int s = a.slot[b];
  IO* out = static_cast<IO*>(a.out) + ((int64_t)b * a.hv + j) * V;
  if (s < 0) {  // padding row
    for (int c = tid; c < V; c += kThreads) out[c] = from_f32<IO>(0.f);
    return;
  }
  const float g = a.log_decay[j];
  if (s >= a.slots || !(g <= 0.f)) {
    if (tid == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
    return;
  }
  float* st = a.state + ((int64_t)s * a.hv + j) * K * V + (int64_t)rg * RPT * V + 4 * cg;
  float4 h[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) h[i] = *reinterpret_cast<const float4*>(st + i * V);
  const IO* qp = row_of<IO>(a.q, b, j) + rg * RPT;
  const IO* kp = row_of<IO>(a.k, b, j) + rg * RPT;
  float qv[RPT], kv[RPT], v[4];
#pragma unroll
  for (int i = 0; i < RPT; i += 4) {
    Quad<IO> x, y;
    x.load(qp + i);
    y.load(kp + i);
    x.open(&qv[i]);
    y.open(&kv[i]);
  }
  Quad<IO> x;
  x.load(row_of<IO>(a.v, b, j) + 4 * cg);
  x.open(v);
  // another row naming the same slot: the two updates would race, so neither is made
  bool dup = false;
  for (int e = tid; e < a.batch; e += kThreads) dup |= (e != b && a.slot[e] == s);
  if (__syncthreads_or(dup)) {
    if (tid == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
    return;
  }
  const float alpha = expf(g);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    h[i].x = fmaf(kv[i], v[0], alpha * h[i].x);
    h[i].y = fmaf(kv[i], v[1], alpha * h[i].y);
    h[i].z = fmaf(kv[i], v[2], alpha * h[i].z);
    h[i].w = fmaf(kv[i], v[3], alpha * h[i].w);
    *reinterpret_cast<float4*>(st + i * V) = h[i];
    o.x = fmaf(h[i].x, qv[i], o.x);
    o.y = fmaf(h[i].y, qv[i], o.y);
    o.z = fmaf(h[i].z, qv[i], o.z);
    o.w = fmaf(h[i].w, qv[i], o.w);
  }
  *reinterpret_cast<float4*>(&part[rg][4 * cg]) = o;
  __syncthreads();
  for (int c = tid; c < V; c += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < RG; ++r) sum += part[r][c];
    out[c] = from_f32<IO>(sum);
  }
}

template <int K, int V> cudaError_t launch(const LinearDecode& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.batch, (unsigned)a.hv);
  return a.bf16 ? launch_ordered(linear_decode_kernel<K, V, __nv_bfloat16>, grid, kThreads, 0, s, a)
                : launch_ordered(linear_decode_kernel<K, V, float>, grid, kThreads, 0, s, a);
}

}  // namespace

cudaError_t linear_decode(const LinearDecode& a, cudaStream_t s) {
  if (a.K == 128) return a.V == 128 ? launch<128, 128>(a, s) : launch<128, 64>(a, s);
  return a.V == 128 ? launch<64, 128>(a, s) : launch<64, 64>(a, s);
}

}  // namespace gdn
