// gdn_kv_attention.cu -- softmax attention of a few query tokens per sequence over the paged
// 8-bit cache.
//
// For query row i of sequence n (rows [cu[n], cu[n + 1]), the last one at the cache's last
// position kv_len[n] - 1) and query head h, over the keys j at or before the row's position (and
// within the window):
//     x_j = scale q . k_j,   o = sum_j softmax(x)_j v_j,   lse = log sum_j exp(x_j),
// kv head h / (hq / hkv).  A row that no key is left for gets o = 0 and lse = -inf.
#include <math_constants.h>

#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kAttThreads = 128;

template <typename IO, int D, bool E4M3>
__global__ void __launch_bounds__(kAttThreads) kv_attention_simple(KvArgs a) {
  constexpr int kWarps = kAttThreads / 32, C = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, kh = h / (a.hq / a.hkv);
  int n = 0;
  int64_t b = 0, e = a.T;
  if (a.cu) {
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    n = lo;
    if (!seq_bounds(a.cu, n, a.T, a.status, b, e) || t < b || t >= e) return;
  } else if (a.N > 1) {
    n = (int)t;
    b = t;
    e = t + 1;
  }
  const int len = a.pos0[n];
  if (len < 0 || len > (int64_t)a.max_pages * a.page) {
    if (threadIdx.x == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
    return;
  }
  const int64_t at = len - (e - b) + (t - b);
  const int64_t j0 = a.window > 0 && at - a.window + 1 > 0 ? at - a.window + 1 : 0;
  const IO* qp = static_cast<const IO*>(a.q) + t * a.q_ts + h * a.q_hs;
  float q[C], o[C], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    q[i] = to_f32(qp[32 * i + lane]);
    o[i] = 0.f;
  }
  for (int64_t j = j0 + warp; j <= at; j += kWarps) {
    const int pid = kv_page_id(a, n, (int)(j / a.page));
    if (pid < 0) continue;
    const int64_t block = (int64_t)pid * a.hkv + kh;
    const int s = (int)(j % a.page);
    const uint8_t* kp = a.k_codes + (block * a.page + s) * D;
    const uint8_t* vp = a.v_codes + (block * a.page + (s & ~3)) * D + (s & 3);
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) x = fmaf(q[i], kv_value<E4M3>(kp[32 * i + lane]), x);
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x *= a.scale * a.k_scale[block];
    const float mn = fmaxf(m, x), f = __expf(m - mn), p = __expf(x - mn), vs = a.v_scale[block];
    l = l * f + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < C; ++i)
      o[i] = fmaf(p * vs, kv_value<E4M3>(vp[4 * (32 * i + lane)]), o[i] * f);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < C; ++i) so[warp][32 * i + lane] = o[i];
  __syncthreads();
  float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  float f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = M > -CUDART_INF_F ? __expf(sm[w] - M) : 0.f;
    L += sl[w] * f[w];
  }
  IO* out = static_cast<IO*>(a.out) + (t * a.hq + h) * D;
  for (int d = threadIdx.x; d < D; d += kAttThreads) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x = fmaf(so[w][d], f[w], x);
    out[d] = from_f32<IO>(L > 0.f ? x / L : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[t * a.hq + h] = M + logf(L);
}

template <typename IO, int D>
cudaError_t launch_att(const KvArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.T, (unsigned)a.hq);
  if (a.e4m3) kv_attention_simple<IO, D, true><<<grid, kAttThreads, 0, s>>>(a);
  else kv_attention_simple<IO, D, false><<<grid, kAttThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename IO>
cudaError_t launch_att_io(const KvArgs& a, cudaStream_t s) {
  switch (a.D) {
    case 64: return launch_att<IO, 64>(a, s);
    case 128: return launch_att<IO, 128>(a, s);
    default: return launch_att<IO, 256>(a, s);
  }
}

}  // namespace

size_t kv_attention_workspace(const KvArgs&) { return 0; }

cudaError_t kv_attention(const KvArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_att_io<__nv_bfloat16>(a, s) : launch_att_io<float>(a, s);
}

}  // namespace gdn
