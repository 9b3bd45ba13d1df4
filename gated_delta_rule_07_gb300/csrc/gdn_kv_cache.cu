// gdn_kv_cache.cu -- new keys and values quantised into the paged 8-bit cache, and ranges of it
// read back.
//
// A page's scale covers all its tokens of one head.  For the tokens that a call adds to a page,
//     s = max(amax / qmax, the page's scale if it already holds tokens of its sequence),
//     code = round(x / s)  (x times the fp32 reciprocal of s),
// and where s grew the page's earlier codes become round(code s_old / s).  A page that the call
// starts takes its scale from its new tokens alone, whatever its last owner left.
//
// One CTA per (touched page, head, keys or values): it needs the page's whole amax before it can
// write the first code, and pages are independent.  Bound by HBM for prompts (each new element
// is read once and written as one byte), by latency for single tokens.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kKvThreads = 256;

template <typename IO>
__device__ __forceinline__ float kv_ld(const IO* p) { return to_f32(*p); }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// the byte of token t, channel d in a (page, head) block
template <int D, bool VALUES> __device__ __forceinline__ int64_t code_at(int t, int d) {
  return VALUES ? (int64_t)(t & ~3) * D + 4 * d + (t & 3) : (int64_t)t * D + d;
}

template <typename IO, int D, bool E4M3, bool VALUES>
__device__ void append_block(const KvArgs& a, const KvSpan& s, int pid) {
  __shared__ float red[kKvThreads / 32];
  const int h = blockIdx.y, tid = threadIdx.x;
  const int64_t block = (int64_t)pid * a.hkv + h;
  uint8_t* codes = (VALUES ? a.v_codes : a.k_codes) + block * a.page * D;
  float* scale = (VALUES ? a.v_scale : a.k_scale) + block;
  const int64_t ts = VALUES ? a.v_ts : a.k_ts;
  const IO* x = static_cast<const IO*>(VALUES ? a.v : a.k) + s.row * ts +
                h * (VALUES ? a.v_hs : a.k_hs);
  const int n = (s.hi - s.lo) * D;
  float amax = 0.f;
  bool bad = false;
  for (int e = tid; e < n; e += kKvThreads) {
    const float v = kv_ld(x + (e / D) * ts + e % D);
    if (finite(v)) amax = fmaxf(amax, fabsf(v));
    else bad = true;
  }
  if (bad) set_status(a.status, GDN_ERR_DEVICE_RANGE);
#pragma unroll
  for (int off = 16; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (tid % 32 == 0) red[tid / 32] = amax;
  const float held = s.lo > 0 ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKvThreads / 32; ++i) amax = fmaxf(amax, red[i]);
  const float now = fmaxf(held, amax >= kKvTiny ? amax * (float)(1.0 / kv_qmax<E4M3>()) : 0.f);
  const float inv = now > 0.f ? 1.f / now : 0.f;
  if (now > held && held > 0.f) {  // the page's earlier codes on the new scale
    const float ratio = held * inv;
    for (int e = tid; e < s.lo * D; e += kKvThreads) {
      uint8_t* c = codes + code_at<D, VALUES>(e / D, e % D);
      *c = (uint8_t)kv_code<E4M3>(kv_value<E4M3>(*c) * ratio);
    }
  }
  for (int e = tid; e < n; e += kKvThreads) {
    const float v = kv_ld(x + (e / D) * ts + e % D);
    const float y = finite(v) ? v * inv : (now > 0.f ? v : 0.f);
    codes[code_at<D, VALUES>(s.lo + e / D, e % D)] = (uint8_t)kv_code<E4M3>(y);
  }
  if (tid == 0) *scale = now;
}

template <typename IO, int D, bool E4M3>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(KvArgs a) {
  KvSpan s;
  if (!kv_span(a, blockIdx.x, s)) return;
  const int pid = kv_page_id(a, s.n, s.page_i);
  if (pid < 0) return;
  if (blockIdx.z) append_block<IO, D, E4M3, true>(a, s, pid);
  else append_block<IO, D, E4M3, false>(a, s, pid);
}

template <typename IO, int D, bool E4M3>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvArgs a) {
  KvSpan s;
  if (!kv_span(a, blockIdx.x, s)) return;
  const int pid = kv_page_id(a, s.n, s.page_i);
  if (pid < 0) return;
  const int h = blockIdx.y;
  const int64_t block = (int64_t)pid * a.hkv + h;
  const bool values = blockIdx.z;
  const uint8_t* codes = (values ? a.v_codes : a.k_codes) + block * a.page * D;
  const float scale = (values ? a.v_scale : a.k_scale)[block];
  IO* out = static_cast<IO*>(values ? a.v_out : a.k_out) + (s.row * a.hkv + h) * D;
  for (int e = threadIdx.x; e < (s.hi - s.lo) * D; e += kKvThreads) {
    const int t = s.lo + e / D, d = e % D;
    const uint32_t c = codes[values ? code_at<D, true>(t, d) : code_at<D, false>(t, d)];
    out[(int64_t)(e / D) * a.hkv * D + d] = from_f32<IO>(kv_value<E4M3>(c) * scale);
  }
}

template <typename IO, int D>
cudaError_t launch_kv(const KvArgs& a, bool append, cudaStream_t s) {
  const int64_t slots = a.cu == nullptr && a.N > 1 ? a.N : a.T / a.page + 2 * (int64_t)a.N;
  const dim3 grid((unsigned)slots, (unsigned)a.hkv, 2);
  if (append) {
    if (a.e4m3) kv_append_kernel<IO, D, true><<<grid, kKvThreads, 0, s>>>(a);
    else kv_append_kernel<IO, D, false><<<grid, kKvThreads, 0, s>>>(a);
  } else {
    if (a.e4m3) kv_read_kernel<IO, D, true><<<grid, kKvThreads, 0, s>>>(a);
    else kv_read_kernel<IO, D, false><<<grid, kKvThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_kv_io(const KvArgs& a, bool append, cudaStream_t s) {
  switch (a.D) {
    case 64: return launch_kv<IO, 64>(a, append, s);
    case 128: return launch_kv<IO, 128>(a, append, s);
    default: return launch_kv<IO, 256>(a, append, s);
  }
}

}  // namespace

cudaError_t kv_append(const KvArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_kv_io<__nv_bfloat16>(a, true, s) : launch_kv_io<float>(a, true, s);
}
cudaError_t kv_read(const KvArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_kv_io<__nv_bfloat16>(a, false, s) : launch_kv_io<float>(a, false, s);
}

}  // namespace gdn
