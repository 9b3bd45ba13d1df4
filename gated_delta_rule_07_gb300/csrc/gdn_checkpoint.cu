// gdn_checkpoint.cu -- activations held in 8 bits between the forward and the backward pass.
//
// Per row (one head of one token): s = amax / qmax, code = round(x / s), value = code s, with the
// cache's codes, arithmetic and treatment of values that are not finite (gdn_kv.cuh).  A row's scale is
// its own, so nothing waits for another row: the kernels stream, bound by HBM.  A lane holds eight
// elements of a row (a 16-byte load in bf16, two in fp32, an 8-byte piece of codes), a warp four groups
// of rows at once, all of them asked for before the first is used.  (q, k, v of 32768 tokens, 268 million
// elements, bf16 and int8: packed in 157 us, with 79% of the issue slots used, where HBM takes 120;
// opened in 116.  Two groups a warp: packed in 171, eight: 182.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_elements.cuh"
#include "gdn_kv.cuh"
#include "gdn_linear.h"
#include "gdn_stream_order.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 4;   // of rows in flight a warp

constexpr int rows_of_block(int D) { return kThreads / (D / 8) * kGroups; }

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Offset in x of row `row` (its heads are neighbours in the packed tensors, strided in x).
__device__ __forceinline__ int64_t offset_of(const CheckpointArgs::Rows& t, int64_t row) {
  if (t.packed) return row * t.D;
  const uint32_t r = (uint32_t)row, token = r / (uint32_t)t.heads;
  return (int64_t)token * t.ts + (int64_t)(r - token * (uint32_t)t.heads) * t.hs;
}

// The largest magnitude of a lane's eight elements; not finite where one of them is not.
__device__ __forceinline__ float largest(const Quad<float> (&q)[2]) {
  float f[8], m = 0.f;
  q[0].open(f);
  q[1].open(f + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = f[i] == f[i] ? fmaxf(m, fabsf(f[i])) : INFINITY;
  return m;
}
__device__ __forceinline__ float largest(const Quad<__nv_bfloat16> (&q)[2]) {
  const uint32_t w[4] = {q[0].v.x, q[0].v.y, q[1].v.x, q[1].v.y};
  __nv_bfloat162 m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
  const __nv_bfloat162 r = __hmax2_nan(__hmax2_nan(m[0], m[1]), __hmax2_nan(m[2], m[3]));
  const float2 f = __bfloat1622float2(r);
  return f.x == f.x && f.y == f.y ? fmaxf(f.x, f.y) : INFINITY;
}
// The codes of eight finite elements of a row, whose largest gives qmax: none is beyond it by more than
// the rounding of fp32, and none is rounded beyond it.  int8: a value of magnitude up to 127, added to
// 3 2^22, has its nearest integer (ties to even) in the sum's low bits, which are its code.
template <bool E4M3> __device__ __forceinline__ uint2 codes_of(const float* f, float inv) {
  // (the product is rounded by itself, as the definition has it: no packed or fused form)
  float2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = make_float2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (E4M3) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[2 * i].y), "f"(y[2 * i].x));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[2 * i + 1].y), "f"(y[2 * i + 1].x));
      r[i] = (uint32_t)lo | (uint32_t)hi << 16;
    } else {
      const float big = 12582912.f;
      const float2 a = make_float2(__fadd_rn(y[2 * i].x, big), __fadd_rn(y[2 * i].y, big));
      const float2 b = make_float2(__fadd_rn(y[2 * i + 1].x, big), __fadd_rn(y[2 * i + 1].y, big));
      const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
      const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
      r[i] = __byte_perm(lo, hi, 0x5410);
    }
  }
  return make_uint2(r[0], r[1]);
}

template <int D, typename IO, bool E4M3>
__device__ __forceinline__ void pack_rows(const CheckpointArgs::Rows& t, int64_t block,
                                          int32_t* status) {
  constexpr int LANES = D / 8, RPG = kThreads / LANES;  // lanes a row, rows a group of the block
  const int sub = threadIdx.x % LANES;
  const int64_t row0 = block * rows_of_block(D) + threadIdx.x / LANES;
  const IO* x = static_cast<const IO*>(t.x);
  Quad<IO> q[kGroups][2];
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t row = row0 + k * RPG;
    if (row < t.rows) {
      const IO* p = x + offset_of(t, row) + 8 * sub;
      q[k][0].load(p);
      q[k][1].load(p + 4);
    } else {
      q[k][0].clear();
      q[k][1].clear();
    }
  }
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t row = row0 + k * RPG;
    float f[8], amax = largest(q[k]);
    q[k][0].open(f);
    q[k][1].open(f + 4);
    const bool bad = !is_finite(amax);
    if (bad) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, is_finite(f[i]) ? fabsf(f[i]) : 0.f);
    }
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const float scale = amax >= kKvTiny ? amax * (float)(1.0 / kv_qmax<E4M3>()) : 0.f;
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    uint2 codes;
    if (!bad) {
      codes = codes_of<E4M3>(f, inv);
    } else {
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        c[i] = kv_code<E4M3>(is_finite(f[i]) ? f[i] * inv
                             : f[i] == f[i]  ? copysignf(kv_qmax<E4M3>(), f[i]) : 0.f);
      codes = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                         c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    }
    if (row < t.rows) {
      if (bad) set_status(status, GDN_ERR_DEVICE_RANGE);
      *reinterpret_cast<uint2*>(t.codes + row * D + 8 * sub) = codes;
      if (sub == 0) t.scale[row] = scale;
    }
    __syncwarp();
  }
}

template <int D, typename IO, bool E4M3>
__device__ __forceinline__ void open_rows(const CheckpointArgs::Rows& t, int64_t block) {
  constexpr int LANES = D / 8, RPG = kThreads / LANES;
  const int sub = threadIdx.x % LANES;
  const int64_t row0 = block * rows_of_block(D) + threadIdx.x / LANES;
  IO* x = static_cast<IO*>(t.x);
  uint2 c[kGroups];
  float scale[kGroups];
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t row = row0 + k * RPG;
    c[k] = make_uint2(0u, 0u);
    scale[k] = 0.f;
    if (row < t.rows) {
      c[k] = __ldg(reinterpret_cast<const uint2*>(t.codes + row * D + 8 * sub));
      scale[k] = __ldg(t.scale + row);
    }
  }
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t row = row0 + k * RPG;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = kv_value<E4M3>(c[k].x >> (8 * i) & 0xffu) * scale[k];
      f[4 + i] = kv_value<E4M3>(c[k].y >> (8 * i) & 0xffu) * scale[k];
    }
    if (row < t.rows) {
      IO* p = x + offset_of(t, row) + 8 * sub;
      put4(p, f);
      put4(p + 4, f + 4);
    }
  }
}

template <bool PACK, bool E4M3, typename IO>
__device__ __forceinline__ void rows_of(const CheckpointArgs::Rows& t, int64_t block, int32_t* status) {
  if (t.D == 64) {
    if (PACK) pack_rows<64, IO, E4M3>(t, block, status); else open_rows<64, IO, E4M3>(t, block);
  } else if (t.D == 128) {
    if (PACK) pack_rows<128, IO, E4M3>(t, block, status); else open_rows<128, IO, E4M3>(t, block);
  } else {
    if (PACK) pack_rows<256, IO, E4M3>(t, block, status); else open_rows<256, IO, E4M3>(t, block);
  }
}

template <bool PACK, bool E4M3>
__global__ void __launch_bounds__(kThreads) checkpoint_kernel(const __grid_constant__ CheckpointArgs a) {
  stream_order();
  int i = 0;
  while (i + 1 < a.count && (int64_t)blockIdx.x >= a.first[i + 1]) ++i;
  const CheckpointArgs::Rows& t = a.t[i];
  const int64_t block = (int64_t)blockIdx.x - a.first[i];
  if (t.bf16)
    rows_of<PACK, E4M3, __nv_bfloat16>(t, block, a.status);
  else
    rows_of<PACK, E4M3, float>(t, block, a.status);
}

template <bool PACK> cudaError_t launch(CheckpointArgs& a, cudaStream_t s) {
  a.first[0] = 0;
  for (int i = 0; i < a.count; ++i) {
    const int64_t per = rows_of_block(a.t[i].D);
    a.first[i + 1] = a.first[i] + (a.t[i].rows + per - 1) / per;
  }
  if (a.first[a.count] == 0) return cudaSuccess;
  const dim3 grid((unsigned)a.first[a.count]);
  return a.e4m3 ? launch_ordered(checkpoint_kernel<PACK, true>, grid, kThreads, 0, s, a)
                : launch_ordered(checkpoint_kernel<PACK, false>, grid, kThreads, 0, s, a);
}

}  // namespace

cudaError_t checkpoint_pack(CheckpointArgs& a, cudaStream_t s) { return launch<true>(a, s); }
cudaError_t checkpoint_open(CheckpointArgs& a, cudaStream_t s) { return launch<false>(a, s); }

}  // namespace gdn
