// gdn_qk_rope.cu -- queries and keys of a softmax-attention layer: RMS norm per head, the norm's
// weight, and the rotation by position, in one pass; and the gradients of that pass.
//
// A row is one head of one token, x of D numbers.  With r = 1 / sqrt(mean(x^2) + eps):
//     y_d = x_d r (w_d + offset),
// and on the first R of the D dimensions the pairs (a, b) = (y_i, y_{i + R/2}) (style "half") or
// (y_{2i}, y_{2i + 1}) (style "pairs") are turned by the angle of the token's position,
//     (a, b) -> (a c_i - b s_i, b c_i + a s_i),   c, s = the position's row of the table.
// Backward, with dy the turned-back gradient (the turn is orthogonal) and n = x r:
//     dw_d = sum over rows of dy_d n_d,   dn = dy (w + offset),   dx = r (dn - n mean(dn n)).
//
// Bound by HBM: every element is read once and written once (the gradient reads two and writes
// one).  A row is held by D / 8 lanes, eight consecutive elements each (16 bytes of bf16), so a
// row's mean is a shuffle over those lanes and its rotation partner's elements are one lane's
// registers away; nothing goes through shared memory.  Statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attention.h"
#include "gdn_common.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kVec = 8;  // elements a lane holds of a row

// eight elements as loaded
template <typename IO> struct Pack8;
template <> struct Pack8<__nv_bfloat16> { uint4 u; };
template <> struct Pack8<float> { float4 a, b; };

__device__ __forceinline__ void load8(Pack8<__nv_bfloat16>& p, const __nv_bfloat16* s) {
  p.u = __ldg(reinterpret_cast<const uint4*>(s));
}
__device__ __forceinline__ void load8(Pack8<float>& p, const float* s) {
  p.a = __ldg(reinterpret_cast<const float4*>(s));
  p.b = __ldg(reinterpret_cast<const float4*>(s) + 1);
}
__device__ __forceinline__ void open8(const Pack8<__nv_bfloat16>& p, float* f) {
  const uint32_t u[4] = {p.u.x, p.u.y, p.u.z, p.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the top half of an fp32
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void open8(const Pack8<float>& p, float* f) {
  f[0] = p.a.x; f[1] = p.a.y; f[2] = p.a.z; f[3] = p.a.w;
  f[4] = p.b.x; f[5] = p.b.y; f[6] = p.b.z; f[7] = p.b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* d, const float* f) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(d) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* d, const float* f) {
  reinterpret_cast<float4*>(d)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(d)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ Pack8<__nv_bfloat16> shfl8(const Pack8<__nv_bfloat16>& p, int src) {
  Pack8<__nv_bfloat16> r;
  r.u.x = __shfl_sync(0xffffffffu, p.u.x, src);
  r.u.y = __shfl_sync(0xffffffffu, p.u.y, src);
  r.u.z = __shfl_sync(0xffffffffu, p.u.z, src);
  r.u.w = __shfl_sync(0xffffffffu, p.u.w, src);
  return r;
}
__device__ __forceinline__ Pack8<float> shfl8(const Pack8<float>& p, int src) {
  Pack8<float> r;
  r.a.x = __shfl_sync(0xffffffffu, p.a.x, src);
  r.a.y = __shfl_sync(0xffffffffu, p.a.y, src);
  r.a.z = __shfl_sync(0xffffffffu, p.a.z, src);
  r.a.w = __shfl_sync(0xffffffffu, p.a.w, src);
  r.b.x = __shfl_sync(0xffffffffu, p.b.x, src);
  r.b.y = __shfl_sync(0xffffffffu, p.b.y, src);
  r.b.z = __shfl_sync(0xffffffffu, p.b.z, src);
  r.b.w = __shfl_sync(0xffffffffu, p.b.w, src);
  return r;
}

// eight floats of a 16-byte aligned row, or all `otherwise` where there is none
__device__ __forceinline__ void floats8(const float* s, float otherwise, float* f) {
  if (s) {
    Pack8<float> p;
    load8(p, s);
    open8(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = otherwise;
  }
}

// A lane's part in the rotation: its cosines and signed sines, and the lane that holds the other
// element of each of its pairs.  out_i = y_i cs_i + other_i sn_i, where `other` is the partner
// lane's element i ("half") or this lane's element i ^ 1 ("pairs"); lanes past R turn nothing.
struct Turn {
  float cs[kVec], sn[kVec];
  int partner;
};
template <int LPR>
__device__ __forceinline__ Turn make_turn(const float* row, int R, bool pairs, int lane,
                                          float sign) {
  Turn t;
  const int l = lane % LPR, d0 = kVec * l;
  t.partner = lane;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    t.cs[i] = 1.f;
    t.sn[i] = 0.f;
  }
  if (d0 >= R) return t;
  if (pairs) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + d0 / 2));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + R / 2 + d0 / 2));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.cs[2 * i] = t.cs[2 * i + 1] = cc[i];
      t.sn[2 * i] = -sign * ss[i];
      t.sn[2 * i + 1] = sign * ss[i];
    }
  } else {
    const bool low = d0 < R / 2;
    t.partner = low ? lane + R / (2 * kVec) : lane - R / (2 * kVec);
    const int at = low ? d0 : d0 - R / 2;
    floats8(row + at, 1.f, t.cs);
    floats8(row + R / 2 + at, 0.f, t.sn);
#pragma unroll
    for (int i = 0; i < kVec; ++i) t.sn[i] *= low ? -sign : sign;
  }
  return t;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// A warp takes `U` steps of 32 / LPR heads of one token.  Units: token x head group, token major.
template <typename IO, int D, int U>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(QkRopeArgs a) {
  constexpr int LPR = D / kVec, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int H = a.hq + a.hkv, groups = (H + RPW * U - 1) / (RPW * U);
  const int64_t units = a.T * groups;
  const int64_t step = (int64_t)gridDim.x * (kRopeThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32; u < units;
       u += step) {
    const int64_t t = u / groups;
    const int h0 = (int)(u - t * groups) * RPW * U + sub;
    Pack8<IO> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * RPW;
      const IO* p = h < a.hq ? static_cast<const IO*>(a.q) + t * a.q_ts + h * a.q_hs
                             : static_cast<const IO*>(a.k) + t * a.k_ts + (h - a.hq) * a.k_hs;
      if (h < H) load8(x[i], p + kVec * l);
      else x[i] = Pack8<IO>{};
    }
    const int pos = a.pos[t];
    if (pos < 0 || pos >= a.max_pos) {  // (the same for the whole warp)
      if (lane == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
      continue;
    }
    const Turn turn = make_turn<LPR>(a.table + (int64_t)pos * a.R, a.R, a.pairs, lane, 1.f);
    const int pl = turn.partner % LPR;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * RPW;
      float f[kVec], w[kVec], o[kVec], s2 = 0.f;
      open8(x[i], f);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s2 = fmaf(f[j], f[j], s2);
      const float r = rsqrtf(row_sum<LPR>(s2) * (1.f / D) + a.eps);
      const float* wt = h < a.hq ? a.wq : a.wk;
      floats8(wt ? wt + kVec * l : nullptr, 1.f - a.offset, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) f[j] *= r * (w[j] + a.offset);
      if (a.pairs) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = fmaf(f[j], turn.cs[j], f[j ^ 1] * turn.sn[j]);
      } else {
        float g[kVec];
        open8(shfl8(x[i], turn.partner), g);
        floats8(wt ? wt + kVec * pl : nullptr, 1.f - a.offset, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          o[j] = fmaf(f[j], turn.cs[j], g[j] * (r * (w[j] + a.offset)) * turn.sn[j]);
      }
      if (h < H) {
        IO* dst = h < a.hq ? static_cast<IO*>(a.q_out) + (t * a.hq + h) * D
                           : static_cast<IO*>(a.k_out) + (t * a.hkv + h - a.hq) * D;
        store8(dst + kVec * l, o);
      }
    }
  }
}

// Gradients.  Each warp walks its units in a fixed order and keeps its share of both weights'
// gradients in registers; a CTA's warps join theirs in shared memory and write one partial sum
// per CTA, which qk_rope_dw_kernel adds up in CTA order: the same bits on every run.
template <typename IO, int D, int U>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_backward_kernel(QkRopeArgs a) {
  constexpr int LPR = D / kVec, RPW = 32 / LPR, kWarps = kRopeThreads / 32;
  __shared__ float part[kWarps][2][D];
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR, warp = threadIdx.x / 32;
  const int H = a.hq + a.hkv, groups = (H + RPW * U - 1) / (RPW * U);
  const int64_t units = a.T * groups;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  float dw[2][kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) dw[0][j] = dw[1][j] = 0.f;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < units; u += step) {
    const int64_t t = u / groups;
    const int h0 = (int)(u - t * groups) * RPW * U + sub;
    Pack8<IO> x[U], g[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * RPW;
      const bool isq = h < a.hq;
      const IO* p = isq ? static_cast<const IO*>(a.q) + t * a.q_ts + h * a.q_hs
                        : static_cast<const IO*>(a.k) + t * a.k_ts + (h - a.hq) * a.k_hs;
      const IO* d = isq ? static_cast<const IO*>(a.dq_out) + (t * a.hq + h) * D
                        : static_cast<const IO*>(a.dk_out) + (t * a.hkv + h - a.hq) * D;
      if (h < H) {
        load8(x[i], p + kVec * l);
        load8(g[i], d + kVec * l);
      } else {
        x[i] = Pack8<IO>{};
        g[i] = Pack8<IO>{};
      }
    }
    const int pos = a.pos[t];
    if (pos < 0 || pos >= a.max_pos) {
      if (lane == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
      continue;
    }
    const Turn turn = make_turn<LPR>(a.table + (int64_t)pos * a.R, a.R, a.pairs, lane, -1.f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * RPW;
      const bool isq = h < a.hq;
      float f[kVec], d[kVec], dy[kVec], w[kVec], s2 = 0.f, dot = 0.f;
      open8(x[i], f);
      open8(g[i], d);
      if (a.pairs) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) dy[j] = fmaf(d[j], turn.cs[j], d[j ^ 1] * turn.sn[j]);
      } else {
        float e[kVec];
        open8(shfl8(g[i], turn.partner), e);
#pragma unroll
        for (int j = 0; j < kVec; ++j) dy[j] = fmaf(d[j], turn.cs[j], e[j] * turn.sn[j]);
      }
      const float* wt = isq ? a.wq : a.wk;
      floats8(wt ? wt + kVec * l : nullptr, 1.f - a.offset, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        s2 = fmaf(f[j], f[j], s2);
        w[j] = dy[j] * (w[j] + a.offset);  // dn
        dot = fmaf(w[j], f[j], dot);
      }
      const float r = rsqrtf(row_sum<LPR>(s2) * (1.f / D) + a.eps);
      const float m = row_sum<LPR>(dot) * (1.f / D) * r;  // mean(dn n)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float n = f[j] * r;
        const float c = dy[j] * n;
        dw[0][j] += isq ? c : 0.f;
        dw[1][j] += isq ? 0.f : c;
        f[j] = r * (w[j] - n * m);
      }
      if (h < H) {
        IO* dst = isq ? static_cast<IO*>(a.dq) + (t * a.hq + h) * D
                      : static_cast<IO*>(a.dk) + (t * a.hkv + h - a.hq) * D;
        store8(dst + kVec * l, f);
      }
    }
  }
  // a warp's rows (lanes with the same l), then the CTA's warps
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float s = dw[which][j];
#pragma unroll
      for (int off = LPR; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (sub == 0) part[warp][which][kVec * l + j] = s;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kRopeThreads) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += part[i][c / D][c % D];
    a.partial[(int64_t)blockIdx.x * 2 * D + c] = s;
  }
}

// dw[c] = sum over CTAs of partial[cta][c]: a warp per 32 columns takes every eighth CTA
__global__ void __launch_bounds__(256) qk_rope_dw_kernel(QkRopeArgs a, int ctas) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float s = 0.f;
#pragma unroll 4
  for (int i = warp; i < ctas; i += 8) s += a.partial[(int64_t)i * 2 * a.D + c];
  part[warp][lane] = s;
  __syncthreads();
  if (warp) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += part[i][lane];
  if (c < a.D) a.dwq[c] = s;
  else a.dwk[c - a.D] = s;
}

// A warp takes four steps of heads a unit where there are units enough to fill the GPU's warps
// several times over, one step where there are few.
bool many(const QkRopeArgs& a) {
  const int rpw = 32 * kVec / a.D;
  return a.T * ((a.hq + a.hkv + 4 * rpw - 1) / (4 * rpw)) >= 4 * kRopeCtas * (kRopeThreads / 32);
}

template <typename IO, int D, int U>
int rope_ctas(const QkRopeArgs& a) {
  constexpr int RPW = 32 * kVec / D;
  const int64_t units = a.T * ((a.hq + a.hkv + RPW * U - 1) / (RPW * U));
  const int64_t c = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  return (int)(c < kRopeCtas ? c : kRopeCtas);
}

template <typename IO, int D, int U>
cudaError_t launch_rope(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  const int ctas = rope_ctas<IO, D, U>(a);
  if (!backward) {
    // forward: no per-CTA state, so every unit gets a warp of its own
    constexpr int RPW = 32 * kVec / D;
    const int64_t units = a.T * ((a.hq + a.hkv + RPW * U - 1) / (RPW * U));
    const int64_t c = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    qk_rope_kernel<IO, D, U><<<(unsigned)(c < 0x7fffffff ? c : 0x7fffffff), kRopeThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  qk_rope_backward_kernel<IO, D, U><<<ctas, kRopeThreads, 0, s>>>(a);
  qk_rope_dw_kernel<<<2 * D / 32, 256, 0, s>>>(a, ctas);
  return cudaGetLastError();
}

template <typename IO, int D>
cudaError_t launch_rope_u(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  return many(a) ? launch_rope<IO, D, 4>(a, backward, s) : launch_rope<IO, D, 1>(a, backward, s);
}
template <typename IO>
cudaError_t launch_rope_io(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  switch (a.D) {
    case 64: return launch_rope_u<IO, 64>(a, backward, s);
    case 128: return launch_rope_u<IO, 128>(a, backward, s);
    default: return launch_rope_u<IO, 256>(a, backward, s);
  }
}

}  // namespace

cudaError_t qk_rope(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  return a.bf16 ? launch_rope_io<__nv_bfloat16>(a, backward, s)
                : launch_rope_io<float>(a, backward, s);
}

}  // namespace gdn
