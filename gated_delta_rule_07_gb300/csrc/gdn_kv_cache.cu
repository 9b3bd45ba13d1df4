// gdn_kv_cache.cu -- new keys and values quantised into the paged 8-bit cache, and ranges of it
// read back.
//
// A page's scale covers all its tokens of one head.  For the tokens that a call adds to a page,
//     s = max(amax / qmax, the page's scale if it already holds tokens of its sequence),
//     code = round(x / s)  (x times the fp32 reciprocal of s),
// and where s grew the page's earlier codes become round(code s_old / s).  A page that the call
// starts takes its scale from its new tokens alone, whatever its last owner left.
//
// Append: a CTA per touched page, head (or a few, one after the other) and keys or values: it needs
// the page's whole amax before it can write the first code, and pages are independent.  The page's
// new values are read once and wait in registers for the amax (the number of registers is a template
// parameter: page x D / 256 values a thread).  Keys: a thread takes 8 channels of a token (16 bytes
// of bf16 in, 8 out); values: 4 tokens of 4 channels, one 16-byte piece of the value layout.  Heads
// are the fastest grid index, so that CTAs running together read whole token rows.  Read back: a
// CTA per page and head or two, its keys and values cut into equal runs for its warps.
//
// Prompts are bound by HBM and, nearly as much, by the instructions that form the codes; single
// tokens by latency: launch, sequence table, block table, data.  Measured (GB300), bf16, int8: 7
// prompts of up to 8192 rows, 8 heads of 128, appended in 60.7 us and read back in 48.5 us, 5.39 TB/s
// of algorithmic bytes together (79% of a copy's 6.80 TB/s); one row of each of 96 sequences, 2 heads
// of 256, in 4.8 us, their last pages read back in 5.9 us.
#include <cuda_fp16.h>

#include "gdn_elements.cuh"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kKvThreads = 256;

// ------------------------------------------------------------------------- elements and codes

// eight: one 16-byte load of bf16, two of fp32
template <typename IO>
__device__ __forceinline__ void load8(Quad<IO>* q, const IO* p) {
  if constexpr (sizeof(IO) == 2) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    q[0].v = make_uint2(v.x, v.y);
    q[1].v = make_uint2(v.z, v.w);
  } else {
    q[0].load(p);
    q[1].load(p + 4);
  }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// The largest magnitude so far, as bits without the sign: their order is that of the magnitudes, with
// infinities and NaN above the finite ones.  bf16: of the even and of the odd elements.
__device__ __forceinline__ void take_bits(const Quad<float>& q, uint32_t& m) {
  m = max(max(m, __float_as_uint(q.v.x) & 0x7fffffffu), __float_as_uint(q.v.y) & 0x7fffffffu);
  m = max(max(m, __float_as_uint(q.v.z) & 0x7fffffffu), __float_as_uint(q.v.w) & 0x7fffffffu);
}
__device__ __forceinline__ void take_bits(const Quad<__nv_bfloat16>& q, uint32_t& m) {
  m = __vmaxu2(__vmaxu2(m, q.v.x & 0x7fff7fffu), q.v.y & 0x7fff7fffu);
}
template <typename IO> __device__ __forceinline__ float bits_value(uint32_t m) {
  if constexpr (sizeof(IO) == 4) return __uint_as_float(m);
  else return __uint_as_float(max(m & 0xffff0000u, m << 16));
}
// the largest finite magnitude
template <typename IO> __device__ __forceinline__ void take_finite(const Quad<IO>& q, float& amax) {
  float f[4];
  q.open(f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (finite(f[i])) amax = fmaxf(amax, fabsf(f[i]));
}

// Elements that are not finite, once the page's scale is known: a NaN becomes 0, an infinity the
// value of the largest code, `lim` (0 where the page has no scale; rounded to bf16 it is at most
// 2^-9 off, which rounds to the same code).
template <typename IO> __device__ __forceinline__ void mend(Quad<IO>& q, float lim) {
  float f[4];
  q.open(f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!finite(f[i])) f[i] = f[i] == f[i] ? copysignf(lim, f[i]) : 0.f;
  q.close(f);
}

// The codes of four elements, the first in the low byte.
template <bool E4M3> __device__ __forceinline__ uint32_t encode4(const float* f, float inv) {
  if constexpr (E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1] * inv), "f"(f[0] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3] * inv), "f"(f[2] * inv));
    return lo | ((uint32_t)hi << 16);
  } else {
    // |x inv| <= 127.3: adding 1.5 2^23 leaves the rounded integer in the low byte
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(__fadd_rn(__fmul_rn(f[i], inv), 12582912.f));
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
  }
}

// four codes on a new scale
template <bool E4M3> __device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r |= kv_code<E4M3>(kv_value<E4M3>((w >> (8 * i)) & 0xffu) * ratio) << (8 * i);
  return r;
}

// ------------------------------------------------------------------------------------- append

// The page's new scale: its amax joined over the CTA, against the scale it holds.  `red`: a word
// a warp, not the one before's.
struct NewScale {
  float held, now, inv, lim;
};
template <bool E4M3>
__device__ __forceinline__ NewScale new_scale(float amax, bool bad, float held, float* red,
                                              int32_t* status) {
  const int tid = threadIdx.x;
  if (bad) set_status(status, GDN_ERR_DEVICE_RANGE);
#pragma unroll
  for (int off = 16; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (tid % 32 == 0) red[tid / 32] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKvThreads / 32; ++i) amax = fmaxf(amax, red[i]);
  NewScale s;
  s.held = held;
  s.now = fmaxf(held, amax >= kKvTiny ? amax * (float)(1.0 / kv_qmax<E4M3>()) : 0.f);
  s.inv = s.now > 0.f ? 1.f / s.now : 0.f;
  s.lim = fminf(s.now * kv_qmax<E4M3>(), 3.3895313892515355e38f);  // (bf16's largest)
  return s;
}

// A page's new keys of one head: IT pieces of 8 channels a thread.
template <typename IO, int D, bool E4M3, int IT> struct NewKeys {
  Quad<IO> q[IT][2];
  float held;

  __device__ __forceinline__ void load(const KvArgs& a, const KvSpan& s, int64_t block, int h) {
    const int tid = threadIdx.x, pieces = (s.hi - s.lo) * (D / 8);
    const IO* x = static_cast<const IO*>(a.k) + s.row * a.k_ts + h * a.k_hs;
    held = s.lo > 0 ? a.k_scale[block] : 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i && i * kKvThreads >= pieces) break;
      const int e = tid + i * kKvThreads;
      q[i][0].clear();
      q[i][1].clear();
      if (e < pieces) load8(q[i], x + (e / (D / 8)) * a.k_ts + 8 * (e % (D / 8)));
    }
  }
  __device__ __forceinline__ void store(const KvArgs& a, const KvSpan& s, int64_t block, float* red) {
    const int tid = threadIdx.x, pieces = (s.hi - s.lo) * (D / 8);
    uint8_t* codes = a.k_codes + block * a.page * D;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i && i * kKvThreads >= pieces) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) take_bits(q[i][j], top);
    }
    float amax = bits_value<IO>(top), f[4];
    const bool bad = !finite(amax);
    if (bad) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (!i || i * kKvThreads < pieces) take_finite(q[i][j], amax);
    }
    const NewScale n = new_scale<E4M3>(amax, bad, held, red, a.status);
    if (n.now > n.held && n.held > 0.f) {  // the page's earlier codes on the new scale
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int e = tid; e < s.lo * (D / 4); e += kKvThreads)
        w[e] = rescale4<E4M3>(w[e], n.held * n.inv);
    }
    if (bad) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (!i || i * kKvThreads < pieces) mend(q[i][j], n.lim);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i && i * kKvThreads >= pieces) break;
      const int e = tid + i * kKvThreads;
      if (e < pieces) {
        uint2 w;
        q[i][0].open(f);
        w.x = encode4<E4M3>(f, n.inv);
        q[i][1].open(f);
        w.y = encode4<E4M3>(f, n.inv);
        *reinterpret_cast<uint2*>(codes + s.lo * D + 8 * e) = w;
      }
    }
    if (tid == 0) a.k_scale[block] = n.now;
  }
};

// A page's new values of one head: IT pieces of 4 tokens x 4 channels a thread (a piece at an end
// of the span may hold earlier tokens' codes, or none yet).
template <typename IO, int D, bool E4M3, int IT> struct NewValues {
  Quad<IO> q[IT][4];
  uint4 old;  // codes beside the new ones in the first piece
  float held;

  __device__ __forceinline__ void load(const KvArgs& a, const KvSpan& s, int64_t block, int h) {
    const int tid = threadIdx.x, g0 = s.lo / 4;
    const int pieces = ((s.hi + 3) / 4 - g0) * (D / 4);
    const uint8_t* codes = a.v_codes + block * a.page * D;
    const IO* x = static_cast<const IO*>(a.v) + s.row * a.v_ts + h * a.v_hs;
    held = s.lo > 0 ? a.v_scale[block] : 0.f;
    old = make_uint4(0u, 0u, 0u, 0u);
    if (s.lo % 4 && tid < D / 4)
      old = *reinterpret_cast<const uint4*>(codes + (int64_t)g0 * 4 * D + 16 * tid);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i && i * kKvThreads >= pieces) break;
      const int e = tid + i * kKvThreads, t0 = 4 * (g0 + e / (D / 4)), d = 4 * (e % (D / 4));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        q[i][t].clear();
        if (e < pieces && t0 + t >= s.lo && t0 + t < s.hi)
          q[i][t].load(x + (t0 + t - s.lo) * a.v_ts + d);
      }
    }
  }
  __device__ __forceinline__ void store(const KvArgs& a, const KvSpan& s, int64_t block, float* red) {
    const int tid = threadIdx.x, g0 = s.lo / 4;
    const int pieces = ((s.hi + 3) / 4 - g0) * (D / 4);
    uint8_t* codes = a.v_codes + block * a.page * D;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i && i * kKvThreads >= pieces) break;
#pragma unroll
      for (int t = 0; t < 4; ++t) take_bits(q[i][t], top);
    }
    float amax = bits_value<IO>(top), f[4];
    const bool bad = !finite(amax);
    if (bad) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (!i || i * kKvThreads < pieces) take_finite(q[i][t], amax);
    }
    const NewScale n = new_scale<E4M3>(amax, bad, held, red, a.status);
    const bool grew = n.now > n.held && n.held > 0.f;
    if (grew) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int e = tid; e < g0 * D; e += kKvThreads) w[e] = rescale4<E4M3>(w[e], n.held * n.inv);
    }
    if (bad) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (!i || i * kKvThreads < pieces) mend(q[i][t], n.lim);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i && i * kKvThreads >= pieces) break;
      const int e = tid + i * kKvThreads;
      if (e < pieces) {
        uint32_t w[4], o[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {  // w[t]: token t's codes of the four channels
          q[i][t].open(f);
          w[t] = encode4<E4M3>(f, n.inv);
        }
        // transpose 4 x 4 bytes: a word of four tokens for each channel
        const uint32_t a01 = __byte_perm(w[0], w[1], 0x5140), b01 = __byte_perm(w[0], w[1], 0x7362);
        const uint32_t a23 = __byte_perm(w[2], w[3], 0x5140), b23 = __byte_perm(w[2], w[3], 0x7362);
        o[0] = __byte_perm(a01, a23, 0x5410);
        o[1] = __byte_perm(a01, a23, 0x7632);
        o[2] = __byte_perm(b01, b23, 0x5410);
        o[3] = __byte_perm(b01, b23, 0x7632);
        if (i == 0 && s.lo % 4 && tid < D / 4) {  // earlier tokens in the first piece
          const uint32_t keep = (1u << (8 * (s.lo % 4))) - 1u;
          uint32_t was[4] = {old.x, old.y, old.z, old.w};
          if (grew) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {  // (rotated, so that the loop is one copy of the code)
              const uint32_t r = rescale4<E4M3>(was[0], n.held * n.inv);
              was[0] = was[1];
              was[1] = was[2];
              was[2] = was[3];
              was[3] = r;
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) o[c] = (o[c] & ~keep) | (was[c] & keep);
        }
        *reinterpret_cast<uint4*>(codes + (int64_t)g0 * 4 * D + 16 * e) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    if (tid == 0) a.v_scale[block] = n.now;
  }
};

// Heads [h0, h1) of a page.  (Two heads in flight at a time cost more registers than they
// hid: prompts took a tenth longer.)
template <typename New>
__device__ __forceinline__ void append_heads(const KvArgs& a, const KvSpan& s, int pid, int h0,
                                             int h1, float (*red)[kKvThreads / 32]) {
  const int64_t block = (int64_t)pid * a.hkv;
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    New x;
    x.load(a, s, block + h, h);
    x.store(a, s, block + h, red[h & 1]);
  }
}

// CTAs an SM holds at least: 64 registers a thread where the waiting values leave room (prompts of 7 x
// 8192 rows take 116 us with the read back with the compiler's own number, 109 so).
template <typename IO, int IT> constexpr int append_resident() {
  constexpr int words = IT * sizeof(IO);  // x 4: registers of waiting values
  return words <= 8 ? 4 : words <= 16 ? 2 : 1;
}

// IT: pages of at most 4096 IT new values.  Blocks: (slot, group of `per` heads, keys or values).
template <typename IO, int D, bool E4M3, int IT>
__global__ void __launch_bounds__(kKvThreads, append_resident<IO, IT>())
kv_append_kernel(KvArgs a, int per) {
  __shared__ float red[2][kKvThreads / 32];
  __shared__ KvFound found;
  const int groups = (a.hkv + per - 1) / per, slot = blockIdx.x / (2 * groups);
  const int which = blockIdx.x - slot * 2 * groups;
  stream_order();
  kv_find(a, slot, found);
  if (found.pid < 0) return;
  const KvSpan s = found.span;
  const int h0 = which / 2 * per, h1 = h0 + per < a.hkv ? h0 + per : a.hkv;
  if (which & 1) append_heads<NewValues<IO, D, E4M3, IT>>(a, s, found.pid, h0, h1, red);
  else append_heads<NewKeys<IO, D, E4M3, 2 * IT>>(a, s, found.pid, h0, h1, red);
}

// --------------------------------------------------------------------------------------- read

// four values of a word's codes
template <bool E4M3>
__device__ __forceinline__ void decode4(uint32_t w, float scale, float* f) {
  if constexpr (E4M3) {  // (kv_value's bits for two codes at a time)
    const uint32_t x = __byte_perm(w, 0, 0x1404), y = __byte_perm(w, 0, 0x3424);
    const uint32_t lo = (x & 0x80008000u) | ((x >> 1) & 0x3f803f80u);
    const uint32_t hi = (y & 0x80008000u) | ((y >> 1) & 0x3f803f80u);
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = p.x * 256.f * scale; f[1] = p.y * 256.f * scale;
    f[2] = q.x * 256.f * scale; f[3] = q.y * 256.f * scale;
  } else {  // 2^23 + (code + 128) in an fp32's mantissa
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.f) * scale;
  }
}
constexpr int kReadUnroll = 4;  // loads a thread has in flight

// Blocks: (slot, group of `per` heads).  The group's keys and values are cut into runs of
// kReadUnroll pieces a lane, and the runs dealt out to the CTA's warps.
template <typename IO, int D, bool E4M3>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvArgs a, int per) {
  constexpr int E = 16 / sizeof(IO), RUN = kReadUnroll * 32;
  __shared__ KvFound found;
  const int groups = (a.hkv + per - 1) / per, slot = blockIdx.x / groups;
  const int lane = threadIdx.x & 31, h0 = (blockIdx.x - slot * groups) * per;
  stream_order();
  kv_find(a, slot, found);
  if (found.pid < 0) return;
  const KvSpan s = found.span;
  const int heads = h0 + per < a.hkv ? per : a.hkv - h0;
  const int64_t block = (int64_t)found.pid * a.hkv + h0;
  const int64_t ts = (int64_t)a.hkv * D, out0 = (s.row * a.hkv + h0) * D;
  const int k_pieces = (s.hi - s.lo) * (D / E), k_runs = (k_pieces + RUN - 1) / RUN;
  const int g0 = s.lo / 4, v_pieces = ((s.hi + 3) / 4 - g0) * (D / 4);
  const int v_runs = (v_pieces + RUN - 1) / RUN;
  for (int r = threadIdx.x / 32; r < heads * (k_runs + v_runs); r += kKvThreads / 32) {
    if (r < heads * k_runs) {  // keys: 16 bytes of output a piece
      const int h = r / k_runs, e0 = (r - h * k_runs) * RUN + lane;
      const uint8_t* codes = a.k_codes + ((block + h) * a.page + s.lo) * D;
      const float scale = a.k_scale[block + h];
      IO* out = static_cast<IO*>(a.k_out) + out0 + h * D;
      uint32_t w[kReadUnroll][E / 4];
#pragma unroll
      for (int i = 0; i < kReadUnroll; ++i) {
        const int e = e0 + i * 32;
        if (e < k_pieces) {
          if constexpr (E == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(codes + E * e));
            w[i][0] = v.x;
            w[i][1] = v.y;
          } else {
            w[i][0] = __ldg(reinterpret_cast<const uint32_t*>(codes + E * e));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kReadUnroll; ++i) {
        const int e = e0 + i * 32;
        if (e >= k_pieces) break;
        IO* dst = out + (e / (D / E)) * ts + E * (e % (D / E));
        float f[4];
        decode4<E4M3>(w[i][0], scale, f);
        if constexpr (E == 8) {
          const uint2 x = bf16x4(f);
          decode4<E4M3>(w[i][1], scale, f);
          const uint2 y = bf16x4(f);
          *reinterpret_cast<uint4*>(dst) = make_uint4(x.x, x.y, y.x, y.y);
        } else {
          put4(dst, f);
        }
      }
    } else {  // values: 4 tokens x 4 channels a piece
      const int q = r - heads * k_runs, h = q / v_runs, e0 = (q - h * v_runs) * RUN + lane;
      const uint8_t* codes = a.v_codes + ((block + h) * a.page + 4 * g0) * D;
      const float scale = a.v_scale[block + h];
      IO* out = static_cast<IO*>(a.v_out) + out0 + h * D;
      uint4 w[kReadUnroll];
#pragma unroll
      for (int i = 0; i < kReadUnroll; ++i) {
        const int e = e0 + i * 32;
        if (e < v_pieces) w[i] = __ldg(reinterpret_cast<const uint4*>(codes + 16 * e));
      }
#pragma unroll
      for (int i = 0; i < kReadUnroll; ++i) {
        const int e = e0 + i * 32;
        if (e >= v_pieces) break;
        const int t0 = 4 * (g0 + e / (D / 4)), d = 4 * (e % (D / 4));
        float f[4][4];
        decode4<E4M3>(w[i].x, scale, f[0]);
        decode4<E4M3>(w[i].y, scale, f[1]);
        decode4<E4M3>(w[i].z, scale, f[2]);
        decode4<E4M3>(w[i].w, scale, f[3]);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (t0 + t >= s.lo && t0 + t < s.hi) {
            const float g[4] = {f[0][t], f[1][t], f[2][t], f[3][t]};
            put4(out + (t0 + t - s.lo) * ts + d, g);
          }
      }
    }
  }
}

// ---------------------------------------------------------------------------------- launching

template <typename IO, int D, bool E4M3>
cudaError_t launch_kv(const KvArgs& a, bool append, cudaStream_t s) {
  const int64_t slots =
      a.cu == nullptr && a.N > 1 ? a.N : (a.T >> a.page_shift) + 2 * (int64_t)a.N;
  // registers for the values that a page can add: one row a sequence needs one piece
  const int values = a.cu == nullptr && a.N > 1 ? D : a.page * D;
  // A CTA takes several heads of its page, one after the other, where that leaves the GPU four
  // rounds of CTAs (of the 608 that its 152 SMs hold): the page is looked up once for them.
  // Prompts of 7 x 8192 rows, 8 heads of 128: append 80 us with one head a CTA, 68 with two, 64
  // with four; read 53 us with one, 47 with two.  A step of 96 rows, 2 heads of 256, is quicker with
  // one: 10.6 us for both, 12.5 with all heads in a CTA.
  const int64_t single = slots * (append ? 2 : 1) * a.hkv, many = single / (4 * 608);
  const int most = append ? 4 : 2, per = many < 1 ? 1 : many < most ? (int)many : most;
  const int64_t ctas = slots * (append ? 2 : 1) * ((a.hkv + per - 1) / per);
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto go = [&](void (*kern)(KvArgs, int)) {
    return launch_ordered(kern, dim3((unsigned)ctas), kKvThreads, 0, s, a, per);
  };
  if (!append) return go(kv_read_kernel<IO, D, E4M3>);
  // (pages of 128 tokens at most: D / 32 pieces.  Small pages, 5 sequences of 700 rows, 3 heads of 64
  // in pages of 16: 8.6 us with the read back, 8.9 with room for more.  Between 8192 and 16384 values
  // the room costs nothing: prompts of pages of 8192 take 109 us with room for 16384, 112 without.)
  if (values <= 4096) return go(kv_append_kernel<IO, D, E4M3, 1>);
  if constexpr (D == 256) {
    if (values > 16384) return go(kv_append_kernel<IO, D, E4M3, 8>);
  }
  return go(kv_append_kernel<IO, D, E4M3, (D == 64 ? 2 : 4)>);
}

template <typename IO>
cudaError_t launch_kv_io(const KvArgs& a, bool append, cudaStream_t s) {
  switch (a.D) {
    case 64: return a.e4m3 ? launch_kv<IO, 64, true>(a, append, s) : launch_kv<IO, 64, false>(a, append, s);
    case 128: return a.e4m3 ? launch_kv<IO, 128, true>(a, append, s) : launch_kv<IO, 128, false>(a, append, s);
    default: return a.e4m3 ? launch_kv<IO, 256, true>(a, append, s) : launch_kv<IO, 256, false>(a, append, s);
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
