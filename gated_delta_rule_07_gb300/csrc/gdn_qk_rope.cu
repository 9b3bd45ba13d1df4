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
// one).  A row is held by D / 8 lanes, two groups of four elements each: the two halves of four
// pairs ("half": d = 4 l and R/2 + 4 l; eight neighbours for "pairs" and past R), so that a pair
// is within one lane, a row's mean is a shuffle over its lanes, and nothing of the forward goes
// through shared memory.  Statistics are fp32.
//
// Measured (GB300, whose copies reach 6.80 TB/s), bf16: forward of 16384 tokens of 32 + 8 heads of
// 128, 59.4 us, 5.79 TB/s of algorithmic bytes (85% of the copies; fp32 107 us, 94%); of 24 tokens of
// 16 + 2 heads of 256, 1.8 us in a graph, a launch's time.  Gradients of 8192 tokens of 16 + 2 heads of
// 256 in 42.5 us, 5.38 TB/s (79%; 16384 tokens of 40 heads of 128 in fp32 167 us, 90%): 71% of the issue
// slots are used, the sums of the weights' gradients and the copies into the ring on top of the
// forward's work.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attention.h"
#include "gdn_common.cuh"
#include "gdn_elements.cuh"
#include "gdn_stream_order.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kVec = 8;  // elements a lane holds of a row

// A lane's place in a row of the forward: where its two groups of four begin.
struct Place {
  int d0, d1;
  bool turned;
};
template <bool PAIRS>
__device__ __forceinline__ Place place_of(int l, int R) {
  Place p;
  p.turned = kVec * l < R;
  const bool halves = !PAIRS && p.turned;
  p.d0 = halves ? 4 * l : kVec * l;
  p.d1 = halves ? R / 2 + 4 * l : kVec * l + 4;
  return p;
}

// A lane's eight elements as four pairs: a[i], b[i] turn together.
template <bool PAIRS, typename IO>
__device__ __forceinline__ void open_pairs(const Quad<IO>* q, float* a, float* b) {
  if constexpr (PAIRS) {
    float f[kVec];
    q[0].open(f);
    q[1].open(f + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = f[2 * i];
      b[i] = f[2 * i + 1];
    }
  } else {
    q[0].open(a);
    q[1].open(b);
  }
}
template <bool PAIRS, typename IO>
__device__ __forceinline__ void put_pairs(IO* row, const Place& p, const float* a, const float* b) {
  if constexpr (PAIRS) {
    const float f[kVec] = {a[0], b[0], a[1], b[1], a[2], b[2], a[3], b[3]};
    put4(row + p.d0, f);
    put4(row + p.d1, f + 4);
  } else {
    put4(row + p.d0, a);
    put4(row + p.d1, b);
  }
}
// four elements of a weight (plus the offset), or ones
__device__ __forceinline__ void weight4(const float* w, int d, float offset, float* f) {
  if (w) {
    Quad<float> q;
    q.load(w + d);
    q.open(f);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = w ? f[i] + offset : 1.f;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// Work: a unit is a token's run of `steps` x 32 / LPR query heads, or key heads.  A warp takes one
// unit: the rotation's and the weight's factors are the same for all its rows and are formed once.
struct RopeUnits {
  int steps;         // row steps of a unit
  int per_q, per_k;  // units of a token's query heads, key heads
};

template <typename IO, int D, bool PAIRS, int U>
__global__ void __launch_bounds__(kRopeThreads, sizeof(IO) == 2 ? 4 : 2)
qk_rope_kernel(QkRopeArgs a, RopeUnits un) {
  constexpr int LPR = D / kVec, RPW = 32 / LPR;
  stream_order();
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int64_t u = (int64_t)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32;
  const int per_token = un.per_q + un.per_k;
  const int64_t t = u < 0x7fffffff ? (uint32_t)u / (uint32_t)per_token : u / per_token;
  if (t >= a.T) return;
  int first = (int)(u - t * per_token);
  const bool isq = first < un.per_q;
  if (!isq) first -= un.per_q;
  const int heads = isq ? a.hq : a.hkv;
  const int h1 = min(heads, (first + 1) * un.steps * RPW);
  const Place p = place_of<PAIRS>(l, a.R);
  int h = first * un.steps * RPW + sub;
  const int64_t hs = isq ? a.q_hs : a.k_hs;
  // the next row to load, its second group's distance, the distance of a step's row
  const IO* src = static_cast<const IO*>(isq ? a.q : a.k) + t * (isq ? a.q_ts : a.k_ts) + h * hs +
                  p.d0;
  const int dd = p.d1 - p.d0;
  const int64_t rs = RPW * hs;
  IO* dst = static_cast<IO*>(isq ? a.q_out : a.k_out) + (t * heads + h) * D;
  Quad<IO> x[U][2];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    x[i][0].clear();
    x[i][1].clear();
    if (h + i * RPW < h1) {
      x[i][0].load(src);
      x[i][1].load(src + dd);
    }
    src += rs;
  }
  const int pos = a.pos[t];
  float w[kVec], wa[4], wb[4], c[4], s[4];
  weight4(isq ? a.wq : a.wk, p.d0, a.offset, w);
  weight4(isq ? a.wq : a.wk, p.d1, a.offset, w + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wa[i] = PAIRS ? w[2 * i] : w[i];
    wb[i] = PAIRS ? w[2 * i + 1] : w[4 + i];
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (pos < 0 || pos >= a.max_pos) {  // (the same for the whole warp)
    if (lane == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
    return;
  }
  if (p.turned) {
    const float* row = a.table + (int64_t)pos * a.R + 4 * l;
    Quad<float> q;
    q.load(row);
    q.open(c);
    q.load(row + a.R / 2);
    q.open(s);
  }
  // out_a = r (a wa c - b wb s), out_b = r (b wb c + a wa s)
  float aa[4], ab[4], ba[4], bb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    aa[i] = wa[i] * c[i];
    ab[i] = wb[i] * -s[i];
    bb[i] = wb[i] * c[i];
    ba[i] = wa[i] * s[i];
  }
  const int rounds = (h1 - (h - sub) + U * RPW - 1) / (U * RPW);
  for (int round = 0; round < rounds; ++round) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float f[4], g[4], o[4], s2 = 0.f;
      open_pairs<PAIRS>(x[i], f, g);
      if (h + (i + U) * RPW < h1) {  // the next round's row
        x[i][0].load(src);
        x[i][1].load(src + dd);
      }
      src += rs;
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = fmaf(f[j], f[j], fmaf(g[j], g[j], s2));
      const float r = rsqrtf(row_sum<LPR>(s2) * (1.f / D) + a.eps);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] = r * fmaf(f[j], aa[j], g[j] * ab[j]);
        g[j] = r * fmaf(g[j], bb[j], f[j] * ba[j]);
      }
      if (h + i * RPW < h1) put_pairs<PAIRS>(dst + i * RPW * D, p, o, g);
    }
    h += U * RPW;
    dst += U * RPW * D;
  }
}

// Gradients.  A CTA has query rows or key rows, a warp walks tokens in a fixed order and keeps its
// share of the weight's gradient in registers; a CTA's warps join theirs in shared memory and
// write one partial sum per CTA, which qk_rope_dw_kernel adds up in a fixed order: the same bits
// on every run.  A thread's rows come through a ring of its own in shared memory (cp.async), so
// that the next is on its way without holding registers.  8192 tokens of 18 heads of 256 take 42.8 us
// with two slots, 45.0 with three, 45.7 with four (the L1 cache gets what the ring leaves).
constexpr int kRopeRing = 2;
template <typename IO> constexpr int rope_ring_bytes() {
  return kRopeRing * 4 * kRopeThreads * 4 * (int)sizeof(IO);
}
template <int BYTES>
__device__ __forceinline__ void ring_copy(uint32_t dst, const void* src, bool ok) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src),
                 "r"(ok ? 8 : 0) : "memory");
}

template <typename IO, int D, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads, sizeof(IO) == 2 ? 3 : 2)
qk_rope_backward_kernel(QkRopeArgs a, int ctas_q) {
  constexpr int LPR = D / kVec, RPW = 32 / LPR, kWarps = kRopeThreads / 32;
  constexpr int QB = 4 * sizeof(IO);  // bytes of a group of four
  __shared__ __align__(16) float part[kWarps][D];
  extern __shared__ __align__(16) char ring[];  // [slot][x0, x1, g0, g1][thread]
  stream_order();
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR, warp = threadIdx.x / 32;
  const bool isq = (int)blockIdx.x < ctas_q;
  const int heads = isq ? a.hq : a.hkv, T = (int)a.T;  // (T fits 31 bits)
  const int64_t rs = RPW * (isq ? a.q_hs : a.k_hs), ts = isq ? a.q_ts : a.k_ts;
  const Place p = place_of<PAIRS>(l, a.R);
  const int dd = p.d1 - p.d0;
  const IO* const xs = static_cast<const IO*>(isq ? a.q : a.k) + sub * (isq ? a.q_hs : a.k_hs) + p.d0;
  const IO* const gs = static_cast<const IO*>(isq ? a.dq_out : a.dk_out) + sub * D + p.d0;
  IO* const dst = static_cast<IO*>(isq ? a.dq : a.dk) + sub * D;
  float w[kVec], wa[4], wb[4], dwa[4], dwb[4];
  weight4(isq ? a.wq : a.wk, p.d0, a.offset, w);
  weight4(isq ? a.wq : a.wk, p.d1, a.offset, w + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    wa[j] = PAIRS ? w[2 * j] : w[j];
    wb[j] = PAIRS ? w[2 * j + 1] : w[4 + j];
    dwa[j] = dwb[j] = 0.f;
  }
  const int stride = (int)(isq ? ctas_q : gridDim.x - ctas_q) * kWarps;
  int t = (int)(isq ? blockIdx.x : blockIdx.x - ctas_q) * kWarps + warp;
  auto after = [&](int tt) { return tt < T - stride ? tt + stride : T; };

  // the copies walk the rows of the warp's tokens ahead of the sums
  int ft = t, fh = sub, fslot = 0;
  const IO *xp = xs + (int64_t)(t < T ? t : 0) * ts, *gp = gs + (int64_t)(t < T ? t : 0) * heads * D;
  const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * QB;
  auto fetch = [&] {
    const bool ok = ft < T && fh < heads;
    const uint32_t at = ring0 + fslot * (4 * kRopeThreads * QB);
    // (a copy that reads nothing still names an address inside the tensor)
    ring_copy<QB>(at, ok ? xp : xs - sub * (isq ? a.q_hs : a.k_hs), ok);
    ring_copy<QB>(at + kRopeThreads * QB, ok ? xp + dd : xs - sub * (isq ? a.q_hs : a.k_hs), ok);
    ring_copy<QB>(at + 2 * kRopeThreads * QB, ok ? gp : gs - sub * D, ok);
    ring_copy<QB>(at + 3 * kRopeThreads * QB, ok ? gp + dd : gs - sub * D, ok);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    fslot = fslot == kRopeRing - 1 ? 0 : fslot + 1;
    fh += RPW;
    xp += rs;
    gp += RPW * D;
    if (fh - sub >= heads && ft < T) {  // the warp's next token (the same step for all its lanes)
      ft = after(ft);
      fh = sub;
      const int64_t tt = ft < T ? ft : 0;
      xp = xs + tt * ts;
      gp = gs + tt * heads * D;
    }
  };
#pragma unroll
  for (int i = 0; i < kRopeRing - 1; ++i) fetch();
  int slot = 0, pos = t < T ? a.pos[t] : 0;
  while (t < T) {
    const int next = after(t);
    const bool good = pos >= 0 && pos < a.max_pos;
    if (!good && lane == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = 1.f;
      s[j] = 0.f;
    }
    if (p.turned) {
      const float* row = a.table + (int64_t)(good ? pos : 0) * a.R + 4 * l;
      Quad<float> q;
      q.load(row);
      q.open(c);
      q.load(row + a.R / 2);
      q.open(s);
    }
    if (next < T) pos = a.pos[next];
    IO* out = dst + (int64_t)t * heads * D;
    for (int h = sub; h - sub < heads; h += RPW) {
      fetch();
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kRopeRing - 1) : "memory");
      Quad<IO> q[2];
      float xa[4], xb[4], ya[4], yb[4], s2 = 0.f, dot = 0.f;
      const char* at = ring + slot * (4 * kRopeThreads * QB) + threadIdx.x * QB;
      q[0].v = *reinterpret_cast<const decltype(q[0].v)*>(at);
      q[1].v = *reinterpret_cast<const decltype(q[0].v)*>(at + kRopeThreads * QB);
      open_pairs<PAIRS>(q, xa, xb);
      q[0].v = *reinterpret_cast<const decltype(q[0].v)*>(at + 2 * kRopeThreads * QB);
      q[1].v = *reinterpret_cast<const decltype(q[0].v)*>(at + 3 * kRopeThreads * QB);
      open_pairs<PAIRS>(q, ya, yb);
      slot = slot == kRopeRing - 1 ? 0 : slot + 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // dy: turned back
        const float da = ya[j];
        ya[j] = fmaf(da, c[j], yb[j] * s[j]);
        yb[j] = fmaf(yb[j], c[j], -da * s[j]);
        s2 = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], s2));
        dot = fmaf(ya[j] * wa[j], xa[j], fmaf(yb[j] * wb[j], xb[j], dot));
      }
      const float r = rsqrtf(row_sum<LPR>(s2) * (1.f / D) + a.eps);
      const float m = row_sum<LPR>(dot) * (1.f / D) * r;  // mean(dn n)
      // (past the last head there is no row: zeros, whose n is not a number where eps is 0)
      const bool live = good && h < heads;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float na = xa[j] * r, nb = xb[j] * r;
        if (live) {
          dwa[j] = fmaf(ya[j], na, dwa[j]);
          dwb[j] = fmaf(yb[j], nb, dwb[j]);
        }
        xa[j] = r * fmaf(ya[j], wa[j], -na * m);
        xb[j] = r * fmaf(yb[j], wb[j], -nb * m);
      }
      if (live) put_pairs<PAIRS>(out, p, xa, xb);
      out += RPW * D;
    }
    t = next;
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  // a warp's rows (lanes with the same l), then the CTA's warps
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
      dwa[j] += __shfl_xor_sync(0xffffffffu, dwa[j], off);
      dwb[j] += __shfl_xor_sync(0xffffffffu, dwb[j], off);
    }
  if (sub == 0) put_pairs<PAIRS>(part[warp], p, dwa, dwb);
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kRopeThreads) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += part[i][d];
    a.partial[(int64_t)blockIdx.x * D + d] = sum;
  }
}

// dw = the sum of the query CTAs' (key CTAs') partial sums.  A block has eight columns of one of
// them, its threads every 128th CTA each: few dependent steps, in a fixed order.
__global__ void __launch_bounds__(1024) qk_rope_dw_kernel(QkRopeArgs a, int ctas_q, int ctas) {
  __shared__ float part[32][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, sub = lane / 8;
  const int blocks = a.D / 8;
  const bool isq = (int)blockIdx.x < blocks;
  const int c = (isq ? blockIdx.x : blockIdx.x - blocks) * 8 + lane % 8;
  stream_order();
  float s = 0.f;
#pragma unroll 4
  for (int i = (isq ? 0 : ctas_q) + 4 * warp + sub; i < (isq ? ctas_q : ctas); i += 128)
    s += a.partial[(int64_t)i * a.D + c];
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if (sub == 0) part[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += part[i][lane];
    (isq ? a.dwq : a.dwk)[c] = sum;
  }
}

int div_up(int64_t x, int64_t y) { return (int)((x + y - 1) / y); }

template <typename IO, int D, bool PAIRS, int U>
cudaError_t launch_forward(const QkRopeArgs& a, RopeUnits un, cudaStream_t s) {
  const int64_t units = a.T * (un.per_q + un.per_k);
  const int64_t ctas = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_ordered(qk_rope_kernel<IO, D, PAIRS, U>, dim3((unsigned)ctas), kRopeThreads, 0, s, a,
                        un);
}

template <typename IO, int D, bool PAIRS>
cudaError_t launch_rope(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  constexpr int RPW = 32 * kVec / D, kWarps = kRopeThreads / 32;
  if (!backward) {
    // Heads of a unit: sixteen steps, four, or one, the most that leaves 4096 units (27 warps an SM).
    // 16384 tokens of 40 heads of 128 take 59.4 us with sixteen, 62.1 with four, 121.5 with one;
    // 1024 such tokens 5.4, 5.2 and 7.3; 256 tokens of 18 heads of 256 take 5.2, 3.0 and 2.7.
    RopeUnits un;
    for (un.steps = 16;; un.steps /= 4) {
      un.per_q = div_up(a.hq, un.steps * RPW);
      un.per_k = div_up(a.hkv, un.steps * RPW);
      if (un.steps == 1 || a.T * (un.per_q + un.per_k) >= 4096) break;
    }
    return un.steps == 1 ? launch_forward<IO, D, PAIRS, 1>(a, un, s)
                         : launch_forward<IO, D, PAIRS, 4>(a, un, s);
  }
  // Three CTAs an SM at most, shared between query and key rows by their number (8192 tokens of 18
  // heads of 256: 42.8 us; two an SM 48.6, four 53.2); where tokens are few, a warp two of them
  // (1531 tokens of 9 heads of 64, fp32: 6.5 us; one 7.1, four 7.9).
  const int most = div_up(a.T, 2 * kWarps);
  int64_t ctas_q = (int64_t)kRopeCtas * a.hq / (a.hq + a.hkv);
  ctas_q = ctas_q < 1 ? 1 : ctas_q > kRopeCtas - 1 ? kRopeCtas - 1 : ctas_q;
  int64_t ctas_k = kRopeCtas - ctas_q;
  if (ctas_q > most) ctas_q = most;
  if (ctas_k > most) ctas_k = most;
  const auto kern = qk_rope_backward_kernel<IO, D, PAIRS>;
  constexpr int smem = rope_ring_bytes<IO>();
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, smem, ready);
  if (e != cudaSuccess) return e;
  e = launch_ordered(kern, dim3((unsigned)(ctas_q + ctas_k)), kRopeThreads, smem, s, a, (int)ctas_q);
  if (e != cudaSuccess) return e;
  return launch_ordered(qk_rope_dw_kernel, dim3(2 * D / 8), 1024, 0, s, a, (int)ctas_q,
                        (int)(ctas_q + ctas_k));
}
template <typename IO, int D>
cudaError_t launch_rope_style(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  return a.pairs ? launch_rope<IO, D, true>(a, backward, s) : launch_rope<IO, D, false>(a, backward, s);
}
template <typename IO>
cudaError_t launch_rope_io(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  switch (a.D) {
    case 64: return launch_rope_style<IO, 64>(a, backward, s);
    case 128: return launch_rope_style<IO, 128>(a, backward, s);
    default: return launch_rope_style<IO, 256>(a, backward, s);
  }
}

}  // namespace

cudaError_t qk_rope(const QkRopeArgs& a, bool backward, cudaStream_t s) {
  return a.bf16 ? launch_rope_io<__nv_bfloat16>(a, backward, s)
                : launch_rope_io<float>(a, backward, s);
}

}  // namespace gdn
