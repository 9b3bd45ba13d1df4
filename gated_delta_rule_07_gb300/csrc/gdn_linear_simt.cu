// gdn_linear_simt.cu -- linear attention with a decay for each head (gdn_linear.h) in fp32 on the CUDA
// cores, for fp32 I/O and for bf16 rows that tensor maps cannot describe (broadcast ones); and the scan
// over a sequence's segments, which both families use.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_elements.cuh"
#include "gdn_linear.cuh"
#include "gdn_stream_order.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int C = 64;        // tokens of a chunk
constexpr int kTile = 32;    // tokens that the state kernel stages at a time

template <typename IO>
__device__ __forceinline__ const IO* head_rows(const LinearRows& r, int head) {
  return static_cast<const IO*>(r.p) + (int64_t)(head / r.share) * r.hs;
}

// Rows t0 .. t0 + n of D elements into dst (rows of `stride` floats), zeros behind them; row i times
// its weight a^{|w0 + w1 i|}.
template <int ROWS, int D, typename IO, bool WEIGHTED>
__device__ __forceinline__ void stage(float* dst, int stride, const IO* src, int64_t ts, int64_t t0,
                                      int n, float log2a, int w0, int w1) {
#pragma unroll 8
  for (int i0 = 0; i0 < ROWS * (D / 4); i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    Quad<IO> q;
    float f[4];
    if (r < n)
      q.load(src + (t0 + r) * ts + c);
    else
      q.clear();
    q.open(f);
    if (WEIGHTED) {
      const float w = r < n ? linear::power(log2a, w0 + w1 * r) : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] *= w;
    }
    put4(dst + r * stride + c, f);
  }
}

__global__ void __launch_bounds__(1024) linear_check_kernel(LinearShape s) {
  stream_order();
  linear::usable(s);
}

// ------------------------------------------------------------------ a segment's own state

// One block a (slot, value head): the K x V sums in registers, 32 tokens staged at a time.  (Half of K a
// block: 195 us for four sequences of 2048 tokens, 16 heads of 128, against 167.)
template <int K, int V, typename IO>
__global__ void __launch_bounds__(kThreads) linear_state_kernel(LinearState a) {
  constexpr int MK = K / 16, MV = V / 16;
  __shared__ __align__(16) float xs[kTile][K], ys[kTile][V];
  stream_order();
  if (!linear::usable(a.s)) return;
  int n;
  int64_t t0, t1;
  const int64_t slot = blockIdx.x;
  const int head = blockIdx.y;
  if (!linear::slot_tokens(a.s, slot, n, t0, t1)) return;
  const float log2a = linear::log2_decay(a.s, head);
  const IO* x = head_rows<IO>(a.x, head);
  const IO* y = head_rows<IO>(a.y, head);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[MK][MV] = {};
  for (int64_t t = t0; t < t1; t += kTile) {
    const int m = (int)(t1 - t < kTile ? t1 - t : kTile);
    // forward: a token decays on its way to the segment's last; backward: to before the first
    const int w0 = a.reverse ? (int)(t - t0) + 1 : (int)(t1 - 1 - t), w1 = a.reverse ? 1 : -1;
    stage<kTile, K, IO, false>(&xs[0][0], K, x, a.x.ts, t, m, 0.f, 0, 0);
    stage<kTile, V, IO, true>(&ys[0][0], V, y, a.y.ts, t, m, log2a, w0, w1);
    __syncthreads();
#pragma unroll 4
    for (int r = 0; r < kTile; ++r) {
      float u[MK], w[MV];
#pragma unroll
      for (int i = 0; i < MK; i += 4) *reinterpret_cast<float4*>(&u[i]) =
          *reinterpret_cast<const float4*>(&xs[r][ty * MK + i]);
#pragma unroll
      for (int i = 0; i < MV; i += 4) *reinterpret_cast<float4*>(&w[i]) =
          *reinterpret_cast<const float4*>(&ys[r][16 * i + 4 * tx]);
#pragma unroll
      for (int i = 0; i < MK; ++i)
#pragma unroll
        for (int j = 0; j < MV; ++j) acc[i][j] = fmaf(u[i], w[j], acc[i][j]);
    }
    __syncthreads();
  }
  float* u = a.states + (slot * a.s.hv + head) * K * V;
#pragma unroll
  for (int i = 0; i < MK; ++i)
#pragma unroll
    for (int j = 0; j < MV; j += 4) put4(u + (ty * MK + i) * V + 16 * j + 4 * tx, &acc[i][j]);
}

// ------------------------------------------------------------------ the scan over segments

// Loads that wait for nothing between them.  (Sixteen: 10 us for 65536 tokens of 32 heads, 13 with branches
// around plain loads; four: 27 and 12 for gradients of 8 x 4096 tokens.)
__device__ __forceinline__ void load_if(float4& v, const float* p, bool yes) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.s32 p, %5, 0;\n@p ld.global.v4.f32 {%0, %1, %2, %3}, [%4];\n}\n"
               : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w)
               : "l"(p), "r"((int)yes)
               : "memory");
}
// One thread carries four elements of a state through its sequence's segments; the segments' sums are
// read `kAhead` at a time, for each step waits for the one before only in registers.  A backward pass has
// two scans, which run side by side.
struct ScanPair {
  LinearScan of[2];
};
template <int kAhead>
__global__ void __launch_bounds__(kThreads) linear_scan_kernel(const __grid_constant__ ScanPair both,
                                                               int blocks) {
  stream_order();
  const LinearScan& a = both.of[blockIdx.z / blocks];
  if (!linear::usable(a.s)) return;
  const int n = blockIdx.x, head = blockIdx.y;
  const int64_t size = (int64_t)a.s.K * a.s.V;
  const int64_t at = ((int64_t)(blockIdx.z % blocks) * kThreads + threadIdx.x) * 4;
  if (at >= size) return;
  const int64_t b = a.s.cu ? a.s.cu[n] : 0, e = a.s.cu ? a.s.cu[n + 1] : a.s.T;
  const int count = (int)((e - b + a.s.seg - 1) / a.s.seg);
  const int64_t slot0 = b / a.s.seg + n;
  const float log2a = linear::log2_decay(a.s, head);
  const float whole = linear::power(log2a, a.s.seg);
  const float rest = linear::power(log2a, (int)(e - b) - (count - 1) * a.s.seg);  // the last segment's
  const int64_t mine = ((int64_t)n * a.s.hv + head) * size + at;
  float4 h = a.first ? *reinterpret_cast<const float4*>(a.first + mine) : make_float4(0, 0, 0, 0);
  float* u = a.states + (slot0 * a.s.hv + head) * size + at;
  const int64_t step = (int64_t)a.s.hv * size;
  for (int i0 = 0; i0 < count; i0 += kAhead) {
    float4 add[kAhead] = {};
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = a.reverse ? count - 1 - (i0 + k) : i0 + k;
      if constexpr (kAhead > 4)
        load_if(add[k], u + i * step, i0 + k < count);
      else if (i0 + k < count)
        add[k] = *reinterpret_cast<const float4*>(u + i * step);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = a.reverse ? count - 1 - (i0 + k) : i0 + k;
      if (i0 + k < count) {
        *reinterpret_cast<float4*>(u + i * step) = h;
        const float w = i == count - 1 ? rest : whole;
        h.x = fmaf(w, h.x, add[k].x);
        h.y = fmaf(w, h.y, add[k].y);
        h.z = fmaf(w, h.z, add[k].z);
        h.w = fmaf(w, h.w, add[k].w);
      }
    }
  }
  if (a.last) *reinterpret_cast<float4*>(a.last + mine) = h;
}

// ------------------------------------------------------------------ the pass

// One block a (slot, value head) walks the segment's chunks of 64 tokens with S in shared memory.  What
// several value heads add to one output head goes to fp32 rows of their own, which a kernel behind sums in
// the heads' order.  (Walked one after another by one block: 104 us for the two such passes of four ragged
// sequences of up to 500 tokens, three value heads to each of two key heads, instead of 39.)
//
// 49152 multiply-adds a token at A = B = 128 make it the CUDA cores' to bound, if their operands come
// cheaply: a thread has four neighbouring columns of several rows (of P, two columns of eight), so that a
// warp reads the rows' operand as broadcasts and four steps of it at once.  (Threads of 4 x 4 and 64
// columns a block: 571 us for four sequences of 2048 tokens, 16 heads of 128; so 407, where the segments
// fill fewer SMs.)
template <int A, int B> constexpr int pass_smem() {
  return (2 * C * (A + 4) + C * B + A * B + C * (C + 4) + C + 4) * 4;
}
template <int A, int B, typename IO>
__global__ void __launch_bounds__(kThreads, 1) linear_pass_kernel(LinearPass a) {
  constexpr int CL = B / 4, RG = kThreads / CL;  // threads of a row, groups of rows
  constexpr int MO = C / RG, MS = A / RG;        // rows a thread of the output, of S
  extern __shared__ __align__(16) float smem[];
  float* zs = smem;                    // [C][A + 4]
  float* xs = zs + C * (A + 4);        // [C][A + 4]
  float* ys = xs + C * (A + 4);        // [C][B]
  float* S = ys + C * B;               // [A][B]
  float* P = S + A * B;                // [C][C + 4]
  float* power = P + C * (C + 4);      // [C + 1]: a^i
  stream_order();
  if (!linear::accepted(a.s)) return;
  int n;
  int64_t t0, t1;
  const int64_t slot = blockIdx.x;
  if (!linear::slot_tokens(a.s, slot, n, t0, t1)) return;
  const int head = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rg = threadIdx.x / CL, col = threadIdx.x % CL * 4;
  const int chunks = (int)((t1 - t0 + C - 1) / C);
  const int64_t ots = (int64_t)a.s.hv * B;
  IO* out = static_cast<IO*>(a.out) + (int64_t)head * B + col;
  float* apart = a.out_share > 1 ? a.partial + (int64_t)head * B + col : nullptr;
  const float log2a = linear::log2_decay(a.s, head);
  const IO* z = head_rows<IO>(a.z, head);
  const IO* x = head_rows<IO>(a.x, head);
  const IO* y = head_rows<IO>(a.y, head);
  const float* st = a.states + (slot * a.s.hv + head) * A * B;
  const float enter = a.reverse ? 1.f : linear::power(log2a, 1);
  for (int i = threadIdx.x; i < A * B; i += kThreads) {
    // (the faster index along the stored rows)
    const int r = a.transposed ? i % A : i / B, c = a.transposed ? i / A : i % B;
    S[r * B + c] = (a.transposed ? st[c * A + r] : st[i]) * enter;
  }
  if (threadIdx.x <= C) power[threadIdx.x] = linear::power(log2a, threadIdx.x);
  for (int ci = 0; ci < chunks; ++ci) {
    const int64_t t = t0 + (int64_t)(a.reverse ? chunks - 1 - ci : ci) * C;
    const int m = (int)(t1 - t < C ? t1 - t : C);
    stage<C, A, IO, false>(zs, A + 4, z, a.z.ts, t, m, 0.f, 0, 0);
    stage<C, A, IO, false>(xs, A + 4, x, a.x.ts, t, m, 0.f, 0, 0);
    stage<C, B, IO, false>(ys, B, y, a.y.ts, t, m, 0.f, 0, 0);
    __syncthreads();
    {  // P[i][j] = a^{|i - j|} z_i . x_j where j is at or before i; a warp has eight rows
      float p[8][2] = {};
#pragma unroll 2
      for (int k = 0; k < A; k += 4) {
        float4 w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = *reinterpret_cast<const float4*>(xs + (lane + 32 * j) * (A + 4) + k);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 u = *reinterpret_cast<const float4*>(zs + (8 * warp + i) * (A + 4) + k);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            p[i][j] = fmaf(u.x, w[j].x, fmaf(u.y, w[j].y, fmaf(u.z, w[j].z, fmaf(u.w, w[j].w, p[i][j]))));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * warp + i, c = lane + 32 * j, gap = a.reverse ? c - r : r - c;
          P[r * (C + 4) + c] = gap >= 0 && c < m ? p[i][j] * power[gap] : 0.f;
        }
    }
    __syncthreads();
    float o[MO][4] = {};
    auto times = [&](const float* u, int stride, const float* w, int steps) {  // o += rows of u by w
#pragma unroll 2
      for (int k = 0; k < steps; k += 4) {
        float4 v[4];
#pragma unroll
        for (int l = 0; l < 4; ++l) v[l] = *reinterpret_cast<const float4*>(w + (k + l) * B + col);
#pragma unroll
        for (int i = 0; i < MO; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(u + (rg * MO + i) * stride + k);
          const float e[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            o[i][0] = fmaf(e[l], v[l].x, o[i][0]);
            o[i][1] = fmaf(e[l], v[l].y, o[i][1]);
            o[i][2] = fmaf(e[l], v[l].z, o[i][2]);
            o[i][3] = fmaf(e[l], v[l].w, o[i][3]);
          }
        }
      }
    };
    times(zs, A + 4, S, A);
#pragma unroll
    for (int i = 0; i < MO; ++i) {
      const int r = rg * MO + i;
      const float w = power[a.reverse ? (r < m ? m - 1 - r : 0) : r];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] *= w;
    }
    times(P, C + 4, ys, C);
#pragma unroll
    for (int i = 0; i < MO; ++i) {
      const int r = rg * MO + i;
      if (r >= m) continue;
      const int64_t row = (t + r) * ots;
      if (apart)
        put4(apart + row, o[i]);
      else
        put4(out + row, o[i]);
    }
    __syncthreads();
    if (ci + 1 < chunks) {  // S <- a^m S + sum_j a^{steps to the chunk's end} x_j y_j^T
      const float w = power[m];
      float* const mine = S + rg * MS * B + col;
      float acc[MS][4];
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(mine + i * B);
        acc[i][0] = w * v.x; acc[i][1] = w * v.y; acc[i][2] = w * v.z; acc[i][3] = w * v.w;
      }
#pragma unroll 2
      for (int k = 0; k < m; ++k) {
        const float wk = power[a.reverse ? k + 1 : m - k];
        float4 v = *reinterpret_cast<const float4*>(ys + k * B + col);
        v.x *= wk; v.y *= wk; v.z *= wk; v.w *= wk;
#pragma unroll
        for (int i = 0; i < MS; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(xs + k * (A + 4) + rg * MS + i);
          const float e[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            acc[i + l][0] = fmaf(e[l], v.x, acc[i + l][0]);
            acc[i + l][1] = fmaf(e[l], v.y, acc[i + l][1]);
            acc[i + l][2] = fmaf(e[l], v.z, acc[i + l][2]);
            acc[i + l][3] = fmaf(e[l], v.w, acc[i + l][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MS; ++i) put4(mine + i * B, acc[i]);
      __syncthreads();
    }
  }
}

// out [T, heads, B] = the sum of the share's fp32 rows, in the heads' order; four elements a thread.  Rows
// behind the last sequence are left as they are.
template <typename IO>
__global__ void __launch_bounds__(kThreads) linear_sum_kernel(LinearPass a) {
  stream_order();
  if (!linear::accepted(a.s)) return;
  const int64_t rows = (a.s.cu ? a.s.cu[a.s.N] : a.s.T) * (a.s.hv / a.out_share);
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x, row = at / (a.B / 4);
  const int c = (int)(at - row * (a.B / 4)) * 4;
  if (row >= rows) return;
  float f[4] = {};
  for (int g = 0; g < a.out_share; ++g) {
    const float4 v = *reinterpret_cast<const float4*>(a.partial + (row * a.out_share + g) * a.B + c);
    f[0] += v.x; f[1] += v.y; f[2] += v.z; f[3] += v.w;
  }
  put4(static_cast<IO*>(a.out) + row * a.B + c, f);
}

template <int K, int V>
cudaError_t launch_state(const LinearState& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.s.slots, (unsigned)a.s.hv);
  return a.s.bf16 ? launch_ordered(linear_state_kernel<K, V, __nv_bfloat16>, grid, kThreads, 0, s, a)
                  : launch_ordered(linear_state_kernel<K, V, float>, grid, kThreads, 0, s, a);
}

template <int A, int B, typename IO> cudaError_t launch_pass(const LinearPass& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(linear_pass_kernel<A, B, IO>, pass_smem<A, B>(), done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.s.slots, (unsigned)a.s.hv);
  const cudaError_t done_pass =
      launch_ordered(linear_pass_kernel<A, B, IO>, grid, kThreads, pass_smem<A, B>(), s, a);
  if (done_pass != cudaSuccess || a.out_share == 1) return done_pass;
  const int64_t threads = a.s.T * (a.s.hv / a.out_share) * (B / 4);
  return launch_ordered(linear_sum_kernel<IO>, dim3((unsigned)((threads + kThreads - 1) / kThreads)),
                        kThreads, 0, s, a);
}
template <typename IO> cudaError_t launch_pass_of(const LinearPass& a, cudaStream_t s) {
  if (a.A == 128) return a.B == 128 ? launch_pass<128, 128, IO>(a, s) : launch_pass<128, 64, IO>(a, s);
  return a.B == 128 ? launch_pass<64, 128, IO>(a, s) : launch_pass<64, 64, IO>(a, s);
}

}  // namespace

cudaError_t linear_check(const LinearShape& a, cudaStream_t s) {
  return launch_ordered(linear_check_kernel, dim3(1), 1024, 0, s, a);
}

cudaError_t linear_state_simt(const LinearState& a, cudaStream_t s) {
  if (a.s.K == 128) return a.s.V == 128 ? launch_state<128, 128>(a, s) : launch_state<128, 64>(a, s);
  return a.s.V == 128 ? launch_state<64, 128>(a, s) : launch_state<64, 64>(a, s);
}

cudaError_t linear_scan(const LinearScan* scans, int count, cudaStream_t s) {
  const LinearShape& shape = scans[0].s;
  const int blocks = (shape.K * shape.V / 4 + kThreads - 1) / kThreads;
  ScanPair both;
  both.of[0] = scans[0];
  both.of[1] = scans[count - 1];
  const dim3 grid((unsigned)shape.N, (unsigned)shape.hv, (unsigned)(blocks * count));
  // Sixteen ahead for sequences of many segments (16384 tokens of 32 heads, 9 segments: 17 us for the two
  // scans of a backward pass, 38 four at a time), four for those of a few, where the registers cost more
  // (eight ragged sequences: 16 us, 54).
  if (shape.T / shape.seg >= 4 * (int64_t)shape.N)
    return launch_ordered(linear_scan_kernel<16>, grid, kThreads, 0, s, both, blocks);
  return launch_ordered(linear_scan_kernel<4>, grid, kThreads, 0, s, both, blocks);
}

cudaError_t linear_pass_simt(const LinearPass& a, cudaStream_t s) {
  return a.s.bf16 ? launch_pass_of<__nv_bfloat16>(a, s) : launch_pass_of<float>(a, s);
}

}  // namespace gdn
