// gdn_kv_attention.cuh -- what the attention kernels over the 8-bit cache share: the work plan, the
// codes as fp16, and the join of partial results.
//
// Work: units of UNIT keys, of all sequences, kv heads and row tiles in one line, cut into equal
// runs, one a CTA: ragged lengths balance, and one long sequence fills the GPU.  Items cut between
// CTAs leave partial sums (M, X, sum, unnormalised o), joined in order by a second small kernel.
//
// Range.  The weights of o are 2^(y - M), y = x + log2(value scale) (x: scores in log2), and reach
// o whatever the scales are.  The sum is of 2^(x - X) and has a reference of its own, X = M - B: B is
// the smallest log2 of a value scale met so far (within kBelow), so that a term is a weight times
// 2^(B - log2(value scale)) <= 2^kBelow and neither small scales nor many keys overflow it.  A page of
// scale 0 weighs as one of 2^(B - kZero), whose codes (zeros, where an append wrote them) weigh less
// than fp32 tells beside any other page's; before the first other page B is 0, and then moves M
// instead of the sum.  Terms are lost only below 2^-126: value scales of one sequence and head may
// differ by 2^100 (beside pages of scale 0, by 2^70).
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>

#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kAttWarps = 4, kAttThreads = 32 * kAttWarps;
constexpr int kMaxCtas = 912;  // CTAs at most, six an SM (the workspace holds two parts of each)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The reference M of a row's weights 2^(y - M) stands kHead below the largest score where it was
// last moved, and moves when a score exceeds it by kSlack (log2): weights stay within fp16's range,
// and one 2^-22 of the largest still has all of fp16's bits.
constexpr float kHead = 8.f, kSlack = 15.f;
constexpr float kNone = -1e30f;  // the reference before any key
constexpr float kBelow = 8.f;    // how far a value scale may lie below 2^B before B follows
constexpr float kZero = 40.f;    // how far below 2^B a value scale of 0 stands
constexpr float kLeastScale = 1.17549435e-38f;  // value scales below it count as 0

// ------------------------------------------------------------------------------ the work plan

struct Item {          // what a sequence asks for
  int64_t row0;        // its first packed row
  int m, len;          // query rows (tokens), keys
  int tile0, tiles;    // tiles of UNIT keys that some row sees
  int row_tiles;       // tiles of ROWS of the m * group rows of a kv head
};

// An item is a kv head and row tile of a sequence.  Its units: IDLE ones for its start (queries,
// joining warps), then its tiles of UNIT keys.
template <int ROWS, int UNIT, int IDLE> struct Work {
  static constexpr int unit = UNIT, idle = IDLE, rows = ROWS;
static __device__ __forceinline__ bool item_of(const KvArgs& a, int n, Item& it) {
  int64_t b, e;
  if (a.cu == nullptr && a.N > 1) {
    b = n;
    e = n + 1;
  } else if (!seq_bounds(a.cu, n, a.T, a.status, b, e)) {
    return false;
  }
  if (e <= b) return false;
  const int len = a.pos0[n];
  if (len < 0 || len > (int64_t)a.max_pages * a.page) {
    set_status(a.status, GDN_ERR_DEVICE_INPUT);
    return false;
  }
  it.row0 = b;
  it.m = (int)(e - b);
  it.len = len;
  const int64_t lo = a.window > 0 ? (int64_t)len - it.m - a.window + 1 : 0;
  it.tile0 = lo > 0 ? (int)(lo / UNIT) : 0;
  it.tiles = (len + UNIT - 1) / UNIT - it.tile0;
  if (it.tiles < 1) it.tiles = 1;  // no key at all: a unit that sees nothing writes the zeros
  it.row_tiles = (int)(((int64_t)it.m * a.group + ROWS - 1) / ROWS);
  return true;
}
static __device__ __forceinline__ int64_t units_of(const KvArgs& a, const Item& it) {
  return (int64_t)(it.tiles + IDLE) * it.row_tiles * a.hkv;
}
};
// x / y for x >= 0, y > 0 (a quotient that fits an int)
__device__ __forceinline__ int quotient(int64_t x, int64_t y) {
  int q = (int)__fdividef((float)x, (float)y);
  while ((int64_t)q * y > x) --q;
  while ((int64_t)(q + 1) * y <= x) ++q;
  return q;
}
// x / group for the small x of a row tile (group_mul = 2^32 / group, rounded up)
__device__ __forceinline__ int over_group(const KvArgs& a, int x) {
  return a.group == 1 ? x : (int)__umulhi((uint32_t)x, a.group_mul);
}

// An item that ends in this CTA and began in CTA `first` before it (first < 0: there is none).
struct Desc {
  int64_t row0;                 // the sequence's first packed row
  int first, head, rows;        // kv head, live rows of the row tile
  int token0, rem;              // row r of the tile: token token0 + (rem + r) / group
  int unused;
};

// A CTA's run of units: [u, u1) of the line, `per` a CTA, beginning `off` units into sequence n.
struct Run {
  int64_t per, u, u1, off;
  int n;
};

// Finds this CTA's run (false: it has none) and clears its descriptor.  Sequences beyond a CTA's
// threads are walked twice: once for the total, once to find the run's start.
template <typename W, int THREADS = kAttThreads>
__device__ __forceinline__ bool plan_run(const KvArgs& a, int min_units, Desc* descs, Run& run) {
  __shared__ int64_t scan[THREADS / 32];
  __shared__ int64_t start_off;
  __shared__ int start_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  stream_order();
  int64_t total = 0, per = 0, u = 0;
  for (int pass = a.N <= THREADS; pass < 2; ++pass) {
    int64_t before = 0;
    for (int n0 = 0; n0 < a.N; n0 += THREADS) {
      Item it;
      const int n = n0 + tid;
      const int64_t w = n < a.N && W::item_of(a, n, it) ? W::units_of(a, it) : 0;
      int64_t s = w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += y;
      }
      if (lane == 31) scan[warp] = s;
      __syncthreads();
      int64_t all = 0;
#pragma unroll
      for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) s += scan[i];
        all += scan[i];
      }
      s += before;  // units up to and with sequence n
      before += all;
      if (n0 + THREADS >= a.N) total = before;
      if (pass) {
        if (per == 0) {
          // (a run may be a little longer than its share: the same in every CTA)
          per = (int64_t)((float)total * (1.000002f / (float)gridDim.x)) + 1;
          per = per > min_units ? per : min_units;
          u = blockIdx.x * per;
        }
        if (u < s && u >= s - w) {
          start_n = n;
          start_off = u - (s - w);
        }
      }
      __syncthreads();
    }
  }
  const int64_t u1 = u + per < total ? u + per : total;
  if (tid == 0) descs[blockIdx.x].first = -1;
  if (u >= u1) return false;
  run = Run{per, u, u1, start_off, start_n};
  return true;
}

// ---------------------------------------------------------------------------------- operands

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// four codes to two registers of fp16 pairs
template <bool E4M3>
__device__ __forceinline__ void open_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; "
        "cvt.rn.f16x2.e4m3x2 %1, b;}" : "=r"(lo), "=r"(hi) : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;  // code + 128; 0x6400 | u is 1024 + u
    const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x64806480u));
  }
}

__device__ __forceinline__ void load16(const float* p, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
    f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[8 * i + 2 * e] = __uint_as_float(u[e] << 16);
      f[8 * i + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                            *reinterpret_cast<const uint32_t*>(&y));
}

// A row of queries as fp16: times the power of two `down` that brings its largest magnitude into
// [2^14, 2^15), and `up` = 1 / down.  fp16's smallest step is then 2^-38 of that magnitude: bf16
// elements down to 2^-31 of it are exact, and smaller ones (or the second part of an fp32 one) are
// off by 2^-39 of it at most.
struct RowScale {
  float down, up;
};
__device__ __forceinline__ RowScale row_scale(float amax) {
  int ex = (int)((__float_as_uint(amax) >> 23) & 0xff);
  ex = ex == 0 ? 127 : min(max(ex, 16), 254);  // (both factors normal numbers)
  return RowScale{__uint_as_float((uint32_t)(254 + 14 - ex) << 23),
                  __uint_as_float((uint32_t)(ex - 14) << 23)};
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 open_half(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float log2_fast(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---------------------------------------------------------------------------------- the join

// Joins the partial results of the item that ended in CTA `cta` and began in CTA d.first before it.
// A thread takes four channels of a row and every `groups`-th partial, in CTA order; the groups
// join in shared memory, in order.  Columns (rows x D / 4) are spread over blockIdx.y.
constexpr int kJoinThreads = 256;
// A partial result's references and sum (o beside it).
struct alignas(16) Part {
  float m, x, sum, unused;
};
// 2^(M - X), what an o over its sum still lacks (an o of zeros may have any M)
__device__ __forceinline__ float value_scale(float m, float x) { return exp2_fast(fminf(m - x, 127.f)); }

template <typename IO, int D, int ROWS>
__device__ __forceinline__ void join_item(const KvArgs& a, const float* part_o,
                                          const Part* parts, int cta, const Desc& d, int groups,
                                          float4* so, Part* sml) {
  const int cols = kJoinThreads / groups, g = threadIdx.x / cols;
  const int col = blockIdx.y * cols + threadIdx.x % cols, row = col / (D / 4);
  const int dim = 4 * (col % (D / 4));
  const bool live = row < d.rows;
  const int count = live ? cta - d.first + 1 : 0;
  // CTA first + i left its part in its second slot where the item began there, else in its first
  const int64_t slot0 = 2 * (int64_t)d.first * ROWS + row;
  float m = kNone, mx = kNone, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = g; i < count; i += groups) {
    const int64_t slot = slot0 + (2 * i + (i == 0)) * ROWS;
    const Part ml = parts[slot];
    const float4 x = *reinterpret_cast<const float4*>(part_o + slot * D + dim);
    const float now = fmaxf(m, ml.m), f = exp2_fast(ml.m - now), k = exp2_fast(m - now);
    const float now_x = fmaxf(mx, ml.x);
    m = now;
    L = fmaf(ml.sum, exp2_fast(ml.x - now_x), L * exp2_fast(mx - now_x));
    mx = now_x;
    o.x = fmaf(x.x, f, o.x * k);
    o.y = fmaf(x.y, f, o.y * k);
    o.z = fmaf(x.z, f, o.z * k);
    o.w = fmaf(x.w, f, o.w * k);
  }
  if (groups > 1) {
    so[threadIdx.x] = o;
    sml[threadIdx.x] = Part{m, mx, L, 0.f};
    __syncthreads();
    if (g) return;
    for (int i = 1; i < groups; ++i) {
      m = fmaxf(m, sml[i * cols + threadIdx.x].m);
      mx = fmaxf(mx, sml[i * cols + threadIdx.x].x);
    }
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    L = 0.f;
    for (int i = 0; i < groups; ++i) {
      const Part ml = sml[i * cols + threadIdx.x];
      const float4 x = so[i * cols + threadIdx.x];
      const float f = exp2_fast(ml.m - m);
      L = fmaf(ml.sum, exp2_fast(ml.x - mx), L);
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    }
  }
  if (!live) return;
  const int tk = over_group(a, d.rem + row);
  const int64_t at =
      (d.row0 + d.token0 + tk) * a.hq + d.head * a.group + d.rem + row - tk * a.group;
  const float inv = L > 0.f ? 1.f / L : 0.f, up = value_scale(m, mx);
  store4(static_cast<IO*>(a.out) + at * D + dim,
         make_float4(o.x * inv * up, o.y * inv * up, o.z * inv * up, o.w * inv * up));
  if (a.lse && dim == 0) a.lse[at] = (mx + log2f(L)) * kLn2;
}

// SEVERAL: block blockIdx.x joins the items that ended in the CTAs blockIdx.x, + gridDim.x, ..;
// else the one that ended in CTA blockIdx.x, if any did.  (Six blocks an SM: 32 ragged sequences of
// up to 8192 keys are joined in 4.4 us so, in 4.8 with the compiler's own 48 registers; with
// SEVERAL, one sequence of 1500 keys takes 9.7 us with six, 9.5 without.)
template <typename IO, int D, int ROWS, bool SEVERAL>
__global__ void __launch_bounds__(kJoinThreads, SEVERAL ? 5 : 6)
kv_attention_join(KvArgs a, const float* part_o, const Part* parts, const Desc* descs, int ctas,
                  int groups) {
  __shared__ float4 so[kJoinThreads];
  __shared__ Part sml[kJoinThreads];
  stream_order();
  if constexpr (SEVERAL) {
    __shared__ int ending[kMaxCtas], items;
    if (threadIdx.x == 0) items = 0;
    __syncthreads();
    // (in any order: items do not depend on each other)
    for (int c = blockIdx.x + threadIdx.x * gridDim.x; c < ctas; c += kJoinThreads * gridDim.x)
      if (descs[c].first >= 0) ending[atomicAdd(&items, 1)] = c;
    __syncthreads();
    for (int i = 0; i < items; ++i) {
      const Desc d = descs[ending[i]];
      join_item<IO, D, ROWS>(a, part_o, parts, ending[i], d, groups, so, sml);
      __syncthreads();
    }
  } else {
    const Desc d = descs[blockIdx.x];
    if (d.first >= 0)
      join_item<IO, D, ROWS>(a, part_o, parts, (int)blockIdx.x, d, groups, so, sml);
  }
}

// --------------------------------------------------------------------------------- launching

struct Workspace {  // two partial results of each CTA, a descriptor of each
  float* part_o;
  Part* parts;
  Desc* descs;
  Workspace(const KvArgs& a, int rows) {
    part_o = a.workspace;
    parts = reinterpret_cast<Part*>(part_o + (int64_t)2 * kMaxCtas * rows * a.D);
    descs = reinterpret_cast<Desc*>(parts + (int64_t)2 * kMaxCtas * rows);
  }
  static size_t bytes(const KvArgs& a, int rows) {
    const size_t r = (size_t)2 * kMaxCtas * rows;
    return r * a.D * sizeof(float) + r * sizeof(Part) + kMaxCtas * sizeof(Desc);
  }
};

// as many CTAs as run together, or as the block table's width can give min_units units
template <typename W> int grid_ctas(const KvArgs& a, int resident, int min_units) {
  const int64_t row_tiles = (a.T + a.N - 1) / a.N * a.group / W::rows + 1;
  const int64_t most = (((int64_t)a.max_pages << a.page_shift) / W::unit + 1 + W::idle) * a.hkv *
                       a.N * row_tiles / min_units + 1;
  const int ctas = resident < kMaxCtas ? resident : kMaxCtas;
  return ctas < most ? ctas : (int)most;
}

template <typename IO, int D, int ROWS>
cudaError_t launch_join(const KvArgs& a, const Workspace& ws, int ctas, cudaStream_t s) {
  // Few long items: a block for each CTA would mostly find nothing to join, and setting those up
  // takes time (one sequence of 60000 keys, 2 kv heads: 27.1 us with a block a CTA, 19.8 with four
  // an item; 32 sequences of up to 8192 keys, 8 kv heads: 19.1 with a block a CTA, 20.7 with four an
  // item).
  const int64_t items = (int64_t)a.N * a.hkv, parts = ctas / items;
  const bool few = 4 * items < ctas;
  // An item has about `parts` partials where the sequences are alike, several times as many where
  // some are longer: four groups of threads for each and more from 16 partials on, so that a thread
  // takes a few.  Those 32 sequences take 19.1 us so, 21.8 with one group; four of 9000 keys and 24
  // rows 17.9, and 21.5 with groups for every partial.  Where most items have none (256 sequences of up
  // to 500 keys) more groups only cost blocks: 28.5 us with four, 27.6 with one.
  constexpr int all_cols = ROWS * (D / 4);
  int groups = all_cols < kJoinThreads ? kJoinThreads / all_cols : 1;
  while (groups < (few ? 64 : 16) && ((parts > 0 && groups < 4) || 4 * groups < parts)) groups *= 2;
  const auto go = [&](auto kern, int blocks) {
    return launch_ordered(kern, dim3(blocks, all_cols * groups / kJoinThreads), kJoinThreads, 0, s, a,
                          (const float*)ws.part_o, (const Part*)ws.parts,
                          (const Desc*)ws.descs, ctas, groups);
  };
  if (few) return go(kv_attention_join<IO, D, ROWS, true>, (int)(4 * items));
  return go(kv_attention_join<IO, D, ROWS, false>, ctas);
}

}  // namespace
}  // namespace gdn
