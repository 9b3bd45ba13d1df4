// gdn_kv_attention.cu -- softmax attention of a few query tokens per sequence over the paged
// 8-bit cache.
//
// For query row i of sequence n (rows [cu[n], cu[n + 1]), the last one at the cache's last
// position kv_len[n] - 1) and query head h, over the keys j at or before the row's position (and
// within the window):
//     x_j = scale q . k_j,   o = sum_j softmax(x)_j v_j,   lse = log sum_j exp(x_j),
// kv head h / (hq / hkv).  A row that no key is left for gets o = 0 and lse = -inf.
//
// Bound by HBM: with g query heads a kv head and m rows, 2 D bytes of codes feed 4 g m D flops.
// The kernel streams the codes once, straight into registers:
//   * Products.  Rows (query tokens x the heads of a kv head) are the N = 8 side of
//     mma.m16n8k16 (fp16 operands, fp32 sums); keys are the M side of S^T = K Q^T and the channels
//     the M side of O^T = V^T P^T.  Every code is then needed by one lane of one warp: no shared
//     memory, no barrier, no copy in the way.  Which of a product's contraction indices a lane
//     holds is free as long as both operands agree, so a lane's 16 contiguous bytes of a key row
//     are its operands of four products (the queries are laid out to match), and the value
//     layout's words of four tokens are those of the second product; the weights get from the
//     first's result layout to the second's operand layout by an 8 x 8 transpose (movmatrix).
//   * Codes are exact in fp16: int8 by way of 1024 + u in an fp16's mantissa, e4m3 by moving its
//     bits (times 2^-8; no code becomes a NaN, so bytes past a length are harmless under a weight
//     of 0).  Queries are scaled by a power of two per row into fp16's range: exact for bf16; fp32
//     ones are split into two fp16 parts, and the weights too, for fp32 accuracy.
//   * Softmax, one pass: the running maximum is of y = x log2 e + log2(value scale), so that the
//     weights w = 2^(y - M) already carry their page's value scale and stay in fp16's range
//     whatever the scales are; the sum takes w / value scale.  The maximum only moves (and the
//     sums are only rescaled) when a tile exceeds it by 2^6: weights stay below 2^6.
//   * Work.  Units of 16 keys, of all sequences, kv heads and row tiles in one line, cut into
//     equal runs, one a CTA: ragged lengths balance, one long sequence fills the GPU.  A CTA's
//     warps take its run's units in turn and join at the end of each item; items cut between CTAs
//     leave partial sums (M, sum, unnormalised o), joined in order by a second small kernel.
#include <cuda_fp16.h>
#include <math_constants.h>

#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;      // keys of a unit
constexpr int kMinUnits = 16;  // units of a CTA at least
constexpr int kItemUnits = 8;  // units that starting an item is worth (queries, joining warps)
constexpr int kMaxCtas = 608;  // CTAs at most (the workspace holds two partial results of each)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 6.f;  // the maximum moves when exceeded by this (log2)
constexpr float kNone = -1e30f;  // the maximum before any key

// ------------------------------------------------------------------------------ the work plan

struct Item {          // what a sequence asks for
  int64_t row0;        // its first packed row
  int m, len;          // query rows (tokens), keys
  int tile0, tiles;    // units of 16 keys that some row sees
  int row_tiles;       // tiles of the m * group rows of a kv head
};

template <int ROWS>
__device__ __forceinline__ bool item_of(const KvArgs& a, int n, Item& it) {
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
  it.tile0 = lo > 0 ? (int)(lo / kTile) : 0;
  it.tiles = (len + kTile - 1) / kTile - it.tile0;
  if (it.tiles < 1) it.tiles = 1;  // no key at all: a unit that sees nothing writes the zeros
  it.row_tiles = (int)(((int64_t)it.m * a.group + ROWS - 1) / ROWS);
  return true;
}
// its units: an item (a kv head and row tile of it) is kItemUnits idle ones, then its tiles
__device__ __forceinline__ int64_t units_of(const KvArgs& a, const Item& it) {
  return (int64_t)(it.tiles + kItemUnits) * it.row_tiles * a.hkv;
}
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

// ---------------------------------------------------------------------------------- operands

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// four codes to two registers of fp16 pairs (int8: the codes; e4m3: the values times 2^-8)
template <bool E4M3>
__device__ __forceinline__ void open_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    const uint32_t x = __byte_perm(w, 0, 0x1404), y = __byte_perm(w, 0, 0x3424);
    lo = (x & 0x80008000u) | ((x >> 1) & 0x3f803f80u);
    hi = (y & 0x80008000u) | ((y >> 1) & 0x3f803f80u);
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

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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

// ------------------------------------------------------------------------------------ kernel

// NT: tiles of 8 rows that a warp carries.  SPLIT (fp32 I/O): queries and weights in two parts.
template <int D, int NT, bool SPLIT> struct Shape {
  static constexpr int rows = 8 * NT, parts = SPLIT ? 2 : 1;
  // queries stay in registers where they are few, else each product reads them from shared memory
  static constexpr bool q_regs = !SPLIT && D * NT <= 128;
  static constexpr int q_bytes = parts * rows * D * 2;
  static constexpr int pad = D + 4;  // floats of a row of partial sums (conflict-free)
  static constexpr int o_bytes = kWarps * rows * pad * 4;
  static constexpr int smem = q_bytes > o_bytes ? q_bytes : o_bytes;
  // registers decide the resident CTAs: the sums alone are D NT / 4 of them
  static constexpr int ctas = D * NT <= 128 ? 4 : D * NT <= 256 ? 3 : 2;
};

template <typename IO, int D, int NT, bool E4M3>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT, sizeof(IO) == 4>::ctas))
kv_attention_kernel(KvArgs a, float* part_o, float2* part_ml, Desc* descs) {
  constexpr bool SPLIT = sizeof(IO) == 4;
  using S = Shape<D, NT, SPLIT>;
  constexpr int ROWS = S::rows, KC = D / 64, VC = D / 32, STEPS = D / 16;
  extern __shared__ __align__(16) char smem[];
  __shared__ int64_t scan[kWarps];
  __shared__ int64_t start_off;
  __shared__ int start_n;
  __shared__ float q_scale[ROWS];
  __shared__ float2 warp_ml[kWarps][ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int r = lane >> 2, c = lane & 3;

  // the plan: all units, this CTA's run [u, u1) of them, the sequence that u falls into (sequences
  // beyond a CTA's threads are walked twice: once for the total, once to find the run's start)
  int64_t total = 0, per = 0, u = 0;
  for (int pass = a.N <= kThreads; pass < 2; ++pass) {
    int64_t before = 0;
    for (int n0 = 0; n0 < a.N; n0 += kThreads) {
      Item it;
      const int n = n0 + tid;
      const int64_t w = n < a.N && item_of<ROWS>(a, n, it) ? units_of(a, it) : 0;
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
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) s += scan[i];
        all += scan[i];
      }
      s += before;  // units up to and with sequence n
      before += all;
      if (n0 + kThreads >= a.N) total = before;
      if (pass) {
        if (per == 0) {
          // (a run may be a little longer than its share: the same in every CTA)
          per = (int64_t)((float)total * (1.000002f / (float)gridDim.x)) + 1;
          per = per > kMinUnits ? per : kMinUnits;
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
  asm volatile("griddepcontrol.launch_dependents;");
  if (u >= u1) return;

  int n = start_n;
  int64_t off = start_off;
  while (u < u1 && n < a.N) {
    Item it;
    if (!item_of<ROWS>(a, n, it) || off >= units_of(a, it)) {
      ++n;
      off = 0;
      continue;
    }
    // one item: kv head, row tile, and this CTA's tiles [ta, tb) of it
    const int span = it.tiles + kItemUnits;
    const int which = quotient(off, span);
    const int at0 = (int)(off - (int64_t)which * span);  // place in the item, idle units first
    const int at1 = (int)(span < at0 + (u1 - u) ? span : at0 + (u1 - u));
    const int64_t item_u = u - at0;
    u += at1 - at0;
    off += at1 - at0;
    const int ta = max(at0 - kItemUnits, 0), tb = max(at1 - kItemUnits, 0);
    if (ta >= tb) continue;
    const int head = (uint32_t)which / (uint32_t)it.row_tiles;
    const int row_base = (which - head * it.row_tiles) * ROWS;
    const int rows = min(ROWS, it.m * a.group - row_base);  // live rows of the tile
    // row r of the tile is token token0 + (rem + r) / group, query head head group + the remainder
    const int token0 = (uint32_t)row_base / (uint32_t)a.group, rem = row_base - token0 * a.group;

    // the first tiles are on their way before the queries are
    const int* table = a.table + (int64_t)n * a.max_pages;
    auto page_of = [&](int tile) {  // a tile's page id (-1: none; its keys are left out)
      const int key = (it.tile0 + tile) * kTile;
      if (tile >= tb || key >= it.len) return -1;
      const int pid = __ldg(table + (key >> a.page_shift));
      if (pid >= 0 && pid < a.num_pages) return pid;
      if (lane == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
      return -1;
    };
    uint4 kb[2][KC], vb[VC];
    float ks = 0.f, vs = 0.f;
    // key rows of the lane: tokens 4 (r / 2) + r % 2 and two on, so that the first product's
    // result rows are the tokens whose weights the second's operand words hold
    const int tok = 4 * (r >> 1) + (r & 1);
    const uint8_t* const kp = a.k_codes + tok * D + 16 * c;
    const uint8_t* const vp = a.v_codes + 4 * c * D + 16 * r;
    auto bytes_of = [&](int pid, int tile) {  // where the tile's keys and its values begin
      const int slot = ((it.tile0 + tile) * kTile) & (a.page - 1);
      return ((int64_t)pid * a.hkv + head) * (a.page * D) + slot * D;
    };
    auto load_k = [&](int pid, int tile) {
      if (pid < 0) return;
      const uint8_t* p = kp + bytes_of(pid, tile);
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        kb[0][j] = ld_stream(p + 64 * j);
        kb[1][j] = ld_stream(p + 2 * D + 64 * j);
      }
      const int64_t block = (int64_t)pid * a.hkv + head;
      ks = __ldg(a.k_scale + block);
      vs = __ldg(a.v_scale + block);
    };
    auto load_v = [&](int pid, int tile) {
      if (pid < 0) return;
      const uint8_t* p = vp + bytes_of(pid, tile);
#pragma unroll
      for (int j = 0; j < VC; ++j) vb[j] = ld_stream(p + 128 * j);
    };
#pragma unroll
    for (int j = 0; j < KC; ++j) kb[0][j] = kb[1][j] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < VC; ++j) vb[j] = make_uint4(0, 0, 0, 0);
    int tile = ta + warp, pid = page_of(tile), pid_next = page_of(tile + kWarps);
    load_k(pid, tile);
    load_v(pid, tile);

    // queries: scaled by a power of two into [1, 2), fp16, in the order the products take them.  A
    // thread has 16 dims of a row, 64 j + 16 cc on: lane (row % 8, cc)'s share of products 4 j ..
    // 4 j + 3
#pragma unroll 1
    for (int i = tid; i < ROWS * STEPS; i += kThreads) {
      const int row = i / STEPS, chunk = i % STEPS;
      const int tk = over_group(a, rem + row), gq = rem + row - tk * a.group;
      const bool live = row < rows;
      const IO* q = static_cast<const IO*>(a.q) + (it.row0 + (live ? token0 + tk : 0)) * a.q_ts +
                    (int64_t)(head * a.group + (live ? gq : 0)) * a.q_hs + 16 * chunk;
      float f[16], amax = 0.f;
      load16(q, f);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        f[e] = live ? f[e] : 0.f;
        amax = fmaxf(amax, fabsf(f[e]));
      }
      // (the row's threads are neighbours; whole warps run here: ROWS STEPS is a multiple of 32)
#pragma unroll
      for (int o = 1; o < STEPS; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      int ex = (int)((__float_as_uint(amax) >> 23) & 0xff);
      ex = ex == 0 ? 127 : min(max(ex, 2), 252);
      const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
      if (chunk == 0) q_scale[row] = __uint_as_float((uint32_t)ex << 23) * (a.scale * kLog2e);
      uint4* at = reinterpret_cast<uint4*>(smem) +
                  ((row / 8) * (STEPS / 2) + 2 * (chunk / 4)) * 32 + 4 * (row % 8) + chunk % 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = f[8 * h + 2 * e] * down, y = f[8 * h + 2 * e + 1] * down;
          hi[e] = pack_half(x, y);
          const float2 z = open_half(hi[e]);
          lo[e] = pack_half(x - z.x, y - z.y);
        }
        at[32 * h] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (SPLIT)
          at[ROWS * D / 8 + 32 * h] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    __syncthreads();
    uint4 qr[S::q_regs ? NT : 1][S::q_regs ? STEPS / 2 : 1];
    if constexpr (S::q_regs) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < STEPS / 2; ++s)
          qr[t][s] = reinterpret_cast<const uint4*>(smem)[(t * (STEPS / 2) + s) * 32 + lane];
    }
    // this lane's columns: rows 8 t + 2 c + e, the last key each sees, its scale
    int last[NT][2];
    float qs[NT][2], M[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * t + 2 * c + e;
        last[t][e] = row < rows ? it.len - it.m + token0 + over_group(a, rem + row) : -1;
        qs[t][e] = q_scale[row];
        M[t][e] = kNone;
        l[t][e] = 0.f;
      }
    // keys that every row sees: [all_lo, all_hi] (none where some row is not live)
    const int all_hi = rows == ROWS ? it.len - it.m + token0 : -1;
    const int64_t all_lo = a.window > 0 ? (int64_t)it.len - it.m + token0 +
                                              over_group(a, rem + rows - 1) - a.window + 1
                                        : INT64_MIN;
    float acc[NT][2 * VC][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2 * VC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][i][e] = 0.f;

    for (; tile < tb; tile += kWarps) {
      const int pid_after = page_of(tile + 2 * kWarps);
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&kb[0][j]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&kb[1][j]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // two products of the four in 16 bytes
          uint32_t x[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            open_codes<E4M3>(w0[2 * h + i], x[i][0], x[i][2]);
            open_codes<E4M3>(w1[2 * h + i], x[i][1], x[i][3]);
          }
#pragma unroll
          for (int part = 0; part < S::parts; ++part)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              uint4 q;
              if constexpr (S::q_regs)
                q = qr[t][2 * j + h];
              else
                q = reinterpret_cast<const uint4*>(smem + part * ROWS * D * 2)
                    [(t * (STEPS / 2) + 2 * j + h) * 32 + lane];
              mma16816(s[t], x[0][0], x[0][1], x[0][2], x[0][3], q.x, q.y);
              mma16816(s[t], x[1][0], x[1][1], x[1][2], x[1][3], q.z, q.w);
            }
        }
      }
      const float k_now = ks * (E4M3 ? 256.f : 1.f), v_now = vs * (E4M3 ? 256.f : 1.f);
      load_k(pid_next, tile + kWarps);

      // scores in log2, with the page's value scale; a page of zero values weighs as 2^-100
      const float lv = v_now > 0.f ? log2_fast(v_now) : -100.f;
      const float rv = exp2_fast(-lv);
      const int key = (it.tile0 + tile) * kTile + tok;
      const int first = (it.tile0 + tile) * kTile;
      const bool open = pid >= 0 && first + kTile - 1 <= all_hi && first >= all_lo;
      bool moves = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = fmaf(s[t][e], k_now * qs[t][e & 1], lv);
          if (!open) {
            const int kk = key + (e & 2), la = last[t][e & 1];
            const bool seen = pid >= 0 && kk <= la && (a.window == 0 || (int64_t)kk > (int64_t)la - a.window);
            y = seen ? y : -CUDART_INF_F;
          }
          s[t][e] = y;
        }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) moves |= fmaxf(s[t][e], s[t][e + 2]) > M[t][e] + kSlack;
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[t][e], s[t][e + 2]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m, M[t][e]);
            const float f = exp2_fast(M[t][e] - m);
            M[t][e] = m;
            l[t][e] *= f;
#pragma unroll
            for (int i = 0; i < 2 * VC; ++i) {
              acc[t][i][e] *= f;
              acc[t][i][e + 2] *= f;
            }
          }
      }
      uint32_t p[NT][S::parts][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = exp2_fast(s[t][e] - M[t][e & 1]);
          l[t][e & 1] = fmaf(w[e], rv, l[t][e & 1]);
        }
        const uint32_t h0 = pack_half(w[0], w[1]), h1 = pack_half(w[2], w[3]);
        p[t][0][0] = transpose8x8(h0);
        p[t][0][1] = transpose8x8(h1);
        if constexpr (SPLIT) {
          const float2 x = open_half(h0), y = open_half(h1);
          p[t][1][0] = transpose8x8(pack_half(w[0] - x.x, w[1] - x.y));
          p[t][1][1] = transpose8x8(pack_half(w[2] - y.x, w[3] - y.y));
        }
      }
#pragma unroll
      for (int j = 0; j < VC; ++j) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&vb[j]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[4];
          open_codes<E4M3>(w[2 * h], x[0], x[2]);
          open_codes<E4M3>(w[2 * h + 1], x[1], x[3]);
#pragma unroll
          for (int part = 0; part < S::parts; ++part)
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma16816(acc[t][2 * j + h], x[0], x[1], x[2], x[3], p[t][part][0], p[t][part][1]);
        }
      }
      load_v(pid_next, tile + kWarps);
      pid = pid_next;
      pid_next = pid_after;
    }

    // join the warps: each leaves its maxima and sums, then its o on the common maximum
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (r == 0) warp_ml[warp][8 * t + 2 * c + e] = make_float2(M[t][e], x);
      }
    __syncthreads();  // (the queries in shared memory are no longer needed either)
    float* so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * t + 2 * c + e;
        float m = M[t][e];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_ml[w][row].x);
        const float f = exp2_fast(M[t][e] - m);
#pragma unroll
        for (int j = 0; j < VC; ++j)
          *reinterpret_cast<float4*>(so + (warp * ROWS + row) * S::pad + 32 * j + 4 * r) =
              make_float4(acc[t][2 * j][e] * f, acc[t][2 * j][e + 2] * f,
                          acc[t][2 * j + 1][e] * f, acc[t][2 * j + 1][e + 2] * f);
      }
    const bool begins = ta == 0, ends = tb == it.tiles, whole = begins && ends;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (begins ? 1 : 0);
    if (tid < rows) {  // the rows' sums
      float m = kNone, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_ml[w][tid].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        L = fmaf(warp_ml[w][tid].y, exp2_fast(warp_ml[w][tid].x - m), L);
      q_scale[tid] = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
      if (!whole) {
        part_ml[slot * ROWS + tid] = make_float2(m, L);
      } else if (a.lse) {
        const int tk = over_group(a, rem + tid);
        a.lse[(it.row0 + token0 + tk) * a.hq + head * a.group + rem + tid - tk * a.group] =
            (m + log2f(L)) * kLn2;
      }
    }
    if (ends && !begins && tid == 0) {
      Desc d;
      d.row0 = it.row0;
      d.first = quotient(item_u + kItemUnits, per);
      d.head = head;
      d.rows = rows;
      d.token0 = token0;
      d.rem = rem;
      d.unused = 0;
      descs[blockIdx.x] = d;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = 4 * (i % (D / 4));
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(so + (w * ROWS + row) * S::pad + d);
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
      }
      const float inv = q_scale[row];
      o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (whole) {
        const int tk = over_group(a, rem + row);
        const int64_t at =
            (it.row0 + token0 + tk) * a.hq + head * a.group + rem + row - tk * a.group;
        store4(static_cast<IO*>(a.out) + at * D + d, o);
      } else {
        *reinterpret_cast<float4*>(part_o + (slot * ROWS + row) * D + d) = o;
      }
    }
    __syncthreads();
  }
}

// Joins the partial results of the item that ended in CTA blockIdx.x and began in an earlier one.
// A thread takes four channels of a row and every `groups`-th partial, in CTA order; the groups
// join in shared memory, in order.  Columns (rows x D / 4) are spread over blockIdx.y.
constexpr int kJoinThreads = 256;
template <typename IO, int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join(KvArgs a, const float* part_o,
                                                                  const float2* part_ml,
                                                                  const Desc* descs, int groups) {
  constexpr int ROWS = 8 * NT;
  __shared__ float4 so[kJoinThreads];
  __shared__ float2 sml[kJoinThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Desc d = descs[blockIdx.x];
  if (d.first < 0) return;
  const int cols = kJoinThreads / groups, g = threadIdx.x / cols;
  const int col = blockIdx.y * cols + threadIdx.x % cols, row = col / (D / 4);
  const int dim = 4 * (col % (D / 4));
  const bool live = row < d.rows;
  const int count = live ? (int)blockIdx.x - d.first + 1 : 0;
  // CTA first + i left its part in its second slot where the item began there, else in its first
  const int64_t slot0 = 2 * (int64_t)d.first * ROWS + row;
  float m = kNone, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = g; i < count; i += groups) {
    const int64_t slot = slot0 + (2 * i + (i == 0)) * ROWS;
    const float2 ml = part_ml[slot];
    const float4 x = *reinterpret_cast<const float4*>(part_o + slot * D + dim);
    const float now = fmaxf(m, ml.x), f = exp2_fast(ml.x - now), k = exp2_fast(m - now);
    m = now;
    L = fmaf(ml.y, f, L * k);
    o.x = fmaf(x.x, f, o.x * k);
    o.y = fmaf(x.y, f, o.y * k);
    o.z = fmaf(x.z, f, o.z * k);
    o.w = fmaf(x.w, f, o.w * k);
  }
  if (groups > 1) {
    so[threadIdx.x] = o;
    sml[threadIdx.x] = make_float2(m, L);
    __syncthreads();
    if (g) return;
    for (int i = 1; i < groups; ++i) m = fmaxf(m, sml[i * cols + threadIdx.x].x);
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    L = 0.f;
    for (int i = 0; i < groups; ++i) {
      const float2 ml = sml[i * cols + threadIdx.x];
      const float4 x = so[i * cols + threadIdx.x];
      const float f = exp2_fast(ml.x - m);
      L = fmaf(ml.y, f, L);
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
  const float inv = L > 0.f ? 1.f / L : 0.f;
  store4(static_cast<IO*>(a.out) + at * D + dim,
         make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (a.lse && dim == 0) a.lse[at] = (m + log2f(L)) * kLn2;
}

// --------------------------------------------------------------------------------- launching

// Tiles of 8 rows a warp carries: as many as the average sequence's rows of a kv head fill (a row
// tile more reads the cache once more), within the registers (D NT <= 512).
int row_tiles(const KvArgs& a) {
  const int64_t rows = (a.T + a.N - 1) / a.N * a.group;
  return rows <= 8 ? 1 : rows <= 16 || a.D == 256 ? 2 : 4;
}

template <typename IO, int D, int NT, bool E4M3>
cudaError_t launch(const KvArgs& a, cudaStream_t s) {
  using S = Shape<D, NT, sizeof(IO) == 4>;
  const auto kern = kv_attention_kernel<IO, D, NT, E4M3>;
  static const cudaError_t ready =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem);
  if (ready != cudaSuccess) return ready;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // as many CTAs as run together, or as the block table's width can give kMinUnits units
  const int64_t rows = (a.T + a.N - 1) / a.N * a.group / S::rows + 1;
  const int64_t most = (((int64_t)a.max_pages << a.page_shift) / kTile + kItemUnits) * a.hkv * a.N *
                       rows / kMinUnits + 1;
  int ctas = sms * S::ctas < kMaxCtas ? sms * S::ctas : kMaxCtas;
  if (ctas > most) ctas = (int)most;
  float* part_o = a.workspace;
  float2* part_ml = reinterpret_cast<float2*>(part_o + (int64_t)2 * kMaxCtas * S::rows * D);
  Desc* descs = reinterpret_cast<Desc*>(part_ml + (int64_t)2 * kMaxCtas * S::rows);
  kern<<<ctas, kThreads, S::smem, s>>>(a, part_o, part_ml, descs);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // launched while the first kernel drains; it waits for its end before it reads anything
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // partials of an item, if the sequences are alike: a thread takes about eight of them
  const int64_t parts = ctas / ((int64_t)a.N * a.hkv);
  constexpr int all_cols = S::rows * (D / 4);
  int groups = all_cols < kJoinThreads ? kJoinThreads / all_cols : 1;
  while (groups < 16 && 8 * groups < parts) groups *= 2;
  cfg.gridDim = dim3(ctas, all_cols * groups / kJoinThreads);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attention_join<IO, D, NT>, a, (const float*)part_o,
                            (const float2*)part_ml, (const Desc*)descs, groups);
}

template <typename IO, int D, bool E4M3>
cudaError_t launch_rows(const KvArgs& a, cudaStream_t s) {
  switch (row_tiles(a)) {
    case 1: return launch<IO, D, 1, E4M3>(a, s);
    case 2: return launch<IO, D, 2, E4M3>(a, s);
    default:
      if constexpr (D <= 128) return launch<IO, D, 4, E4M3>(a, s);
      else return launch<IO, D, 2, E4M3>(a, s);
  }
}
template <typename IO, bool E4M3>
cudaError_t launch_d(const KvArgs& a, cudaStream_t s) {
  switch (a.D) {
    case 64: return launch_rows<IO, 64, E4M3>(a, s);
    case 128: return launch_rows<IO, 128, E4M3>(a, s);
    default: return launch_rows<IO, 256, E4M3>(a, s);
  }
}

}  // namespace

size_t kv_attention_workspace(const KvArgs& a) {
  const size_t rows = (size_t)2 * kMaxCtas * 8 * row_tiles(a);
  return rows * a.D * sizeof(float) + rows * sizeof(float2) + kMaxCtas * sizeof(Desc);
}

cudaError_t kv_attention(const KvArgs& a, cudaStream_t s) {
  if (a.bf16) return a.e4m3 ? launch_d<__nv_bfloat16, true>(a, s) : launch_d<__nv_bfloat16, false>(a, s);
  return a.e4m3 ? launch_d<float, true>(a, s) : launch_d<float, false>(a, s);
}

}  // namespace gdn
