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
//   * Codes are exact in fp16: int8 by way of 1024 + u in an fp16's mantissa, e4m3 by the
//     conversion instruction (its NaN codes, which only bytes past a length can hold, are taken out
//     of the values there; a weight of 0 would not hide them).  Queries are scaled by a power of two
//     per row to the top of fp16's range (row_scale).  Weights are rounded to fp16, 2^-11 each, an
//     eighth of what the output's rounding to bf16 costs; the weights' sum, which lse is made of,
//     takes them in fp32.  fp32 queries and weights are split into two fp16 parts, 22 bits.
//   * Softmax, one pass: the running maximum is of y = x log2 e + log2(value scale), so that the
//     weights w = 2^(y - M) already carry their page's value scale and stay in fp16's range
//     whatever the scales are; the sum takes w / value scale, on a reference of its own.  The
//     reference M follows the running maximum and only moves (and the sums are only rescaled) when
//     a tile exceeds it by 2^15: weights stay below that, fp16's range.
//   * Work.  Units of 16 keys, of all sequences, kv heads and row tiles in one line, cut into
//     equal runs, one a CTA: ragged lengths balance, one long sequence fills the GPU.  A CTA's
//     warps take its run's units in turn and join at the end of each item; items cut between CTAs
//     leave partial sums (M, sum, unnormalised o), joined in order by a second small kernel.
//
// Measured (GB300, device time; share of a copy's 6.80 TB/s), eight query heads a kv head unless said
// otherwise: 64 sequences of up to 65536 keys, 4 kv heads of 128: int8 585 us (94%), e4m3 563 us (98%:
// the conversion is one instruction; opened by shifts it was 726); 16 x 32768 keys 79 us (83%); fp32
// I/O, 16 x 30000 keys, 80 us (74%: twice the products, tensor pipe 29% busy, and 125 registers leave
// sixteen warps an SM to wait for the loads); 16 x 30000 keys, heads of 256, 8 rows 72 us (83%), 16
// rows 54 us for half the bytes (55%: registers leave two CTAs an SM); heads of 64 in pages of 16, 16 x
// 60000 keys, 82 us (72%: a warp's tile of 16 keys is 2 KB, so the softmax's instructions weigh twice
// as much a byte).  One sequence of 1500 keys takes 9.5 us and 32 ragged ones of up to 8192 19.1 us:
// launch, plan, an item's start and end, and the join are about 9 us of either.  A deeper ring of tiles
// in shared memory was slower (64 x 65536: 825 us, at any depth): its copies take more issue than the
// loads here.
#include "gdn_kv_attention.cuh"

namespace gdn {
namespace {

constexpr int kWarps = kAttWarps, kThreads = kAttThreads;
constexpr int kTile = 16;      // keys of a unit
// Units of a CTA at least: one sequence of 1500 keys takes 9.5 us with 8, 11.9 with 16, 16.3 with 32;
// with 4 it takes 8.7, but one of 8000 keys 12.7 us against 11.0 (more parts to join).
constexpr int kMinUnits = 8;
// Units that starting an item is worth (queries, joining warps): 32 ragged sequences of up to 8192
// keys take 19.2 us with 8, 19.9 with 16, 42.6 with 1.
constexpr int kItemUnits = 8;

// ---------------------------------------------------------------------------------- operands

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
  // Registers decide the resident CTAs: the sums alone are D NT / 4 of them.  Heads of 64 have small
  // tiles and need more warps for as many bytes on their way: 16 x 60000 keys, bf16, 82.6 us with
  // six CTAs an SM, 90.4 with five or four; fp32 (with spills at six), 16 x 30000: 54.1, 53.5, 56.5.
  // Heads of 128 spill with five: 64 x 65536 keys 782 us, 585 with four.
  static constexpr int ctas =
      D * NT <= 64 ? (SPLIT ? 5 : 6) : D * NT <= 128 ? 4 : D * NT <= 256 ? 3 : 2;
};

template <typename IO, int D, int NT, bool E4M3>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT, sizeof(IO) == 4>::ctas))
kv_attention_kernel(KvArgs a, float* part_o, Part* parts, Desc* descs) {
  constexpr bool SPLIT = sizeof(IO) == 4;
  using S = Shape<D, NT, SPLIT>;
  using W = Work<S::rows, kTile, kItemUnits>;
  constexpr int ROWS = S::rows, KC = D / 64, VC = D / 32, STEPS = D / 16;
  extern __shared__ __align__(16) char smem[];
  __shared__ float q_scale[ROWS], row_up[ROWS];
  __shared__ float2 warp_mx[kWarps][ROWS];
  __shared__ float warp_sum[kWarps][ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int r = lane >> 2, c = lane & 3;

  Run run;
  if (!plan_run<W>(a, kMinUnits, descs, run)) return;
  const int64_t per = run.per, u1 = run.u1;
  int64_t u = run.u, off = run.off;
  int n = run.n;
  while (u < u1 && n < a.N) {
    Item it;
    if (!W::item_of(a, n, it) || off >= W::units_of(a, it)) {
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
    auto has_page = [&](int tile) { return tile < tb && (it.tile0 + tile) * kTile < it.len; };
    auto entry_of = [&](int tile) {  // the table's entry, loaded a tile before it is looked at
      return has_page(tile) ? __ldg(table + ((it.tile0 + tile) * kTile >> a.page_shift)) : -1;
    };
    auto page_of = [&](int entry, int tile) {  // a tile's page id (-1: none; its keys are left out)
      if (!has_page(tile)) return -1;
      if (entry >= 0 && entry < a.num_pages) return entry;
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
    int tile = ta + warp;
    const int entry0 = entry_of(tile);
    int entry = entry_of(tile + kWarps), pid = page_of(entry0, tile);
    load_k(pid, tile);
    load_v(pid, tile);

    // queries: scaled by a power of two, fp16, in the order the products take them.  A thread has 16
    // dims of a row, 64 j + 16 cc on: lane (row % 8, cc)'s share of products 4 j .. 4 j + 3
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
      const RowScale rs = row_scale(amax);
      const float down = rs.down;
      if (chunk == 0) q_scale[row] = rs.up * (a.scale * kLog2e);
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

    // B, and the value scale below which it moves: any at first, until a page of values is met
    float base = 0.f, low = CUDART_INF_F;
    for (; tile < tb; tile += kWarps) {
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
      const float k_now = ks, v_now = vs;
      const int pid_next = page_of(entry, tile + kWarps);
      load_k(pid_next, tile + kWarps);
      entry = entry_of(tile + 2 * kWarps);

      // scores in log2, with the page's value scale (the same for the whole warp)
      float lv = log2_fast(v_now);
      if (v_now < low) {
        if (v_now < kLeastScale) {
          lv = base - kZero;
        } else {
          const float f = exp2_fast(lv - base);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (low < CUDART_INF_F) l[t][e] *= f;
              else M[t][e] += lv;
            }
          base = lv;
          low = fmaxf(v_now * exp2_fast(-kBelow), kLeastScale);
        }
      }
      const float rv = exp2_fast(base - lv);
      const int key = (it.tile0 + tile) * kTile + tok;
      const int first = (it.tile0 + tile) * kTile;
      const bool open = pid >= 0 && first + kTile - 1 <= all_hi && first >= all_lo;
      bool moves = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
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
        for (int e = 0; e < 2; ++e) moves |= fmaxf(s[t][e], s[t][e + 2]) > M[t][e] + kSlack;
      }
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[t][e], s[t][e + 2]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m - kHead, M[t][e]);
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
      if (E4M3 && !open) {  // bytes past the length: no NaN under their weights of 0
        const int keep = min(max(it.len - first - 4 * c, 0), 4);
        const uint32_t mask = keep == 4 ? 0xffffffffu : (1u << (8 * keep)) - 1u;
#pragma unroll
        for (int j = 0; j < VC; ++j) {
          vb[j].x &= mask;
          vb[j].y &= mask;
          vb[j].z &= mask;
          vb[j].w &= mask;
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
            for (int t = 0; t < NT; ++t) {
              mma16816(acc[t][2 * j + h], x[0], x[1], x[2], x[3], p[t][part][0], p[t][part][1]);
            }
        }
      }
      load_v(pid_next, tile + kWarps);
      pid = pid_next;
    }

    // join the warps: each leaves its references and sums, then its o on the common reference
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const float mx = M[t][e] - base;
        if (!(low < CUDART_INF_F)) M[t][e] = kNone;  // no values: o does not count
        if (r == 0) {
          warp_mx[warp][8 * t + 2 * c + e] = make_float2(M[t][e], mx);
          warp_sum[warp][8 * t + 2 * c + e] = x;
        }
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
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_mx[w][row].x);
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
      float m = kNone, mx = kNone, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        m = fmaxf(m, warp_mx[w][tid].x);
        mx = fmaxf(mx, warp_mx[w][tid].y);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        L = fmaf(warp_sum[w][tid], exp2_fast(warp_mx[w][tid].y - mx), L);
      q_scale[tid] = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
      row_up[tid] = whole ? value_scale(m, mx) : 1.f;
      if (!whole) {
        parts[slot * ROWS + tid] = Part{m, mx, L, 0.f};
      } else if (a.lse) {
        const int tk = over_group(a, rem + tid);
        a.lse[(it.row0 + token0 + tk) * a.hq + head * a.group + rem + tid - tk * a.group] =
            (mx + log2f(L)) * kLn2;
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
      const float inv = q_scale[row], up = row_up[row];
      o = make_float4(o.x * inv * up, o.y * inv * up, o.z * inv * up, o.w * inv * up);
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

// --------------------------------------------------------------------------------- launching

// rows of a kv head in the average sequence
int64_t average_rows(const KvArgs& a) { return (a.T + a.N - 1) / a.N * a.group; }

// More than sixteen rows: the tcgen05 kernel, where it is built.  int8, 4 kv heads of 128: 24
// sequences of 20000 keys with 8 .. 40 rows take 124 us there and 160 here, with 8 .. 64 rows 153 and
// 250, but with 8 or 16 rows 111 and 108; 16 x 20000 keys with 16 rows 75 and 69; one sequence of
// 1500 keys with 16 rows 13.0 and 9.4.  Heads of 64 gain less: 24 x 20000 keys with 8 .. 40 rows take 99
// us there and 106 here, 40 ragged sequences of up to 9000 keys with 8 .. 24 rows 29 and 23.
bool use_tc(const KvArgs& a) { return a.bf16 && a.D <= 128 && average_rows(a) > 16; }

// Tiles of 8 rows a warp carries: as many as the average sequence's rows fill (a row tile more
// reads the cache once more), within the registers (D NT <= 512).  16 x 30000 keys, 4 kv heads of
// 128, fp32: 8 rows take 80 us with one tile (two: 121); 16 rows 115 with two (one: 147, four: 210);
// 32 rows 194 with four (two: 216).
int row_tiles(const KvArgs& a) {
  const int64_t rows = average_rows(a);
  return rows <= 8 ? 1 : rows <= 16 || a.D == 256 ? 2 : 4;
}

template <typename IO, int D, int NT, bool E4M3>
cudaError_t launch(const KvArgs& a, cudaStream_t s) {
  using S = Shape<D, NT, sizeof(IO) == 4>;
  using W = Work<S::rows, kTile, kItemUnits>;
  const auto kern = kv_attention_kernel<IO, D, NT, E4M3>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, S::smem, ready);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ctas = grid_ctas<W>(a, sms * S::ctas, kMinUnits);
  const Workspace ws(a, S::rows);
  e = launch_ordered(kern, dim3(ctas), kThreads, S::smem, s, a, ws.part_o, ws.parts, ws.descs);
  if (e != cudaSuccess) return e;
  return launch_join<IO, D, S::rows>(a, ws, ctas, s);
}

template <typename IO, int D, bool E4M3>
cudaError_t launch_rows(const KvArgs& a, cudaStream_t s) {
  const int tiles = row_tiles(a);
  if (tiles == 1) return launch<IO, D, 1, E4M3>(a, s);
  if constexpr (D == 256) return launch<IO, D, 2, E4M3>(a, s);
  // (bf16 with more rows of smaller heads runs on tcgen05)
  else if constexpr (sizeof(IO) == 2) return launch<IO, D, 2, E4M3>(a, s);
  else return tiles == 2 ? launch<IO, D, 2, E4M3>(a, s) : launch<IO, D, 4, E4M3>(a, s);
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
  return use_tc(a) ? kv_attention_tc_workspace(a) : Workspace::bytes(a, 8 * row_tiles(a));
}

cudaError_t kv_attention(const KvArgs& a, cudaStream_t s) {
  if (use_tc(a)) return kv_attention_tc(a, s);
  if (a.bf16) return a.e4m3 ? launch_d<__nv_bfloat16, true>(a, s) : launch_d<__nv_bfloat16, false>(a, s);
  return a.e4m3 ? launch_d<float, true>(a, s) : launch_d<float, false>(a, s);
}

}  // namespace gdn
