// gdn_kv_attention_tc.cu -- attention over the paged 8-bit cache where a kv head has more than sixteen
// query rows a sequence (large groups, drafted tokens): bf16 I/O, D <= 128, on tcgen05.
//
// With few rows, opening a code costs more than using it, so here each code is opened once for up
// to 64 rows: a CTA takes 128 keys a step, writes them as fp16 operand tiles into shared memory and
// leaves the products to the tensor core,
//     S^T [128 keys x 64 rows] = K Q^T,      O^T [D x 64 rows] += V^T P^T,
// both with fp32 sums in Tensor Memory: keys (channels) are its 128 lanes, rows its columns.
//   * Operands are in the 128-byte-swizzle layout.  Keys: a lane opens 16 channels of a key (two
//     16-byte stores); values: two of the cache's words of four tokens open to eight neighbouring
//     keys of a channel (one 16-byte store), so neither needs a transpose.
//   * A thread is a key in the softmax (two warps share a key's rows): it has the key's scores, and
//     writes its weights as part of one operand row.  As in the kernel for few rows the reference
//     of the weights only moves when a step exceeds it; only then is the sum in Tensor Memory
//     rescaled.  The sums of the weights stay in the threads' registers until the item ends.
//   * One CTA an SM, its warps in four parts that hand steps to each other by mbarriers, each
//     buffer twice: eight warps load codes (a step ahead, in registers) and open them; eight turn
//     scores into weights; one thread issues the products, S^T of a step before O^T of the last;
//     one warp looks pages and scales up, a few steps ahead, for all of them.  So opening, softmax
//     and products of different steps run side by side, and each part's chain of instructions a
//     step, which is what bounds the kernel, is short.
// Work is cut as in the other kernel, in units of 128 keys.
//
// A step of 128 keys of 128 channels moves 32 KB of codes from HBM (1220 cycles at the SM's share of
// a copy's rate) and about 170 KB through shared memory (the opened tiles written and read again by
// the products, weights, queries: about 1350 cycles).  It takes about 2100: the opening warps wait
// some 650 of them for codes that were asked for a step ahead (a second step ahead does not fit 96
// registers a thread), and the products' issue takes 950, mostly for shared memory.
// Measured (GB300): 24 sequences of up to 20000 keys, 4 kv heads of 128, 8 .. 40 rows: 124 us (51% of
// the copy's rate; tensor pipe 21% busy; e4m3 122); 8 .. 64 rows 153 us; heads of 64, 99 us.  Bringing
// codes to L2 four steps ahead made 123, 152 and 98 us of an earlier form 119, 166 and 101: left out.
#include "gdn_kv_attention.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kOpenWarps = 8, kSoftWarps = 8;  // then one that issues, one that looks pages up
constexpr int kTcThreads = 32 * (kOpenWarps + kSoftWarps + 2);
constexpr int kAhead = 8;        // steps whose pages are known at a time
constexpr int kCols = 64;        // columns of S^T and O^T: an item's query rows, at most
constexpr int kKeys = 128;       // keys of a step, lanes of S^T
constexpr int kTcMinUnits = 2;   // steps of a CTA at least (4 x 9000 keys: 1 to 4 within 5%)
// Steps that starting an item is worth: 40 ragged sequences of up to 9000 keys, 8 .. 24 rows, heads
// of 64, take 29.5 us with 5, 35.5 with 3, 29.8 with 7; 24 x 20000 keys 124 us with any of them.
constexpr int kTcItemUnits = 5;
constexpr long long kWaitCycles = 2000000000LL;  // limit of a bounded wait: about a second

constexpr int kSumPad = 136;     // floats between rows of key sums (conflict-free)

struct TcSmem {  // byte offsets, each operand tile on a 1024-byte boundary
  static constexpr int tile = 128 * 128 * 2;
  static constexpr int K = 0;                 // 2 x [128 keys][D], 64-channel blocks
  static constexpr int V = K + 2 * tile;      // 2 x [128 channels][128 keys], 64-key blocks
  static constexpr int P = V + 2 * tile;      // 2 x [128 keys][64 rows]
  static constexpr int p_tile = 128 * 64 * 2;
  static constexpr int Q = P + 2 * p_tile;    // [64 rows][D], 64-channel blocks
  // float4 {a0, a1, b0, b1} of a pair of rows: score scale, minus the reference
  static constexpr int row_ab = Q + 64 * 128 * 2;
  static constexpr int row_f = row_ab + 64 * 8;      // float: rescaling of a row
  static constexpr int row_d = row_f + 64 * 4;       // float: minus a row's reference before it moved
  static constexpr int row_last = row_d + 64 * 4;    // int: the last key a row sees
  static constexpr int wmax = row_last + 64 * 4;     // float [4 quarters][64]
  static constexpr int runs = wmax + 4 * 64 * 4;     // PageRun [kAhead][8]
  static constexpr int bars = runs + kAhead * 8 * 32;  // mbarriers, see below
  static constexpr int tmem = bars + (10 + 2 * kAhead) * 8;
  static constexpr int failed = tmem + 4;
  static constexpr int item = failed + 4;            // ItemState
  static constexpr int bytes = item + 64 + 1024;     // (the base is rounded up to 1024)
  static constexpr int sums = K;  // float [rows][kSumPad], then [rows][D], at the end of an item
};
// A step's run of 16 keys, all within a page: where its codes begin (< 0: it has no page), its key
// scale, log2 of its value scale, 2^B over that scale.  And the same for all runs of the step: B,
// whether a page of values has been met, and 1, or where B moved (rare) what the sums so far are
// multiplied by (0: B is the first, and moves the references); 2^B over the scale is then given as 0,
// so that the step's weights reach the sums only when those have moved.
struct alignas(16) PageRun {
  int64_t from;
  float base;
  int valued;
  float ks, lv, rv, again;
};
// What the item loop needs again after an item (kept out of the registers in between).
struct ItemState {
  int64_t u, off, per, u1, row0, first_u;
  int n;
};
static_assert(sizeof(PageRun) == 32 && sizeof(ItemState) <= 64, "TcSmem");
// The mbarriers.  Two of each, for the steps that use a buffer in turn: its keys, values, weights
// are in place; S^T is done, so the key tile is free again; O^T is done, so the value and weight
// tiles are.  kAhead of each: S^T has been read (and the step's runs); the step's runs are in place.
enum { kKeysIn = 0, kValuesIn = 2, kWeightsIn = 4, kScoresDone = 6, kSumDone = 8 };
constexpr int kScoresRead = 10, kPagesIn = kScoresRead + kAhead;

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// sixteen columns of this warp's lanes, loaded and waited for
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// true in one thread of a converged warp
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// two fp32 in a 64-bit register: one instruction for both
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Bounded wait: sleeps in hardware; gives up after about a second, or when another thread has.
__device__ __forceinline__ void wait_one(uint32_t bar, uint32_t parity, volatile int* failed) {
  bool done = mbar_try(bar, parity);
  if (!done) {
    const long long began = clock64();
    while (!done && !*failed) {
      done = mbar_try(bar, parity);
      if (!done && clock64() - began > kWaitCycles) *failed = 1;
    }
  }
}
// the same for a warp
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, volatile int* failed) {
  wait_one(bar, parity, failed);
  __syncwarp();  // (Tensor Memory is read by converged warps)
}
// barrier of the softmax warps that also ORs a predicate
__device__ __forceinline__ bool soft_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 1, %2, p;\n"
      "selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r) : "r"((uint32_t)v), "n"(32 * kSoftWarps) : "memory");
  return r != 0;
}

// sixteen streamed bytes where `ok`, else zeros (without a branch, or a copy that would wait)
__device__ __forceinline__ void ld_stream_or_zero(uint4& v, const uint8_t* p, bool ok) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %5, 0;\nmov.b32 %0, 0;\nmov.b32 %1, 0;\nmov.b32 %2, 0;\n"
      "mov.b32 %3, 0;\n@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"((uint32_t)ok));
}
// the queries are in place: the softmax warps to the one that issues the products
__device__ __forceinline__ void queries_in() {
  asm volatile("barrier.cta.sync 2, %0;" ::"n"(32 * (kSoftWarps + 1)) : "memory");
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <int D, bool E4M3, int ROWS>
__global__ void __launch_bounds__(kTcThreads, 1)
kv_attention_tc_kernel(KvArgs a, float* part_o, Part* parts, Desc* descs) {
  using TcWork = Work<ROWS, kKeys, kTcItemUnits>;
  constexpr int KC = D / 64, VC = D / 64;
  extern __shared__ char smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  char* const sm = smem_raw + (base - raw);
  float4* const row_ab = reinterpret_cast<float4*>(sm + TcSmem::row_ab);
  float* const row_f = reinterpret_cast<float*>(sm + TcSmem::row_f);
  float* const row_d = reinterpret_cast<float*>(sm + TcSmem::row_d);
  int* const row_last = reinterpret_cast<int*>(sm + TcSmem::row_last);
  float* const wmax = reinterpret_cast<float*>(sm + TcSmem::wmax);
  PageRun* const runs = reinterpret_cast<PageRun*>(sm + TcSmem::runs);
  volatile ItemState* const state = reinterpret_cast<volatile ItemState*>(sm + TcSmem::item);
  volatile int* const failed = reinterpret_cast<volatile int*>(sm + TcSmem::failed);
  const uint32_t bars = base + TcSmem::bars;
  auto score_scale = [&](int row) -> float& {
    return reinterpret_cast<float*>(row_ab)[4 * (row >> 1) + (row & 1)];
  };
  auto minus_ref = [&](int row) -> float& {
    return reinterpret_cast<float*>(row_ab)[4 * (row >> 1) + 2 + (row & 1)];
  };
  auto bar = [&](int which, uint32_t step) { return bars + 8 * (which + (step & 1)); };
  auto read_bar = [&](uint32_t step) { return bars + 8 * (kScoresRead + step % kAhead); };
  auto pages_bar = [&](uint32_t step) { return bars + 8 * (kPagesIn + step % kAhead); };
  // a step's buffers are used every other step: the parity of its own use of a barrier
  auto parity = [](uint32_t step) { return (step >> 1) & 1; };
  auto parity_ahead = [](uint32_t step) { return (step / kAhead) & 1; };

  if (warp == kOpenWarps + kSoftWarps) {
    tmem_alloc(base + TcSmem::tmem, 256);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(bars + 8 * (kKeysIn + b), kOpenWarps);
      mbar_init(bars + 8 * (kValuesIn + b), kOpenWarps);
      mbar_init(bars + 8 * (kWeightsIn + b), kSoftWarps);
      mbar_init(bars + 8 * (kScoresDone + b), 1);
      mbar_init(bars + 8 * (kSumDone + b), 1);
    }
    for (int b = 0; b < kAhead; ++b) {
      mbar_init(bars + 8 * (kScoresRead + b), kSoftWarps);
      mbar_init(bars + 8 * (kPagesIn + b), 1);
    }
    *failed = 0;
  }
  // (what the tiles hold past D or past the live rows only reaches lanes and columns of the products
  // that nobody reads)
  fence_before_sync();
  {
    Run run = {};
    const bool any = plan_run<TcWork, kTcThreads>(a, kTcMinUnits, descs, run);
    if (tid == 0) {
      state->u = run.u;
      state->off = run.off;
      state->per = run.per;
      state->u1 = any ? run.u1 : run.u;  // (no units: nothing to do)
      state->n = run.n;
    }
  }
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(sm + TcSmem::tmem);  // S^T, S^T, O^T

  uint32_t step0 = 0;  // steps of the items before this one
  while (!*failed) {
    const int64_t u = state->u, off = state->off, u1 = state->u1;
    const int n = state->n;
    if (u >= u1 || n >= a.N) break;
    __syncthreads();  // (the state is read before it moves on)
    Item it;
    if (!TcWork::item_of(a, n, it) || off >= TcWork::units_of(a, it)) {
      if (tid == 0) {
        state->n = n + 1;
        state->off = 0;
      }
      __syncthreads();
      continue;
    }
    const int span = it.tiles + kTcItemUnits;
    const int which = quotient(off, span);
    const int at0 = (int)(off - (int64_t)which * span);
    const int at1 = (int)(span < at0 + (u1 - u) ? span : at0 + (u1 - u));
    const int ta = max(at0 - kTcItemUnits, 0), tb = max(at1 - kTcItemUnits, 0);
    if (tid == 32 * kOpenWarps) {  // (a softmax warp: those read it at the item's end)
      state->u = u + at1 - at0;
      state->off = off + at1 - at0;
      state->row0 = it.row0;
      state->first_u = u - at0 + kTcItemUnits;
    }
    if (ta >= tb) {
      __syncthreads();
      continue;
    }
    const int head = (uint32_t)which / (uint32_t)it.row_tiles;
    const int row_base = (which - head * it.row_tiles) * ROWS;
    const int rows = min(ROWS, it.m * a.group - row_base);
    const int token0 = (uint32_t)row_base / (uint32_t)a.group, rem = row_base - token0 * a.group;

    if (warp < kOpenWarps) {
      // ------------------------------------------------------------------ opening the codes
      // A warp opens sixteen keys.  Keys: a lane has key 8 j + r of them, channels 64 h + 16 c;
      // values: the eight keys from 8 g on, channels 64 i + 4 x .. + 3.  Eight neighbouring lanes
      // then write to eight different 16-byte columns (for the values with the channels' order
      // turned in every other pair of lanes), and read from two lines.
      const int r = lane >> 2, c4 = lane & 3, g = lane & 1, x = lane >> 1;
      const bool turn = x & 2;
      const uint32_t k_at = base + TcSmem::K + (16 * warp + r) * 128;
      const uint32_t k_c0 = ((2 * c4) ^ r) << 4, k_c1 = ((2 * c4 + 1) ^ r) << 4;
      const uint32_t v_at = base + TcSmem::V + (warp >> 2) * 16384 + 4 * x * 128;
      const int v_chunk = 2 * (warp & 3) + g, v_row = 4 * (x & 1);
      const uint8_t* const kp = a.k_codes + r * D + 16 * c4;
      const uint8_t* const vp = a.v_codes + 8 * g * D + 16 * x;
      uint4 kb[2][KC], vb[VC][2];
      auto load_k = [&](int64_t from, int j, int h) {
        ld_stream_or_zero(kb[j][h], kp + from + 8 * D * j + 64 * h, from >= 0);
      };
      auto load_v = [&](int64_t from, int i, int t) {
        ld_stream_or_zero(vb[i][t], vp + from + 256 * i + 4 * D * t, from >= 0);
      };
      auto from_of = [&](uint32_t step) {  // (once its pages are in)
        return *reinterpret_cast<volatile int64_t*>(&runs[step % kAhead * 8 + warp].from);
      };
      wait_bar(pages_bar(step0), parity_ahead(step0), failed);
      {
        const int64_t from = from_of(step0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < KC; ++h) load_k(from, j, h);
#pragma unroll
        for (int i = 0; i < VC; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) load_v(from, i, t);
      }
      // A register's codes of the next step are asked for as soon as this step's are taken.
      auto next_from = [&](int tile, uint32_t step) -> int64_t {
        if (tile >= tb) return -1;
        wait_bar(pages_bar(step), parity_ahead(step), failed);
        return from_of(step);
      };
      int64_t from = next_from(ta + 1, step0 + 1);
      uint32_t step = step0;
      for (int tile = ta; tile < tb; ++tile, ++step) {
        const uint32_t at = (step & 1) * TcSmem::tile;
        if (step >= 2) wait_bar(bar(kScoresDone, step), parity(step - 2), failed);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < KC; ++h) {
            uint32_t y[8];
            const uint4 w = kb[j][h];
            open_codes<E4M3>(w.x, y[0], y[1]);
            open_codes<E4M3>(w.y, y[2], y[3]);
            open_codes<E4M3>(w.z, y[4], y[5]);
            open_codes<E4M3>(w.w, y[6], y[7]);
            load_k(from, j, h);
            const uint32_t to = k_at + at + h * 16384 + j * 1024;
            sts16(to + k_c0, y[0], y[1], y[2], y[3]);
            sts16(to + k_c1, y[4], y[5], y[6], y[7]);
          }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kKeysIn, step));
        const int left = it.len - (it.tile0 + tile) * kKeys - 16 * warp;  // keys up to the length
        if (E4M3 && left < 16) {  // bytes past the length: no NaN under their weights of 0
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int keep = min(max(left - 8 * g - 4 * t, 0), 4);
            const uint32_t mask = keep == 4 ? 0xffffffffu : (1u << (8 * keep)) - 1u;
#pragma unroll
            for (int i = 0; i < VC; ++i) {
              vb[i][t].x &= mask;
              vb[i][t].y &= mask;
              vb[i][t].z &= mask;
              vb[i][t].w &= mask;
            }
          }
        }
        if (step >= 2) wait_bar(bar(kSumDone, step), parity(step - 2), failed);
#pragma unroll
        for (int i = 0; i < VC; ++i) {
          uint32_t w[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            w[t][0] = turn ? vb[i][t].z : vb[i][t].x;
            w[t][1] = turn ? vb[i][t].w : vb[i][t].y;
            w[t][2] = turn ? vb[i][t].x : vb[i][t].z;
            w[t][3] = turn ? vb[i][t].y : vb[i][t].w;
            load_v(from, i, t);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int ch = e ^ (turn ? 2 : 0);  // the channel of four that this store has
            uint32_t y[4];
            open_codes<E4M3>(w[0][e], y[0], y[1]);
            open_codes<E4M3>(w[1][e], y[2], y[3]);
            sts16(v_at + at + i * 8192 + ch * 128 + ((v_chunk ^ (v_row + ch)) << 4), y[0], y[1], y[2],
                  y[3]);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kValuesIn, step));
        from = next_from(tile + 2, step + 2);
      }
    } else if (warp < kOpenWarps + kSoftWarps) {
      // ------------------------------------------------------------------ scores to weights
      // Tensor Memory: lanes (keys, channels) 32 quarter + lane; columns (rows) 32 i + 16 half
      // + 0 .. 15
      const int sw = warp - kOpenWarps, quarter = sw & 3, half = sw >> 2;
      const int tm_lane = 32 * quarter + lane, own = 2 * quarter + (lane >> 4), st = 32 * sw + lane;
      const uint32_t tm_q = tm + ((uint32_t)(quarter * 32) << 16), tm_o = tm_q + 128;
      // queries: scaled by a power of two, fp16; a thread has 16 channels of a row
#pragma unroll 1
      for (int i = st; i < ROWS * (D / 16); i += 32 * kSoftWarps) {
        const int row = i / (D / 16), chunk = i % (D / 16);
        const int tk = over_group(a, rem + row), gq = rem + row - tk * a.group;
        const bool live = row < rows;
        float f[16], amax = 0.f;
        load16(static_cast<const __nv_bfloat16*>(a.q) + (it.row0 + (live ? token0 + tk : 0)) * a.q_ts +
                   (int64_t)(head * a.group + (live ? gq : 0)) * a.q_hs + 16 * chunk, f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          f[e] = live ? f[e] : 0.f;
          amax = fmaxf(amax, fabsf(f[e]));
        }
#pragma unroll
        for (int o = 1; o < D / 16; o <<= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const RowScale rs = row_scale(amax);
        const float down = rs.down;
        if (chunk == 0) {
          // (a row that is not live has a reference that nothing exceeds: weights 0)
          score_scale(row) = rs.up * (a.scale * kLog2e);
          minus_ref(row) = live ? -kNone : kNone;
          row_last[row] = live ? it.len - it.m + token0 + tk : -1;
        }
        const uint32_t at = base + TcSmem::Q + (chunk / 4) * (kCols * 128) + row * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = pack_half(f[8 * h + 2 * e] * down, f[8 * h + 2 * e + 1] * down);
          sts16(at + (((2 * (chunk % 4) + h) ^ (row & 7)) << 4), y[0], y[1], y[2], y[3]);
        }
      }
      fence_async_smem();
      queries_in();
      // keys that every live row sees: [all_lo, all_hi]
      const int all_hi = it.len - it.m + token0;
      const int64_t lo = (int64_t)all_hi + over_group(a, rem + rows - 1) - a.window + 1;
      const int all_lo = a.window > 0 && lo > 0 ? (int)lo : 0;
      uint64_t l[ROWS / 4];  // sums of the weights of this thread's key, two rows a register
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) l[i] = 0;
      uint32_t step = step0;
      for (int tile = ta; tile < tb; ++tile, ++step) {
        const int first = (it.tile0 + tile) * kKeys, key = first + tm_lane;
        const bool open = first + kKeys - 1 <= all_hi && first >= all_lo;
        const uint32_t tm_s = tm_q + 64 * (step & 1);
        const uint32_t p_at = base + TcSmem::P + (step & 1) * TcSmem::p_tile + tm_lane * 128;
        // S^T of this step is done, so is O^T of the one before the last (issued before it): the
        // weight tile is free.  The keys were in place before S^T was begun, so the pages were.
        wait_bar(bar(kScoresDone, step), parity(step), failed);
        fence_after_sync();
        const float4 run = *reinterpret_cast<const float4*>(&runs[step % kAhead * 8 + own].ks);
        const float ks = run.x, lv = run.y, rv = run.z;
        const uint64_t ks2 = pair(ks, ks), lv2 = pair(lv, lv);
        uint64_t rv2 = pair(rv, rv);
        auto seen = [&](int la) {
          return key <= la && (a.window == 0 || key > la - a.window);
        };
        // A score above its row's reference by more than kSlack counts as kSlack here; if there is
        // one, its part is taken out of the sums again, the references move, and the weights are
        // formed once more (`again`), when only such scores are left to add to the sums.
        float top = 0.f;  // the largest score above its row's reference
        auto weights = [&](bool again) {
#pragma unroll
          for (int cc = 0; cc < ROWS / 32; ++cc) {
            const int c = 2 * cc + half;
            if (16 * c >= rows) break;
            uint32_t s[16], p[8];
            tmem_ld16(tm_s + 16 * c, s);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const ulonglong2 ab = *reinterpret_cast<const ulonglong2*>(row_ab + 8 * c + i / 2);
              const uint64_t s2 = pair(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
              const uint64_t a2 = mul2(ks2, ab.x);
              float y0, y1;
              unpair(fma2(s2, a2, add2(lv2, ab.y)), y0, y1);
              if (!open) {
                const int2 la = *reinterpret_cast<const int2*>(row_last + 16 * c + i);
                y0 = seen(la.x) ? y0 : -CUDART_INF_F;
                y1 = seen(la.y) ? y1 : -CUDART_INF_F;
              }
              top = fmaxf(top, fmaxf(y0, y1));
              const float w0 = exp2_fast(fminf(y0, kSlack)), w1 = exp2_fast(fminf(y1, kSlack));
              uint64_t& l2 = l[8 * cc + i / 2];
              if (again) {
                // (the very comparison of the first time, against the reference of then)
                const uint64_t was = *reinterpret_cast<const uint64_t*>(row_d + 16 * c + i);
                float z0, z1;
                unpair(fma2(s2, a2, add2(lv2, was)), z0, z1);
                l2 = fma2(pair(y0 > -CUDART_INF_F && z0 > kSlack ? w0 : 0.f,
                               y1 > -CUDART_INF_F && z1 > kSlack ? w1 : 0.f), rv2, l2);
              } else {
                l2 = fma2(pair(w0, w1), rv2, l2);
              }
              p[i / 2] = pack_half(w0, w1);
            }
            sts16(p_at + (((2 * c) ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
            sts16(p_at + (((2 * c + 1) ^ (lane & 7)) << 4), p[4], p[5], p[6], p[7]);
          }
        };
        // (an item's first step has no reference yet: it goes straight there)
        const bool starts = tile == ta;
        if (!starts) weights(false);
        if (starts || soft_or(top > kSlack || run.w != 1.f)) {
          // the rows' references move to this step's maxima; O^T of the last step has to be done
          // (that of this one waits for the weights)
          float first_base = 0.f;
          if (run.w != 1.f) {  // B has moved (not in an item's first step)
            const float base = runs[step % kAhead * 8].base;
            if (run.w > 0.f) {
#pragma unroll
              for (int i = 0; i < ROWS / 4; ++i) l[i] = mul2(l[i], pair(run.w, run.w));
            } else {
              first_base = base;
            }
            const float x = lv > -CUDART_INF_F ? exp2_fast(base - lv) : 0.f;
            rv2 = pair(x, x);
          }
          const bool fresh = starts || run.w != 1.f;  // no weight of the step is in the sums
          if (!starts) wait_bar(bar(kSumDone, step - 1), parity(step - 1), failed);
          fence_after_sync();
#pragma unroll
          for (int cc = 0; cc < ROWS / 32; ++cc) {
            const int c = 2 * cc + half;
            if (16 * c >= rows) break;
            uint32_t s[16];
            tmem_ld16(tm_s + 16 * c, s);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const ulonglong2 ab = *reinterpret_cast<const ulonglong2*>(row_ab + 8 * c + i / 2);
              const int2 la = *reinterpret_cast<const int2*>(row_last + 16 * c + i);
              const uint64_t s2 = pair(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
              const uint64_t a2 = mul2(ks2, ab.x);
              float y0, y1, z0, z1;
              unpair(fma2(s2, a2, add2(lv2, ab.y)), z0, z1);
              unpair(fma2(s2, a2, lv2), y0, y1);
              const bool in0 = seen(la.x), in1 = seen(la.y);
              const float over = fresh ? 0.f : -exp2_fast(kSlack);
              l[8 * cc + i / 2] = fma2(pair(in0 && z0 > kSlack ? over : 0.f,
                                            in1 && z1 > kSlack ? over : 0.f), rv2, l[8 * cc + i / 2]);
              y0 = in0 ? y0 : -CUDART_INF_F;
              y1 = in1 ? y1 : -CUDART_INF_F;
              y0 = warp_max(y0);
              y1 = warp_max(y1);
              if (lane == 0) {
                wmax[quarter * ROWS + 16 * c + i] = y0;
                wmax[quarter * ROWS + 16 * c + i + 1] = y1;
              }
            }
          }
          soft_or(false);
          if (st < rows) {
            const float was = -minus_ref(st) + first_base;
            float m = was;
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, wmax[q * ROWS + st] - kHead);
            row_f[st] = exp2_fast(was - m);
            row_d[st] = -was;
            minus_ref(st) = -m;
          }
          soft_or(false);
#pragma unroll
          for (int cc = 0; cc < ROWS / 32; ++cc) {
            const int c = 2 * cc + half;
            if (16 * c >= rows) break;
            uint32_t s[16];
            if (!starts) tmem_ld16(tm_o + 16 * c, s);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float f0 = 16 * c + i < rows ? row_f[16 * c + i] : 1.f;
              const float f1 = 16 * c + i + 1 < rows ? row_f[16 * c + i + 1] : 1.f;
              l[8 * cc + i / 2] = mul2(l[8 * cc + i / 2], pair(f0, f1));
              if (!starts) {
                s[i] = __float_as_uint(__uint_as_float(s[i]) * f0);
                s[i + 1] = __float_as_uint(__uint_as_float(s[i + 1]) * f1);
              }
            }
            if (!starts) tmem_st16(tm_o + 16 * c, s);
          }
          weights(!fresh);
        }
        fence_async_smem();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kWeightsIn, step));
          mbar_arrive(read_bar(step));
        }
      }
      // the item's end: sums over the keys (threads), then o
      const bool begins = ta == 0, ends = tb == it.tiles, whole = begins && ends;
      const int64_t row0 = state->row0;
      const float base_now = runs[(step - 1) % kAhead * 8].base;
      const bool valued = runs[(step - 1) % kAhead * 8].valued;
      wait_bar(bar(kSumDone, step - 1), parity(step - 1), failed);
      fence_after_sync();
      float* const sums = reinterpret_cast<float*>(sm + TcSmem::sums);
#pragma unroll
      for (int cc = 0; cc < ROWS / 32; ++cc)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int row = 32 * cc + 16 * half + i;
          float l0, l1;
          unpair(l[8 * cc + i / 2], l0, l1);
          if (row < rows) sums[row * kSumPad + tm_lane] = l0;
          if (row + 1 < rows) sums[(row + 1) * kSumPad + tm_lane] = l1;
        }
      soft_or(false);
      const int64_t slot = 2 * (int64_t)blockIdx.x + (begins ? 1 : 0);
#pragma unroll 1
      for (int row = st >> 3; row < ROWS; row += 4 * kSoftWarps) {  // eight threads a row
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) L += sums[row * kSumPad + 8 * i + (st & 7)];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (row < rows && (st & 7) == 0) {
          const float m = -minus_ref(row), mx = m - base_now;
          row_f[row] = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
          if (!whole) {
            parts[slot * ROWS + row] = Part{valued ? m : kNone, mx, L, 0.f};
          } else if (a.lse) {
            const int tk = over_group(a, rem + row);
            a.lse[(row0 + token0 + tk) * a.hq + head * a.group + rem + row - tk * a.group] =
                (mx + log2f(L)) * kLn2;
          }
        }
      }
      if (ends && !begins && st == 0) {
        Desc d;
        d.row0 = row0;
        d.first = quotient(state->first_u, state->per);
        d.head = head;
        d.rows = rows;
        d.token0 = token0;
        d.rem = rem;
        d.unused = 0;
        descs[blockIdx.x] = d;
      }
      float* const o_at = sums + ROWS * kSumPad;  // [ROWS][D]
#pragma unroll 1
      for (int c = half; 16 * c < rows; c += 2) {  // this thread's channel, sixteen rows at a time
        uint32_t s[16];
        tmem_ld16(tm_o + 16 * c, s);
        if (tm_lane < D) {
#pragma unroll
          for (int i = 0; i < 16; ++i) o_at[(16 * c + i) * D + tm_lane] = __uint_as_float(s[i]);
        }
        __syncwarp();
      }
      soft_or(false);
      const float up = !whole ? 1.f : valued ? exp2_fast(base_now) : 0.f;
#pragma unroll 1
      for (int i = st; i < rows * (D / 4); i += 32 * kSoftWarps) {
        const int row = i / (D / 4), d = 4 * (i % (D / 4));
        float4 o = *reinterpret_cast<const float4*>(o_at + row * D + d);
        const float inv = row_f[row];
        o = make_float4(o.x * inv * up, o.y * inv * up, o.z * inv * up, o.w * inv * up);
        if (whole) {
          const int tk = over_group(a, rem + row);
          const int64_t at =
              (row0 + token0 + tk) * a.hq + head * a.group + rem + row - tk * a.group;
          store4(static_cast<__nv_bfloat16*>(a.out) + at * D + d, o);
        } else {
          *reinterpret_cast<float4*>(part_o + (slot * ROWS + row) * D + d) = o;
        }
      }
      fence_before_sync();
    } else if (warp == kOpenWarps + kSoftWarps) {
      // ------------------------------------------------------------------ the products
      queries_in();
      {
        const uint32_t id = idesc_f16(128, 64, 0, 0), id_pv = idesc_f16(128, 64, 0, 1);
        const uint64_t dk = sdesc(base + TcSmem::K, 16, 1024), dq = sdesc(base + TcSmem::Q, 16, 1024);
        const uint64_t dv = sdesc(base + TcSmem::V, 16, 1024);
        const uint64_t dp = sdesc(base + TcSmem::P, 128 * 128, 1024);
        const int steps = tb - ta;
        for (int i = 0; i <= steps; ++i) {
          const uint32_t step = step0 + i;
          if (i < steps) {  // S^T of this step
            wait_bar(bar(kKeysIn, step), parity(step), failed);
            if (step >= 2) wait_bar(read_bar(step - 2), parity_ahead(step - 2), failed);
            fence_after_sync();
            const uint64_t k = dk + (step & 1) * (TcSmem::tile >> 4);
            if (elected()) {
#pragma unroll
              for (int s = 0; s < D / 16; ++s)
                mma_ss(tm + 64 * (step & 1), k + (((s >> 2) * 16384 + (s & 3) * 32) >> 4),
                       dq + (((s >> 2) * (kCols * 128) + (s & 3) * 32) >> 4), id, s > 0);
              mma_commit(bar(kScoresDone, step));
            }
            __syncwarp();
          }
          if (i > 0) {  // O^T of the last
            const uint32_t prev = step - 1;
            wait_bar(bar(kValuesIn, prev), parity(prev), failed);
            wait_bar(bar(kWeightsIn, prev), parity(prev), failed);
            fence_after_sync();
            const uint64_t v = dv + (prev & 1) * (TcSmem::tile >> 4);
            const uint64_t p = dp + (prev & 1) * (TcSmem::p_tile >> 4);
            if (elected()) {
#pragma unroll
              for (int s = 0; s < kKeys / 16; ++s)
                mma_ss(tm + 128, v + (((s >> 2) * 16384 + (s & 3) * 32) >> 4), p + ((s * 2048) >> 4),
                       id_pv, i > 1 || s > 0);
              mma_commit(bar(kSumDone, prev));
            }
            __syncwarp();
          }
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ pages and scales
      // Four steps at a time, eight lanes each, a lane a run of 16 keys; the table's entries four
      // steps ahead of their scales' use.  (One step at a time the loads' latency is the warp's pace:
      // 132 us for 24 x 20000 keys when it was tried, 128 four at a time.)
      constexpr int kBatch = 4;
      const int* table = a.table + (int64_t)n * a.max_pages;
      const int mine = lane >> 3, at = 16 * (lane & 7);
      auto has_page = [&](int tile) { return tile < tb && (it.tile0 + tile) * kKeys + at < it.len; };
      auto entry_of = [&](int tile) {
        const int key = (it.tile0 + tile) * kKeys + at;
        return has_page(tile) ? __ldg(table + (key >> a.page_shift)) : -1;
      };
      int entry = entry_of(ta + mine);
      // B, and the value scale below which it moves: any at first, until a page of values is met
      float base = 0.f, low = CUDART_INF_F;
      uint32_t step = step0;
      for (int tile = ta; tile < tb; tile += kBatch, step += kBatch) {
        const int next = entry_of(tile + kBatch + mine);
        PageRun run;
        run.from = -1;
        run.ks = 0.f;
        float vs = 0.f;
        if (has_page(tile + mine)) {
          if (entry >= 0 && entry < a.num_pages) {
            const int64_t block = (int64_t)entry * a.hkv + head;
            const int slot = ((it.tile0 + tile + mine) * kKeys + at) & (a.page - 1);
            vs = __ldg(a.v_scale + block);
            run.from = block * (a.page * D) + slot * D;
            run.ks = __ldg(a.k_scale + block);
          } else {
            set_status(a.status, GDN_ERR_DEVICE_INPUT);
          }
        }
        entry = next;
        const bool zeros = !(vs >= kLeastScale);
        run.again = 1.f;
        run.base = base;
        run.valued = low < CUDART_INF_F;
        if (__any_sync(0xffffffffu, !zeros && vs < low)) {  // B, step by step
          float least = zeros ? CUDART_INF_F : vs;  // of the step's eight runs
#pragma unroll
          for (int o = 1; o < 8; o <<= 1)
            least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const float x = __shfl_sync(0xffffffffu, least, 8 * i);
            float again = 1.f;
            if (x < low) {
              const float lx = log2_fast(x);
              if (tile + i > ta)
                again = low < CUDART_INF_F ? fmaxf(exp2_fast(lx - base), kLeastScale) : 0.f;
              base = lx;
              low = fmaxf(x * exp2_fast(-kBelow), kLeastScale);
            }
            if (mine == i) {
              run.again = again;
              run.base = base;
              run.valued = low < CUDART_INF_F;
            }
          }
        }
        run.lv = zeros ? run.base - kZero : log2_fast(vs);
        run.rv = run.again == 1.f ? exp2_fast(run.base - run.lv) : 0.f;
        if (run.from < 0) {  // keys without a page weigh nothing
          run.lv = -CUDART_INF_F;
          run.rv = 0.f;
        }
        // the slots' last users: the softmax of kAhead steps before
        const int steps = min(kBatch, tb - tile);
        for (int i = 0; i < steps; ++i)
          if (step + i >= kAhead) wait_bar(read_bar(step + i), parity_ahead(step + i - kAhead), failed);
        if (mine < steps) runs[(step + mine) % kAhead * 8 + (lane & 7)] = run;
        __syncwarp();
        if (lane < steps) mbar_arrive(pages_bar(step + lane));
      }
    }
    step0 += tb - ta;
    __syncthreads();
    fence_after_sync();
  }
  if (tid == 0 && *failed) set_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
  fence_before_sync();
  __syncthreads();
  if (warp == kOpenWarps + kSoftWarps) tmem_dealloc(tm, 256);
}

template <int D, bool E4M3, int ROWS>
cudaError_t launch_tc(const KvArgs& a, cudaStream_t s) {
  using TcWork = Work<ROWS, kKeys, kTcItemUnits>;
  const auto kern = kv_attention_tc_kernel<D, E4M3, ROWS>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, TcSmem::bytes, ready);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ctas = grid_ctas<TcWork>(a, sms, kTcMinUnits);
  const Workspace ws(a, ROWS);
  e = launch_ordered(kern, dim3(ctas), kTcThreads, TcSmem::bytes, s, a, ws.part_o, ws.parts,
                     ws.descs);
  if (e != cudaSuccess) return e;
  return launch_join<__nv_bfloat16, D, ROWS>(a, ws, ctas, s);
}

// Rows of an item: 32 where the average sequence's rows of a kv head fit, which leaves the softmax's
// threads half the sums to hold; else 64 (a row tile more reads and opens the codes once more).
// 24 x 20000 keys with 22 rows on average take 124 us with 32 (145 with 64), with 36 rows 153 us with
// 64 (161 with 32).
int item_rows(const KvArgs& a) { return (a.T + a.N - 1) / a.N * a.group <= 32 ? 32 : 64; }

template <int D, bool E4M3>
cudaError_t launch_tc_rows(const KvArgs& a, cudaStream_t s) {
  return item_rows(a) == 32 ? launch_tc<D, E4M3, 32>(a, s) : launch_tc<D, E4M3, 64>(a, s);
}

}  // namespace

size_t kv_attention_tc_workspace(const KvArgs& a) { return Workspace::bytes(a, item_rows(a)); }

cudaError_t kv_attention_tc(const KvArgs& a, cudaStream_t s) {
  if (a.D == 64) return a.e4m3 ? launch_tc_rows<64, true>(a, s) : launch_tc_rows<64, false>(a, s);
  return a.e4m3 ? launch_tc_rows<128, true>(a, s) : launch_tc_rows<128, false>(a, s);
}

}  // namespace gdn
