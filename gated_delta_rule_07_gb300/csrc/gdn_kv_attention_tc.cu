// gdn_kv_attention_tc.cu -- attention over the paged 8-bit cache where a kv head has more than eight
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
//   * One CTA an SM, its warps in three parts that hand steps to each other by mbarriers, each
//     buffer twice: eight warps load codes (a step ahead, in registers) and open them; eight turn
//     scores into weights; a thread of the first part issues the products, S^T of a step before
//     O^T of the last (a warp of its own would leave each thread 96 registers, not 128).
//     So opening, softmax and products of different steps run side by side.  (All in one part, two
//     CTAs an SM, took 2.5 times as long: each step's chain of waits in a row.)
// Work is cut as in the other kernel, in units of 128 keys.
#include "gdn_kv_attention.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kOpenWarps = 8, kSoftWarps = 8;
constexpr int kTcThreads = 32 * (kOpenWarps + kSoftWarps);
constexpr int kRows = 64;        // query rows of an item: columns of S^T and O^T
constexpr int kKeys = 128;       // keys of a step, lanes of S^T
constexpr int kTcMinUnits = 2;   // steps of a CTA at least
constexpr int kTcItemUnits = 3;  // steps that starting an item is worth
constexpr long long kWaitCycles = 2000000000LL;  // limit of a bounded wait: about a second
using TcWork = Work<kRows, kKeys, kTcItemUnits>;

struct TcSmem {  // byte offsets, each operand tile on a 1024-byte boundary
  static constexpr int tile = 128 * 128 * 2;
  static constexpr int K = 0;                 // 2 x [128 keys][D], 64-channel blocks
  static constexpr int V = K + 2 * tile;      // 2 x [128 channels][128 keys], 64-key blocks
  static constexpr int P = V + 2 * tile;      // 2 x [128 keys][64 rows]
  static constexpr int p_tile = 128 * 64 * 2;
  static constexpr int Q = P + 2 * p_tile;    // [64 rows][D], 64-channel blocks
  static constexpr int row_c = Q + 64 * 128 * 2;     // float2 {score scale, reference} of a row
  static constexpr int row_f = row_c + 64 * 8;       // float: rescaling of a row
  static constexpr int row_d = row_f + 64 * 4;       // float: a row's reference before its last move
  static constexpr int row_last = row_d + 64 * 4;    // int: the last key a row sees
  static constexpr int wmax = row_last + 64 * 4;     // float [4 quarters][64]
  static constexpr int bars = wmax + 4 * 64 * 4;     // mbarriers, two of each of the six below
  static constexpr int tmem = bars + 12 * 8;
  static constexpr int failed = tmem + 4;
  static constexpr int bytes = failed + 4 + 1024;    // (the base is rounded up to 1024)
  static constexpr int sums = K;  // float [64][129], at the end of an item
};
// The mbarriers of a buffer: its keys (values, weights) are in place; S^T is done, so the key tile
// is free again; O^T is done, so the value and weight tiles are; S^T has been read.
enum { kKeysIn = 0, kValuesIn = 2, kWeightsIn = 4, kScoresDone = 6, kSumDone = 8, kScoresRead = 10 };

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// sixteen columns of this warp's lanes, loaded and waited for
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  uint32_t none[16] = {};
  tmem_ld16_nw(taddr, r);
  tmem_wait_ld16x2(r, none);
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

template <int D, bool E4M3>
__global__ void __launch_bounds__(kTcThreads, 1)
kv_attention_tc_kernel(KvArgs a, float* part_o, float2* part_ml, Desc* descs) {
  constexpr int KC = D / 64, VC = D / 64;
  extern __shared__ char smem_raw[];
  Run run;
  if (!plan_run<TcWork, kTcThreads>(a, kTcMinUnits, descs, run)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  char* const sm = smem_raw + (base - raw);
  float2* const row_c = reinterpret_cast<float2*>(sm + TcSmem::row_c);
  float* const row_f = reinterpret_cast<float*>(sm + TcSmem::row_f);
  float* const row_d = reinterpret_cast<float*>(sm + TcSmem::row_d);
  int* const row_last = reinterpret_cast<int*>(sm + TcSmem::row_last);
  float* const wmax = reinterpret_cast<float*>(sm + TcSmem::wmax);
  volatile int* const failed = reinterpret_cast<volatile int*>(sm + TcSmem::failed);
  const uint32_t bars = base + TcSmem::bars;
  auto bar = [&](int which, uint32_t step) { return bars + 8 * (which + (step & 1)); };
  // a step's buffers are used every other step: the parity of its own use of a barrier
  auto parity = [](uint32_t step) { return (step >> 1) & 1; };

  if (warp == 0) {
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
      mbar_init(bars + 8 * (kScoresRead + b), kSoftWarps);
    }
    *failed = 0;
  }
  // (what the tiles hold past D or past the live rows only reaches lanes and columns of the products
  // that nobody reads)
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(sm + TcSmem::tmem);  // S^T, S^T, O^T

  uint32_t step0 = 0;  // steps of the items before this one
  int n = run.n;
  int64_t u = run.u, off = run.off;
  while (u < run.u1 && n < a.N && !*failed) {
    Item it;
    if (!TcWork::item_of(a, n, it) || off >= TcWork::units_of(a, it)) {
      ++n;
      off = 0;
      continue;
    }
    const int span = it.tiles + kTcItemUnits;
    const int which = quotient(off, span);
    const int at0 = (int)(off - (int64_t)which * span);
    const int at1 = (int)(span < at0 + (run.u1 - u) ? span : at0 + (run.u1 - u));
    const int64_t item_u = u - at0;
    u += at1 - at0;
    off += at1 - at0;
    const int ta = max(at0 - kTcItemUnits, 0), tb = max(at1 - kTcItemUnits, 0);
    if (ta >= tb) continue;
    const int head = (uint32_t)which / (uint32_t)it.row_tiles;
    const int row_base = (which - head * it.row_tiles) * kRows;
    const int rows = min(kRows, it.m * a.group - row_base);
    const int token0 = (uint32_t)row_base / (uint32_t)a.group, rem = row_base - token0 * a.group;

    // Page ids of a step's run of 16 keys.  The table's entry is loaded a step before it is looked
    // at.
    const int* table = a.table + (int64_t)n * a.max_pages;
    auto has_page = [&](int tile, int run16) {
      return tile < tb && (it.tile0 + tile) * kKeys + 16 * run16 < it.len;
    };
    auto entry_of = [&](int tile, int run16) {
      const int key = (it.tile0 + tile) * kKeys + 16 * run16;
      return has_page(tile, run16) ? __ldg(table + (key >> a.page_shift)) : -1;
    };
    auto page_of = [&](int entry, int tile, int run16) {  // -1: none
      if (!has_page(tile, run16)) return -1;
      if (entry >= 0 && entry < a.num_pages) return entry;
      if (lane == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
      return -1;
    };
    // keys that every live row sees: [all_lo, all_hi]
    const int all_hi = it.len - it.m + token0;
    const int64_t all_lo = a.window > 0 ? (int64_t)it.len - it.m + token0 +
                                              over_group(a, rem + rows - 1) - a.window + 1
                                        : INT64_MIN;
    const bool begins = ta == 0, ends = tb == it.tiles, whole = begins && ends;

    // queries: scaled by a power of two into [1, 2), fp16; a thread has 16 channels of a row
#pragma unroll 1
    for (int i = tid; i < kRows * (D / 16); i += kTcThreads) {
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
      int ex = (int)((__float_as_uint(amax) >> 23) & 0xff);
      ex = ex == 0 ? 127 : min(max(ex, 2), 252);
      const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
      if (chunk == 0) {
        // (a row that is not live has a reference that nothing exceeds: weights 0)
        row_c[row] = make_float2(__uint_as_float((uint32_t)ex << 23) * (a.scale * kLog2e),
                                 live ? kNone : -kNone);
        row_last[row] = live ? it.len - it.m + token0 + tk : -1;
      }
      const uint32_t at = base + TcSmem::Q + (chunk / 4) * (kRows * 128) + row * 128;
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
    __syncthreads();

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
      // The products, issued by one thread (of warp 0): S^T of a step, and O^T, begun or added to.
      auto issue_scores = [&](uint32_t step) {
        if (lane == 0) {
          wait_one(bar(kKeysIn, step), parity(step), failed);
          if (step >= 2) wait_one(bar(kScoresRead, step), parity(step - 2), failed);
          fence_after_sync();
          const uint32_t k = base + TcSmem::K + (step & 1) * TcSmem::tile;
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_ss(tm + 64 * (step & 1), sdesc(k + (s >> 2) * 16384 + (s & 3) * 32, 16, 1024),
                   sdesc(base + TcSmem::Q + (s >> 2) * (kRows * 128) + (s & 3) * 32, 16, 1024),
                   idesc_f16(128, 64, 0, 0), s > 0);
          mma_commit(bar(kScoresDone, step));
        }
        __syncwarp();
      };
      auto issue_sum = [&](uint32_t step, bool begin) {
        if (lane == 0) {
          wait_one(bar(kValuesIn, step), parity(step), failed);
          wait_one(bar(kWeightsIn, step), parity(step), failed);
          fence_after_sync();
          const uint32_t v = base + TcSmem::V + (step & 1) * TcSmem::tile;
          const uint32_t p = base + TcSmem::P + (step & 1) * TcSmem::p_tile;
#pragma unroll
          for (int s = 0; s < kKeys / 16; ++s)
            mma_ss(tm + 128, sdesc(v + (s >> 2) * 16384 + (s & 3) * 32, 16, 1024),
                   sdesc(p + s * 2048, 128 * 128, 1024), idesc_f16(128, 64, 0, 1), !begin || s > 0);
          mma_commit(bar(kSumDone, step));
        }
        __syncwarp();
      };
      uint4 kb[2][KC], vb[VC][2];
      int64_t from = 0;  // where the warp's keys, and its values, begin
      auto load_k = [&](int pid, int tile) {
        const int slot = ((it.tile0 + tile) * kKeys + 16 * warp) & (a.page - 1);
        from = ((int64_t)pid * a.hkv + head) * (a.page * D) + slot * D;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < KC; ++h)
            kb[j][h] = pid >= 0 ? ld_stream(kp + from + 8 * D * j + 64 * h)
                                : make_uint4(0u, 0u, 0u, 0u);
      };
      auto load_v = [&](int pid) {
#pragma unroll
        for (int i = 0; i < VC; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            vb[i][t] = pid >= 0 ? ld_stream(vp + from + 256 * i + 4 * D * t)
                                : make_uint4(0u, 0u, 0u, 0u);
      };
      {
        const int pid = page_of(entry_of(ta, warp), ta, warp);
        load_k(pid, ta);
        load_v(pid);
      }
      int entry = entry_of(ta + 1, warp);
      uint32_t step = step0;
      for (int tile = ta; tile < tb; ++tile, ++step) {
        const int first = (it.tile0 + tile) * kKeys;
        const int pid = page_of(entry, tile + 1, warp);
        entry = entry_of(tile + 2, warp);
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
            const uint32_t to = k_at + at + h * 16384 + j * 1024;
            sts16(to + k_c0, y[0], y[1], y[2], y[3]);
            sts16(to + k_c1, y[4], y[5], y[6], y[7]);
          }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kKeysIn, step));
        load_k(pid, tile + 1);
        if (warp == 0) issue_scores(step);
        if (E4M3 && first + kKeys > it.len) {  // bytes past the length: no NaN under weights of 0
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int keep = min(max(it.len - first - 16 * warp - 8 * g - 4 * t, 0), 4);
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
        load_v(pid);
        if (warp == 0 && tile > ta) issue_sum(step - 1, tile == ta + 1);
      }
      if (warp == 0) issue_sum(step - 1, tb == ta + 1);
    } else {
      // ------------------------------------------------------------------ scores to weights
      // Tensor Memory: lanes (keys, channels) 32 quarter + lane; columns (rows) 32 i + 16 half
      // + 0 .. 15
      const int sw = warp - kOpenWarps, quarter = sw & 3, half = sw >> 2;
      const int tm_lane = 32 * quarter + lane, own = 2 * quarter + (lane >> 4), st = 32 * sw + lane;
      const uint32_t tm_q = tm + ((uint32_t)(quarter * 32) << 16), tm_o = tm_q + 128;
      float l[kRows / 2];  // sums of the weights of this thread's key and rows
#pragma unroll
      for (int i = 0; i < kRows / 2; ++i) l[i] = 0.f;
      float ks = 0.f, vs = 0.f;  // this thread's key: its scales (vs < 0: it has no page)
      auto load_scales = [&](int pid) {
        const int64_t block = (int64_t)pid * a.hkv + head;
        ks = pid >= 0 ? __ldg(a.k_scale + block) : 0.f;
        vs = pid >= 0 ? __ldg(a.v_scale + block) : -1.f;
      };
      load_scales(page_of(entry_of(ta, own), ta, own));
      int entry = entry_of(ta + 1, own);
      uint32_t step = step0;
      for (int tile = ta; tile < tb; ++tile, ++step) {
        const int first = (it.tile0 + tile) * kKeys, key = first + tm_lane;
        const bool open = first + kKeys - 1 <= all_hi && first >= all_lo;
        const uint32_t tm_s = tm_q + 64 * (step & 1);
        const uint32_t p_at = base + TcSmem::P + (step & 1) * TcSmem::p_tile + tm_lane * 128;
        // a page of zero values weighs as 2^-100; keys without a page not at all
        const float k_now = ks;
        const float lv = vs > 0.f ? log2_fast(vs) : vs < 0.f ? -CUDART_INF_F : -100.f;
        const float rv = vs < 0.f ? 0.f : exp2_fast(-lv);
        load_scales(page_of(entry, tile + 1, own));
        entry = entry_of(tile + 2, own);
        if (step >= 2) wait_bar(bar(kSumDone, step), parity(step - 2), failed);  // (the weight tile)
        wait_bar(bar(kScoresDone, step), parity(step), failed);
        fence_after_sync();
        auto seen = [&](int la) {
          return key <= la && (a.window == 0 || (int64_t)key > (int64_t)la - a.window);
        };
        // A score above its row's reference by more than kSlack counts as kSlack here; if there is
        // one, its part is taken out of the sums again, the references move, and the weights are
        // formed once more (`again`), when only such scores are left to add to the sums.
        float top = 0.f;  // the largest score above its row's reference
        auto weights = [&](bool again) {
#pragma unroll
          for (int cc = 0; cc < kRows / 32; ++cc) {
            const int c = 2 * cc + half;
            if (16 * c >= rows) break;
            uint32_t s[16], p[8];
            tmem_ld16(tm_s + 16 * c, s);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float4 rc = *reinterpret_cast<const float4*>(row_c + 16 * c + i);
              float y0 = fmaf(__uint_as_float(s[i]), k_now * rc.x, lv - rc.y);
              float y1 = fmaf(__uint_as_float(s[i + 1]), k_now * rc.z, lv - rc.w);
              if (!open) {
                const int2 la = *reinterpret_cast<const int2*>(row_last + 16 * c + i);
                y0 = seen(la.x) ? y0 : -CUDART_INF_F;
                y1 = seen(la.y) ? y1 : -CUDART_INF_F;
              }
              top = fmaxf(top, fmaxf(y0, y1));
              const float w0 = exp2_fast(fminf(y0, kSlack)), w1 = exp2_fast(fminf(y1, kSlack));
              float &l0 = l[16 * cc + i], &l1 = l[16 * cc + i + 1];
              if (again) {
                // (the very comparison of the first time, against the reference of then)
                const float2 was = *reinterpret_cast<const float2*>(row_d + 16 * c + i);
                const float z0 = fmaf(__uint_as_float(s[i]), k_now * rc.x, lv - was.x);
                const float z1 = fmaf(__uint_as_float(s[i + 1]), k_now * rc.z, lv - was.y);
                l0 = y0 > -CUDART_INF_F && z0 > kSlack ? fmaf(w0, rv, l0) : l0;
                l1 = y1 > -CUDART_INF_F && z1 > kSlack ? fmaf(w1, rv, l1) : l1;
              } else {
                l0 = fmaf(w0, rv, l0);
                l1 = fmaf(w1, rv, l1);
              }
              p[i / 2] = pack_half(w0, w1);
            }
            sts16(p_at + (((2 * c) ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
            sts16(p_at + (((2 * c + 1) ^ (lane & 7)) << 4), p[4], p[5], p[6], p[7]);
          }
        };
        weights(false);
        if (soft_or(top > kSlack)) {
          // the rows' references move to this step's maxima; O^T of the last step has to be done
          // (that of this one waits for the weights)
          if (tile > ta) wait_bar(bar(kSumDone, step - 1), parity(step - 1), failed);
          fence_after_sync();
#pragma unroll
          for (int cc = 0; cc < kRows / 32; ++cc) {
            const int c = 2 * cc + half;
            if (16 * c >= rows) break;
            uint32_t s[16];
            tmem_ld16(tm_s + 16 * c, s);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 rc = row_c[16 * c + i];
              const bool in = seen(row_last[16 * c + i]);
              const float z = fmaf(__uint_as_float(s[i]), k_now * rc.x, lv - rc.y);
              if (in && z > kSlack) l[16 * cc + i] = fmaf(-exp2_fast(kSlack), rv, l[16 * cc + i]);
              float y = in ? fmaf(__uint_as_float(s[i]), k_now * rc.x, lv) : -CUDART_INF_F;
#pragma unroll
              for (int o = 16; o; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
              if (lane == 0) wmax[quarter * kRows + 16 * c + i] = y;
            }
          }
          soft_or(false);
          if (st < rows) {
            const float was = row_c[st].y;
            float m = was;
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, wmax[q * kRows + st] - kHead);
            row_f[st] = exp2_fast(was - m);
            row_d[st] = was;
            row_c[st].y = m;
          }
          soft_or(false);
#pragma unroll
          for (int cc = 0; cc < kRows / 32; ++cc) {
            const int c = 2 * cc + half;
            if (16 * c >= rows) break;
            uint32_t s[16];
            if (tile > ta) tmem_ld16(tm_o + 16 * c, s);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float f = 16 * c + i < rows ? row_f[16 * c + i] : 1.f;
              l[16 * cc + i] *= f;
              if (tile > ta) s[i] = __float_as_uint(__uint_as_float(s[i]) * f);
            }
            if (tile > ta) tmem_st16(tm_o + 16 * c, s);
          }
          weights(true);
        }
        fence_async_smem();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kWeightsIn, step));
          mbar_arrive(bar(kScoresRead, step));
        }
      }
      // the item's end: sums over the keys (threads), then o
      wait_bar(bar(kSumDone, step - 1), parity(step - 1), failed);
      fence_after_sync();
      float* const sums = reinterpret_cast<float*>(sm + TcSmem::sums);
#pragma unroll
      for (int cc = 0; cc < kRows / 32; ++cc)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * cc + 16 * half + i < rows)
            sums[(32 * cc + 16 * half + i) * 129 + tm_lane] = l[16 * cc + i];
      soft_or(false);
      const int64_t slot = 2 * (int64_t)blockIdx.x + (begins ? 1 : 0);
      if (st < rows) {
        float L = 0.f;
#pragma unroll 8
        for (int i = 0; i < kKeys; ++i) L += sums[st * 129 + i];
        const float m = row_c[st].y;
        row_f[st] = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
        if (!whole) {
          part_ml[slot * kRows + st] = make_float2(m, L);
        } else if (a.lse) {
          const int tk = over_group(a, rem + st);
          a.lse[(it.row0 + token0 + tk) * a.hq + head * a.group + rem + st - tk * a.group] =
              (m + log2f(L)) * kLn2;
        }
      }
      if (ends && !begins && st == 0) {
        Desc d;
        d.row0 = it.row0;
        d.first = quotient(item_u + kTcItemUnits, run.per);
        d.head = head;
        d.rows = rows;
        d.token0 = token0;
        d.rem = rem;
        d.unused = 0;
        descs[blockIdx.x] = d;
      }
      soft_or(false);
#pragma unroll 1
      for (int c = half; 16 * c < rows; c += 2) {  // this thread's channel, sixteen rows at a time
        uint32_t s[16];
        tmem_ld16(tm_o + 16 * c, s);
        if (tm_lane < D) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = 16 * c + i;
            if (row >= rows) break;
            const float o = __uint_as_float(s[i]) * row_f[row];
            if (whole) {
              const int tk = over_group(a, rem + row);
              const int64_t at =
                  (it.row0 + token0 + tk) * a.hq + head * a.group + rem + row - tk * a.group;
              static_cast<__nv_bfloat16*>(a.out)[at * D + tm_lane] = __float2bfloat16_rn(o);
            } else {
              part_o[(slot * kRows + row) * D + tm_lane] = o;
            }
          }
        }
        __syncwarp();
      }
      fence_before_sync();
    }
    step0 += tb - ta;
    __syncthreads();
    fence_after_sync();
  }
  if (tid == 0 && *failed) set_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tm, 256);
}

template <int D, bool E4M3>
cudaError_t launch_tc(const KvArgs& a, cudaStream_t s) {
  const auto kern = kv_attention_tc_kernel<D, E4M3>;
  static const cudaError_t ready =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem::bytes);
  if (ready != cudaSuccess) return ready;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ctas = grid_ctas<TcWork>(a, sms, kTcMinUnits);
  const Workspace ws(a, kRows);
  kern<<<ctas, kTcThreads, TcSmem::bytes, s>>>(a, ws.part_o, ws.part_ml, ws.descs);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<__nv_bfloat16, D, kRows>(a, ws, ctas, s);
}

}  // namespace

size_t kv_attention_tc_workspace(const KvArgs& a) { return Workspace::bytes(a, kRows); }

cudaError_t kv_attention_tc(const KvArgs& a, cudaStream_t s) {
  if (a.D == 64) return a.e4m3 ? launch_tc<64, true>(a, s) : launch_tc<64, false>(a, s);
  return a.e4m3 ? launch_tc<128, true>(a, s) : launch_tc<128, false>(a, s);
}

}  // namespace gdn
