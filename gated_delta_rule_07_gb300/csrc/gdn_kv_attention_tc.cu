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
//   * A thread is a key in the softmax: it has the key's scores of all rows, and writes its row of
//     weights as one operand row.  As in the kernel for few rows the reference of the weights only
//     moves when a step exceeds it; only then is the sum in Tensor Memory rescaled.  The sums of the weights
//     stay in the threads' registers until the item ends.
//   * The next step's codes are loaded into registers while this one's products run; two CTAs an SM
//     fill each other's waits.
// Work is cut as in the other kernel, in units of 128 keys.
#include "gdn_kv_attention.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kRows = 64;        // query rows of an item: columns of S^T and O^T
constexpr int kKeys = 128;       // keys of a step, lanes of S^T
constexpr int kTcMinUnits = 2;   // steps of a CTA at least
constexpr int kTcItemUnits = 2;  // steps that starting an item is worth
constexpr int kTcCtas = 2;       // resident CTAs of an SM
constexpr long long kWaitCycles = 2000000000LL;  // limit of a bounded wait: about a second
using TcWork = Work<kRows, kKeys, kTcItemUnits>;

struct TcSmem {  // byte offsets, each operand tile on a 1024-byte boundary
  static constexpr int K = 0;                   // [128 keys][D], 64-channel blocks
  static constexpr int V = K + 128 * 128 * 2;   // [128 channels][128 keys], 64-key blocks
  static constexpr int P = V + 128 * 128 * 2;   // [128 keys][64 rows]
  static constexpr int Q = P + 128 * 64 * 2;    // [64 rows][D], 64-channel blocks
  static constexpr int row_c = Q + 64 * 128 * 2;     // float2 {score scale, maximum} of a row
  static constexpr int row_f = row_c + 64 * 8;       // float: rescaling of a row
  static constexpr int row_last = row_f + 64 * 4;    // int: the last key a row sees
  static constexpr int wmax = row_last + 64 * 4;     // float [4 warps][64]
  static constexpr int bar_s = wmax + 4 * 64 * 4;    // mbarriers: S^T done, O^T done
  static constexpr int bar_o = bar_s + 8;
  static constexpr int tmem = bar_o + 8;
  static constexpr int failed = tmem + 4;
  static constexpr int bytes = failed + 4 + 1024;    // (the base is rounded up to 1024)
  static constexpr int sums = K;  // float [64][129], at the end of an item
};

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
// bounded wait: sleeps in hardware, gives up after about a second
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
  const long long began = clock64();
  bool done = mbar_try(bar, parity);
  while (!done && clock64() - began <= kWaitCycles) done = mbar_try(bar, parity);
  __syncwarp();  // (Tensor Memory is read by converged warps)
  return done;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kAttThreads, kTcCtas)
kv_attention_tc_kernel(KvArgs a, float* part_o, float2* part_ml, Desc* descs) {
  constexpr int KC = D / 64, VC = D / 32;
  extern __shared__ char smem_raw[];
  Run run;
  if (!plan_run<TcWork>(a, kTcMinUnits, descs, run)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  char* const sm = smem_raw + (base - raw);
  float2* const row_c = reinterpret_cast<float2*>(sm + TcSmem::row_c);
  float* const row_f = reinterpret_cast<float*>(sm + TcSmem::row_f);
  int* const row_last = reinterpret_cast<int*>(sm + TcSmem::row_last);
  float* const wmax = reinterpret_cast<float*>(sm + TcSmem::wmax);
  volatile int* const failed = reinterpret_cast<volatile int*>(sm + TcSmem::failed);
  const uint32_t bar_s = base + TcSmem::bar_s, bar_o = base + TcSmem::bar_o;

  if (warp == 0) {
    tmem_alloc(base + TcSmem::tmem, 128);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(bar_s, 1);
    mbar_init(bar_o, 1);
    *failed = 0;
  }
  // (what the tiles hold past D or past the live rows only reaches lanes and columns of the products
  // that nobody reads)
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(sm + TcSmem::tmem);
  const uint32_t tm_s = tm + ((uint32_t)(warp * 32) << 16), tm_o = tm_s + 64;
  const uint32_t id = idesc_f16(128, 64, 0, 0), id_pv = idesc_f16(128, 64, 0, 1);
  uint32_t phase_s = 0, phase_o = 0;

  // a lane's places.  Keys: key 8 j + r of the warp's 32, channels 64 h + 16 c; values: the eight
  // keys from 8 g on of the warp's 32, channels 32 i + 4 x .. + 3.  Eight neighbouring lanes then
  // write to eight different 16-byte columns, and read from two lines of keys, four of values.
  const int r = lane >> 2, c4 = lane & 3, g = lane & 3, x = lane >> 2;
  const uint32_t k_at = base + TcSmem::K + (32 * warp + r) * 128;
  const uint32_t k_c0 = ((2 * c4) ^ r) << 4, k_c1 = ((2 * c4 + 1) ^ r) << 4;
  const uint32_t v_at = base + TcSmem::V + (warp >> 1) * 16384 + 4 * x * 128;
  const int v_chunk = 4 * (warp & 1) + g, v_row = 4 * (x & 1);
  const uint8_t* const kp = a.k_codes + r * D + 16 * c4;
  const uint8_t* const vp = a.v_codes + 8 * (g & 1) * D + 16 * x;

  int n = run.n;
  int64_t u = run.u, off = run.off;
  bool ok = true;
  while (u < run.u1 && n < a.N && ok) {
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

    const int* table = a.table + (int64_t)n * a.max_pages;
    // the warp's 32 keys are two runs of 16, each within a page: the page ids (-1: none)
    auto page_of = [&](int tile, int half) {
      const int key = (it.tile0 + tile) * kKeys + 32 * warp + 16 * half;
      if (tile >= tb || key >= it.len) return -1;
      const int pid = __ldg(table + (key >> a.page_shift));
      if (pid >= 0 && pid < a.num_pages) return pid;
      if (lane == 0) set_status(a.status, GDN_ERR_DEVICE_INPUT);
      return -1;
    };
    auto bytes_of = [&](int pid, int tile, int half) {
      const int slot = ((it.tile0 + tile) * kKeys + 32 * warp + 16 * half) & (a.page - 1);
      return ((int64_t)pid * a.hkv + head) * (a.page * D) + slot * D;
    };
    uint4 kb[4][KC], vb[VC][2];
    float ks = 0.f, lv = 0.f;  // this thread's key: its scale, log2 of its value scale
    int pid[2];
    auto load_k = [&](int tile) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = pid[j >> 1];
        const uint8_t* at = kp + bytes_of(p, tile, j >> 1) + 8 * (j & 1) * D;
#pragma unroll
        for (int h = 0; h < KC; ++h)
          kb[j][h] = p >= 0 ? ld_stream(at + 64 * h) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto load_v = [&](int tile) {
      const int p = g & 2 ? pid[1] : pid[0];
      const uint8_t* at = vp + bytes_of(p, tile, g >> 1);
#pragma unroll
      for (int i = 0; i < VC; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          vb[i][t] = p >= 0 ? ld_stream(at + 128 * i + 4 * D * t) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto load_scales = [&] {
      const int p = lane & 16 ? pid[1] : pid[0];
      const int64_t block = (int64_t)p * a.hkv + head;
      ks = p >= 0 ? __ldg(a.k_scale + block) : 0.f;
      const float vs = p >= 0 ? __ldg(a.v_scale + block) : 0.f;
      // a page of zero values weighs as 2^-100; keys without a page not at all
      lv = p < 0 ? -CUDART_INF_F : vs > 0.f ? log2_fast(vs) : -100.f;
    };
    int tile = ta;
    pid[0] = page_of(tile, 0);
    pid[1] = page_of(tile, 1);
    load_k(tile);
    load_v(tile);
    load_scales();

    // queries: scaled by a power of two into [1, 2), fp16; a thread has 16 channels of a row
#pragma unroll 1
    for (int i = tid; i < kRows * (D / 16); i += kAttThreads) {
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
        // (a row that is not live has a maximum that nothing exceeds: weights 0)
        row_c[row] = make_float2(__uint_as_float((uint32_t)ex << 23) * (a.scale * kLog2e),
                                 live ? kNone : -kNone);
        row_last[row] = live ? it.len - it.m + token0 + tk : -1;
      }
      const uint32_t at = base + TcSmem::Q + (chunk / 4) * (kRows * 128) + row * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = pack_half(f[8 * h + 2 * e] * down, f[8 * h + 2 * e + 1] * down);
        sts16(at + (((2 * (chunk % 4) + h) ^ (row & 7)) << 4), x[0], x[1], x[2], x[3]);
      }
    }
    float l[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) l[i] = 0.f;
    // keys that every live row sees: [all_lo, all_hi]
    const int all_hi = it.len - it.m + token0;
    const int64_t all_lo = a.window > 0 ? (int64_t)it.len - it.m + token0 +
                                              over_group(a, rem + rows - 1) - a.window + 1
                                        : INT64_MIN;

    for (; tile < tb && ok; ++tile) {
      const int first = (it.tile0 + tile) * kKeys, key = first + tid;
      const bool open = first + kKeys - 1 <= all_hi && first >= all_lo;
      const int pid_next[2] = {page_of(tile + 1, 0), page_of(tile + 1, 1)};
      // the keys (their tile is free: every thread saw the last step's S^T done)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < KC; ++h) {
          uint32_t x[8];
          const uint4 w = kb[j][h];
          open_codes<E4M3>(w.x, x[0], x[1]);
          open_codes<E4M3>(w.y, x[2], x[3]);
          open_codes<E4M3>(w.z, x[4], x[5]);
          open_codes<E4M3>(w.w, x[6], x[7]);
          const uint32_t at = k_at + h * 16384 + j * 1024;
          sts16(at + k_c0, x[0], x[1], x[2], x[3]);
          sts16(at + k_c1, x[4], x[5], x[6], x[7]);
        }
      fence_async_smem();
      fence_before_sync();
      __syncthreads();
      if (tid == 0) {
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_ss(tm, sdesc(base + TcSmem::K + (s >> 2) * 16384 + (s & 3) * 32, 16, 1024),
                 sdesc(base + TcSmem::Q + (s >> 2) * (kRows * 128) + (s & 3) * 32, 16, 1024), id,
                 s > 0);
        mma_commit(bar_s);
      }
      __syncwarp();
      const float ks_now = ks, lv_now = lv;
      const float rv = exp2_fast(lv_now == -CUDART_INF_F ? 0.f : -lv_now);
      // the values, once the last step's O^T is done with their tile (and the weights')
      if (tile > ta) {
        ok = wait_bar(bar_o, phase_o);
        phase_o ^= 1;
      }
      if (E4M3 && !open) {  // bytes past the length: no NaN under their weights of 0
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int keep = min(max(it.len - first - 32 * warp - 8 * g - 4 * t, 0), 4);
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
#pragma unroll
      for (int i = 0; i < VC; ++i) {
        const uint32_t w0[4] = {vb[i][0].x, vb[i][0].y, vb[i][0].z, vb[i][0].w};
        const uint32_t w1[4] = {vb[i][1].x, vb[i][1].y, vb[i][1].z, vb[i][1].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t o[4];
          open_codes<E4M3>(w0[e], o[0], o[1]);
          open_codes<E4M3>(w1[e], o[2], o[3]);
          sts16(v_at + i * 4096 + e * 128 + ((v_chunk ^ (v_row + e)) << 4), o[0], o[1], o[2], o[3]);
        }
      }
      pid[0] = pid_next[0];
      pid[1] = pid_next[1];
      load_k(tile + 1);
      load_v(tile + 1);
      load_scales();

      // scores to weights: this thread's key, all rows
      ok = wait_bar(bar_s, phase_s) && ok;
      phase_s ^= 1;
      fence_after_sync();
      auto seen = [&](int la) {
        return key <= la && (a.window == 0 || (int64_t)key > (int64_t)la - a.window);
      };
      float top = 0.f;  // the largest score above its row's maximum
#pragma unroll
      for (int c = 0; c < kRows / 16; ++c) {
        if (16 * c >= rows) break;
        uint32_t s[16];
        tmem_ld16(tm_s + 16 * c, s);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float4 rc = *reinterpret_cast<const float4*>(row_c + 16 * c + i);
          float y0 = fmaf(__uint_as_float(s[i]), ks_now * rc.x, lv_now - rc.y);
          float y1 = fmaf(__uint_as_float(s[i + 1]), ks_now * rc.z, lv_now - rc.w);
          if (!open) {
            const int2 la = *reinterpret_cast<const int2*>(row_last + 16 * c + i);
            y0 = seen(la.x) ? y0 : -CUDART_INF_F;
            y1 = seen(la.y) ? y1 : -CUDART_INF_F;
          }
          top = fmaxf(top, fmaxf(y0, y1));
        }
      }
      if (!ok) *failed = 1;
      if (__syncthreads_or(top > kSlack)) {
        // the rows' maxima move to this step's
#pragma unroll
        for (int c = 0; c < kRows / 16; ++c) {
          if (16 * c >= rows) break;
          uint32_t s[16];
          tmem_ld16(tm_s + 16 * c, s);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y = fmaf(__uint_as_float(s[i]), ks_now * row_c[16 * c + i].x, lv_now);
            y = seen(row_last[16 * c + i]) ? y : -CUDART_INF_F;
#pragma unroll
            for (int o = 16; o; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
            if (lane == 0) wmax[warp * kRows + 16 * c + i] = y;
          }
        }
        __syncthreads();
        if (tid < rows) {
          const float was = row_c[tid].y;
          float m = was;
#pragma unroll
          for (int w = 0; w < kAttWarps; ++w) m = fmaxf(m, wmax[w * kRows + tid] - kHead);
          row_f[tid] = exp2_fast(was - m);
          row_c[tid].y = m;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kRows / 16; ++c) {
          if (16 * c >= rows) break;
          uint32_t s[16];
          if (tile > ta) tmem_ld16(tm_o + 16 * c, s);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float f = 16 * c + i < rows ? row_f[16 * c + i] : 1.f;
            l[16 * c + i] *= f;
            if (tile > ta) s[i] = __float_as_uint(__uint_as_float(s[i]) * f);
          }
          if (tile > ta) tmem_st16(tm_o + 16 * c, s);
        }
      }
      // the weights, and their sums
#pragma unroll
      for (int c = 0; c < kRows / 16; ++c) {
        if (16 * c >= rows) break;
        uint32_t s[16], p[8];
        tmem_ld16(tm_s + 16 * c, s);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float4 rc = *reinterpret_cast<const float4*>(row_c + 16 * c + i);
          float y0 = fmaf(__uint_as_float(s[i]), ks_now * rc.x, lv_now - rc.y);
          float y1 = fmaf(__uint_as_float(s[i + 1]), ks_now * rc.z, lv_now - rc.w);
          if (!open) {
            const int2 la = *reinterpret_cast<const int2*>(row_last + 16 * c + i);
            y0 = seen(la.x) ? y0 : -CUDART_INF_F;
            y1 = seen(la.y) ? y1 : -CUDART_INF_F;
          }
          const float w0 = exp2_fast(y0), w1 = exp2_fast(y1);
          l[16 * c + i] = fmaf(w0, rv, l[16 * c + i]);
          l[16 * c + i + 1] = fmaf(w1, rv, l[16 * c + i + 1]);
          p[i / 2] = pack_half(w0, w1);
        }
        const uint32_t at = base + TcSmem::P + tid * 128;
        sts16(at + (((2 * c) ^ (tid & 7)) << 4), p[0], p[1], p[2], p[3]);
        sts16(at + (((2 * c + 1) ^ (tid & 7)) << 4), p[4], p[5], p[6], p[7]);
      }
      fence_async_smem();
      fence_before_sync();
      __syncthreads();
      if (*failed) ok = false;  // (the same for all threads)
      if (tid == 0) {
        fence_after_sync();
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)
          mma_ss(tm + 64, sdesc(base + TcSmem::V + (s >> 2) * 16384 + (s & 3) * 32, 16, 1024),
                 sdesc(base + TcSmem::P + s * 2048, 128 * 128, 1024), id_pv,
                 (tile > ta) || s > 0);
        mma_commit(bar_o);
      }
      __syncwarp();
    }
    // the item's end: sums over the keys (threads), then o
    ok = wait_bar(bar_o, phase_o) && ok;
    phase_o ^= 1;
    if (!ok) *failed = 1;
    fence_after_sync();
    float* const sums = reinterpret_cast<float*>(sm + TcSmem::sums);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < rows) sums[i * 129 + tid] = l[i];
    __syncthreads();
    if (*failed) {
      if (tid == 0) set_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
      break;
    }
    const bool begins = ta == 0, ends = tb == it.tiles, whole = begins && ends;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (begins ? 1 : 0);
    if (tid < rows) {
      float L = 0.f;
#pragma unroll 8
      for (int i = 0; i < kAttThreads; ++i) L += sums[tid * 129 + i];
      const float m = row_c[tid].y;
      row_f[tid] = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
      if (!whole) {
        part_ml[slot * kRows + tid] = make_float2(m, L);
      } else if (a.lse) {
        const int tk = over_group(a, rem + tid);
        a.lse[(it.row0 + token0 + tk) * a.hq + head * a.group + rem + tid - tk * a.group] =
            (m + log2f(L)) * kLn2;
      }
    }
    if (ends && !begins && tid == 0) {
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
    __syncthreads();
#pragma unroll 1
    for (int c = 0; 16 * c < rows; ++c) {  // this thread's channel, sixteen rows at a time
      uint32_t s[16];
      tmem_ld16(tm_o + 16 * c, s);
      if (tid < D) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = 16 * c + i;
          if (row >= rows) break;
          const float o = __uint_as_float(s[i]) * row_f[row];
          if (whole) {
            const int tk = over_group(a, rem + row);
            const int64_t at =
                (it.row0 + token0 + tk) * a.hq + head * a.group + rem + row - tk * a.group;
            static_cast<__nv_bfloat16*>(a.out)[at * D + tid] = __float2bfloat16_rn(o);
          } else {
            part_o[(slot * kRows + row) * D + tid] = o;
          }
        }
      }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tm, 128);
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
  const int ctas = grid_ctas<TcWork>(a, sms * kTcCtas, kTcMinUnits);
  const Workspace ws(a, kRows);
  kern<<<ctas, kAttThreads, TcSmem::bytes, s>>>(a, ws.part_o, ws.part_ml, ws.descs);
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
