// gdn_kv.cuh -- device helpers of the 8-bit paged key/value cache: its layout, its codes and the
// map from packed rows to pages.
//
// A page holds `page` tokens of every kv head.  With h the head and t the token's place in it:
//     keys    byte ((pid hkv + h) page + t) D + d
//     values  byte ((pid hkv + h) page + 4 (t / 4)) D + 4 d + t % 4
// so that four tokens' codes of one value channel are one 32-bit word: the products with the
// values contract over tokens, and a lane's operand registers want neighbouring tokens.
// value of a code = code * scale[pid][h], keys and values each with their own scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attention.h"
#include "gdn_common.cuh"

namespace gdn {

constexpr float kKvTiny = 7.888609052210118e-31f;  // 2^-100: pages below it are stored as zeros

template <bool E4M3> __device__ __forceinline__ constexpr float kv_qmax() {
  return E4M3 ? 448.f : 127.f;
}

// The value a code stands for, before its scale.
template <bool E4M3> __device__ __forceinline__ float kv_value(uint32_t byte) {
  if constexpr (E4M3) {
    // e4m3's exponent and mantissa bits, moved to an fp16's, are the value times 2^-8 (the biases
    // are 7 and 15), subnormals included; a NaN code reads as +-480
    const uint16_t h = (uint16_t)(((byte & 0x80u) << 8) | ((byte & 0x7fu) << 7));
    return __half2float(__ushort_as_half(h)) * 256.f;
  } else {
    return (float)(int8_t)byte;
  }
}

// The code of y (a value over its scale): rounded to nearest, ties to even, within +-qmax.
// A NaN is stored as 0.
template <bool E4M3> __device__ __forceinline__ uint32_t kv_code(float y) {
  y = y == y ? fminf(fmaxf(y, -kv_qmax<E4M3>()), kv_qmax<E4M3>()) : 0.f;
  if constexpr (E4M3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(y));
    return r & 0xffu;
  } else {
    return (uint32_t)__float2int_rn(y) & 0xffu;
  }
}

// A packed range of tokens over pages.  Sequence n's rows [cu[n], cu[n + 1]) stand at positions
// pos0[n] onward; they touch at most rows / page + 2 pages, so "slots" enumerate every (sequence,
// touched page) without a prefix sum: sequence n owns those from cu[n] / page + 2 n on, and all lie
// below T / page + 2 N.  Without cu, a row is a sequence (or all rows are the one sequence).
struct KvSpan {
  int n;          // sequence
  int page_i;     // page of the sequence
  int lo, hi;     // tokens [lo, hi) of the page
  int64_t row;    // the packed row of token lo
};

// Finds slot's span; false where there is none.  One warp's lanes search together.
__device__ __forceinline__ bool kv_span(const KvArgs& a, int64_t slot, KvSpan& s) {
  int n = 0;
  int64_t b, e, k;
  if (a.cu == nullptr && a.N > 1) {  // one row a sequence, one page each
    n = (int)slot;
    b = n;
    e = n + 1;
    k = 0;
  } else {
    if (a.cu) {  // the largest n with cu[n] / page + 2 n <= slot: 32 probes a step
      const int lane = threadIdx.x & 31;
      int lo = 0, hi = a.N - 1;  // the answer is in [lo, hi]
      while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        bool below = false;
        if (at <= hi) {
          const int c = a.cu[at];
          below = (int64_t)(c < 0 ? 0 : c) / a.page + 2 * (int64_t)at <= slot;
        }
        // (a table that is not sorted may send this anywhere in [0, N): it is checked below)
        const int got = __popc(__ballot_sync(0xffffffffu, below));
        const int next = lo + got * step;
        hi = min(hi, next + step - 1);
        lo = min(next, hi);
        if (step == 1) break;
      }
      n = lo;
    }
    if (!seq_bounds(a.cu, n, a.T, a.status, b, e)) return false;
    k = slot - (b / a.page + 2 * (int64_t)n);
  }
  if (k < 0 || e <= b) return false;
  const int64_t p0 = a.pos0 ? a.pos0[n] : 0, p1 = p0 + (e - b);
  if (p0 < 0 || p1 > (int64_t)a.max_pages * a.page) {
    set_status(a.status, GDN_ERR_DEVICE_INPUT);
    return false;
  }
  const int64_t pi = p0 / a.page + k;
  if (pi * a.page >= p1) return false;
  const int64_t first = pi * a.page;
  s.n = n;
  s.page_i = (int)pi;
  s.lo = (int)(p0 > first ? p0 - first : 0);
  s.hi = (int)(p1 < first + a.page ? p1 - first : a.page);
  s.row = b + first + s.lo - p0;
  return true;
}

// The page's id, or -1 (and the status word set) where the block table names none of the pool.
__device__ __forceinline__ int kv_page_id(const KvArgs& a, int n, int page_i) {
  const int pid = a.table[(int64_t)n * a.max_pages + page_i];
  if (pid >= 0 && pid < a.num_pages) return pid;
  set_status(a.status, GDN_ERR_DEVICE_INPUT);
  return -1;
}

}  // namespace gdn
