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
#include "gdn_stream_order.cuh"

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

// The page's id, or -1 (and the status word set) where the block table names none of the pool.
__device__ __forceinline__ int kv_page_id(const KvArgs& a, int n, int page_i) {
  const int pid = a.table[(int64_t)n * a.max_pages + page_i];
  if (pid >= 0 && pid < a.num_pages) return pid;
  set_status(a.status, GDN_ERR_DEVICE_INPUT);
  return -1;
}

// Sequence n's span in its k-th slot; false where it has none (or does not fit).
__device__ __forceinline__ bool kv_span_of(const KvArgs& a, int n, int64_t b, int64_t e, int64_t p0,
                                           int64_t k, KvSpan& s) {
  if (k < 0 || e <= b) return false;
  const int64_t p1 = p0 + (e - b);
  if (p0 < 0 || p1 > (int64_t)a.max_pages << a.page_shift) {
    set_status(a.status, GDN_ERR_DEVICE_INPUT);
    return false;
  }
  const int64_t pi = (p0 >> a.page_shift) + k, first = pi << a.page_shift;
  if (first >= p1) return false;
  s.n = n;
  s.page_i = (int)pi;
  s.lo = (int)(p0 > first ? p0 - first : 0);
  s.hi = (int)(p1 < first + a.page ? p1 - first : a.page);
  s.row = b + first + s.lo - p0;
  return true;
}

// A CTA's span and page id (-1: nothing to do), found together by its threads.  Up to a thread a
// sequence: each looks at its own (one step of loads, and the owner reads the block table), else a
// search by 32 probes a step.
struct KvFound {
  KvSpan span;
  int pid, owner;
};
__device__ __forceinline__ void kv_find(const KvArgs& a, int64_t slot, KvFound& shared) {
  const int tid = threadIdx.x;
  if (a.N <= (int)blockDim.x && (a.cu || a.N == 1)) {
    if (tid == 0) {
      shared.pid = -1;
      shared.owner = a.N;
    }
    __syncthreads();
    KvSpan s;
    bool mine = false;
    if (tid < a.N) {
      const int64_t b = a.cu ? a.cu[tid] : 0, e = a.cu ? a.cu[tid + 1] : a.T;
      const int64_t p0 = a.pos0 ? a.pos0[tid] : 0;
      const int64_t k = slot - ((b >> a.page_shift) + 2 * (int64_t)tid);
      if (b < 0 || e < b || e > a.T)
        set_status(a.status, GDN_ERR_DEVICE_INPUT);
      else
        mine = k < (e >> a.page_shift) - (b >> a.page_shift) + 2 &&
               kv_span_of(a, tid, b, e, p0, k, s);
      // (of a table that does not ascend, several sequences may claim a slot: the first has it)
      if (mine) atomicMin(&shared.owner, tid);
    }
    __syncthreads();
    if (mine && shared.owner == tid) {
      shared.span = s;
      shared.pid = kv_page_id(a, s.n, s.page_i);
    }
    __syncthreads();
    return;
  }
  if (tid < 32) {
    int n = (int)slot;  // (without cu: one row a sequence, one page each)
    int64_t b = n, e = n + 1, k = 0;
    bool ok = true;
    if (a.cu) {  // the largest n with cu[n] / page + 2 n <= slot is in [lo, hi]
      int lo = 0, hi = a.N - 1;
      while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + (tid + 1) * step;
        bool below = false;
        if (at <= hi) {
          const int c = a.cu[at];
          below = (int64_t)((c < 0 ? 0 : c) >> a.page_shift) + 2 * (int64_t)at <= slot;
        }
        // (a table that does not ascend may send this anywhere in [0, N): it is checked below)
        const int next = lo + __popc(__ballot_sync(0xffffffffu, below)) * step;
        hi = min(hi, next + step - 1);
        lo = min(next, hi);
      }
      n = lo;
      ok = seq_bounds(a.cu, n, a.T, a.status, b, e);
      k = slot - ((b >> a.page_shift) + 2 * (int64_t)n);
    }
    KvSpan s;
    ok = ok && kv_span_of(a, n, b, e, a.pos0 ? a.pos0[n] : 0, k, s);
    if (tid == 0) {
      shared.pid = ok ? kv_page_id(a, s.n, s.page_i) : -1;
      if (ok) shared.span = s;
    }
  }
  __syncthreads();
}

}  // namespace gdn
