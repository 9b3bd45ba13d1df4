// gdn_linear.cuh -- what the kernels of linear attention share: the table's checks, a segment's
// tokens, powers of the decay.
#pragma once

#include "gdn_common.cuh"
#include "gdn_linear.h"

namespace gdn {
namespace linear {

// Whether the call's table and decays can be used, decided alike by every block of every kernel of a
// call (so that outputs are written whole or not at all).  Contains a block barrier.
__device__ __forceinline__ bool usable(const LinearShape& s) {
  if (s.refused != nullptr) return *s.refused == 0;
  bool bad = false;
  if (s.cu != nullptr) {
    for (int i = threadIdx.x; i < s.N; i += blockDim.x) {
      const int32_t b = s.cu[i], e = s.cu[i + 1];
      bad |= e < b || e > s.T || (i == 0 && b != 0);
    }
  }
  for (int i = threadIdx.x; i < s.hv; i += blockDim.x) bad |= !(s.log_decay[i] <= 0.f);
  if (!__syncthreads_or(bad)) return true;
  if (threadIdx.x == 0) set_status(s.status, GDN_ERR_DEVICE_INPUT);
  return false;
}

// Tokens [t0, t1) of a slot, and its sequence; false for a slot that no sequence owns.
__device__ __forceinline__ bool slot_tokens(const LinearShape& s, int64_t slot, int& n, int64_t& t0,
                                            int64_t& t1) {
  n = 0;
  if (s.cu != nullptr) {
    int lo = 0, hi = s.N - 1;
    while (lo < hi) {  // the last sequence whose first slot is at or below this one
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)(s.cu[mid] / s.seg) + mid <= slot) lo = mid; else hi = mid - 1;
    }
    n = lo;
  }
  const int64_t b = s.cu ? s.cu[n] : 0, e = s.cu ? s.cu[n + 1] : s.T;
  t0 = b + (slot - (b / s.seg + n)) * s.seg;
  t1 = t0 + s.seg < e ? t0 + s.seg : e;
  return t0 >= b && t0 < e;
}

// log2 of a head's decay.  (A decay of exp(-1e4) and all below it are 0 in fp32 after one step, as
// they have to be; the bound keeps no steps times minus infinity from being NaN.)
__device__ __forceinline__ float log2_decay(const LinearShape& s, int head) {
  return fmaxf(s.log_decay[head], -1e4f) * 1.4426950408889634f;
}
__device__ __forceinline__ float power(float log2a, int steps) { return exp2f(log2a * (float)steps); }

}  // namespace linear
}  // namespace gdn
