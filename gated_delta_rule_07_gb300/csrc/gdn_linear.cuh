// gdn_linear.cuh -- what the kernels of linear attention share: the table's checks, a segment's
// tokens, powers of the decay.
#pragma once

#include "gdn_common.cuh"
#include "gdn_linear.h"

namespace gdn {
namespace linear {

// Whether the call's table and decays can be used: outputs are written whole or not at all.  The call's
// first kernels look at them, each of their blocks for itself, and leave what they find in a word for the
// pass.  (With the look in the passes too, they took 374 us instead of 349 for 65536 tokens, 149 instead of
// 124 for dq and dk of 16384.  The scan is better off with a look of its own: gradients of 8 x 4096 tokens,
// 12 us for the two, 24 by the word.)  Contains a block barrier.
__device__ __forceinline__ bool accepted(const LinearShape& s) { return *s.refused == 0; }
__device__ __forceinline__ bool usable(const LinearShape& s) {
  if (s.looked) return accepted(s);
  bool bad = false;
  if (s.cu != nullptr) {
    for (int i = threadIdx.x; i < s.N; i += blockDim.x) {
      const int32_t b = s.cu[i], e = s.cu[i + 1];
      bad |= e < b || e > s.T || (i == 0 && b != 0);
    }
  }
  for (int i = threadIdx.x; i < s.hv; i += blockDim.x) bad |= !(s.log_decay[i] <= 0.f);
  bad = __syncthreads_or(bad) != 0;
  if (threadIdx.x == 0 && (blockIdx.x | blockIdx.y) == 0) {
    *s.refused = bad ? 1 : 0;
    if (bad) set_status(s.status, GDN_ERR_DEVICE_INPUT);
  }
  return !bad;
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
