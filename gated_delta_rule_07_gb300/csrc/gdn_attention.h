// gdn_attention.h -- launcher interface of the softmax-attention layers' kernels: query/key norms
// with the rotation, and the 8-bit paged key/value cache.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// Query/key norms and rotation, forward and gradients (gdn_qk_norm_rope and its backward).
// Row strides are in elements; outputs and output gradients are contiguous.
constexpr int kRopeCtas = 456;  // CTAs of the gradient kernel at most, one partial weight sum each
struct QkRopeArgs {
  int64_t T, q_ts, q_hs, k_ts, k_hs;
  int hq, hkv, D, R, max_pos;
  bool bf16, pairs;
  float eps, offset;
  const void *q, *k, *dq_out, *dk_out;
  const int32_t* pos;
  const float *table, *wq, *wk;
  void *q_out, *k_out, *dq, *dk;
  float *dwq, *dwk, *partial;  // partial [CTAs, D]: query rows' CTAs first
  int32_t* status;
};
cudaError_t qk_rope(const QkRopeArgs& a, bool backward, cudaStream_t s);

// The paged 8-bit key/value cache (gdn_kv_append, gdn_kv_read, gdn_kv_attention).  pos0: tokens
// already held (append), first position (read), whole length (attention) of each sequence.
struct KvArgs {
  int64_t T, k_ts, k_hs, v_ts, v_hs, q_ts, q_hs;
  int N, hq, hkv, D, page, page_shift, num_pages, max_pages, window;  // page = 1 << page_shift
  int group;           // query heads of a kv head; 2^32 / group, rounded up
  uint32_t group_mul;
  bool bf16, e4m3;
  float scale;
  const void *k, *v, *q;
  const int32_t *table, *pos0, *cu;
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
  void *k_out, *v_out, *out;
  float *lse, *workspace;
  int32_t* status;
};
cudaError_t kv_append(const KvArgs& a, cudaStream_t s);
cudaError_t kv_read(const KvArgs& a, cudaStream_t s);
cudaError_t kv_attention(const KvArgs& a, cudaStream_t s);
size_t kv_attention_workspace(const KvArgs& a);
// its form on tcgen05, for more than sixteen rows a kv head (bf16, D <= 128)
cudaError_t kv_attention_tc(const KvArgs& a, cudaStream_t s);
size_t kv_attention_tc_workspace(const KvArgs& a);

}  // namespace gdn
