// gdn_linear.h -- launcher interface of linear attention with a decay for each head (prompts,
// gradients, single tokens) and of the 8-bit checkpoints.
//
// Per value head, a = exp(log_decay) <= 1:  h_t = a h_{t-1} + k_t v_t^T,  o_t = h_t^T q_t.  With D_t
// the gradient of the state after token t and F_t = D_t + q_t do_t^T (D_{t-1} = a F_t), the gradients
// are dq_t = h_t do_t, dk_t = F_t v_t, dv_t = F_t^T k_t: each of them is the same computation on other
// rows, two of them walking backward in time.  So there is one pass, "targets" z, "sources" x and y:
//     out_i = sum_{j at or before i} a^{|i - j|} (z_i . x_j) y_j  +  a^{steps before i} z_i S
// where "before" is in the direction of the walk and S is what has gathered up to where it stands:
//     output   z   x   y    direction   S at the start of a segment
//     out      q   k   v    forward     a h        (h: the state that enters it)
//     dq       do  v   k    forward     a h^T
//     dk       v   do  q    backward    D^T        (D: the gradient of the state that leaves it)
//     dv       k   q   do   backward    D
// Sequences are cut into segments of a fixed length that run in parallel: a first kernel gathers each
// segment's own state, a scan over a sequence's segments makes the states that they start from, and
// the pass runs over every segment from its state.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct LinearRows {      // [T, heads, D] rows; value head j reads head j / share
  const void* p;
  int64_t ts, hs;        // strides of a token and a head, in elements
  int share;
};

// Segments ("slots"): sequence n owns ceil(L / seg) of them from slot cu[n] / seg + n on, which are
// disjoint for a valid table; all lie below T / seg + N.
struct LinearShape {
  int64_t T, slots;
  int N, hk, hv, K, V, seg;
  bool bf16;
  const float* log_decay;   // [hv]
  const int32_t* cu;        // [N + 1], or null: one sequence
  int32_t* status;
  int32_t* refused;         // 1 where the call's table or decays cannot be used, else 0
  bool looked;              // a kernel ahead has written it
};
// Beyond so many sequences the table is looked at once, ahead of the call's kernels, and not by the first
// one's every block (10000 sequences of 32 heads: 320000 blocks, 40 KB each).
constexpr int kLinearLooked = 512;
cudaError_t linear_check(const LinearShape& a, cudaStream_t s);

// U[slot, head] = sum over its tokens of a^{steps to where the walk leaves} x y^T, [K, V] each.
struct LinearState {
  LinearShape s;
  LinearRows x, y;
  bool reverse;
  float* states;            // [slots, hv, K, V]
  int* tops;                // tensor cores: [slots, hv, 2], the largest finite |x| and |y|, as fp32's bits
};
// The states that the segments start from, in place of U; the walk starts from `first` (null: 0) and
// its end goes to `last` (null: nowhere), [N, hv, K, V] each.
struct LinearScan {
  LinearShape s;
  bool reverse;
  float* states;
  const float* first;
  float* last;
};
struct LinearPass {
  LinearShape s;
  LinearRows z, x, y;
  int A, B;                 // lengths of the rows of z and x, and of y and the output
  bool reverse, transposed; // transposed: S is the transpose of the state as it is stored
  const float* states;
  void* out;                // [T, hv / out_share, B]
  int out_share;            // value heads summed into one output head
  float* partial;           // with out_share > 1: their running sum, T hv / out_share B values (tensor
                            // cores), or each's rows, T hv B values (CUDA cores)
  // tensor cores: entry 2 (slot hv + head) bounds these rows (see LinearState)
  const int *x_top, *y_top;
};

// fp32 arithmetic on the CUDA cores: every dtype and head size.
cudaError_t linear_state_simt(const LinearState& a, cudaStream_t s);
cudaError_t linear_pass_simt(const LinearPass& a, cudaStream_t s);
cudaError_t linear_scan(const LinearScan* scans, int count, cudaStream_t s);  // one, or two of a shape

// The same on the tensor cores: bf16, segments of whole chunks of 128 tokens, T > 0, rows
// that are strided by 16 bytes or more.
cudaError_t linear_state_tc(const LinearState& a, cudaStream_t s);
cudaError_t linear_pass_tc(const LinearPass& a, cudaStream_t s);

struct LinearDecode {
  int batch, slots, hk, hv, K, V;
  bool bf16;
  LinearRows q, k, v;       // a row is a token
  const float* log_decay;
  const int32_t* slot;
  float* state;
  void* out;
  int32_t* status;
};
cudaError_t linear_decode(const LinearDecode& a, cudaStream_t s);

constexpr int kCheckpoints = 8;  // tensors of one call
struct CheckpointArgs {
  int count;
  bool e4m3;
  struct Rows {
    void* x;                // rows, read (pack) or written (open)
    uint8_t* codes;         // [T, heads, D]
    float* scale;           // [T, heads]
    int64_t rows, ts, hs;   // T heads rows
    int heads, D;
    bool bf16, packed;      // packed: x's rows follow one another
  } t[kCheckpoints];
  int64_t first[kCheckpoints + 1];  // blocks before each tensor's
  int32_t* status;
};
cudaError_t checkpoint_pack(CheckpointArgs& a, cudaStream_t s);
cudaError_t checkpoint_open(CheckpointArgs& a, cudaStream_t s);

}  // namespace gdn
