// gdn_linear_tc.cu -- linear attention with a decay for each head (gdn_linear.h) on the fifth-generation
// tensor cores: bf16 I/O.  Tiles are 128 columns wide, two blocks of 64; rows of 64 have the first block
// alone, and products take that many steps or columns fewer.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_linear.cuh"
#include "gdn_sm100.cuh"
#include "gdn_stream_order.cuh"
#include "gdn_tc5_util.cuh"

namespace gdn {
namespace {

using namespace sm100;
using namespace tc5u;

constexpr int D = 128;                            // K and V at most
constexpr long long kWaitCycles = 2000000000LL;   // limit of a bounded wait: about a second

// true in one thread of a converged warp
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// Bounded wait of a warp: sleeps in hardware; gives up after about a second, or when another has.
__device__ __forceinline__ void wait_longer(uint32_t bar, uint32_t parity, volatile int* failed) {
  const long long began = clock64();
  while (!*failed && !mbar_try(bar, parity))
    if (clock64() - began > kWaitCycles) *failed = 1;
}
__device__ __forceinline__ void wait_one(uint32_t bar, uint32_t parity, volatile int* failed) {
  if (!mbar_try(bar, parity)) wait_longer(bar, parity, failed);
}
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, volatile int* failed) {
  wait_one(bar, parity, failed);
  __syncwarp();
}
// A warpgroup's registers a thread, from now on (of the block's, which the groups share).  All warps of
// a group are to come to the same one of these, so roles branch by warpgroups first.
template <int N> __device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N> __device__ __forceinline__ void leave_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
// Bounded wait for work of one's own that is in flight, after another wait has given up.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const long long began = clock64();
  while (!mbar_try(bar, parity) && clock64() - began < kWaitCycles) {
  }
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ float low(uint32_t bf2) { return __uint_as_float(bf2 << 16); }
__device__ __forceinline__ float high(uint32_t bf2) { return __uint_as_float(bf2 & 0xffff0000u); }
// 2^e, 0 below fp32's range
__device__ __forceinline__ float two_to(int e) {
  return __uint_as_float((uint32_t)max(0, min(e, 127) + 127) << 23);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
// packed bf16: the larger magnitudes, of the even and of the odd elements
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// such magnitudes, or zeros where one is infinite
__device__ __forceinline__ uint32_t finite(uint32_t m) { return (m + 0x00800080u) & 0x80008000u ? 0u : m; }
// the larger of such a pair, as bits of fp32 (which have magnitudes' order)
__device__ __forceinline__ int larger_of_two(uint32_t m) {
  return (int)(max(m & 0x7fffu, m >> 16 & 0x7fffu) << 16);
}
// e with |v| < 2^e for the bits of a magnitude of fp32's normal range
__device__ __forceinline__ int exponent_of(int bits) { return (bits >> 23) - 126; }

// ------------------------------------------------------------------ a segment's own state

// U = sum of weighted x y^T over a segment, to fp32 accuracy: y's rows times their powers of the decay
// are split into three bf16 parts (24 bits), x is bf16 as it stands, products and their sums are exact
// or fp32.  64 tokens at a time go through the tensor core into Tensor Memory and from there into a
// register-held U, decayed on the way: the weights stay within a tile, and the tensor core's own sums,
// whose roundings do not average out, stay short.  (However far the share has decayed at the end of its
// sequence: what is behind it may be zeros, and then it is all that there is.)
//
// HBM takes 1340 cycles for a tile of an SM's share, so little may go through shared memory beside the
// tiles themselves (256 of its cycles): y comes out of it transposed (ldmatrix) and the parts go straight to
// Tensor Memory, as the operand whose rows are y's columns; the tensor core reads x alone from shared memory.
// So it makes U^T.  (65536 tokens of 32 heads: 198 us, of HBM's 119, with 69% of the issue slots used, by
// the splitting above all; with parts written back to shared memory 270, whatever the number of warps.)
// Five tiles are on their way or at work; splitting (sixteen warps), the products and the sums (eight
// warps, for Tensor Memory's lanes and their registers) each on another.  896 threads launch with 72
// registers, 504 for the seven warpgroups' warps of an SM's quarter: the sums' two take 96, splitting's
// four keep 64, the last 56.
constexpr int kTile = 64, kSplit = 512, kAdd = 256, kStateThreads = kSplit + kAdd + 128, kStages = 5;
static_assert(kSplit % 128 == 0 && kAdd % 128 == 0, "roles that set registers are whole warpgroups");
constexpr uint32_t kRaw = kTile * D * 2;          // bytes of a tile of one tensor
struct StateSmem {                                // offsets from a 1024-byte boundary
  static constexpr uint32_t X = 0, Y = kRaw, stage = 2 * kRaw, BARS = kStages * stage;
  static constexpr int bytes = BARS + 24 * 8 + 1024;
};

// Four 8 x 8 blocks of 16-bit elements, transposed: a lane gives a row of one (lane / 8) and gets of each
// the elements [lane / 4] [2 (lane % 4)] and the next.
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// Such blocks to 16 lanes and 8 columns of Tensor Memory: rows 0-7 and 8-15 of four columns, of the next four.
__device__ __forceinline__ void tmem_st_blocks(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

template <bool WIDE>  // K = V = 128
__global__ void __launch_bounds__(kStateThreads, 1)
linear_state_tc_kernel(const LinearState a, const __grid_constant__ CUtensorMap mx,
                       const __grid_constant__ CUtensorMap my) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_word, top[2];
  volatile int* failed = &failed_word;
  stream_order();
  if (!linear::usable(a.s)) return;
  const int K = WIDE ? D : a.s.K, V = WIDE ? D : a.s.V;
  const int head = blockIdx.x % a.s.hv;
  const int64_t slot = blockIdx.x / a.s.hv;
  int n;
  int64_t t0, t1;
  if (!linear::slot_tokens(a.s, slot, n, t0, t1)) return;
  const uint32_t base = (saddr(raw_smem) + 1023u) & ~1023u, bars = base + StateSmem::BARS;
  // (one of a stage, or of two in turn)
  const uint32_t full = bars, free_ = full + 8 * kStages, ready = free_ + 8 * kStages, done = ready + 16, taken = done + 16,
                 end = taken + 16;
  auto half = [](int i) { return (uint32_t)(i >> 1) & 1; };
  const int tid = threadIdx.x, warp = tid / 32;
  if (tid == 0) {
    failed_word = 0;
    top[0] = top[1] = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(free_ + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(ready + 8 * i, kSplit);
      mbar_init(done + 8 * i, 1);
      mbar_init(taken + 8 * i, kAdd);
    }
    mbar_init(end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  constexpr int kLoad = (kSplit + kAdd) / 32, kMma = kLoad + 1;
  if (warp == kMma) {
    tmem_alloc(saddr(&tmem_at), 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  constexpr uint32_t tm = 0, tm_parts = 256;  // (all of Tensor Memory): two sums; three parts, twice
  const int begin = (int)t0, length = (int)(t1 - t0), tiles = (length + kTile - 1) / kTile;
  // the i-th tile of the walk, its tokens
  auto first_token = [&](int i) { return begin + (a.reverse ? tiles - 1 - i : i) * kTile; };
  auto tokens = [&](int i) { return min(begin + length - first_token(i), kTile); };
  const float log2a = linear::log2_decay(a.s, head);

  if (warp >= kLoad) {  // (the last warpgroup; the rest of its warps have nothing to do)
    leave_registers<56>();
    if (warp == kLoad) {
      if (tid % 32 == 0) {
        int loaded = 0;
        for (int i = 0, st = 0, round = 0; i < tiles; ++i) {
          if (round) wait_one(free_ + 8 * st, (round - 1) & 1, failed);
          if (*failed) break;
          const uint32_t x = base + st * StateSmem::stage + StateSmem::X,
                         y = base + st * StateSmem::stage + StateSmem::Y;
          const int t = first_token(i);
          mbar_expect_tx(full + 8 * st, (uint32_t)(K + V) * kTile * 2);
#pragma unroll 1
          for (int b = 0; b < K; b += 64)
            tma_box(x + b * (kRaw / 128), &mx, b, head / a.x.share, t, full + 8 * st);
#pragma unroll 1
          for (int b = 0; b < V; b += 64)
            tma_box(y + b * (kRaw / 128), &my, b, head / a.y.share, t, full + 8 * st);
          loaded = i + 1;
          if (++st == kStages) {
            st = 0;
            ++round;
          }
        }
        if (*failed)
          for (int i = loaded > kStages ? loaded - kStages : 0; i < loaded; ++i)
            drain(full + 8 * (i % kStages), (i / kStages) & 1);
      }
      __syncwarp();
    } else if (warp == kMma) {
      // (lanes behind V hold nothing that is read)
      const uint32_t id = idesc_f16(128, K, 0, 1, 1);
      const uint64_t at = sdesc(base, kRaw / 2, 1024);
#pragma unroll 1
      for (int i = 0, st = 0; i < tiles; ++i) {
        wait_bar(ready + 8 * (i & 1), half(i), failed);
        if (i >= 2) wait_bar(taken + 8 * (i & 1), half(i - 2), failed);
        if (*failed) break;
        fence_after_sync();
        const uint64_t x = at + ((st * StateSmem::stage + StateSmem::X) >> 4);
        const uint32_t d = tm + 128 * (i & 1), parts = tm_parts + 96 * (i & 1);
        if (elected()) {
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)  // (the small parts first)
            mma_ts(d, parts + 64 + 8 * ks, x + ks * 128, id, ks > 0);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) mma_ts(d, parts + 32 + 8 * ks, x + ks * 128, id, 1);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) mma_ts(d, parts + 8 * ks, x + ks * 128, id, 1);
          mma_commit(done + 8 * (i & 1));
          mma_commit(free_ + 8 * st);
        }
        __syncwarp();
        st = st + 1 == kStages ? 0 : st + 1;
      }
      if (*failed) {
        if (elected()) {
          mma_commit(end);
          drain(end, 0);
        }
        __syncwarp();
      }
    }
  } else if (warp < kSplit / 32) {
    // ---------------------------------------------------------------- weights and parts
    // A warp has 16 tokens, and the 32 columns whose lanes of Tensor Memory it can write; a thread four of
    // the tokens, and of x two 16-byte pieces of a row to look at.
    leave_registers<64>();
    const int lane = tid % 32, quarter = warp & 3, token0 = 16 * (warp >> 2), pair = token0 + 2 * (lane & 3);
    const int r = tid / 8;
    const int from = token0 + (lane >> 4) * 8 + (lane & 7);  // the row that this lane gives ldmatrix,
    uint32_t source[2];                                      // and where its columns are
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int c = 32 * quarter + 16 * g + (lane >> 3 & 1) * 8;
      source[g] = sw128_offset(kTile, from, c);
    }
    uint32_t x_max = 0, y_max = 0;
    float2 w_whole[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = pair + 8 * k;
      w_whole[k] = make_float2(linear::power(log2a, a.reverse ? t + 1 : kTile - 1 - t),
                               linear::power(log2a, a.reverse ? t + 2 : kTile - 2 - t));
    }
#pragma unroll 1
    for (int i = 0, st = 0, round = 0; i < tiles; ++i) {
      const uint32_t x = base + st * StateSmem::stage + StateSmem::X + 16 * tid,
                     y = base + st * StateSmem::stage + StateSmem::Y;
      const int m = tokens(i);
      float2 w[2] = {w_whole[0], w_whole[1]};
      uint32_t mask[2] = {0xffffffffu, 0xffffffffu};
      if (m < kTile) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = pair + 8 * k;
          mask[k] = (t < m ? 0xffffu : 0u) | (t + 1 < m ? 0xffff0000u : 0u);
          if (!a.reverse)
            w[k] = make_float2(linear::power(log2a, max(0, m - 1 - t)),
                               linear::power(log2a, max(0, m - 2 - t)));
        }
      }
      wait_bar(full + 8 * st, round & 1, failed);
      if (i >= 2) wait_bar(done + 8 * (i & 1), half(i - 2), failed);  // (the parts' columns)
      fence_after_sync();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (32 * quarter >= V) break;
        uint32_t v[4], mid[4];
        float2 f[4];
        load_transposed(y + source[g], v);
        if (m < kTile) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] &= mask[j >> 1];
        }
        const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y_max = larger(y_max, v[j]);
          f[j] = mul2(make_float2(low(v[j]), high(v[j])), w[j >> 1]);
          v[j] = pack_bf2(f[j].x, f[j].y);
          f[j] = __ffma2_rn(make_float2(low(v[j]), high(v[j])), minus, f[j]);
          mid[j] = pack_bf2(f[j].x, f[j].y);
        }
        const uint32_t to = ((uint32_t)(32 * quarter + 16 * g) << 16) + tm_parts + 96 * (i & 1) + token0 / 2;
        tmem_st_blocks(to, v);
        tmem_st_blocks(to + 32, mid);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = __ffma2_rn(make_float2(low(mid[j]), high(mid[j])), minus, f[j]);
          mid[j] = pack_bf2(f[j].x, f[j].y);
        }
        tmem_st_blocks(to + 64, mid);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (64 * b >= K) break;
        if (r < m) {
          const uint4 v = lds16(x + 8192 * b);
          x_max = larger(larger(larger(larger(x_max, v.x), v.y), v.z), v.w);
        } else {  // (another sequence's rows, or none)
          sts16(x + 8192 * b, make_uint4(0, 0, 0, 0));
        }
      }
      __syncwarp();
      if (m < kTile) fence_async_smem();
      tmem_wait_st();
      fence_before_sync();
      mbar_arrive(ready + 8 * (i & 1));
      if (++st == kStages) {
        st = 0;
        ++round;
      }
    }
    // An infinity does not reach the outputs of the chunks before its own, so it is not to scale their rows:
    // a warp that has met one looks at its rows once more, without it.  (Left out tile by tile it took
    // 2% more: 196 us for 65536 tokens of 32 heads, 192 so.)
    if (__any_sync(0xffffffffu, finite(x_max) != x_max || finite(y_max) != y_max)) {
      const __nv_bfloat16* const xp = static_cast<const __nv_bfloat16*>(a.x.p) +
                                      (int64_t)(head / a.x.share) * a.x.hs + 8 * (tid % 8);
      const __nv_bfloat16* const yp = static_cast<const __nv_bfloat16*>(a.y.p) +
                                      (int64_t)(head / a.y.share) * a.y.hs + 32 * quarter + 16 * (lane & 1);
      auto look = [](uint32_t most, const __nv_bfloat16* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int j = 0; j < 4; ++j) most = larger(most, finite(larger(0u, w[j])));
        return most;
      };
      x_max = y_max = 0;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int64_t t = first_token(i);
        const int m = tokens(i), other = token0 + lane / 2;
#pragma unroll 1
        for (int b = 0; b < K && r < m; b += 64) x_max = look(x_max, xp + (t + r) * a.x.ts + b);
#pragma unroll 1
        for (int c = 0; c < 16 && other < m && 32 * quarter < V; c += 8)
          y_max = look(y_max, yp + (t + other) * a.y.ts + c);
      }
      __syncwarp();
    }
    const int most_x = __reduce_max_sync(0xffffffffu, larger_of_two(x_max));
    const int most_y = __reduce_max_sync(0xffffffffu, larger_of_two(y_max));
    if (tid % 32 == 0) {
      atomicMax(top, most_x);
      atomicMax(top + 1, most_y);
    }
  } else {
    // ---------------------------------------------------------------- the sum
    take_registers<96>();
    const int at = tid - kSplit, row = at & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16, cols = (uint32_t)(at >> 7) * 64;
    const float whole = linear::power(log2a, kTile);
    float2 u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int m = tokens(i);
      const float w = m == kTile ? whole : linear::power(log2a, m);
      wait_bar(done + 8 * (i & 1), half(i), failed);
      fence_after_sync();
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        uint32_t p[16];
        tmem_ld16_nw(tm + lanes + 128 * (i & 1) + cols + 2 * c, p);
        tmem_wait_ld16(p);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          u[c + k] = __ffma2_rn(make_float2(w, w), u[c + k],
                                make_float2(__uint_as_float(p[2 * k]), __uint_as_float(p[2 * k + 1])));
      }
      fence_before_sync();
      mbar_arrive(taken + 8 * (i & 1));
    }
    float* out = a.states + (slot * a.s.hv + head) * K * V + (int64_t)cols * V + row;  // (U^T's row)
    if (!*failed && row < V && (int)cols < K) {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        out[2 * c * V] = u[c].x;
        out[(2 * c + 1) * V] = u[c].y;
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (tid < 2) a.tops[2 * (slot * a.s.hv + head) + tid] = top[tid];
  if (warp == kMma) tmem_dealloc(tm, 512);
  if (tid == 0 && *failed) set_status(a.s.status, GDN_ERR_DEVICE_TIMEOUT);
}

// ------------------------------------------------------------------ the pass

// One block walks a segment's chunks of 128 tokens (for every value head that its output head sums).
// Per chunk, with i, j counted in the walk's direction, p_i = a^i and n the chunk's tokens:
//     P = z x^T                       bf16 as loaded, into Tensor Memory
//     W = P a^{i - j}, j <= i         fp16, in P's place: an operand in Tensor Memory
//     O = W y + (p_i z) S             fp16 operands, one fp32 sum; z's beside W
//     S <- a^n S + (a^{n - j} x)^T y  fp16 operands; S fp32 in registers, its fp16 copy in shared memory
// fp16's range is not bf16's, so operands are scaled by powers of two, which come off again in fp32:
// with 2^e_x, 2^e_y above all of a head's x and y in the segment (the state kernel has seen them), 2^e_z
// above a row of z, M = e_x + e_y, and 2^(E + 1) a bound of S and of 128 |x| |y|:
//     y~ = y 2^(14 - e_y)     x~ = a^{n - j} x 2^(15 + e_y - M)     S~ = S 2^(15 - E)
//     z~ = p_i z 2^(14 - e_z)   W~ = W 2^(15 + e_y - e_z - E)         O = O~ 2^(e_z + E - 29)
// so that nothing can overflow that does not in fp32, and each rounding is half a step of fp16 (2^-11) of
// a term, or 2^-38 of what bounds the sum.  (E comes from bounds, not from S: every role has to know it, and
// none is to wait for S.)
//
// What bounds it is shared memory and the hand-offs between its roles: a chunk takes 6000 cycles (65536
// tokens of 32 heads: 345 us), where HBM takes 4300 (238 us).  Its threads read and write shared
// memory in 3150 of them, its tiles arrive in 768 (128 bytes a cycle) and go to the tensor cores in 1536.
// So z's rows go to the tensor core through Tensor Memory, the outputs leave by TMA from y's tile, and a
// sum over value heads is kept in an order of rows that its threads read together.
constexpr int C = 128;
constexpr uint32_t kTileBytes = C * D * 2, kBlock = kTileBytes / 2;  // (a block: 64 columns)
constexpr int kWeightWarps = 4, kStateWarps = 8, kOpenWarps = 4;
constexpr int kPassThreads = 32 * (kWeightWarps + kStateWarps + kOpenWarps + 4);  // (warpgroups)
constexpr int kFirstState = kWeightWarps, kFirstOpen = kFirstState + kStateWarps,
              kLoadWarp = kFirstOpen + kOpenWarps, kMmaWarp = kLoadWarp + 1;
static_assert(kWeightWarps % 4 == 0 && kStateWarps % 4 == 0 && kOpenWarps % 4 == 0,
              "roles that set registers are whole warpgroups");
struct PassSmem {             // offsets from a 1024-byte boundary
  static constexpr uint32_t Z = 0, X = kTileBytes, Y = 2 * kTileBytes, stage = 3 * kTileBytes;
  static constexpr uint32_t S = 2 * stage, POWERS = S + kTileBytes, TARGETS = POWERS + (C + 32) * 4;
  static constexpr uint32_t BARS = TARGETS + 2 * C * 4, MISC = BARS + 30 * 8;
  static constexpr int bytes = MISC + 16 + 1024;
};
static_assert(PassSmem::bytes <= 232448, "shared memory of a block");
// Registers: 640 threads launch with 96 each, 480 for the five warpgroups' warps of an SM's quarter; the
// state's two take 136, the weights keep 88, opening and the last one 56 each: 472.
// barriers: those of a pair alternate from chunk to chunk
enum { kFull = 0, kScores = 2, kValues = 4, kWeights = 6, kFree = 10, kSumsRead = 12,
       kTargets = 14, kOut = 16, kRows = 18, kFullY = 20, kStateIn = 22, kGrown, kTaken, kSums, kStart, kBegun, kEnd };

// Rows of a tile, a thread each.  (A row's logical 16-byte piece p lies at p ^ (row & 7) of its block, so
// that neighbouring rows' threads meet different banks.)
__device__ __forceinline__ uint32_t piece(uint32_t tile, int row, int p) {
  return tile + (p >> 3) * kBlock + row * 128 + ((p & 7 ^ row & 7) << 4);
}
// the largest magnitudes of a row of bf16, of even and odd elements
__device__ __forceinline__ uint32_t row_max_of(uint32_t tile, int row, int width) {
  uint32_t m[4] = {};
#pragma unroll 4
  for (int p = 0; p < width / 8; ++p) {
    const uint4 v = lds16(piece(tile, row, p));
    m[0] = larger(m[0], v.x);
    m[1] = larger(m[1], v.y);
    m[2] = larger(m[2], v.z);
    m[3] = larger(m[3], v.w);
  }
  return larger(larger(m[0], m[1]), larger(m[2], m[3]));
}
// Four pieces of a row of bf16 times f, as packed fp16.
__device__ __forceinline__ void open_pieces(uint32_t tile, int row, int p0, float f, uint4 (&v)[4]) {
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = lds16(piece(tile, row, p0 + p));
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t* w = &v[p].x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = mul2(make_float2(low(w[j]), high(w[j])), ff);
      w[j] = pack_h2(x.x, x.y);
    }
  }
}
// A row in its place; zeros where it is not live.
__device__ __forceinline__ void open_row(uint32_t tile, int row, int width, bool live, float f) {
  if (live) {
#pragma unroll 1
    for (int p0 = 0; p0 < width / 8; p0 += 4) {
      uint4 v[4];
      open_pieces(tile, row, p0, f, v);
#pragma unroll
      for (int p = 0; p < 4; ++p) sts16(piece(tile, row, p0 + p), v[p]);
    }
  } else {
#pragma unroll 1
    for (int p = 0; p < width / 8; ++p) sts16(piece(tile, row, p), make_uint4(0, 0, 0, 0));
  }
  __syncwarp();
}
// Exponents of rows of z: the least one that is told apart (times 2^126, bf16's least value is 2^-7 and has
// all its bits in fp16), and that of a row of zeros.
constexpr int kLeastRow = -112, kNoRow = -120;
// A head's x and y in a segment: 2^ex and 2^ey above their largest magnitudes (of at least 2^-101, and products
// of at least 2^-97: what is left out is below fp32's states), p 2^M above a product of the two, with a
// thousandth more for the roundings of what is bounded by it.
struct Tops {
  int ex, ey, M;
  float p;
};
constexpr float kMore = 1.002f;
// the fraction of a magnitude that exponent_of leaves, in [1/2, 1)
__device__ __forceinline__ float fraction_of(int bits) {
  return __int_as_float((bits & 0x7fffff) | 126 << 23);
}
__device__ __forceinline__ Tops tops_of(const LinearPass& a, int64_t at) {
  const int x = max(a.x_top[2 * at], 26 << 23), y = max(a.y_top[2 * at], 26 << 23);
  Tops t;
  t.ex = exponent_of(x);
  t.ey = exponent_of(y);
  t.M = max(t.ex + t.ey, -97);
  t.p = t.ex + t.ey < -97 ? 1.f : kMore * fraction_of(x) * fraction_of(y);
  return t;
}
// |S| <= b 2^q for what S starts from and what the chunks have added.
struct Bound {
  float b, whole, grown;  // a^C and C p 2^(M - q): what a whole chunk does
  int q, M, least;
  __device__ __forceinline__ void start(int max_s, const Tops& t, float log2a) {
    M = t.M;
    q = max(exponent_of(max_s), M + 7);
    b = kMore * fraction_of(max_s) * two_to(exponent_of(max_s) - q);
    whole = linear::power(log2a, C);
    grown = C * t.p * two_to(max(M - q, -126));  // (not nothing: it may outlive what S starts from)
    least = exponent_of(__float_as_int(C * t.p)) - 1 + M;
  }
  // E: |S| 2^(15 - E) and |W| 2^(15 + e_y - e_z - E) <= 65536 / kMore, which fp16 holds
  __device__ __forceinline__ int E() const { return max(exponent_of(__float_as_int(b)) - 1 + q, least); }
  // (a chunk of fewer tokens is the walk's first or last: it may count as whole where it adds, and
  // decays by what it has)
  __device__ __forceinline__ void grow(float decay) { b = fmaf(decay, b, grown); }
};
__device__ __forceinline__ void tma_out(const CUtensorMap* map, uint32_t src, int x, int head, int t0) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)), "r"(src), "r"(x), "r"(head), "r"(t0)
               : "memory");
}

// REVERSE: the walk goes backward in time.  SUM: an output head has several value heads.
// WIDE: A = B = 128 (faster where that is known: a call of 65536 tokens 552 us, 585 otherwise; gradients of
// 16384 502 and 558).
template <bool REVERSE, bool SUM, bool WIDE>
__global__ void __launch_bounds__(kPassThreads, 1)
linear_pass_tc_kernel(const LinearPass a, const __grid_constant__ CUtensorMap mz,
                      const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                      const __grid_constant__ CUtensorMap mo) {
  extern __shared__ uint8_t raw_smem[];
  stream_order();
  if (!linear::accepted(a.s)) return;
  const int share = SUM ? a.out_share : 1, heads = a.s.hv / share;
  const int A = WIDE ? D : a.A, B = WIDE ? D : a.B;
  const int oh = blockIdx.x % heads;
  const int64_t slot = blockIdx.x / heads;
  int n;
  int64_t t0, t1;
  if (!linear::slot_tokens(a.s, slot, n, t0, t1)) return;
  const uint32_t base = (saddr(raw_smem) + 1023u) & ~1023u;
  uint8_t* const gbase = raw_smem + (base - saddr(raw_smem));
  float* const powers = reinterpret_cast<float*>(gbase + PassSmem::POWERS) + 32;  // [-32, C)
  int* const targets = reinterpret_cast<int*>(gbase + PassSmem::TARGETS);  // e_z of two chunks' rows
  int* const misc = reinterpret_cast<int*>(gbase + PassSmem::MISC);
  volatile int* const failed = misc;       // 0: failed, 1: Tensor Memory, 2-3: max |S| at a head's start
  const uint32_t bars = base + PassSmem::BARS;
  auto bar = [&](int which, int it) { return bars + 8 * (which + (it & 1)); };
  auto one = [&](int which) { return bars + 8 * which; };
  auto half = [](int it) { return (uint32_t)(it >> 1) & 1; };
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    misc[0] = misc[2] = misc[3] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kFull, i), 1);
      mbar_init(bar(kFullY, i), 1);
      mbar_init(bar(kScores, i), 1);
      mbar_init(bar(kFree, i), 1);
      mbar_init(bar(kValues, i), 32 * kOpenWarps);
      mbar_init(bar(kWeights, i), 32 * kWeightWarps);
      mbar_init(bar(kRows, i), 32 * kOpenWarps);
      mbar_init(bar(kTargets, i), 32 * kWeightWarps);
      mbar_init(bar(kSumsRead, i), 32 * kStateWarps);
      mbar_init(bar(kOut, i), 32 * kStateWarps);
    }
    mbar_init(one(kStateIn), 32 * kStateWarps);
    mbar_init(one(kGrown), 1);
    mbar_init(one(kTaken), 32 * kStateWarps);
    mbar_init(one(kSums), 1);
    mbar_init(one(kStart), 32 * kStateWarps);
    mbar_init(one(kBegun), 32 * kWeightWarps);
    mbar_init(one(kEnd), 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) {
    tmem_alloc(saddr(misc + 1), 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  constexpr uint32_t tm = 0;  // (all of Tensor Memory: its first column)
  const uint32_t tm_o = tm + 256, tm_g = tm + 384;  // P twice, O, growth of S
  const int begin = (int)t0, length = (int)(t1 - t0);
  const int chunks = (length + C - 1) / C, total = chunks * share;
  auto first_token = [&](int c) { return begin + (REVERSE ? chunks - 1 - c : c) * C; };
  auto tokens = [&](int c) { return min(begin + length - first_token(c), C); };

  if (warp >= kLoadWarp) {  // (the last warpgroup; the rest of its warps have nothing to do)
    leave_registers<56>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- loads, and the outputs' stores
      if (lane == 0) {
        int loaded = 0, next_c = 0, head = oh * share;  // of the next loads
#pragma unroll 1
        for (int it = -2, c = -2, g = 0; it < total; ++it) {  // (chunk it is given out, it + 2 loaded)
          const bool more = loaded < total;
          const uint32_t st = base + (it & 1) * PassSmem::stage;
          const int t = first_token(next_c);
          if (more) {
            if (it >= 0) wait_one(bar(kFree, it), half(it), failed);
            if (*failed) break;
            const uint32_t b = bar(kFull, it);
            mbar_expect_tx(b, (uint32_t)A * C * 4);
            const int zh = head / a.z.share, xh = head / a.x.share;
#pragma unroll 1
            for (int k = 0; 64 * k < A; ++k) {
              tma_box(st + PassSmem::Z + k * kBlock, &mz, 64 * k, zh, t, b);
              tma_box(st + PassSmem::X + k * kBlock, &mx, 64 * k, xh, t, b);
            }
          }
          if (it >= 0) {
            wait_one(bar(kOut, it), half(it), failed);
            if (*failed) break;
            if (g + 1 == share && tokens(c) == C) {
#pragma unroll 1
              for (int k = 0; 64 * k < B; ++k)
                tma_out(&mo, st + PassSmem::Y + k * kBlock, 64 * k, oh, first_token(c));
              asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
              if (more) bulk_wait_read();
            }
          }
          if (more) {
            const uint32_t b = bar(kFullY, it);
            mbar_expect_tx(b, (uint32_t)B * C * 2);
            const int yh = head / a.y.share;
#pragma unroll 1
            for (int k = 0; 64 * k < B; ++k) tma_box(st + PassSmem::Y + k * kBlock, &my, 64 * k, yh, t, b);
            ++loaded;
            if (++next_c == chunks) {
              next_c = 0;
              ++head;
            }
          }
          if (++c == chunks) {
            c = 0;
            ++g;
          }
        }
        bulk_wait_all();
        if (*failed)
          for (int i = loaded > 2 ? loaded - 2 : 0; i < loaded; ++i) {
            drain(bar(kFull, i), half(i));
            drain(bar(kFullY, i), half(i));
          }
        if (*failed && loaded < total) drain(bar(kFull, loaded), half(loaded));
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- products
      // (growth: lanes behind A hold nothing that is read)
      const uint32_t id_p = idesc_f16(128, 128, 0, 0, 1), id_o = idesc_f16(128, B, 0, 1),
                     id_g = idesc_f16(128, B, 1, 1);
      // rows by features (the contraction's index contiguous), and features or columns by rows
      const uint64_t of_rows = sdesc(base, 16, 1024), of_cols = sdesc(base, kBlock, 1024);
      // A chunk takes two turns: the state's growth, the sums.  The next chunk's scores are made behind the
      // one when its tiles are there already, else behind the other; the first chunk's before all.
      int grown = 0, scored = 0;
#pragma unroll 1
      for (int turn = -1, c = 0; turn < 2 * total && !*failed; ++turn) {
        const int it = turn >> 1;
        const uint64_t x = of_cols + (((it & 1) * PassSmem::stage + PassSmem::X) >> 4),
                       y = of_cols + (((it & 1) * PassSmem::stage + PassSmem::Y) >> 4);
        if (turn >= 0 && !(turn & 1)) {
          wait_bar(bar(kValues, it), half(it), failed);  // (and x)
          if (c + 1 < chunks) {
            if (grown > 0) wait_bar(one(kTaken), (grown - 1) & 1, failed);
            fence_after_sync();
            if (elected()) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks) mma_ss(tm_g, x + ks * 128, y + ks * 128, id_g, ks > 0);
              mma_commit(one(kGrown));
            }
            __syncwarp();
            ++grown;
          }
        } else if (turn >= 0) {
          const uint32_t w = tm + 128 * (it & 1);
          wait_bar(bar(kWeights, it), half(it), failed);
          if (it > 0) wait_bar(bar(kSumsRead, it - 1), half(it - 1), failed);
          fence_after_sync();
          if (elected()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) mma_ts(tm_o, w + 8 * ks, y + ks * 128, id_o, ks > 0);
          }
          __syncwarp();
          wait_bar(bar(kTargets, it), half(it), failed);
          wait_bar(one(kStateIn), it & 1, failed);
          fence_after_sync();
          if (elected()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              if (16 * ks < A) mma_ts(tm_o, w + 64 + 8 * ks, of_cols + (PassSmem::S >> 4) + ks * 128, id_o, 1);
            mma_commit(one(kSums));
            mma_commit(bar(kFree, it));
          }
          __syncwarp();
          c = c + 1 == chunks ? 0 : c + 1;
        }
        if (scored < total && scored <= it + 1 &&
            ((turn & 1) ||
             __shfl_sync(0xffffffffu, mbar_test(bar(kFull, scored), half(scored)), 0))) {
          wait_bar(bar(kFull, scored), half(scored), failed);
          fence_after_sync();
          const uint64_t z = of_rows + (((scored & 1) * PassSmem::stage + PassSmem::Z) >> 4),
                         xr = of_rows + (((scored & 1) * PassSmem::stage + PassSmem::X) >> 4);
          if (elected()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t at = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
              if (16 * ks < A) mma_ss(tm + 128 * (scored & 1), z + at, xr + at, id_p, ks > 0);
            }
            mma_commit(bar(kScores, scored));
          }
          __syncwarp();
          ++scored;
        }
      }
      if (*failed) {
        if (elected()) {
          mma_commit(one(kEnd));
          drain(one(kEnd), 0);
        }
        __syncwarp();
      }
    }
  } else if (warp < kWeightWarps) {
    // ---------------------------------------------------------------- weights; z to Tensor Memory
    leave_registers<88>();
    const int row = tid;  // its lane of Tensor Memory, and row of z
    const uint32_t lanes = (uint32_t)warp * 32 << 16;
    int it = 0;
    for (int g = 0; g < share; ++g) {
      const int64_t at = slot * a.s.hv + oh * share + g;
      const float log2a = linear::log2_decay(a.s, oh * share + g);
      const Tops tops = tops_of(a, at);
      wait_bar(one(kStart), g & 1, failed);
      Bound bound;
      bound.start(((volatile int*)misc)[2 + (g & 1)], tops, log2a);
      // W~'s factor 2^(15 + e_y - e_z - E) in two, the columns' in fp32's range: 2^h, and the rest
      const int h = max(-1, -60 - bound.M);
      named_bar(1, 32 * kWeightWarps);  // (the last head's powers have been read, this one's max |S|)
      if (row == 0) misc[2 + (~g & 1)] = 0;  // for the next head (who used it has read it)
      // a^i 2^(e_y + h), 0 for i < 0
      powers[row] = linear::power(log2a, row) * two_to(tops.ey + h);
      if (row < 32) powers[row - 32] = 0.f;
      named_bar(1, 32 * kWeightWarps);
      mbar_arrive(one(kBegun));
      float2 step[8];  // those of |a 16-column piece's far end - column|
#pragma unroll
      for (int i = 0; i < 8; ++i)
        step[i] = REVERSE ? make_float2(powers[2 * i], powers[2 * i + 1])
                            : make_float2(powers[15 - 2 * i], powers[14 - 2 * i]);
      const float z_whole = linear::power(log2a, REVERSE ? C - 1 - row : row);
      for (int c = 0; c < chunks; ++c, ++it) {
        const int m = tokens(c), E = bound.E();
        bound.grow(m == C ? bound.whole : linear::power(log2a, m));
        wait_bar(bar(kRows, it), half(it), failed);
        wait_bar(bar(kScores, it), half(it), failed);
        fence_after_sync();
        const int ez = targets[C * (it & 1) + row];
        // (where z, x and y together pass fp32's range, what would be lost is made NaN)
        // (and where they are small, the factor takes another power of two)
        const int top = 15 - ez - E - h;
        const float mine = top < -126 && ez != kNoRow ? __int_as_float(0x7fffffff) : two_to(top);
        const bool far = __any_sync(0xffffffffu, ez != kNoRow && top > 127);
        const uint32_t p_at = tm + lanes + 128 * (it & 1);
#pragma unroll 1
        for (int k0 = 0; k0 < C; k0 += 32) {
          // (32 x 32 pieces on the far side of the diagonal, or behind the last token, are not read)
          const int first = 32 * warp;
          uint32_t w[2][8] = {};
          if ((REVERSE ? k0 >= first : k0 <= first) && k0 < m) {
            uint32_t p[2][16];
            tmem_ld16_nw(p_at + k0, p[0]);
            tmem_ld16_nw(p_at + k0 + 16, p[1]);
            tmem_wait_ld16x2(p[0], p[1]);
            if (far) {
              const float more = two_to(max(0, top - 127));
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 16; ++j) p[q][j] = __float_as_uint(__uint_as_float(p[q][j]) * more);
            }
            if (k0 != first) {  // a^|i - j| as a power of the row and one of the column
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int k = k0 + 16 * q;
                const float r = mine * linear::power(log2a, REVERSE ? k - row : row - k - 15);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float2 f = mul2(mul2(make_float2(__uint_as_float(p[q][2 * j]),
                                                         __uint_as_float(p[q][2 * j + 1])),
                                             make_float2(r, r)), step[j]);
                  w[q][j] = pack_h2(f.x, f.y);
                }
              }
            } else {  // across the diagonal
              const float* const at = powers + (REVERSE ? -lane : lane);
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const int t = 16 * q + 2 * j;
                  const float2 f = mul2(mul2(make_float2(__uint_as_float(p[q][2 * j]),
                                                         __uint_as_float(p[q][2 * j + 1])),
                                             make_float2(mine, mine)),
                                        REVERSE ? make_float2(at[t], at[t + 1])
                                                  : make_float2(at[-t], at[-t - 1]));
                  w[q][j] = pack_h2(f.x, f.y);
                }
            }
            if (k0 + 32 > m) {  // (columns of another sequence's rows, or of none)
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const int left = m - k0 - 16 * q - 2 * j;
                  w[q][j] = left > 1 ? w[q][j] : left == 1 ? w[q][j] & 0xffffu : 0u;
                }
            }
          }
          tmem_st8_nw(p_at + k0 / 2, w[0]);
          tmem_st8_nw(p_at + k0 / 2 + 8, w[1]);
        }
        tmem_wait_st();
        fence_before_sync();
        mbar_arrive(bar(kWeights, it));
        // z goes behind W, where P has been read.  (Rows behind the chunk's last token: whatever they
        // hold ends in rows of O that nobody reads.)
        const float z_scale =
            two_to(14 - ez) *
            (!REVERSE || m == C ? z_whole : row < m ? linear::power(log2a, m - 1 - row) : 0.f);
#pragma unroll 1
        for (int p0 = 0; p0 < A / 8; p0 += 4) {
          uint4 v[4];
          open_pieces(base + (it & 1) * PassSmem::stage + PassSmem::Z, row, p0, z_scale, v);
#pragma unroll
          for (int p = 0; p < 4; p += 2) {
            const uint32_t w[8] = {v[p].x, v[p].y, v[p].z, v[p].w,
                                   v[p + 1].x, v[p + 1].y, v[p + 1].z, v[p + 1].w};
            tmem_st8_nw(p_at + 64 + 4 * (p0 + p), w);
          }
        }
        tmem_wait_st();
        fence_before_sync();
        mbar_arrive(bar(kTargets, it));
      }
    }
  } else if (warp < kFirstOpen) {
    // ---------------------------------------------------------------- the state, and the outputs
    take_registers<136>();
    const int st = tid - 32 * kFirstState, row = st & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16, cols = (uint32_t)(st >> 7) * 64;
    const uint32_t copy = base + PassSmem::S + (st >> 7) * kBlock + row * 128;
    const uint32_t turn = (uint32_t)(row & 7);
    const bool mine = (int)cols < B, grows = mine && row < A;
    float2 S[32];
    auto give = [&](int it, int c, int g, int E) {  // (its sums are there)
      const int m = tokens(c), ez = targets[C * (it & 1) + row], e = ez == kNoRow ? 0 : ez + E - 29;
      const int near = max(-126, min(e, 127));
      const float s0 = two_to(near);
      const bool far = __any_sync(0xffffffffu, near != e), live = row < m && !*failed;
      const bool last = !SUM || g + 1 == share;
      if (!mine) {  // (half of the threads have no columns of 64)
        mbar_arrive(bar(kSumsRead, it));
        mbar_arrive(bar(kOut, it));
        return;
      }
      const uint32_t tile = base + (it & 1) * PassSmem::stage + PassSmem::Y + (st >> 7) * kBlock + row * 128;
#pragma unroll 1
      for (int k = 0; k < 64; k += 32) {
        uint32_t o[2][16];
        tmem_ld16_nw(tm_o + lanes + cols + k, o[0]);
        tmem_ld16_nw(tm_o + lanes + cols + k + 16, o[1]);
        tmem_wait_ld16x2(o[0], o[1]);
        if (k == 32) {  // (the next chunk's sums may take their place)
          fence_before_sync();
          mbar_arrive(bar(kSumsRead, it));
        }
        float2 f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          f[i] = mul2(make_float2(__uint_as_float(o[i / 8][2 * i % 16]),
                                  __uint_as_float(o[i / 8][2 * i % 16 + 1])), make_float2(s0, s0));
        if (far) {
          const float s1 = two_to(e - near);
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = mul2(f[i], make_float2(s1, s1));
        }
        if (SUM) {  // the running sum of a chunk: row after row of each four columns
          float4* const sum =
              reinterpret_cast<float4*>(a.partial + ((int64_t)oh * a.s.T + first_token(c)) * B) +
              (int64_t)((cols + k) / 4) * m + row;
          if (g > 0 && live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 before = sum[i * m];
              f[2 * i].x += before.x; f[2 * i].y += before.y;
              f[2 * i + 1].x += before.z; f[2 * i + 1].y += before.w;
            }
          }
          if (!last && live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              sum[i * m] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
          }
        }
        if (last) {
          uint4 b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            b[i] = make_uint4(pack_bf2(f[4 * i].x, f[4 * i].y), pack_bf2(f[4 * i + 1].x, f[4 * i + 1].y),
                              pack_bf2(f[4 * i + 2].x, f[4 * i + 2].y),
                              pack_bf2(f[4 * i + 3].x, f[4 * i + 3].y));
          if (m == C) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sts16(tile + (((k / 8 + i) ^ turn) << 4), b[i]);
          } else if (live) {
            uint4* const out = reinterpret_cast<uint4*>(
                static_cast<__nv_bfloat16*>(a.out) + ((int64_t)(first_token(c) + row) * heads + oh) * B +
                cols + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = b[i];
          }
        }
        __syncwarp();
      }
      fence_async_smem();
      mbar_arrive(bar(kOut, it));
    };
    int grown = 0, c = 0, g = 0, c_before = 0, g_before = 0, E_before = 0, E = 0;
    float log2a = 0.f;
    Bound bound = {};
#pragma unroll 1
    for (int it = 0; it <= total; ++it) {
      if (it < total && c == 0) {
        const int64_t where = slot * a.s.hv + oh * share + g;
        log2a = linear::log2_decay(a.s, oh * share + g);
        const float* from = a.states + where * A * B;
        const Tops tops = tops_of(a, where);
        const float enter = REVERSE ? 1.f : linear::power(log2a, 1);
        uint32_t top = 0;
        if (!grows) {
#pragma unroll
          for (int i = 0; i < 32; ++i) S[i] = make_float2(0.f, 0.f);
        } else if (a.transposed) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            S[i] = make_float2(from[(cols + 2 * i) * A + row], from[(cols + 2 * i + 1) * A + row]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float4 v = *reinterpret_cast<const float4*>(from + row * B + cols + 2 * i);
            S[i] = make_float2(v.x, v.y);
            S[i + 1] = make_float2(v.z, v.w);
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          S[i] = mul2(S[i], make_float2(enter, enter));
          top = max(top, max(__float_as_uint(S[i].x) & 0x7fffffffu, __float_as_uint(S[i].y) & 0x7fffffffu));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        // (the weights have passed the last head's start, and cleared this one's max: with one chunk a
        // head nothing else says so)
        if (g > 0) wait_bar(one(kBegun), (g - 1) & 1, failed);
        if (lane == 0) atomicMax(misc + 2 + (g & 1), (int)top);
        mbar_arrive(one(kStart));
        wait_bar(one(kStart), g & 1, failed);
        bound.start(((volatile int*)misc)[2 + (g & 1)], tops, log2a);
      }
      if (SUM && it > 0 && g_before > 0 && lane % 8 == 0) {  // (the running sum's lines, 8 rows each)
        const int m = tokens(c_before);
        const float4* sum =
            reinterpret_cast<const float4*>(a.partial + ((int64_t)oh * a.s.T + first_token(c_before)) * B) +
            (int64_t)(cols / 4) * m + row;
        if (mine && row < m)
          for (int i = 0; i < 16; ++i) asm volatile("prefetch.global.L1 [%0];" ::"l"(sum + i * m));
      }
      __syncwarp();
      if (it > 0) {  // (the last chunk's use of the copy)
        wait_bar(one(kSums), (it - 1) & 1, failed);
        fence_after_sync();
        give(it - 1, c_before, g_before, E_before);
      }
      if (it < total) {
        E = bound.E();
        const float s = two_to(max(15 - E, -126));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!mine) break;
          float2 f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = mul2(S[4 * k + i], make_float2(s, s));
          if (E > 141) {  // (the factor is below fp32's range, what it makes is not)
            const float s1 = two_to(141 - E);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], make_float2(s1, s1));
          }
          sts16(copy + ((k ^ turn) << 4), make_uint4(pack_h2(f[0].x, f[0].y), pack_h2(f[1].x, f[1].y),
                                                     pack_h2(f[2].x, f[2].y), pack_h2(f[3].x, f[3].y)));
        }
        fence_async_smem();
        mbar_arrive(one(kStateIn));
      }
      if (it < total) {
        const int m = tokens(c);
        const float w = m == C ? bound.whole : linear::power(log2a, m);
        bound.grow(w);
        if (c + 1 < chunks) {
          const float add = two_to(min(bound.M - 29, 127));
          wait_bar(one(kGrown), grown & 1, failed);
          fence_after_sync();
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            // (a warp's rows are all before A, or all behind it)
            if (!grows) break;
            uint32_t p[16];
            tmem_ld16_nw(tm_g + lanes + cols + 2 * k, p);
            tmem_wait_ld16(p);
            if (bound.M > 156) {  // (beyond it, likewise)
              const float more = two_to(bound.M - 156);
#pragma unroll
              for (int i = 0; i < 16; ++i) p[i] = __float_as_uint(__uint_as_float(p[i]) * more);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              S[k + i] = __ffma2_rn(S[k + i], make_float2(w, w),
                                    mul2(make_float2(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1])),
                                         make_float2(add, add)));
          }
          fence_before_sync();
          mbar_arrive(one(kTaken));
          ++grown;
        }
      }
      c_before = c;
      g_before = g;
      E_before = E;
      if (++c == chunks) {
        c = 0;
        ++g;
      }
    }
  } else {
    // ---------------------------------------------------------------- rows opened to fp16
    leave_registers<56>();
    const int row = tid - 32 * kFirstOpen;  // one thread a row
    int it = 0;
    for (int g = 0; g < share; ++g) {
      const int64_t at = slot * a.s.hv + oh * share + g;
      const float log2a = linear::log2_decay(a.s, oh * share + g);
      const Tops tops = tops_of(a, at);
      const float x_scale = two_to(15 + tops.ey - tops.M);
      const float x_whole = linear::power(log2a, REVERSE ? row + 1 : C - row) * x_scale;
      for (int c = 0; c < chunks; ++c, ++it) {
        const int m = tokens(c);
        const bool live = row < m;
        const uint32_t st = base + (it & 1) * PassSmem::stage;
        wait_bar(bar(kFull, it), half(it), failed);
        const uint32_t most = live ? row_max_of(st + PassSmem::Z, row, A) : 0u;
        const int ez = most ? max(exponent_of(larger_of_two(most)), kLeastRow) : kNoRow;
        if (it >= 2) wait_bar(bar(kSumsRead, it - 2), half(it - 2), failed);  // (who reads it there)
        targets[C * (it & 1) + row] = ez;
        mbar_arrive(bar(kRows, it));
        if (c + 1 < chunks) {
          wait_bar(bar(kScores, it), half(it), failed);  // (x as it was has been read)
          open_row(st + PassSmem::X, row, A, live,
                   REVERSE || m == C ? x_whole : live ? linear::power(log2a, m - row) * x_scale : 0.f);
        }
        wait_bar(bar(kFullY, it), half(it), failed);
        open_row(st + PassSmem::Y, row, B, live, two_to(14 - tops.ey));
        fence_async_smem();
        mbar_arrive(bar(kValues, it));
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tm, 512);
  if (tid == 0 && *failed) set_status(a.s.status, GDN_ERR_DEVICE_TIMEOUT);
}

// Rows [T, heads, width] bf16 read in boxes of 64 features of one head and `tokens` tokens (128-byte
// swizzle); tokens past T read as zeros.
cudaError_t rows_map(CUtensorMap* m, const LinearRows& r, int64_t T, int heads, int width, int tokens) {
  EncodeTiled fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  // (The driver's call wants a context on the thread, which a thread's first runtime call alone may not have
  // made: an autograd engine's thread comes here with none.)
  thread_local int bound = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev != bound) {
    e = cudaSetDevice(dev);
    if (e == cudaSuccess) bound = dev;
  }
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)T};
  // (the stride of a dimension of one row means nothing, but has to be one)
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? r.hs * 2 : width * 2),
                                 (cuuint64_t)(T > 1 ? r.ts * 2 : (int64_t)heads * width * 2)};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)tokens}, each[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(r.p), dims, strides, box, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool WIDE> cudaError_t launch_state(const LinearState& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_state_tc_kernel<WIDE>, StateSmem::bytes, done);
  CUtensorMap mx, my;
  if (e == cudaSuccess) e = rows_map(&mx, a.x, a.s.T, a.s.hv / a.x.share, a.s.K, kTile);
  if (e == cudaSuccess) e = rows_map(&my, a.y, a.s.T, a.s.hv / a.y.share, a.s.V, kTile);
  if (e != cudaSuccess) return e;
  return launch_ordered(linear_state_tc_kernel<WIDE>, dim3((unsigned)(a.s.slots * a.s.hv)), kStateThreads,
                        StateSmem::bytes, s, a, mx, my);
}

template <bool REVERSE, bool SUM, bool WIDE> cudaError_t launch_pass(const LinearPass& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_pass_tc_kernel<REVERSE, SUM, WIDE>, PassSmem::bytes, done);
  const int heads = a.s.hv / a.out_share;
  const LinearRows out = {a.out, (int64_t)heads * a.B, a.B, a.out_share};
  CUtensorMap mz, mx, my, mo;
  if (e == cudaSuccess) e = rows_map(&mz, a.z, a.s.T, a.s.hv / a.z.share, a.A, C);
  if (e == cudaSuccess) e = rows_map(&mx, a.x, a.s.T, a.s.hv / a.x.share, a.A, C);
  if (e == cudaSuccess) e = rows_map(&my, a.y, a.s.T, a.s.hv / a.y.share, a.B, C);
  if (e == cudaSuccess) e = rows_map(&mo, out, a.s.T, heads, a.B, C);
  if (e != cudaSuccess) return e;
  return launch_ordered(linear_pass_tc_kernel<REVERSE, SUM, WIDE>, dim3((unsigned)(a.s.slots * heads)),
                        kPassThreads, PassSmem::bytes, s, a, mz, mx, my, mo);
}

}  // namespace

cudaError_t linear_state_tc(const LinearState& a, cudaStream_t s) {
  return a.s.K == D && a.s.V == D ? launch_state<true>(a, s) : launch_state<false>(a, s);
}

cudaError_t linear_pass_tc(const LinearPass& a, cudaStream_t s) {
  const bool wide = a.A == D && a.B == D;
  if (a.out_share > 1) {
    if (a.reverse) return wide ? launch_pass<true, true, true>(a, s) : launch_pass<true, true, false>(a, s);
    return wide ? launch_pass<false, true, true>(a, s) : launch_pass<false, true, false>(a, s);
  }
  if (a.reverse) return wide ? launch_pass<true, false, true>(a, s) : launch_pass<true, false, false>(a, s);
  return wide ? launch_pass<false, false, true>(a, s) : launch_pass<false, false, false>(a, s);
}

}  // namespace gdn
