// gdn_linear_tc.cu -- linear attention with a decay for each head (gdn_linear.h) on the fifth-generation
// tensor cores: bf16 I/O, K = V = 128.
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

constexpr int D = 128;                            // K and V
constexpr long long kWaitCycles = 2000000000LL;   // limit of a bounded wait: about a second

// true in one thread of a converged warp
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// Bounded wait of a warp: sleeps in hardware; gives up after about a second, or when another has.
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, volatile int* failed) {
  bool done = mbar_try(bar, parity);
  if (!done) {
    const long long began = clock64();
    while (!done && !*failed) {
      done = mbar_try(bar, parity);
      if (!done && clock64() - began > kWaitCycles) *failed = 1;
    }
  }
  __syncwarp();
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

// ------------------------------------------------------------------ a segment's own state

// U = sum of weighted x y^T over a segment, to fp32 accuracy: y's rows times their powers of the decay
// are split into three bf16 parts (24 bits), x is bf16 as it stands, products and their sums are exact
// or fp32.  64 tokens at a time go through the tensor core into Tensor Memory and from there into a
// register-held U, decayed on the way: the weights stay within a tile, and the tensor core's own sums,
// whose roundings do not average out, stay short.
constexpr int kTile = 64, kWorkers = 256, kStateThreads = kWorkers + 32;
constexpr uint32_t kRaw = kTile * D * 2;          // bytes of a tile of one tensor
struct StateSmem {                                // offsets from a 1024-byte boundary
  static constexpr uint32_t X = 0, Y = 2 * kRaw, MID = 4 * kRaw, LOW = 5 * kRaw, BARS = 6 * kRaw;
  static constexpr int bytes = BARS + 64 + 1024;
};

__global__ void __launch_bounds__(kStateThreads, 2)
linear_state_tc_kernel(const LinearState a, const __grid_constant__ CUtensorMap mx,
                       const __grid_constant__ CUtensorMap my) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_word;
  volatile int* failed = &failed_word;
  stream_order();
  if (!linear::usable(a.s)) return;
  const int head = blockIdx.x % a.s.hv;
  const int64_t slot = blockIdx.x / a.s.hv;
  int n;
  int64_t t0, t1;
  if (!linear::slot_tokens(a.s, slot, n, t0, t1)) return;
  const uint32_t base = (saddr(raw_smem) + 1023u) & ~1023u;
  const uint32_t full = base + StateSmem::BARS, ready = full + 16, done = ready + 8, end = done + 16;
  const int tid = threadIdx.x, warp = tid / 32;
  if (tid == 0) {
    failed_word = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(done + 8 * i, 1);
    }
    mbar_init(ready, kWorkers);
    mbar_init(end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 8) {
    tmem_alloc(saddr(&tmem_at), 256);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = tmem_at;
  const int tiles = (int)((t1 - t0 + kTile - 1) / kTile);
  // the i-th tile of the walk, its tokens
  auto first_token = [&](int i) { return t0 + (int64_t)(a.reverse ? tiles - 1 - i : i) * kTile; };
  auto tokens = [&](int i) { const int64_t m = t1 - first_token(i); return m < kTile ? (int)m : kTile; };

  if (warp == 8) {
    // ---------------------------------------------------------------- loads and products
    int loaded = 0;
    auto load = [&](int i) {
      if (elected()) {
        const uint32_t bar = full + 8 * (i & 1), x = base + StateSmem::X + (i & 1) * kRaw,
                       y = base + StateSmem::Y + (i & 1) * kRaw;
        const int t = (int)first_token(i);
        mbar_expect_tx(bar, 2 * kRaw);
        for (int b = 0; b < 2; ++b) {
          tma_box(x + b * (kRaw / 2), &mx, 64 * b, head / a.x.share, t, bar);
          tma_box(y + b * (kRaw / 2), &my, 64 * b, head / a.y.share, t, bar);
        }
      }
      __syncwarp();
      loaded = i + 1;
    };
    for (int i = 0; i < 2 && i < tiles; ++i) load(i);
    const uint32_t id = idesc_f16(128, 128, 1, 1, 1);
    for (int i = 0; i < tiles; ++i) {
      wait_bar(ready, i & 1, failed);
      if (*failed) break;
      fence_after_sync();
      const uint32_t x = base + StateSmem::X + (i & 1) * kRaw;
      const uint32_t parts[3] = {base + StateSmem::LOW, base + StateSmem::MID,
                                 base + StateSmem::Y + (i & 1) * kRaw};
      if (elected()) {
#pragma unroll
        for (int p = 0; p < 3; ++p)  // (the small parts first)
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            mma_ss(tm + 128 * (i & 1), sdesc(x + ks * 2048, kRaw / 2, 1024),
                   sdesc(parts[p] + ks * 2048, kRaw / 2, 1024), id, p > 0 || ks > 0);
        mma_commit(done + 8 * (i & 1));
      }
      __syncwarp();
      if (i + 2 < tiles) {
        wait_bar(done + 8 * (i & 1), (i >> 1) & 1, failed);
        if (*failed) break;
        load(i + 2);
      }
    }
    if (*failed) {
      if (elected()) {
        mma_commit(end);
        drain(end, 0);
        for (int i = loaded > 2 ? loaded - 2 : 0; i < loaded; ++i) drain(full + 8 * (i & 1), (i >> 1) & 1);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- weights, parts, the sum
    const float log2a = linear::log2_decay(a.s, head);
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16, cols = (uint32_t)(warp >> 2) * 64;
    float u[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) u[i] = 0.f;
    auto add = [&](int i) {  // tile i into u
      wait_bar(done + 8 * (i & 1), (i >> 1) & 1, failed);
      fence_after_sync();
      const float w = linear::power(log2a, tokens(i));
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        uint32_t p[16];
        tmem_ld16_nw(tm + lanes + 128 * (i & 1) + cols + c, p);
        tmem_wait_ld16(p);
#pragma unroll
        for (int k = 0; k < 16; ++k) u[c + k] = fmaf(w, u[c + k], __uint_as_float(p[k]));
      }
    };
    for (int i = 0; i < tiles; ++i) {
      const uint32_t x = base + StateSmem::X + (i & 1) * kRaw, y = base + StateSmem::Y + (i & 1) * kRaw;
      const int m = tokens(i);
      wait_bar(full + 8 * (i & 1), (i >> 1) & 1, failed);
      if (i > 0) wait_bar(done + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, failed);  // the parts' tiles
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const uint32_t at = 16 * (tid + kWorkers * k);  // a 16-byte piece of a row
        const int r = at / 128 % kTile;
        const float w = linear::power(log2a, a.reverse ? r + 1 : m - 1 - r);
        uint4 v = lds16(y + at), mid, lo;
        uint32_t* pv = &v.x;
        uint32_t* pm = &mid.x;
        uint32_t* pl = &lo.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f0 = r < m ? low(pv[j]) * w : 0.f, f1 = r < m ? high(pv[j]) * w : 0.f;
          pv[j] = pack_bf2(f0, f1);
          f0 -= low(pv[j]);
          f1 -= high(pv[j]);
          pm[j] = pack_bf2(f0, f1);
          pl[j] = pack_bf2(f0 - low(pm[j]), f1 - high(pm[j]));
        }
        sts16(y + at, v);
        sts16(base + StateSmem::MID + at, mid);
        sts16(base + StateSmem::LOW + at, lo);
        if (r >= m) sts16(x + at, make_uint4(0, 0, 0, 0));  // (another sequence's rows, or none)
      }
      fence_async_smem();
      fence_before_sync();
      mbar_arrive(ready);
      if (i > 0) add(i - 1);
    }
    add(tiles - 1);
    float* out = a.states + (slot * a.s.hv + head) * D * D + (int64_t)(tid & 127) * D + cols;
    if (!*failed) {
#pragma unroll
      for (int c = 0; c < 64; c += 4)
        *reinterpret_cast<float4*>(out + c) = make_float4(u[c], u[c + 1], u[c + 2], u[c + 3]);
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 8) tmem_dealloc(tm, 256);
  if (tid == 0 && *failed) set_status(a.s.status, GDN_ERR_DEVICE_TIMEOUT);
}

// ------------------------------------------------------------------ the pass

// One block walks a segment's chunks of 128 tokens (for every value head that its output head sums).
// Per chunk, with i, j counted in the walk's direction, p_i = a^i and n the chunk's tokens:
//     P = z x^T                       bf16 as loaded, into Tensor Memory
//     W = P a^{i - j}, j <= i         fp16, in P's place: an operand in Tensor Memory
//     O = W y + (p_i z) S             fp16 operands, one fp32 sum
//     S <- a^n S + (a^{n - j} x)^T y  fp16 operands; S fp32 in registers, its fp16 copy in shared memory
// fp16's range is not bf16's, so operands are scaled by powers of two, which come off again in fp32:
// a row of y, x or z by that of its largest magnitude, e_y, e_x, e_z; with M = max_j(e_x + e_y) and 2^E
// a bound of S and of 2^(M + 7):
//     y~ = y 2^(14 - e_y)     x~ = a^{n - j} x 2^(15 + e_y - M)     S~ = S 2^(15 - E)
//     z~ = p_i z 2^(14 - e_z)   W~ = W 2^(15 + e_y - e_z - E)         O = O~ 2^(e_z + E - 29)
// so that nothing can overflow that does not in fp32, and each rounding is half a step of fp16 (2^-11) of
// a term, or 2^-38 of what bounds the sum.
constexpr int C = 128;
constexpr uint32_t kTileBytes = C * D * 2, kBlock = kTileBytes / 2;  // (a block: 64 columns)
constexpr int kWeightWarps = 4, kStateWarps = 8, kOpenWarps = 4;
constexpr int kPassThreads = 32 * (kWeightWarps + kStateWarps + kOpenWarps + 2);
constexpr int kFirstState = kWeightWarps, kFirstOpen = kFirstState + kStateWarps,
              kLoadWarp = kFirstOpen + kOpenWarps, kMmaWarp = kLoadWarp + 1;
struct PassTables {           // a chunk's, double-buffered
  int8_t ey[C], ez[C];        // (e_y, e_z clamped to [-113, 127], [-60, 127])
  int M, E;
};
struct PassSmem {             // offsets from a 1024-byte boundary
  static constexpr uint32_t Z = 0, X = kTileBytes, Y = 2 * kTileBytes, stage = 3 * kTileBytes;
  static constexpr uint32_t S = 2 * stage, POWERS = S + kTileBytes, TABLES = POWERS + C * 4;
  static constexpr uint32_t BARS = TABLES + 2 * sizeof(PassTables), MISC = BARS + 20 * 8;
  static constexpr int bytes = MISC + 48 + 1024;
};
static_assert(PassSmem::bytes <= 232448, "shared memory of a block");
// barriers: those of a pair alternate from chunk to chunk
enum { kFull = 0, kScores = 2, kTables = 4, kWeights = 6, kOpened = 8, kFree = 10, kStateIn = 12,
       kGrown, kTaken, kSums, kSumsRead, kStart, kEnd };

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
// e with |v| < 2^e for the largest magnitude in packed bf16 bits; of zeros the least
__device__ __forceinline__ int exponent_of(uint32_t packed_max, int least) {
  const uint32_t m = max(packed_max & 0xffffu, packed_max >> 16);
  return max(min((int)(m >> 7) - 126, 127), least);
}
// packed bf16 times f, as packed fp16
__device__ __forceinline__ uint32_t to_half2(uint32_t bf2, float f) {
  return pack_h2(low(bf2) * f, high(bf2) * f);
}

__global__ void __launch_bounds__(kPassThreads, 1)
linear_pass_tc_kernel(const LinearPass a, const __grid_constant__ CUtensorMap mz,
                      const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my) {
  extern __shared__ uint8_t raw_smem[];
  stream_order();
  if (!linear::usable(a.s)) return;
  const int heads = a.s.hv / a.out_share;
  const int oh = blockIdx.x % heads;
  const int64_t slot = blockIdx.x / heads;
  int n;
  int64_t t0, t1;
  if (!linear::slot_tokens(a.s, slot, n, t0, t1)) return;
  const uint32_t base = (saddr(raw_smem) + 1023u) & ~1023u;
  uint8_t* const gbase = raw_smem + (base - saddr(raw_smem));
  float* const powers = reinterpret_cast<float*>(gbase + PassSmem::POWERS);
  PassTables* const tables = reinterpret_cast<PassTables*>(gbase + PassSmem::TABLES);
  int* const misc = reinterpret_cast<int*>(gbase + PassSmem::MISC);
  volatile int* const failed = misc;       // 0: failed, 1: Tensor Memory, 2-3: max |S| at a head's start,
  int* const row_max = misc + 4;           // 4-11: a chunk's M by warp, twice
  const uint32_t bars = base + PassSmem::BARS;
  auto bar = [&](int which, int it) { return bars + 8 * (which + (it & 1)); };
  auto one = [&](int which) { return bars + 8 * which; };
  auto half = [](int it) { return (uint32_t)(it >> 1) & 1; };
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    misc[0] = misc[2] = misc[3] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kFull, i), 1);
      mbar_init(bar(kScores, i), 1);
      mbar_init(bar(kFree, i), 1);
      mbar_init(bar(kTables, i), 32 * kOpenWarps);
      mbar_init(bar(kWeights, i), 32 * kWeightWarps);
      mbar_init(bar(kOpened, i), 32 * kOpenWarps);
    }
    mbar_init(one(kStateIn), 32 * kStateWarps);
    mbar_init(one(kGrown), 1);
    mbar_init(one(kTaken), 32 * kStateWarps);
    mbar_init(one(kSums), 1);
    mbar_init(one(kSumsRead), 32 * kWeightWarps);
    mbar_init(one(kStart), 32 * kStateWarps);
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
  const uint32_t tm = (uint32_t)misc[1], tm_o = tm + 256, tm_g = tm + 384;  // P twice, O, growth of S
  const int chunks = (int)((t1 - t0 + C - 1) / C), total = chunks * a.out_share;
  auto first_token = [&](int c) { return t0 + (int64_t)(a.reverse ? chunks - 1 - c : c) * C; };
  auto tokens = [&](int c) { const int64_t m = t1 - first_token(c); return m < C ? (int)m : C; };

  if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- loads
    int it = 0;
    for (int g = 0; g < a.out_share && !*failed; ++g) {
      const int head = oh * a.out_share + g;
      for (int c = 0; c < chunks; ++c, ++it) {
        if (it >= 2) wait_bar(bar(kFree, it), half(it - 2), failed);
        if (*failed) break;
        if (elected()) {
          const uint32_t b = bar(kFull, it), st = base + (it & 1) * PassSmem::stage;
          const int t = (int)first_token(c);
          mbar_expect_tx(b, PassSmem::stage);
          for (int k = 0; k < 2; ++k) {
            tma_box(st + PassSmem::Z + k * kBlock, &mz, 64 * k, head / a.z.share, t, b);
            tma_box(st + PassSmem::X + k * kBlock, &mx, 64 * k, head / a.x.share, t, b);
          }
          for (int k = 0; k < 2; ++k)
            tma_box(st + PassSmem::Y + k * kBlock, &my, 64 * k, head / a.y.share, t, b);
        }
        __syncwarp();
      }
    }
    if (*failed && lane == 0)
      for (int i = it > 2 ? it - 2 : 0; i < it; ++i) drain(bar(kFull, i), half(i));
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    const uint32_t id_p = idesc_f16(128, 128, 0, 0, 1), id_o = idesc_f16(128, 128, 0, 1),
                   id_g = idesc_f16(128, 128, 1, 1);
    auto scores = [&](int it) {
      wait_bar(bar(kFull, it), half(it), failed);
      fence_after_sync();
      const uint32_t st = base + (it & 1) * PassSmem::stage;
      if (elected()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t at = (ks >> 2) * kBlock + (ks & 3) * 32;
          mma_ss(tm + 128 * (it & 1), sdesc(st + PassSmem::Z + at, 16, 1024),
                 sdesc(st + PassSmem::X + at, 16, 1024), id_p, ks > 0);
        }
        mma_commit(bar(kScores, it));
      }
      __syncwarp();
    };
    scores(0);
    int grown = 0;
    for (int it = 0, c = 0; it < total && !*failed; ++it, c = c + 1 == chunks ? 0 : c + 1) {
      const uint32_t st = base + (it & 1) * PassSmem::stage;
      if (it + 1 < total) scores(it + 1);
      wait_bar(bar(kTables, it), half(it), failed);
      wait_bar(bar(kOpened, it), half(it), failed);
      if (c + 1 < chunks) {
        if (grown > 0) wait_bar(one(kTaken), (grown - 1) & 1, failed);
        fence_after_sync();
        if (elected()) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss(tm_g, sdesc(st + PassSmem::X + ks * 2048, kBlock, 1024),
                   sdesc(st + PassSmem::Y + ks * 2048, kBlock, 1024), id_g, ks > 0);
          mma_commit(one(kGrown));
        }
        __syncwarp();
        ++grown;
      }
      wait_bar(bar(kWeights, it), half(it), failed);
      if (it > 0) wait_bar(one(kSumsRead), (it - 1) & 1, failed);
      fence_after_sync();
      if (elected()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts(tm_o, tm + 128 * (it & 1) + 8 * ks, sdesc(st + PassSmem::Y + ks * 2048, kBlock, 1024),
                 id_o, ks > 0);
      }
      __syncwarp();
      wait_bar(one(kStateIn), it & 1, failed);
      fence_after_sync();
      if (elected()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss(tm_o, sdesc(st + PassSmem::Z + (ks >> 2) * kBlock + (ks & 3) * 32, 16, 1024),
                 sdesc(base + PassSmem::S + ks * 2048, kBlock, 1024), id_o, 1);
        mma_commit(one(kSums));
        mma_commit(bar(kFree, it));
      }
      __syncwarp();
    }
    if (*failed) {
      if (elected()) {
        mma_commit(one(kEnd));
        drain(one(kEnd), 0);
      }
      __syncwarp();
    }
  } else if (warp < kWeightWarps) {
    // ---------------------------------------------------------------- weights, and the outputs
    const int row = tid;  // its lane of Tensor Memory
    const uint32_t lanes = (uint32_t)warp * 32 << 16;
    const int64_t ots = (int64_t)heads * D;
    float log2a = 0.f;
    auto give = [&](int it, int c, int g) {
      const int m = tokens(c);
      const int64_t at = (first_token(c) + row) * ots + (int64_t)oh * D;
      wait_bar(one(kSums), it & 1, failed);
      fence_after_sync();
      const PassTables& tab = tables[it & 1];
      const int e = tab.ez[row] + tab.E - 29;
      const float s0 = two_to(e / 2), s1 = two_to(e - e / 2);
      const bool live = row < m && !*failed;
#pragma unroll
      for (int k = 0; k < D; k += 32) {
        uint32_t o[2][16];
        tmem_ld16_nw(tm_o + lanes + k, o[0]);
        tmem_ld16_nw(tm_o + lanes + k + 16, o[1]);
        tmem_wait_ld16x2(o[0], o[1]);
        if (live) {
          float f[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i / 16][i % 16]) * s0 * s1;
          if (g > 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 before = *reinterpret_cast<const float4*>(a.partial + at + k + i);
              f[i] += before.x; f[i + 1] += before.y; f[i + 2] += before.z; f[i + 3] += before.w;
            }
          }
          if (g + 1 < a.out_share) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(a.partial + at + k + i) =
                  make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at + k + i) =
                  make_uint4(pack_bf2(f[i], f[i + 1]), pack_bf2(f[i + 2], f[i + 3]),
                             pack_bf2(f[i + 4], f[i + 5]), pack_bf2(f[i + 6], f[i + 7]));
          }
        }
        __syncwarp();
      }
      fence_before_sync();
      mbar_arrive(one(kSumsRead));
    };
    int it = 0, c_before = 0, g_before = 0;  // (a chunk's outputs follow the next one's weights)
    for (int g = 0; g < a.out_share; ++g) {
      log2a = linear::log2_decay(a.s, oh * a.out_share + g);
      named_bar(1, 32 * kWeightWarps);  // (the last head's powers have been read)
      powers[row] = linear::power(log2a, row);
      named_bar(1, 32 * kWeightWarps);
      for (int c = 0; c < chunks; ++c, ++it) {
        const int m = tokens(c);
        wait_bar(bar(kTables, it), half(it), failed);
        wait_bar(bar(kScores, it), half(it), failed);
        fence_after_sync();
        const PassTables& tab = tables[it & 1];
        const int e = 15 - tab.ez[row] - tab.E;
        const float s0 = two_to(e / 2), s1 = two_to(e - e / 2);
        const uint32_t p_at = tm + lanes + 128 * (it & 1);
#pragma unroll 1
        for (int k = 0; k < C; k += 16) {  // (whole pieces of the triangle that are zero are not read)
          const bool none = a.reverse ? k + 15 < 32 * warp : k > 32 * warp + 31;
          uint32_t w[8];
          if (none) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 0u;
          } else {
            uint32_t p[16];
            tmem_ld16_nw(p_at + k, p);
            tmem_wait_ld16(p);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float f[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int s = k + i + j, gap = a.reverse ? s - row : row - s;
                const float v = __uint_as_float(p[i + j]) * s0 * s1 * powers[gap & (C - 1)] *
                                two_to(tab.ey[s]);
                f[j] = gap >= 0 && s < m ? v : 0.f;
              }
              w[i / 2] = pack_h2(f[0], f[1]);
            }
          }
          tmem_st8_nw(p_at + k / 2, w);
        }
        tmem_wait_st();
        fence_before_sync();
        mbar_arrive(bar(kWeights, it));
        if (it > 0) give(it - 1, c_before, g_before);
        c_before = c;
        g_before = g;
      }
    }
    give(total - 1, c_before, g_before);
  } else if (warp < kFirstOpen) {
    // ---------------------------------------------------------------- the state
    const int st = tid - 32 * kFirstState, row = st & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16, cols = (uint32_t)(st >> 7) * 64;
    const uint32_t copy = base + PassSmem::S + (st >> 7) * kBlock + row * 128;
    float S[64];
    int it = 0, grown = 0;
    for (int g = 0; g < a.out_share; ++g) {
      const int head = oh * a.out_share + g;
      const float log2a = linear::log2_decay(a.s, head);
      const float* from = a.states + (slot * a.s.hv + head) * D * D;
      const float enter = a.reverse ? 1.f : linear::power(log2a, 1);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        S[i] = enter * (a.transposed ? from[(cols + i) * D + row] : from[row * D + cols + i]);
        top = max(top, __float_as_uint(S[i]) & 0x7fffffffu);
      }
      atomicMax(misc + 2 + (g & 1), (int)__reduce_max_sync(0xffffffffu, top));
      mbar_arrive(one(kStart));
      for (int c = 0; c < chunks; ++c, ++it) {
        wait_bar(bar(kTables, it), half(it), failed);
        const int M = tables[it & 1].M;
        const float scale = two_to(15 - tables[it & 1].E);
        if (it > 0) wait_bar(one(kSums), (it - 1) & 1, failed);  // (the last chunk's use of the copy)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sts16(copy + ((k ^ (row & 7)) << 4),
                make_uint4(pack_h2(S[8 * k] * scale, S[8 * k + 1] * scale),
                           pack_h2(S[8 * k + 2] * scale, S[8 * k + 3] * scale),
                           pack_h2(S[8 * k + 4] * scale, S[8 * k + 5] * scale),
                           pack_h2(S[8 * k + 6] * scale, S[8 * k + 7] * scale)));
        fence_async_smem();
        mbar_arrive(one(kStateIn));
        if (c + 1 < chunks) {
          const float w = linear::power(log2a, tokens(c)), add = two_to(M - 29);
          wait_bar(one(kGrown), grown & 1, failed);
          fence_after_sync();
#pragma unroll
          for (int k = 0; k < 64; k += 16) {
            uint32_t p[16];
            tmem_ld16_nw(tm_g + lanes + cols + k, p);
            tmem_wait_ld16(p);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              S[k + i] = fmaf(w, S[k + i], __uint_as_float(p[i]) * add);
          }
          fence_before_sync();
          mbar_arrive(one(kTaken));
          ++grown;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- rows opened to fp16
    // One thread a row.  (Its 16-byte pieces are read in an order by which eight neighbouring rows
    // meet different banks: logical piece p of row r lies at p ^ (r & 7) anyway.)
    const int row = tid - 32 * kFirstOpen, ow = row / 32;
    const uint32_t turn = (uint32_t)(row & 7);
    auto piece = [&](int p) { return (uint32_t)((p >> 3) * kBlock + row * 128) + ((p & 7 ^ turn) << 4); };
    int it = 0;
    for (int g = 0; g < a.out_share; ++g) {
      const float log2a = linear::log2_decay(a.s, oh * a.out_share + g);
      double bound = 0.;  // of |S|
      for (int c = 0; c < chunks; ++c, ++it) {
        const int m = tokens(c), i = a.reverse ? m - 1 - row : row;
        const bool live = row < m;
        const uint32_t st = base + (it & 1) * PassSmem::stage;
        wait_bar(bar(kFull, it), half(it), failed);
        uint32_t x_max = 0, y_max = 0, z_max = 0;
#pragma unroll 4
        for (int p = 0; p < 16; ++p) {
          const uint4 x = lds16(st + PassSmem::X + piece(p)), y = lds16(st + PassSmem::Y + piece(p)),
                      z = lds16(st + PassSmem::Z + piece(p));
          const uint32_t* xv = &x.x;
          const uint32_t* yv = &y.x;
          const uint32_t* zv = &z.x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x_max = max_u16x2(x_max, xv[j] & 0x7fff7fffu);
            y_max = max_u16x2(y_max, yv[j] & 0x7fff7fffu);
            z_max = max_u16x2(z_max, zv[j] & 0x7fff7fffu);
          }
        }
        const int ex = live ? exponent_of(x_max, -110) : -110, ey = live ? exponent_of(y_max, -113) : -113;
        const int ez = live ? exponent_of(z_max, -60) : -60;
        const int warp_max = __reduce_max_sync(0xffffffffu, ex + ey);
        // (the chunk before the last has been given out: its table may be written again)
        if (it >= 2) wait_bar(one(kSumsRead), (it - 2) & 1, failed);
        if (lane == 0) row_max[4 * (it & 1) + ow] = warp_max;
        PassTables& tab = tables[it & 1];
        tab.ey[row] = (int8_t)ey;
        tab.ez[row] = (int8_t)ez;
        if (c == 0) wait_bar(one(kStart), g & 1, failed);
        named_bar(2, 32 * kOpenWarps);
        const int* rm = row_max + 4 * (it & 1);
        const int M = max(max(max(rm[0], rm[1]), max(rm[2], rm[3])), -97);
        if (c == 0) {
          bound = __int_as_float(misc[2 + (g & 1)]);
          named_bar(2, 32 * kOpenWarps);
          if (row == 0) misc[2 + (g & 1)] = 0;  // for the head after the next
        }
        const int E = max((__double2hiint(bound) >> 20) - 1022, M + 7);  // (|S| < 2^E)
        if (row == 0) {
          tab.M = M;
          tab.E = E;
        }
        bound = linear::power(log2a, m) * bound + (double)m * two_to(min(M, 120));
        const float y_scale = two_to(14 - ey);
#pragma unroll 4
        for (int p = 0; p < 16; ++p) {
          const uint32_t at = st + PassSmem::Y + piece(p);
          uint4 y = lds16(at);
          y.x = to_half2(y.x, y_scale);
          y.y = to_half2(y.y, y_scale);
          y.z = to_half2(y.z, y_scale);
          y.w = to_half2(y.w, y_scale);
          sts16(at, live ? y : make_uint4(0, 0, 0, 0));
        }
        fence_async_smem();
        mbar_arrive(bar(kTables, it));
        const float z_scale = linear::power(log2a, live ? i : 0) * two_to(14 - ez);
        const float x_scale = linear::power(log2a, live ? m - i : 0) * two_to(15 + ey - M);
        wait_bar(bar(kScores, it), half(it), failed);  // (x and z as they were have been read)
#pragma unroll 2
        for (int p = 0; p < 16; ++p) {
          const uint32_t xa = st + PassSmem::X + piece(p), za = st + PassSmem::Z + piece(p);
          uint4 x = lds16(xa), z = lds16(za);
          x.x = to_half2(x.x, x_scale);
          x.y = to_half2(x.y, x_scale);
          x.z = to_half2(x.z, x_scale);
          x.w = to_half2(x.w, x_scale);
          z.x = to_half2(z.x, z_scale);
          z.y = to_half2(z.y, z_scale);
          z.z = to_half2(z.z, z_scale);
          z.w = to_half2(z.w, z_scale);
          sts16(xa, live ? x : make_uint4(0, 0, 0, 0));
          sts16(za, live ? z : make_uint4(0, 0, 0, 0));
        }
        fence_async_smem();
        mbar_arrive(bar(kOpened, it));
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tm, 512);
  if (tid == 0 && *failed) set_status(a.s.status, GDN_ERR_DEVICE_TIMEOUT);
}

// Rows [T, heads, 128] bf16 read in boxes of 64 features of one head and `tokens` tokens (128-byte
// swizzle); tokens past T read as zeros.
cudaError_t rows_map(CUtensorMap* m, const LinearRows& r, int64_t T, int heads, int tokens) {
  EncodeTiled fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  // (the stride of a dimension of one row means nothing, but has to be one)
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? r.hs * 2 : D * 2),
                                 (cuuint64_t)(T > 1 ? r.ts * 2 : (int64_t)heads * D * 2)};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)tokens}, each[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(r.p), dims, strides, box, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t linear_state_tc(const LinearState& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_state_tc_kernel, StateSmem::bytes, done);
  CUtensorMap mx, my;
  if (e == cudaSuccess) e = rows_map(&mx, a.x, a.s.T, a.s.hv / a.x.share, kTile);
  if (e == cudaSuccess) e = rows_map(&my, a.y, a.s.T, a.s.hv / a.y.share, kTile);
  if (e != cudaSuccess) return e;
  return launch_ordered(linear_state_tc_kernel, dim3((unsigned)(a.s.slots * a.s.hv)), kStateThreads,
                        StateSmem::bytes, s, a, mx, my);
}

cudaError_t linear_pass_tc(const LinearPass& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_pass_tc_kernel, PassSmem::bytes, done);
  CUtensorMap mz, mx, my;
  if (e == cudaSuccess) e = rows_map(&mz, a.z, a.s.T, a.s.hv / a.z.share, C);
  if (e == cudaSuccess) e = rows_map(&mx, a.x, a.s.T, a.s.hv / a.x.share, C);
  if (e == cudaSuccess) e = rows_map(&my, a.y, a.s.T, a.s.hv / a.y.share, C);
  if (e != cudaSuccess) return e;
  return launch_ordered(linear_pass_tc_kernel, dim3((unsigned)(a.s.slots * (a.s.hv / a.out_share))),
                        kPassThreads, PassSmem::bytes, s, a, mz, mx, my);
}

}  // namespace gdn
