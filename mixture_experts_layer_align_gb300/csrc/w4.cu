// 4-bit weights with group scales: matrix-vector products and the expert
// products of the MoE layer for a few tokens.
//
// y[t][r] = sum over groups of scale[r][group] * sum_k x[t][k] (code[r][k] - zero[r][group]).
// At a few tokens the codes' bytes bound it, if turning them into an MMA operand
// does not: at 6.8 TB/s an SM takes in 47 codes a clock.
//
// A thread block has two warpgroups; each owns 128 weight rows and a slice of K
// (they take different rows, or different K of the same rows).  The blocks of a
// cluster share rows and split K further.  TMA brings 256 columns of the codes
// (128 bytes of a row) and of x a stage.  A warpgroup, a thread per row, turns 32
// codes at a time into bf16 (code - zero is a small integer: exact) and puts them
// into tensor memory, where they are the A operand (128 rows) of tcgen05.mma with
// the tokens in N.  The accumulators of each group come back, again a thread per
// row, and are scaled in fp32: no weight is rounded.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;      // weight rows of a warpgroup (64 gate and 64 up rows)
constexpr int kStepK = 256;     // columns of a stage for a warpgroup
constexpr int kCodeBytes = kRows * kStepK / 2;  // its codes
constexpr int kGroupThreads = 128;
constexpr int kThreads = 2 * kGroupThreads + 32;  // and a warp that issues the copies
constexpr unsigned long long kDrainNs = 1000000000ull;

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// The 8 codes of a word, two bf16 at a time: (code - zero) 2^-6.  As a bf16 a
// pattern of 0..255 is that many times 2^-133 (the two lowest exponents share
// their spacing), so a masked nibble needs one fused multiply-add: x 2^127 where
// it lies in bits 0..3 (even codes, low halves), x 2^123 in bits 4..7 (odd codes,
// high halves), - zero 2^-6, all exact.  The byte permutation takes byte i of the
// even and of the odd codes and, for the upper bytes, the sign of an even one: 0.
// nz holds -zero 2^-6 in both halves; the 2^6 is made good when sums are stored.
__device__ __forceinline__ void w4_pairs(uint32_t w, uint32_t nz, uint32_t* v) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = w & 0xf0f0f0f0u;
  v[0] = fma_bf16x2(prmt(even, odd, 0x8480u), 0x7d007f00u, nz);
  v[1] = fma_bf16x2(prmt(even, odd, 0x9591u), 0x7d007f00u, nz);
  v[2] = fma_bf16x2(prmt(even, odd, 0xa6a2u), 0x7d007f00u, nz);
  v[3] = fma_bf16x2(prmt(even, odd, 0xb7b3u), 0x7d007f00u, nz);
}
constexpr uint32_t kNegEight = 0xbe00be00u;  // -8 2^-6, twice

// -z 2^-6 as two bf16.
__device__ __forceinline__ uint32_t w4_neg_zero(uint32_t z) {
  return fma_bf16x2(z * 0x00010001u, 0xff00ff00u, 0x80008000u);
}

__device__ __forceinline__ void load_raw(uint32_t* r, const uint2* p) {
  const uint2 v = __ldg(p);
  r[0] = v.x, r[1] = v.y;
}
__device__ __forceinline__ void load_raw(uint32_t* r, const uint4* p) {
  const uint4 v = __ldg(p);
  r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
}

// acc[i] += s * d[i] for 8 values, two at a time
__device__ __forceinline__ void fma8(float* acc, const uint32_t (&d)[8], float s) {
  uint64_t ss;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "r"(__float_as_uint(s)));
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint32_t lo = __float_as_uint(acc[i]), hi = __float_as_uint(acc[i + 1]);
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "fma.rn.f32x2 a, b, %4, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+r"(lo), "+r"(hi)
        : "r"(d[i]), "r"(d[i + 1]), "l"(ss));
    acc[i] = __uint_as_float(lo);
    acc[i + 1] = __uint_as_float(hi);
  }
}

// mbar_wait with everything but the first try out of line.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* abort,
                                       unsigned long long limit_ns) {
  if (mbar_wait(bar, parity, abort, limit_ns)) return true;
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort,
                                     unsigned long long limit_ns) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, limit_ns);
}

enum W4Mode { kMatvec, kGateUp, kDown };
struct W4Job {
  const void* scales;
  const uint8_t* zeros;
  int scale_bf16;
  int whole_stages;  // K % kStepK == 0 and aligned tensors: a stage's scales in one load
  int mode, K;
  int n_rows;    // rows of the result: N, I or H
  int n_blocks;  // blocks of tokens (an upper bound for the layer)
  int T;
  int x_rows;    // rows of a box of x: 8, or 1 when no block has more tokens
  int split;     // the warpgroups split K (else rows)
  int cluster;   // thread blocks that split K
  void* out;     // matvec: [T][N]; gate/up: h bf16 [aligned row][I]; down: y fp32 [pair][H]
  int out_fp32;
  // layer
  const int32_t* sorted_ids;
  const int32_t* block_expert;
  const int32_t* num_padded;
  const float* wts;
  int P;
  int* err;      // status word, or null
  unsigned long long timeout_ns;
};

template <int PG, int NT>
struct W4Shape {
  static constexpr int kN = NT < 16 ? 16 : NT;  // MMA N (16 at least with 128 rows)
  // Columns of a unit, what is multiplied at a time: as many as leave room for
  // the groups' accumulators in a warpgroup's 128 columns of tensor memory.
  static constexpr int kUnitK = 64 + kN * (4 / PG) <= 128 ? 128
                                : 32 + kN * (PG == 1 ? 2 : 1) <= 128 ? 64 : 32;
  static constexpr int kSub = kUnitK / (32 * PG);  // groups of a unit
  // A unit is converted in parts, each with a slot of tensor memory for its A.
  // With a slot more, the next unit's first part is stored while the MMAs of this
  // one run, and with two sets of accumulators this one's are read during the next
  // one's MMAs, where that fits.
  static constexpr int kParts = kUnitK == 32 ? 1 : 2;
  static constexpr int kPartCols = kUnitK / 2 / kParts;
  static constexpr int kSlots = (kParts + 1) * kPartCols + kN * kSub <= 128 ? kParts + 1 : kParts;
  static constexpr int kSums = kSlots * kPartCols + 2 * kN * kSub <= 128 ? 2 : 1;
  static_assert(kSlots * kPartCols + kSums * kN * kSub <= 128, "tensor memory");
  static_assert(kUnitK % (32 * PG) == 0, "a unit holds whole groups");
  static constexpr int kXSlices = NT <= 16 ? 2 : 1;  // the warpgroups may split K
  static constexpr int kXBytes = NT * kStepK * 2;    // x of a stage, per slice of K
  static constexpr int kPerSm = NT <= 32 ? 2 : 1;
  static constexpr int kStageBytes = 2 * kCodeBytes + kXSlices * kXBytes;
  static constexpr int kStages = (NT <= 32 ? 111 : 222) * 1024 / kStageBytes;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + 1024;
  static_assert(kStages >= 2, "stages");
};

// PG: 32-column pieces of a group (1, 2, 4).  NT: tokens of a block at most.
template <int PG, bool ZP, int NT>
__global__ void __launch_bounds__(kThreads, (W4Shape<PG, NT>::kPerSm))
    w4_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_x,
              const W4Job j) {
  using S = W4Shape<PG, NT>;
  constexpr int kStages = S::kStages;
  constexpr int kUnits = kStepK / S::kUnitK;  // units of a stage
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kStages], s_empty[kStages], s_done[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int CS = j.cluster;
  const int rank = CS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (tid == 0) {
    prefetch_tensormap(&map);
    prefetch_tensormap(&map_x);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 2);
    }
    mbar_init(&s_done[0], 1);
    mbar_init(&s_done[1], 1);
    s_abort = 0;
    fence_mbarrier_init();
  }
  pdl_wait();
  pdl_trigger();

  // which rows and tokens; a block past the layer's last one leaves (all of its
  // cluster does)
  const int job = static_cast<int>(blockIdx.x) / CS;
  const int block = job % j.n_blocks;
  const int rows_wg = j.mode == kGateUp ? kRows / 2 : kRows;  // rows of the result
  const int r0 = job / j.n_blocks * (j.split ? rows_wg : 2 * rows_wg);
  int e = 0, valid;
  if (j.mode == kMatvec) {
    valid = min(NT, j.T - block * NT);
  } else {
    if (block * NT >= __ldg(j.num_padded)) return;
    e = __ldg(j.block_expert + block);
    const int32_t* ids = j.sorted_ids + static_cast<size_t>(block) * NT;
    valid = __popc(__ballot_sync(0xffffffffu, lane < NT && __ldg(ids + min(lane, NT - 1)) < j.P));
    if (NT > 32) valid += __popc(__ballot_sync(0xffffffffu, __ldg(ids + NT - 32 + lane) < j.P));
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, 256);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after_sync();

  // this block's slice of K, in steps of a stage (both warpgroups' columns)
  const int step_k = j.split ? 2 * kStepK : kStepK;
  const int all_steps = (j.K + step_k - 1) / step_k;
  const int step0 = static_cast<int>(static_cast<long long>(rank) * all_steps / CS);
  const int n_steps =
      static_cast<int>(static_cast<long long>(rank + 1) * all_steps / CS) - step0;
  const size_t expert_row = static_cast<size_t>(e) * j.n_rows * (j.mode == kGateUp ? 2 : 1);

  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.f;

  if (warp == 8) {
    if (elect_one()) {
      const int x_boxes = j.x_rows == 1 ? 1 : (valid + 7) / 8;
      const uint32_t box_bytes = static_cast<uint32_t>(j.x_rows) * 128;
      const uint32_t bytes = 2 * kCodeBytes + (j.split ? 8 : 4) * x_boxes * box_bytes;
      int i = 0;
      bool ok = true;
      for (; i < n_steps && ok; ++i) {
        const int slot = i % kStages;
        if (i >= kStages) {
          ok = wait(&s_empty[slot], i / kStages - 1 & 1, &s_abort, j.timeout_ns);
          if (!ok) break;
        }
        uint64_t* bar = &s_full[slot];
        uint8_t* dst = smem + slot * S::kStageBytes;
        mbar_arrive_expect_tx(bar, bytes);
        const int k0 = (step0 + i) * step_k;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int col = (k0 + (j.split ? g * kStepK : 0)) / 2;
          const int row_a = static_cast<int>(expert_row) + r0 + (j.split ? 0 : g * rows_wg);
          const int row_b = row_a + (j.mode == kGateUp ? j.n_rows : kRows / 2);
          tma_load_2d(dst + g * kCodeBytes, &map, bar, col, row_a);
          tma_load_2d(dst + g * kCodeBytes + kCodeBytes / 2, &map, bar, col, row_b);
        }
        // x: [slice][64 columns][token], 128-byte rows
        uint8_t* x = dst + 2 * kCodeBytes;
        for (int c = 0; c < (j.split ? 8 : 4); ++c)
          for (int b = 0; b < x_boxes; ++b)
            tma_load_2d(x + c * (NT * 128) + b * 1024, &map_x, bar, k0 + c * 64,
                        block * NT + b * 8);
      }
      if (!ok) {  // the copies in flight land before the block leaves
        volatile int never = 0;
        for (int n = max(0, i - kStages); n < i; ++n)
          mbar_wait(&s_full[n % kStages], n / kStages & 1, &never, kDrainNs);
      }
    }
  } else {
    const int wg = warp >> 2, row = tid & 127;  // of the warpgroup's 128
    const uint32_t tmem = s_tmem + wg * 128, t_d = tmem + S::kSlots * S::kPartCols;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // this thread's weight row, for its scales (past the result's last one: that one)
    const int out_row = min(r0 + (j.split ? 0 : wg * rows_wg) + row % rows_wg, j.n_rows - 1);
    const size_t grow =
        expert_row + out_row + (j.mode == kGateUp && row >= rows_wg ? j.n_rows : 0);
    const int groups = (j.K + 32 * PG - 1) / (32 * PG);
    constexpr int kGroups = 8 / PG;  // of a stage
    const int k_first = step0 * step_k + (j.split ? wg * kStepK : 0);
    const size_t group0 = grow * groups + k_first / (32 * PG);
    // Scales and zero points of a stage's groups, as they lie in memory: one load
    // each when every row's stage starts on its size (K a multiple of the stage's
    // columns), else group by group.
    uint32_t s_raw[kGroups], z_raw[(kGroups + 3) / 4];
    auto fetch_scales = [&](int step) {
      const int k = k_first + step * step_k;
      if (step >= n_steps || k >= j.K) {  // no columns: their sums are 0, and stay so
#pragma unroll
        for (int i = 0; i < kGroups; ++i) s_raw[i] = 0;
        return;
      }
      const size_t at = group0 + static_cast<size_t>(step) * (step_k / (32 * PG));
      if (j.whole_stages) {
        if (j.scale_bf16) {
          const uint8_t* p = static_cast<const uint8_t*>(j.scales) + at * 2;
          if (PG == 4) s_raw[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
          if (PG == 2) load_raw(s_raw, reinterpret_cast<const uint2*>(p));
          if (PG == 1) load_raw(s_raw, reinterpret_cast<const uint4*>(p));
        } else {
          const uint8_t* p = static_cast<const uint8_t*>(j.scales) + at * 4;
          if (PG == 4) load_raw(s_raw, reinterpret_cast<const uint2*>(p));
          if (PG <= 2) load_raw(s_raw, reinterpret_cast<const uint4*>(p));
          if (PG == 1) load_raw(s_raw + 4, reinterpret_cast<const uint4*>(p) + 1);
        }
        if (ZP) {
          if (PG == 4) z_raw[0] = __ldg(reinterpret_cast<const uint16_t*>(j.zeros + at));
          if (PG == 2) z_raw[0] = __ldg(reinterpret_cast<const uint32_t*>(j.zeros + at));
          if (PG == 1) load_raw(z_raw, reinterpret_cast<const uint2*>(j.zeros + at));
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const bool on = k + i * (32 * PG) < j.K;
        if (j.scale_bf16) {
          const uint32_t v = on ? __ldg(static_cast<const uint16_t*>(j.scales) + at + i) : 0;
          s_raw[i / 2] = i % 2 ? s_raw[i / 2] | v << 16 : v;
        } else {
          s_raw[i] = on ? __ldg(static_cast<const uint32_t*>(j.scales) + at + i) : 0;
        }
        if (ZP) {
          const uint32_t v = on ? __ldg(j.zeros + at + i) : 0;
          z_raw[i / 4] = i % 4 ? z_raw[i / 4] | v << (8 * (i % 4)) : v;
        }
      }
    };
#pragma unroll
    for (int i = 0; i < (kGroups + 3) / 4; ++i) z_raw[i] = 0;
    fetch_scales(0);

    bool ok = true;  // once a wait gives up, the loop runs out without waits and MMAs
    float s_step[kGroups], s_old[S::kSub];
    uint32_t z_step[(kGroups + 3) / 4];
    uint32_t a_first = 0;  // A slot of the unit's first part, in columns
    auto next_slot = [&](uint32_t c) {
      return c == (S::kSlots - 1) * S::kPartCols ? 0u : c + S::kPartCols;
    };
    auto wait_done = [&](int u) {  // unit u's MMAs
      ok = ok && wait(&s_done[wg], u & 1, &s_abort, j.timeout_ns);
      tc_fence_after_sync();
    };
    // adds unit u's sums, scaled
    auto flush = [&](int u, const float (&s)[S::kSub]) {
      const uint32_t at = t_d + lanes + (S::kSums == 2 ? (u & 1) * (S::kN * S::kSub) : 0);
#pragma unroll
      for (int i = 0; i < S::kSub; ++i)
#pragma unroll
        for (int t0 = 0; t0 < NT; t0 += 16) {
          uint32_t d[2][8];
          tmem_ld8_async(at + i * S::kN + t0, d[0]);
          if (NT > 8) tmem_ld8_async(at + i * S::kN + t0 + 8, d[1]);
          tmem_wait_ld();
          fma8(acc + t0, d[0], s[i]);
          if (NT > 8) fma8(acc + t0 + 8, d[1], s[i]);
        }
    };
    // one unit, the h-th of its stage
    auto unit = [&](int u, int slot, auto which) {
      constexpr int h = decltype(which)::value;
      constexpr int kChunks = S::kPartCols / 16;  // 32-column chunks of a part
      const uint8_t* stage = smem + slot * S::kStageBytes;
      const uint8_t* codes = stage + wg * kCodeBytes + row * 128;
      uint32_t nz[S::kSub];
      float s[S::kSub];
#pragma unroll
      for (int i = 0; i < S::kSub; ++i) {
        const int g = h * S::kSub + i;
        s[i] = s_step[g];
        nz[i] = ZP ? w4_neg_zero((z_step[g / 4] >> (8 * (g % 4))) & 0xffu) : kNegEight;
      }
      uint32_t v[kChunks][16];
      auto convert = [&](int part) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c = part * kChunks + i;  // 32 columns of the row: 16 words of A
          const uint4 q = *reinterpret_cast<const uint4*>(
              codes + ((h * (S::kUnitK / 32) + c) ^ (row & 7)) * 16);
          w4_pairs(q.x, nz[c / PG], v[i]);
          w4_pairs(q.y, nz[c / PG], v[i] + 4);
          w4_pairs(q.z, nz[c / PG], v[i] + 8);
          w4_pairs(q.w, nz[c / PG], v[i] + 12);
        }
      };
      const uint32_t a_last = S::kParts == 2 ? next_slot(a_first) : a_first;
      auto store = [&](uint32_t slot_cols) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) tmem_st16(tmem + lanes + slot_cols + i * 16, v[i]);
      };
      constexpr bool kEarly = S::kSlots > S::kParts;
      convert(0);
      if (kEarly) {  // this slot's last MMAs were unit u - 2's
        store(a_first);
        if (S::kParts == 2) convert(1);
      }
      if (u > 0) {
        wait_done(u - 1);
        if (S::kSums == 1) flush(u - 1, s_old);
      }
      if (!kEarly) {
        store(a_first);
        if (S::kParts == 2) convert(1);
      }
      if (S::kParts == 2) store(a_last);
      tmem_wait_st();
      tc_fence_before_sync();
      named_barrier(1 + wg, kGroupThreads);  // A is in place, and the codes are read
      if ((warp & 3) == 0 && elect_one()) {
        tc_fence_after_sync();
        if (ok) {
          const uint32_t idesc = umma_idesc(true, kRows, S::kN);
          uint64_t db = sdesc_kmajor_sw128(smem_addr(stage) + 2 * kCodeBytes +
                                           (j.split ? wg * S::kXBytes : 0));
          if (NT == 8) db &= ~(0x3fffull << 32);  // rows 8..15 are rows 0..7 again
          const uint32_t d = t_d + (S::kSums == 2 ? (u & 1) * (S::kN * S::kSub) : 0);
#pragma unroll
          for (int i = 0; i < S::kUnitK / 16; ++i) {
            // 16 columns: 32 bytes further in a token's 128-byte row, or its next row
            const int i16 = h * (S::kUnitK / 16) + i;
            const uint64_t b = db + (i16 % 4) * 2 + (i16 / 4) * (NT * 128 / 16);
            const uint32_t a = tmem + (i * 8 < S::kPartCols ? a_first : a_last) +
                               i * 8 % S::kPartCols;
            umma_bf16_ts(d + i / (2 * PG) * S::kN, a, b, idesc, i % (2 * PG) != 0);
          }
          umma_commit(&s_done[wg]);
          if (h == kUnits - 1) umma_commit(&s_empty[slot]);
        }
      }
      a_first = next_slot(a_last);
      if (S::kSums == 2 && u > 0) flush(u - 1, s_old);
#pragma unroll
      for (int i = 0; i < S::kSub; ++i) s_old[i] = s[i];
    };
    int slot = 0, phase = 0;
    for (int step = 0; step < n_steps; ++step) {
      ok = ok && wait(&s_full[slot], phase, &s_abort, j.timeout_ns);
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        s_step[i] = __uint_as_float(!j.scale_bf16 ? s_raw[i]
                                    : i % 2       ? s_raw[i / 2] & 0xffff0000u
                                                  : s_raw[i / 2] << 16);
#pragma unroll
      for (int i = 0; i < (kGroups + 3) / 4; ++i) z_step[i] = z_raw[i];
      fetch_scales(step + 1);
      const int u = step * kUnits;
      unit(u, slot, std::integral_constant<int, 0>{});
      unit(u + 1, slot, std::integral_constant<int, 1>{});
      if constexpr (kUnits >= 4) {
        unit(u + 2, slot, std::integral_constant<int, 2>{});
        unit(u + 3, slot, std::integral_constant<int, 3>{});
      }
      if constexpr (kUnits == 8) {
        unit(u + 4, slot, std::integral_constant<int, 4>{});
        unit(u + 5, slot, std::integral_constant<int, 5>{});
        unit(u + 6, slot, std::integral_constant<int, 6>{});
        unit(u + 7, slot, std::integral_constant<int, 7>{});
      }
      if (++slot == kStages) slot = 0, phase ^= 1;
    }
    wait_done(n_steps * kUnits - 1);
    flush(n_steps * kUnits - 1, s_old);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (s_abort) {
    if (tid == 0 && j.err != nullptr) atomicOr(j.err, kDevErrTimeout);
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = __int_as_float(0x7fc00000);  // a wrong sum shows
  }
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(s_tmem, 256);
  }
  // the sums over the slices of K, warpgroups then ranks, in the stages' space:
  // red[warpgroup][token][row]
  float* red = reinterpret_cast<float*>(smem);
  if (warp < 8) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      red[((warp >> 2) * NT + t) * kRows + (tid & 127)] = 64.f * acc[t];
  }
  __syncwarp();
  if (CS > 1) cluster_sync();
  else __syncthreads();
  const uint32_t red_at = smem_addr(red);
  auto sum = [&](int wg, int t, int row) {
    const int at = (wg * NT + t) * kRows + row;
    float v = 0.f;
    for (int i = 0; i < CS; ++i) {
      if (CS == 1) {
        v = j.split ? red[at] + red[at + NT * kRows] : red[at];
      } else {
        const uint32_t a = mapa_shared(red_at + at * 4, i);
        v += ld_cluster_f32(a);
        if (j.split) v += ld_cluster_f32(a + NT * kRows * 4);
      }
    }
    return v;
  };
  const int rows_out = j.split ? rows_wg : 2 * rows_wg;
  for (int i = rank * kThreads + tid; i < rows_out * valid; i += CS * kThreads) {
    const int t = i / rows_out, r = i % rows_out;
    if (r0 + r >= j.n_rows) continue;
    const int wg = r / rows_wg, rw = r % rows_wg;
    if (j.mode == kMatvec) {
      const float v = sum(wg, t, rw);
      const size_t o = (static_cast<size_t>(block) * NT + t) * j.n_rows + r0 + r;
      if (j.out_fp32) static_cast<float*>(j.out)[o] = v;
      else static_cast<__nv_bfloat16*>(j.out)[o] = __float2bfloat16_rn(v);
    } else if (j.mode == kGateUp) {
      const float gate = sum(wg, t, rw), up = sum(wg, t, rw + rows_wg);
      static_cast<__nv_bfloat16*>(
          j.out)[(static_cast<size_t>(block) * NT + t) * j.n_rows + r0 + r] =
          __float2bfloat16_rn(gate / (1.f + expf(-gate)) * up);
    } else {
      const int pair = __ldg(j.sorted_ids + static_cast<size_t>(block) * NT + t);
      static_cast<float*>(j.out)[static_cast<size_t>(pair) * j.n_rows + r0 + r] =
          __ldg(j.wts + pair) * sum(wg, t, rw);
    }
  }
  __syncwarp();
  if (CS > 1) cluster_sync();  // no block leaves while another reads its sums
}

// xs[row] = x[pair / k] for the aligned rows that hold a pair.
__global__ void __launch_bounds__(256)
    w4_gather_kernel(const __nv_bfloat16* __restrict__ x, int k, int H, int P,
                     const int32_t* __restrict__ sorted_ids, const int32_t* __restrict__ num_padded,
                     __nv_bfloat16* __restrict__ xs) {
  pdl_wait();
  pdl_trigger();
  const int rows = __ldg(num_padded), n8 = H / 8;
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const int pair = __ldg(sorted_ids + r);
    if (pair >= P) continue;
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(pair / k) * H);
    uint4* dst = reinterpret_cast<uint4*>(xs + static_cast<size_t>(r) * H);
    for (int i = threadIdx.x; i < n8; i += blockDim.x) dst[i] = __ldg(src + i);
  }
}

// out[t] = sum of its k weighted rows, in slot order.
__global__ void __launch_bounds__(256)
    w4_combine_kernel(const float* __restrict__ y, int T, int k, int H,
                      __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const long long n = static_cast<long long>(T) * (H / 4);
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const long long t = i / (H / 4);
    const int c = static_cast<int>(i - t * (H / 4)) * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < k; ++j) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(y + (t * k + j) * H + c));
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
    *reinterpret_cast<uint2*>(out + t * H + c) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  }
}

// How the warpgroups of a job are laid out: row tiles times slices of K, so that
// there is about one for each of the four that an SM holds, each with a stage's
// columns at least.
void choose_split(W4Job& j, int nt, int num_sms) {
  const int rows_wg = j.mode == kGateUp ? kRows / 2 : kRows;
  const long long tiles = (static_cast<long long>(j.n_rows) + rows_wg - 1) / rows_wg * j.n_blocks;
  const int steps = (j.K + kStepK - 1) / kStepK;
  int slices = 1;
  while (slices < (nt <= 16 ? 16 : 8) && 2 * slices <= steps && tiles * 2 * slices <= 4ll * num_sms) slices *= 2;
  j.split = slices > 1 && nt <= 16 ? 1 : 0;
  j.cluster = j.split ? slices / 2 : slices;
}

template <int PG, bool ZP, int NT>
cudaError_t launch(const CUtensorMap& map, const CUtensorMap& map_x, const W4Job& job, int num_sms,
                   cudaStream_t st) {
  using S = W4Shape<PG, NT>;
  cudaError_t e = checked(cudaFuncSetAttribute(w4_kernel<PG, ZP, NT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(S::kSmem)),
                          "smem attribute");
  if (e != cudaSuccess) return e;
  W4Job j = job;
  j.whole_stages = j.K % kStepK == 0 && reinterpret_cast<uintptr_t>(j.scales) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(j.zeros) % 8 == 0;
  choose_split(j, NT, num_sms);
  const int rows = (j.mode == kGateUp ? kRows / 2 : kRows) * (j.split ? 1 : 2);
  const long long tiles = (static_cast<long long>(j.n_rows) + rows - 1) / rows * j.n_blocks;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * j.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(j.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = j.cluster > 1 ? 2 : 1;
  return checked(cudaLaunchKernelEx(&cfg, w4_kernel<PG, ZP, NT>, map, map_x, j), "kernel launch");
}

template <int PG, bool ZP>
cudaError_t launch_tokens(const CUtensorMap& map, const CUtensorMap& map_x, const W4Job& j, int nt,
                          int num_sms, cudaStream_t st) {
  if (nt == 8) return launch<PG, ZP, 8>(map, map_x, j, num_sms, st);
  if (nt == 16) return launch<PG, ZP, 16>(map, map_x, j, num_sms, st);
  if (nt == 32) return launch<PG, ZP, 32>(map, map_x, j, num_sms, st);
  return launch<PG, ZP, 64>(map, map_x, j, num_sms, st);
}

cudaError_t launch_job(const CUtensorMap& map, const CUtensorMap& map_x, int group, const W4Job& j,
                       int nt, int num_sms, cudaStream_t st) {
  if (j.zeros != nullptr)
    return group == 32   ? launch_tokens<1, true>(map, map_x, j, nt, num_sms, st)
           : group == 64 ? launch_tokens<2, true>(map, map_x, j, nt, num_sms, st)
                         : launch_tokens<4, true>(map, map_x, j, nt, num_sms, st);
  return group == 32   ? launch_tokens<1, false>(map, map_x, j, nt, num_sms, st)
         : group == 64 ? launch_tokens<2, false>(map, map_x, j, nt, num_sms, st)
                       : launch_tokens<4, false>(map, map_x, j, nt, num_sms, st);
}

}  // namespace

int w4_block_rows(int T) { return T <= 8 ? 8 : T <= 16 ? 16 : T <= 32 ? 32 : 64; }

cudaError_t launch_w4_matvec(const CUtensorMap& map, const CUtensorMap& map_x, int T, int K, int N,
                             const W4View& w, void* out, bool out_fp32,
                             unsigned long long timeout_ns, int num_sms, cudaStream_t st) {
  const int nt = w4_block_rows(T);
  W4Job j{};
  j.scales = w.scales;
  j.zeros = w.zeros;
  j.scale_bf16 = w.scale_bf16;
  j.mode = kMatvec;
  j.K = K;
  j.n_rows = N;
  j.n_blocks = (T + nt - 1) / nt;
  j.T = T;
  j.x_rows = w4_x_box_rows(T);
  j.out = out;
  j.out_fp32 = out_fp32 ? 1 : 0;
  j.timeout_ns = timeout_ns;
  return launch_job(map, map_x, w.group, j, nt, num_sms, st);
}

cudaError_t launch_w4_layer(const CUtensorMap& map13, const CUtensorMap& map_x,
                            const CUtensorMap& map2, const CUtensorMap& map_h,
                            const W4LayerParams& p, int num_sms, cudaStream_t st) {
  const int nt = w4_block_rows(p.T);
  const long long P = static_cast<long long>(p.T) * p.k;
  W4Job j{};
  j.n_blocks = static_cast<int>(std::min(P, (P + std::min<long long>(p.E, P) * (nt - 1)) / nt));
  cudaError_t e = launch_pdl(
      w4_gather_kernel, dim3(static_cast<int>(std::min<long long>(P, 4 * num_sms))), dim3(256), 0,
      st, p.x, p.k, p.H, static_cast<int>(P), p.sorted_ids, p.num_padded, p.xs);
  if (e != cudaSuccess) return e;
  j.scales = p.w13.scales;
  j.zeros = p.w13.zeros;
  j.scale_bf16 = p.w13.scale_bf16;
  j.mode = kGateUp;
  j.K = p.H;
  j.n_rows = p.I;
  j.T = p.T;
  j.x_rows = w4_x_box_rows(p.T);
  j.out = p.h;
  j.sorted_ids = p.sorted_ids;
  j.block_expert = p.block_expert;
  j.num_padded = p.num_padded;
  j.wts = p.wts;
  j.P = static_cast<int>(P);
  j.err = p.err;
  j.timeout_ns = p.timeout_ns;
  e = launch_job(map13, map_x, p.w13.group, j, nt, num_sms, st);
  if (e != cudaSuccess) return e;
  j.scales = p.w2.scales;
  j.zeros = p.w2.zeros;
  j.scale_bf16 = p.w2.scale_bf16;
  j.mode = kDown;
  j.K = p.I;
  j.n_rows = p.H;
  j.out = p.y;
  e = launch_job(map2, map_h, p.w2.group, j, nt, num_sms, st);
  if (e != cudaSuccess) return e;
  const long long n = static_cast<long long>(p.T) * (p.H / 4);
  return launch_pdl(w4_combine_kernel,
                    dim3(static_cast<int>(std::min<long long>((n + 255) / 256, 2048))), dim3(256),
                    0, st, static_cast<const float*>(p.y), p.T, p.k, p.H, p.out);
}

}  // namespace moe
