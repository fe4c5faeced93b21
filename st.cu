// 4-bit weights with group scales: matrix-vector products and the expert
// products of the MoE layer for a few tokens.
//
// y[t][r] = sum over groups of scale[r][group] * sum_k x[t][k] (code[r][k] - zero[r][group]).
// At a few tokens the codes' bytes bound it, if turning them into an MMA operand
// does not: at 6.8 TB/s an SM takes in 47 codes a clock.
//
// A thread block owns 128 weight rows and a slice of K; the blocks of a cluster
// share rows and split K.  TMA brings 256 columns of the rows (128 bytes each) a
// stage; four warps, a thread per row, turn 32 codes at a time into bf16 (code -
// zero is a small integer: exact) and put them into tensor memory, where they
// are the A operand (128 rows) of tcgen05.mma with the tokens in N; x goes to
// shared memory.  The accumulators of each group come back, again a thread per
// row, and are scaled in fp32: no weight is rounded.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

__device__ long long g_st[64*32];
#define ST(i) if(blockIdx.x==100&&u>=8&&u<24&&lane==0&&warp==0) g_st[(u-8)*16+(i)]=clock64();
#define SC(i) if(blockIdx.x==100&&u>=8&&u<24) g_st[(u-8)*16+(i)]=clock64();
namespace moe {
namespace {

constexpr int kRows = 128;       // weight rows of a thread block (64 gate and 64 up rows)
constexpr int kStepK = 256;      // columns of a stage
constexpr int kStageBytes = kRows * kStepK / 2;
constexpr int kWorkers = 128;    // threads that convert: one per row
constexpr int kThreads = kWorkers + 32;

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// The 8 codes of a word as four pairs of bf16, (code i - zero, code i + 4 - zero)
// 2^-6.  As a bf16 a pattern of 0..255 is that many times 2^-133 (the two lowest
// exponents share their spacing), so a masked nibble needs one fused
// multiply-add: x 2^127 (bits 0..3) or 2^123 (bits 4..7), - zero 2^-6, all exact.
// nz holds -zero 2^-6 in both halves; the 2^6 is made good when sums are stored.
__device__ __forceinline__ void w4_pairs(uint32_t w, uint32_t nz, uint32_t* v) {
  const uint32_t h = w >> 8;
  v[0] = fma_bf16x2(w & 0x000f000fu, 0x7f007f00u, nz);
  v[1] = fma_bf16x2(w & 0x00f000f0u, 0x7d007d00u, nz);
  v[2] = fma_bf16x2(h & 0x000f000fu, 0x7f007f00u, nz);
  v[3] = fma_bf16x2(h & 0x00f000f0u, 0x7d007d00u, nz);
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

enum W4Mode { kMatvec, kGateUp, kDown };
struct W4Job {
  const void* scales;
  const uint8_t* zeros;
  int scale_bf16;
  int whole_stages;  // K % kStepK == 0 and aligned tensors: a stage's scales in one load
  int mode, K;
  int n_rows;    // rows of the result: N, I or H
  int n_blocks;  // blocks of tokens (an upper bound for the layer)
  const __nv_bfloat16* x;  // tokens, or h by pair (down)
  int T;
  void* out;     // matvec: [T][N]; gate/up: h bf16 [pair][I]; down: y fp32 [pair][H]
  int out_fp32;
  int cluster;   // thread blocks that split K
  // layer
  const int32_t* sorted_ids;
  const int32_t* block_expert;
  const int32_t* num_padded;
  const float* wts;
  int P, k;
  int* err;      // status word, or null
  unsigned long long timeout_ns;
};

template <int PG, int NT>
struct W4Shape {
  static constexpr int kN = NT < 16 ? 16 : NT;  // MMA N (16 at least with 128 rows)
  // columns of a unit: what is converted and multiplied at a time, with two
  // buffers for the converted codes and two for the sums
  static constexpr int kUnitK = NT == 64 && PG == 1 ? 32 : 64;
  static constexpr int kUnits = 128 / kUnitK;  // units of a 128-column block
  static constexpr int kFlush = 32 * PG > kUnitK ? 32 * PG / kUnitK : 1;  // units of a group
  static constexpr int kSub = kUnitK > 32 * PG ? kUnitK / (32 * PG) : 1;  // groups of a unit
  static constexpr int kUsed = kUnitK + 2 * kN * kSub;
  static constexpr int kTmem = kUsed <= 128 ? 128 : 256;
  static_assert(kUsed <= 256, "tensor memory of a thread block");
  // x of a block, two buffers; eight tokens stand for both eight-row halves of N
  static constexpr int kXBytes = NT * 128 * 2;
  static constexpr int kPerSm = NT == 8 ? 4 : kTmem == 128 ? 3 : 2;
  static constexpr int kStages = kPerSm == 4 ? 3 : kPerSm == 3 ? (NT == 16 ? 4 : 3) : 5;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + 2 * kXBytes + 1024;
};

// PG: 32-column pieces of a group (1, 2, 4).  NT: tokens of a block at most.
template <int PG, bool ZP, int NT>
__global__ void __launch_bounds__(kThreads, (W4Shape<PG, NT>::kPerSm))
    w4_kernel(const __grid_constant__ CUtensorMap map, const W4Job j) {
  using S = W4Shape<PG, NT>;
  constexpr int kUnits = S::kUnits, kStages = S::kStages;
  constexpr int kHalfBytes = NT * 128;  // x of 64 columns
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kStages], s_ready[2], s_done[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* s_x = smem + kStages * kStageBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int CS = j.cluster;
  const int rank = CS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (tid == 0) {
    prefetch_tensormap(&map);
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_ready[i], kWorkers / 32);  // a unit's A and x are in place
      mbar_init(&s_done[i], 1);               // its MMAs are done
    }
    s_abort = 0;
    fence_mbarrier_init();
  }
  pdl_wait();
  pdl_trigger();

  // which rows and tokens; a block past the layer's last one leaves (all of its
  // cluster does)
  const int job = static_cast<int>(blockIdx.x) / CS;
  const int block = job % j.n_blocks;
  const int r0 = job / j.n_blocks * (j.mode == kGateUp ? kRows / 2 : kRows);
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
  if (warp == 4) {
    tmem_alloc(&s_tmem, S::kTmem);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem, t_a = tmem, t_d = tmem + S::kUnitK;
  const size_t row_a = (j.mode == kGateUp ? static_cast<size_t>(e) * 2 : static_cast<size_t>(e)) *
                           j.n_rows + r0;
  const size_t row_b = row_a + (j.mode == kGateUp ? j.n_rows : kRows / 2);

  // this block's slice of K, in stages and 128-column blocks
  const int all_steps = (j.K + kStepK - 1) / kStepK;
  const int step0 = static_cast<int>(static_cast<long long>(rank) * all_steps / CS);
  const int step1 = static_cast<int>(static_cast<long long>(rank + 1) * all_steps / CS);
  const int n_steps = step1 - step0;
  const int k0 = step0 * kStepK, k1 = min(step1 * kStepK, j.K);
  const int n_blks = (k1 - k0 + 127) / 128;

  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.f;

  if (warp == 4) {
    if (elect_one()) {
      auto issue = [&](int step) {
        uint64_t* bar = &s_full[step % kStages];
        uint8_t* dst = smem + step % kStages * kStageBytes;
        mbar_arrive_expect_tx(bar, kStageBytes);
        const int col = (step0 + step) * (kStepK / 2);
        tma_load_2d(dst, &map, bar, col, static_cast<int>(row_a));
        tma_load_2d(dst + kStageBytes / 2, &map, bar, col, static_cast<int>(row_b));
      };
      int issued = min(kStages, n_steps);
      for (int i = 0; i < issued; ++i) issue(i);
      const uint32_t idesc = umma_idesc(true, kRows, S::kN);
      uint64_t db = sdesc_kmajor_sw128(smem_addr(s_x));
      if (NT == 8) db &= ~(0x3fffull << 32);  // rows 8..15 are rows 0..7 again
      bool ok = true;
      for (int blk = 0; blk < n_blks && ok; ++blk) {
#pragma unroll
        for (int h = 0; h < kUnits; ++h) {
          const int u = blk * kUnits + h, buf = h % 2;
          ok = mbar_wait_asleep(&s_ready[buf], u / 2 & 1, &s_abort, j.timeout_ns);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t d = t_d + (u / S::kFlush & 1) * (S::kN * S::kSub);
#pragma unroll
          for (int i = 0; i < S::kUnitK / 16; ++i) {
            // 16 columns of the block: 32 bytes further in a token's 128-byte row, or
            // in the second half of the rows
            const int i16 = h * (S::kUnitK / 16) + i;
            const uint64_t b = db + (blk & 1) * (S::kXBytes / 16) + (i16 % 4) * 2 +
                               (i16 / 4) * (kHalfBytes / 16);
            umma_bf16_ts(d + i / (2 * PG) * S::kN, t_a + buf * (S::kUnitK / 2) + i * 8, b, idesc,
                         i16 % (2 * PG) != 0);
          }
          umma_commit(&s_done[buf]);
        }
        // every warp has read the block's codes: its stage is free after the second one
        if (ok && blk % 2 == 1 && issued < n_steps) issue(issued++);
      }
      if (!ok) {
        s_abort = 1;
        if (j.err != nullptr) atomicOr(j.err, kDevErrTimeout);
        // the copies in flight land before the block leaves
        volatile int never = 0;
        for (int i = max(0, issued - kStages); i < issued; ++i)
          mbar_wait_asleep(&s_full[i % kStages], i / kStages & 1, &never, j.timeout_ns);
      }
    }
  } else {
    const int row = tid;  // of the block's 128
    const size_t grow =
        min((row < kRows / 2 ? row_a : row_b - kRows / 2) + row,
            // a row past the result's last one takes that one's scales
            static_cast<size_t>(j.mode == kGateUp ? 2 * e + (row >= kRows / 2) : e) * j.n_rows +
                j.n_rows - 1);
    const int groups = (j.K + 32 * PG - 1) / (32 * PG);
    float s_step[8 / PG];
    uint32_t z_step[(8 / PG + 3) / 4];
    const size_t group0 = grow * groups + k0 / (32 * PG);
    // tokens: 16-byte piece tid % 16 of a block of tokens tid / 16, tid / 16 + 8, ...
    constexpr int kRounds = NT / 8;
    const int piece = tid % 16;
    const __nv_bfloat16* xp[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int t = min(tid / 16 + i * 8, valid - 1);
      size_t at;
      if (j.mode == kMatvec) {
        at = static_cast<size_t>(block) * NT + t;
      } else {
        const int pair = __ldg(j.sorted_ids + static_cast<size_t>(block) * NT + t);
        at = j.mode == kGateUp ? pair / j.k : pair;
      }
      xp[i] = j.x + at * j.K + k0 + piece * 8;
    }
    uint4 x_nx[kRounds];
    auto fetch_x = [&](int blk) {
      const bool on = k0 + blk * 128 + piece * 8 < k1;
#pragma unroll
      for (int i = 0; i < kRounds; ++i)
        x_nx[i] = on ? __ldg(reinterpret_cast<const uint4*>(xp[i] + blk * 128))
                     : make_uint4(0, 0, 0, 0);
    };
    // Scales and zero points of a stage's kGroups groups, as they lie in memory:
    // one load each when every row's stage starts on its size (K a multiple of
    // the stage's columns), else group by group.
    constexpr int kGroups = 8 / PG;
    uint32_t s_raw[kGroups], z_raw[(kGroups + 3) / 4];
    auto fetch_scales = [&](int step) {
      const size_t at = group0 + static_cast<size_t>(step) * kGroups;
      if (step >= n_steps) return;
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
        const bool on = k0 + (step * kGroups + i) * (32 * PG) < k1;
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
    fetch_scales(0);
    fetch_x(0);
    constexpr int kBlkGroups = 4 / PG;  // groups of a block
    float s_cur[kBlkGroups], s_old[kBlkGroups];  // scales of this block and the one before
    // waits for unit u's MMAs
    auto wait_done = [&](int u) {
      const bool ok = mbar_wait_asleep(&s_done[u & 1], u / 2 & 1, &s_abort, j.timeout_ns);
      tc_fence_after_sync();
      return ok;
    };
    // adds the sums of the groups that unit u has finished, scaled by s[0 ..]
    const uint32_t d_at = t_d + (static_cast<uint32_t>(warp * 32) << 16);
    auto flush = [&](int u, const float* s) {
      const uint32_t at = d_at + (u / S::kFlush & 1) * (S::kN * S::kSub);
#pragma unroll
      for (int i = 0; i < S::kSub; ++i)
#pragma unroll
        for (int t0 = 0; t0 < NT; t0 += 16) {
          uint32_t d[2][8];
          tmem_ld8_async(at + i * S::kN + t0, d[0]);
          if (NT > 8) tmem_ld8_async(at + i * S::kN + t0 + 8, d[1]);
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < (NT > 8 ? 16 : 8); ++t)
            acc[t0 + t] = fmaf(s[i], __uint_as_float(d[t / 8][t % 8]), acc[t0 + t]);
        }
    };
    // the scales of unit h of a block (h < 0: of the block before), where it ends a group
    auto scales_of = [&](int h) -> const float* {
      const int g = (h < 0 ? h + kUnits : h) / S::kFlush * S::kSub;
      return (h < 0 ? s_old : s_cur) + g;
    };
    const uint32_t a_at = t_a + (static_cast<uint32_t>(warp * 32) << 16);
    bool ok = true;
    // one 128-column block, the hb-th of its stage
    auto block = [&](int blk, int slot, auto half) {
      constexpr int hb = decltype(half)::value;
      const uint8_t* codes = smem + slot * kStageBytes + row * 128;
      uint32_t nz[kBlkGroups];
#pragma unroll
      for (int i = 0; i < kBlkGroups; ++i) {
        const int g = hb * kBlkGroups + i;
        s_old[i] = s_cur[i];
        s_cur[i] = s_step[g];
        nz[i] = ZP ? w4_neg_zero((z_step[g / 4] >> (8 * (g % 4))) & 0xffu) : kNegEight;
      }
#pragma unroll
      for (int h = 0; h < kUnits; ++h) {
        const int u = blk * kUnits + h, buf = h % 2;
        uint32_t v[S::kUnitK / 32][16];
#pragma unroll
        for (int i = 0; i < S::kUnitK / 32; ++i) {
          const int c = h * (S::kUnitK / 32) + i;  // 32 columns of the row: 16 words of A
          const uint4 q = *reinterpret_cast<const uint4*>(codes + ((hb * 4 + c) ^ (row & 7)) * 16);
          w4_pairs(q.x, nz[c / PG], v[i]);
          w4_pairs(q.y, nz[c / PG], v[i] + 4);
          w4_pairs(q.z, nz[c / PG], v[i] + 8);
          w4_pairs(q.w, nz[c / PG], v[i] + 12);
        }
        if (u >= 2) {  // the MMAs that read this A buffer, and their sums
          if (!wait_done(u - 2)) return false;
          if ((h + kUnits - 2) % kUnits % S::kFlush == S::kFlush - 1) flush(u - 2, scales_of(h - 2));
        }
#pragma unroll
        for (int i = 0; i < S::kUnitK / 32; ++i)
          tmem_st16(a_at + buf * (S::kUnitK / 2) + i * 16, v[i]);
        if (h == 0) {
          ST(3)
      // x, its columns in the order of the codes: (0,4), (1,5), (2,6), (3,7)
          uint8_t* to = s_x + (blk & 1) * S::kXBytes + piece / 8 * kHalfBytes;
#pragma unroll
          for (int i = 0; i < kRounds; ++i) {
            const int t = tid / 16 + i * 8;
            const uint4 x = x_nx[i];
            uint4 p;
            p.x = __byte_perm(x.x, x.z, 0x5410);
            p.y = __byte_perm(x.x, x.z, 0x7632);
            p.z = __byte_perm(x.y, x.w, 0x5410);
            p.w = __byte_perm(x.y, x.w, 0x7632);
            *reinterpret_cast<uint4*>(to + t * 128 + ((piece % 8) ^ (t & 7)) * 16) = p;
          }
          fetch_x(blk + 1);
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_ready[buf]);
      }
      return true;
    };
    int slot = 0, phase = 0;
    for (int step = 0; step < n_steps; ++step) {
      ok = mbar_wait_asleep(&s_full[slot], phase, &s_abort, j.timeout_ns);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        s_step[i] = __uint_as_float(!j.scale_bf16 ? s_raw[i]
                                    : i % 2       ? s_raw[i / 2] & 0xffff0000u
                                                  : s_raw[i / 2] << 16);
#pragma unroll
      for (int i = 0; i < (kGroups + 3) / 4; ++i) z_step[i] = z_raw[i];
      fetch_scales(step + 1);
      ok = block(2 * step, slot, std::integral_constant<int, 0>{});
      if (!ok) break;
      if (2 * step + 1 < n_blks) ok = block(2 * step + 1, slot, std::integral_constant<int, 1>{});
      if (!ok) break;
      if (++slot == kStages) slot = 0, phase ^= 1;
    }
    // the last two units
    if (ok) {
#pragma unroll
      for (int h = kUnits - 2; h < kUnits; ++h) {
        const int u = (n_blks - 1) * kUnits + h;
        ok = wait_done(u);
        if (!ok) break;
        if (h % S::kFlush == S::kFlush - 1) flush(u, scales_of(h));
      }
    }
    if (!ok) {
      s_abort = 1;
      if (j.err != nullptr && lane == 0) atomicOr(j.err, kDevErrTimeout);
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = __int_as_float(0x7fc00000);  // a wrong sum shows
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, S::kTmem);
  }
  // the sums over the cluster's slices of K, in rank order, in the stages' space:
  // red[token][row]
  float* red = reinterpret_cast<float*>(smem);
  if (warp < 4) {
#pragma unroll
    for (int t = 0; t < NT; ++t) red[t * kRows + tid] = 64.f * acc[t];
  }
  if (CS > 1) cluster_sync();
  else __syncthreads();
  const uint32_t red_at = smem_addr(red);
  auto sum = [&](int t, int row) {
    if (CS == 1) return red[t * kRows + row];
    float v = 0.f;
    for (int i = 0; i < CS; ++i)
      v += ld_cluster_f32(mapa_shared(red_at + (t * kRows + row) * 4, i));
    return v;
  };
  const int rows_out = j.mode == kGateUp ? kRows / 2 : kRows;
  for (int i = rank * kThreads + tid; i < rows_out * valid; i += CS * kThreads) {
    const int t = i / rows_out, r = i % rows_out;
    if (r0 + r >= j.n_rows) continue;
    if (j.mode == kMatvec) {
      const float v = sum(t, r);
      const size_t o = (static_cast<size_t>(block) * NT + t) * j.n_rows + r0 + r;
      if (j.out_fp32) static_cast<float*>(j.out)[o] = v;
      else static_cast<__nv_bfloat16*>(j.out)[o] = __float2bfloat16_rn(v);
    } else {
      const int pair = __ldg(j.sorted_ids + static_cast<size_t>(block) * NT + t);
      const size_t o = static_cast<size_t>(pair) * j.n_rows + r0 + r;
      if (j.mode == kGateUp) {
        const float gate = sum(t, r), up = sum(t, r + kRows / 2);
        static_cast<__nv_bfloat16*>(j.out)[o] =
            __float2bfloat16_rn(gate / (1.f + expf(-gate)) * up);
      } else {
        static_cast<float*>(j.out)[o] = __ldg(j.wts + pair) * sum(t, r);
      }
    }
  }
  __syncwarp();
  if (CS > 1) cluster_sync();  // no block leaves while another reads its sums
}

}}

using namespace moe;
#include <cstdio>
#include <vector>
#include <cudaTypedefs.h>
template<int PG,int NT> void go(int T,int group,int NN){ int K=8192,N=NN; uint8_t*c;void*sc;__nv_bfloat16*x;void*o;cudaMalloc(&c,(size_t)N*K/2);cudaMalloc(&sc,(size_t)N*K/8);cudaMalloc(&x,K*256);cudaMalloc(&o,(size_t)N*256);
 cudaMemset(c,1,(size_t)N*K/2);cudaMemset(sc,0,(size_t)N*K/8);cudaMemset(x,0,K*256);
 void* p=nullptr; cudaDriverEntryPointQueryResult q; cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled",&p,12000,cudaEnableDefault,&q);
 auto enc=(PFN_cuTensorMapEncodeTiled_v12000)p; CUtensorMap map; cuuint64_t dims[2]={(cuuint64_t)K/2,(cuuint64_t)N},str[1]={(cuuint64_t)K/2};cuuint32_t box[2]={128,64},es[2]={1,1};
 enc(&map,CU_TENSOR_MAP_DATA_TYPE_UINT8,2,c,dims,str,box,es,CU_TENSOR_MAP_INTERLEAVE_NONE,CU_TENSOR_MAP_SWIZZLE_128B,CU_TENSOR_MAP_L2_PROMOTION_L2_256B,CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
 W4Job j{}; j.scales=sc;j.scale_bf16=1;j.whole_stages=1;j.mode=kMatvec;j.K=K;j.n_rows=N;j.n_blocks=1;j.x=x;j.T=T;j.out=o;j.cluster=1;j.timeout_ns=1000000000ull;
 cudaFuncSetAttribute(w4_kernel<PG,false,NT>,cudaFuncAttributeMaxDynamicSharedMemorySize,(int)W4Shape<PG,NT>::kSmem);
 for(int r=0;r<2;r++) w4_kernel<PG,false,NT><<<N/128,kThreads,W4Shape<PG,NT>::kSmem>>>(map,j);
 printf("NT %d PG %d %s\n",NT,PG,cudaGetErrorString(cudaDeviceSynchronize()));
 static long long h[64*32]; cudaMemcpyFromSymbol(h,g_st,sizeof h);
 for(int u=0;u<8;u++){ long long b=h[u*16]; for(int i=0;i<13;i++) if(i!=9) printf("%6lld",h[u*16+i]-b); printf(" | next %lld\n",h[(u+1)*16]-b);} }
int main(){ go<4,8>(1,128,128*152); go<4,8>(1,128,256*152);go<4,8>(1,128,512*152);}
