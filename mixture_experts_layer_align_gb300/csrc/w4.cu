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

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;       // weight rows of a thread block (64 gate and 64 up rows)
constexpr int kStepK = 256;      // columns of a stage
constexpr int kStages = 3;
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

enum W4Mode { kMatvec, kGateUp, kDown };
struct W4Job {
  const void* scales;
  const uint8_t* zeros;
  int scale_bf16;
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
  // columns of a unit: what is converted, multiplied and accumulated at a time
  static constexpr int kUnitK = NT == 64 && PG == 1 ? 64 : 128;
  static constexpr int kSub = kUnitK / (32 * PG);  // groups, so accumulators, of a unit
  static constexpr int kACols = kUnitK / 2;
  static constexpr int kUsed = kACols + kN * kSub;
  static constexpr int kTmem = kUsed <= 128 ? 128 : 256;
  static_assert(kUsed <= 256, "tensor memory of a thread block");
  static constexpr int kXBytes = kN * kUnitK * 2;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + kXBytes + 1024;
  static constexpr int kPerSm = NT <= 16 ? 4 : NT == 32 ? 3 : 2;
};

// PG: 32-column pieces of a group (1, 2, 4).  NT: tokens of a block at most.
template <int PG, bool ZP, int NT>
__global__ void __launch_bounds__(kThreads, (W4Shape<PG, NT>::kPerSm))
    w4_kernel(const __grid_constant__ CUtensorMap map, const W4Job j) {
  using S = W4Shape<PG, NT>;
  constexpr int kUnits = kStepK / S::kUnitK;  // units of a stage
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kStages], s_a_full, s_d_full;
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
    mbar_init(&s_a_full, kWorkers / 32);
    mbar_init(&s_d_full, 1);
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
  const uint32_t tmem = s_tmem, t_a = tmem, t_d = tmem + S::kACols;
  const size_t row_a = (j.mode == kGateUp ? static_cast<size_t>(e) * 2 : static_cast<size_t>(e)) *
                           j.n_rows + r0;
  const size_t row_b = row_a + (j.mode == kGateUp ? j.n_rows : kRows / 2);

  // this block's slice of K, in stages and units
  const int all_steps = (j.K + kStepK - 1) / kStepK;
  const int step0 = static_cast<int>(static_cast<long long>(rank) * all_steps / CS);
  const int step1 = static_cast<int>(static_cast<long long>(rank + 1) * all_steps / CS);
  const int n_steps = step1 - step0;
  const int k0 = step0 * kStepK, k1 = min(step1 * kStepK, j.K);
  const int n_units = (k1 - k0 + S::kUnitK - 1) / S::kUnitK;

  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.f;

  if (warp == 4) {
    if (lane == 0) {
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
      const uint64_t db = sdesc_kmajor_sw128(smem_addr(s_x));
      bool ok = true;
      for (int u = 0; u < n_units; ++u) {
        ok = mbar_wait(&s_a_full, u & 1, &s_abort, j.timeout_ns);
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int i = 0; i < S::kUnitK / 16; ++i) {
          // 16 columns: 32 bytes further in a token's 128-byte row, or its next row block
          const uint64_t b = db + (i % 4) * 2 + (i / 4) * (S::kN * 128 / 16);
          umma_bf16_ts(t_d + i / (2 * PG) * S::kN, t_a + i * 8, b, idesc, i % (2 * PG) != 0);
        }
        umma_commit(&s_d_full);
        // every warp has read the unit's codes: its stage is free after the last one
        if ((u + 1) % kUnits == 0 && issued < n_steps) issue(issued++);
      }
      if (!ok) {
        s_abort = 1;
        if (j.err != nullptr) atomicOr(j.err, kDevErrTimeout);
        // the copies in flight land before the block leaves
        volatile int never = 0;
        for (int i = max(0, issued - kStages); i < issued; ++i)
          mbar_wait(&s_full[i % kStages], i / kStages & 1, &never, j.timeout_ns);
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
    const size_t group0 = grow * groups + k0 / (32 * PG);
    // tokens: 16-byte piece tid % (kUnitK / 8) of token tid / (kUnitK / 8), ...
    constexpr int kPieces = S::kUnitK / 8, kPerRound = kWorkers / kPieces;
    constexpr int kRounds = (NT + kPerRound - 1) / kPerRound;
    const int piece = tid % kPieces;
    const __nv_bfloat16* xp[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int t = min(tid / kPieces + i * kPerRound, valid - 1);
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
    auto fetch_x = [&](int u) {
      const bool on = u < n_units && k0 + u * S::kUnitK + piece * 8 < k1;
#pragma unroll
      for (int i = 0; i < kRounds; ++i)
        x_nx[i] = on ? __ldg(reinterpret_cast<const uint4*>(xp[i] + u * S::kUnitK))
                     : make_uint4(0, 0, 0, 0);
    };
    float s_nx[S::kSub];
    uint32_t z_nx[S::kSub];
    auto fetch_scales = [&](int u) {
#pragma unroll
      for (int i = 0; i < S::kSub; ++i) {
        const int g = u * S::kSub + i;
        if (u < n_units && k0 + g * (32 * PG) < k1) {
          s_nx[i] = j.scale_bf16
                        ? __uint_as_float(static_cast<uint32_t>(__ldg(
                              static_cast<const uint16_t*>(j.scales) + group0 + g)) << 16)
                        : __ldg(static_cast<const float*>(j.scales) + group0 + g);
          if (ZP) z_nx[i] = __ldg(j.zeros + group0 + g);
        } else {
          s_nx[i] = 0.f;
          if (ZP) z_nx[i] = 0;
        }
      }
    };
    fetch_scales(0);
    fetch_x(0);
    float s_cur[S::kSub];
    // adds the finished accumulators of unit u, scaled
    auto flush = [&](int u) {
      if (!mbar_wait(&s_d_full, u & 1, &s_abort, j.timeout_ns)) return false;
      tc_fence_after_sync();
      const uint32_t at = t_d + (static_cast<uint32_t>(warp * 32) << 16);
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
            acc[t0 + t] = fmaf(s_cur[i], __uint_as_float(d[t / 8][t % 8]), acc[t0 + t]);
        }
      return true;
    };
    const uint32_t a_at = t_a + (static_cast<uint32_t>(warp * 32) << 16);
    bool ok = true;
    for (int u = 0; u < n_units; ++u) {
      const int step = u / kUnits;
      if (u % kUnits == 0) {
        ok = mbar_wait(&s_full[step % kStages], step / kStages & 1, &s_abort, j.timeout_ns);
        if (!ok) break;
      }
      const uint8_t* codes = smem + step % kStages * kStageBytes + row * 128;
      float s[S::kSub];
      uint32_t nz[S::kSub];
#pragma unroll
      for (int i = 0; i < S::kSub; ++i) {
        s[i] = s_nx[i];
        nz[i] = ZP ? w4_neg_zero(z_nx[i]) : kNegEight;
      }
      fetch_scales(u + 1);
      // 32 columns of the row: 16 words of A
      auto convert = [&](int c, uint32_t (&v)[16]) {
        const uint4 q = *reinterpret_cast<const uint4*>(
            codes + ((u % kUnits * (S::kUnitK / 32) + c) ^ (row & 7)) * 16);
        w4_pairs(q.x, nz[c / PG], v);
        w4_pairs(q.y, nz[c / PG], v + 4);
        w4_pairs(q.z, nz[c / PG], v + 8);
        w4_pairs(q.w, nz[c / PG], v + 12);
      };
      uint32_t v0[16], v1[16];
      convert(0, v0);
      convert(1, v1);
      if (u > 0) {
        ok = flush(u - 1);  // and the MMAs that read A and x are done
        if (!ok) break;
      }
      tmem_st16(a_at, v0);
      tmem_st16(a_at + 16, v1);
      if (S::kUnitK == 128) {
        convert(2, v0);
        convert(3, v1);
        tmem_st16(a_at + 32, v0);
        tmem_st16(a_at + 48, v1);
      }
      // x, its columns in the order of the codes: (0,4), (1,5), (2,6), (3,7)
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int t = tid / kPieces + i * kPerRound;
        const uint4 x = x_nx[i];
        uint4 v;
        v.x = __byte_perm(x.x, x.z, 0x5410);
        v.y = __byte_perm(x.x, x.z, 0x7632);
        v.z = __byte_perm(x.y, x.w, 0x5410);
        v.w = __byte_perm(x.y, x.w, 0x7632);
        *reinterpret_cast<uint4*>(s_x + piece / 8 * (S::kN * 128) + t * 128 +
                                  ((piece % 8) ^ (t & 7)) * 16) = v;
      }
      fetch_x(u + 1);
      fence_proxy_async_smem();
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_a_full);
#pragma unroll
      for (int i = 0; i < S::kSub; ++i) s_cur[i] = s[i];
    }
    if (ok && n_units > 0) ok = flush(n_units - 1);
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

// Thread blocks that split K: as many as there is room for at a time, each with a
// stage at least.
int choose_cluster(int K, long long tiles, int per_sm, int num_sms) {
  const int steps = (K + kStepK - 1) / kStepK;
  int c = 1;
  while (c < 8 && 2 * c <= steps && tiles * 2 * c <= static_cast<long long>(per_sm) * num_sms) c *= 2;
  return c;
}

template <int PG, bool ZP, int NT>
cudaError_t launch(const CUtensorMap& map, const W4Job& job, int num_sms, cudaStream_t st) {
  using S = W4Shape<PG, NT>;
  cudaError_t e = checked(cudaFuncSetAttribute(w4_kernel<PG, ZP, NT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(S::kSmem)),
                          "smem attribute");
  if (e != cudaSuccess) return e;
  W4Job j = job;
  const int rows = j.mode == kGateUp ? kRows / 2 : kRows;
  const long long tiles = (static_cast<long long>(j.n_rows) + rows - 1) / rows * j.n_blocks;
  j.cluster = choose_cluster(j.K, tiles, S::kPerSm, num_sms);
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
  return checked(cudaLaunchKernelEx(&cfg, w4_kernel<PG, ZP, NT>, map, j), "kernel launch");
}

template <int PG, bool ZP>
cudaError_t launch_tokens(const CUtensorMap& map, const W4Job& j, int nt, int num_sms,
                          cudaStream_t st) {
  if (nt == 8) return launch<PG, ZP, 8>(map, j, num_sms, st);
  if (nt == 16) return launch<PG, ZP, 16>(map, j, num_sms, st);
  if (nt == 32) return launch<PG, ZP, 32>(map, j, num_sms, st);
  return launch<PG, ZP, 64>(map, j, num_sms, st);
}

cudaError_t launch_job(const CUtensorMap& map, int group, const W4Job& j, int nt, int num_sms,
                       cudaStream_t st) {
  if (j.zeros != nullptr)
    return group == 32   ? launch_tokens<1, true>(map, j, nt, num_sms, st)
           : group == 64 ? launch_tokens<2, true>(map, j, nt, num_sms, st)
                         : launch_tokens<4, true>(map, j, nt, num_sms, st);
  return group == 32   ? launch_tokens<1, false>(map, j, nt, num_sms, st)
         : group == 64 ? launch_tokens<2, false>(map, j, nt, num_sms, st)
                       : launch_tokens<4, false>(map, j, nt, num_sms, st);
}

}  // namespace

int w4_block_rows(int T) { return T <= 8 ? 8 : T <= 16 ? 16 : T <= 32 ? 32 : 64; }

cudaError_t launch_w4_matvec(const CUtensorMap& map, const __nv_bfloat16* x, int T, int K, int N,
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
  j.x = x;
  j.T = T;
  j.out = out;
  j.out_fp32 = out_fp32 ? 1 : 0;
  j.timeout_ns = timeout_ns;
  return launch_job(map, w.group, j, nt, num_sms, st);
}

cudaError_t launch_w4_layer(const CUtensorMap& map13, const CUtensorMap& map2,
                            const W4LayerParams& p, int num_sms, cudaStream_t st) {
  const int nt = w4_block_rows(p.T);
  const long long P = static_cast<long long>(p.T) * p.k;
  W4Job j{};
  j.scales = p.w13.scales;
  j.zeros = p.w13.zeros;
  j.scale_bf16 = p.w13.scale_bf16;
  j.mode = kGateUp;
  j.K = p.H;
  j.n_rows = p.I;
  j.n_blocks = static_cast<int>(std::min(P, (P + std::min<long long>(p.E, P) * (nt - 1)) / nt));
  j.x = p.x;
  j.T = p.T;
  j.out = p.h;
  j.sorted_ids = p.sorted_ids;
  j.block_expert = p.block_expert;
  j.num_padded = p.num_padded;
  j.wts = p.wts;
  j.P = static_cast<int>(P);
  j.k = p.k;
  j.err = p.err;
  j.timeout_ns = p.timeout_ns;
  cudaError_t e = launch_job(map13, p.w13.group, j, nt, num_sms, st);
  if (e != cudaSuccess) return e;
  j.scales = p.w2.scales;
  j.zeros = p.w2.zeros;
  j.scale_bf16 = p.w2.scale_bf16;
  j.mode = kDown;
  j.K = p.I;
  j.n_rows = p.H;
  j.x = p.h;
  j.out = p.y;
  e = launch_job(map2, p.w2.group, j, nt, num_sms, st);
  if (e != cudaSuccess) return e;
  const long long n = static_cast<long long>(p.T) * (p.H / 4);
  return launch_pdl(w4_combine_kernel,
                    dim3(static_cast<int>(std::min<long long>((n + 255) / 256, 2048))), dim3(256),
                    0, st, static_cast<const float*>(p.y), p.T, p.k, p.H, p.out);
}

}  // namespace moe
