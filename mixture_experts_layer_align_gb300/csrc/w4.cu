// 4-bit weights with group scales: matrix-vector products and the expert
// products of the MoE layer for a few tokens.
//
//   y[t][r] = sum over groups of scale[r][g] * sum_k x[t][k] (code[r][k] - zero[r][g])
//           = sum over groups of scale[r][g] * (D[r][g][t] - zero[r][g] X[g][t]),
//   D = sum_k code x, X = sum_k x.
// At a few tokens the codes' bytes bound it, if turning them into an MMA operand
// does not: at 6.8 TB/s an SM takes in 47 codes a clock.  So they are hardly
// turned at all.  A byte 0..15 read as E4M3 is that many times 2^-9 (the two lowest
// exponents share their spacing): the nibbles of a word, spread over bytes by two
// masks and a shift, are the A operand of tcgen05.mma kind::f8f6f4.  x becomes three
// E5M2 pieces whose sum it is, one MMA each into the same accumulator:
// a power of two brings the largest |x| of a token to 2^14 .. 2^15, where x is
// an fp16 value of 8 significant bits; a piece is the top byte of what is left (a
// sign, 5 exponent and 2 mantissa bits: E5M2, three significant bits), so the third
// leaves nothing but what lies 2^-31 below the largest.  Products are exact and
// sums are fp32 (the MMA was checked to keep addends 2^-23 below the sum).
//
// x, and h, is split once for a call, by a kernel of its own, into the image that
// shared memory needs.  A thread block owns 128
// weight rows and a slice of K; the blocks of a cluster share rows and split K.  TMA
// brings 256 columns of the codes (128 bytes of a row) a stage, and x block by block
// of 128 columns.  Four warps, a thread per row, spread the codes of a unit into
// tensor memory (A, 128 rows) and, while its MMAs run, scale the sums of the unit
// before, again a thread per row, in fp32; a fifth warp issues the copies and MMAs.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;      // weight rows of a thread block (64 gate and 64 up rows)
constexpr int kStepK = 256;     // columns of a stage
constexpr int kStageBytes = kRows * kStepK / 2;
constexpr int kRowThreads = 128;  // one per row
constexpr int kThreads = kRowThreads + 32;
constexpr int kBlockK = 128;    // columns of a block of x
constexpr int kPieces = 3;
constexpr int kSplitThreads = 512;
constexpr int kXSlots = 4;      // blocks of x in shared memory

// nt tokens, split: for each block of 128 columns kPieces x [nt][128 bytes], the
// 16-byte chunks of token t's row at chunk ^ t % 8 (the 128-byte swizzle) and in each
// 8 columns the order of the spread codes, 0 2 4 6 1 3 5 7; then for each block (an
// even number of them) fp32 [128 / group][nt], 2^-9 times the sums of the scaled x;
// then fp32 [nt], the factors that undo the scaling of x and of the codes.
__host__ __device__ constexpr int x_piece_bytes(int nt) { return nt * kBlockK; }
struct XLayout {
  int n_cols, nt, per_block;  // blocks of columns, tokens, sums of a block
  __host__ __device__ XLayout(int K, int nt_, int group)
      : n_cols((K + kBlockK - 1) / kBlockK), nt(nt_), per_block(kBlockK / group * nt_) {}
  __host__ __device__ size_t sums() const {
    return static_cast<size_t>(n_cols) * kPieces * x_piece_bytes(nt);
  }
  __host__ __device__ size_t factors() const {
    return sums() + static_cast<size_t>(n_cols + n_cols % 2) * per_block * 4;
  }
  __host__ __device__ size_t bytes() const { return factors() + nt * 4; }  // a multiple of 16
};

__device__ __forceinline__ void load_raw(uint32_t* r, const uint2* p) {
  const uint2 v = __ldg(p);
  r[0] = v.x, r[1] = v.y;
}
__device__ __forceinline__ void load_raw(uint32_t* r, const uint4* p) {
  const uint4 v = __ldg(p);
  r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Larger of two pairs of bf16 magnitudes, NaN if either is.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A warp waits for phase `parity` of `bar`; false, for all of it, after a limited
// number of tries (seconds).  The first look is apart from the loop: it nearly
// always finds the phase over, and a loop costs three times its branch.
constexpr uint32_t kWaitTries = 1u << 24;
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
#pragma unroll 1
  for (uint32_t n = kWaitTries; n != 0; --n)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return false;
}

// Instruction descriptor: D fp32, A E4M3, B E5M2, both K-major, M = 128.
__device__ constexpr uint32_t w4_idesc(int N) {
  return (1u << 4) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | ((128u >> 4) << 24);
}

// x, split: a thread block for each token.  Layer: the rows of the pairs in
// sorted_ids, row pair / k of x.  A token with infinities or NaN gets the factor NaN:
// its sums, not numbers then, are formed again from x itself.
__global__ void __launch_bounds__(kSplitThreads)
    w4_split_kernel(const __nv_bfloat16* __restrict__ x, int T, int K, int nt, int group,
                    uint8_t* __restrict__ xq, const int32_t* __restrict__ sorted_ids,
                    const int32_t* __restrict__ num_padded, int P, int k) {
  __shared__ float s_max[kSplitThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int block = blockIdx.x / nt, t = blockIdx.x % nt;
  long long row = blockIdx.x;
  if (sorted_ids != nullptr) {
    if (row >= __ldg(num_padded)) return;
    const int pair = __ldg(sorted_ids + row);
    if (pair >= P) return;
    row = pair / k;
  } else if (row >= T) {
    return;
  }
  const XLayout lay(K, nt, group);
  const uint4* src = reinterpret_cast<const uint4*>(x + row * K);
  uint8_t* to = xq + block * lay.bytes();
  const int tid = threadIdx.x, n8 = K / 8;
  constexpr int kKeep = 4;  // loads kept from the first pass
  uint4 keep[kKeep];
  uint32_t m = 0;
  auto top = [&](const uint4& w) {
    m = max_bf16x2(m, max_bf16x2(max_bf16x2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                 max_bf16x2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    keep[i] = tid + i * kSplitThreads < n8 ? __ldg(src + tid + i * kSplitThreads) : make_uint4(0, 0, 0, 0);
    top(keep[i]);
  }
  for (int i = tid + kKeep * kSplitThreads; i < n8; i += kSplitThreads) top(__ldg(src + i));
  m = max_bf16x2(m, m >> 16 | m << 16);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
  // (magnitudes as integers order like the numbers, NaN above all)
  if (tid % 32 == 0) s_max[tid / 32] = __uint_as_float(m << 16);
  __syncthreads();
  uint32_t top_bits = 0;
#pragma unroll
  for (int i = 0; i < kSplitThreads / 32; ++i) top_bits = max(top_bits, __float_as_uint(s_max[i]));
  const bool finite = top_bits < 0x7f800000u;
  // biased exponent of the largest; at least 14, so that the scale stays finite
  const int ex = max(finite ? static_cast<int>(top_bits >> 23) : 0, 14);
  const float scale = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);  // 2^(141 - ex)
  const uint64_t scale2 = pack2(scale, scale);
  if (tid == 0)
    reinterpret_cast<float*>(to + lay.factors())[t] =
        finite ? __uint_as_float(static_cast<uint32_t>(ex - 5) << 23) : __int_as_float(0x7fc00000);
  float* sums = reinterpret_cast<float*>(to + lay.sums());
  const int n8_pad = lay.n_cols * (kBlockK / 8);
#pragma unroll 1
  for (int i = tid; i < n8_pad; i += kSplitThreads) {  // whole half warps: a block is 16 threads
    uint4 w = i < n8 && finite ? (i < kSplitThreads       ? keep[0]
                                  : i < 2 * kSplitThreads ? keep[1]
                                  : i < 3 * kSplitThreads ? keep[2]
                                  : i < 4 * kSplitThreads ? keep[3]
                                                   : __ldg(src + i))
                               : make_uint4(0, 0, 0, 0);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    float sum = 0.f;
    uint32_t h[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float lo, hi;
      unpack2(mul2(pack2(bf16_lo(ww[n]), bf16_hi(ww[n])), scale2), lo, hi);
      sum += lo + hi;
      h[n] = cvt_f16x2(lo, hi);
    }
    const int blk = i / 16, c8 = i % 16;
    uint8_t* p = to + static_cast<size_t>(blk) * kPieces * x_piece_bytes(nt) + t * 128 +
                 ((c8 / 2) ^ (t & 7)) * 16 + c8 % 2 * 8;
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      const uint32_t a = __byte_perm(h[0], h[1], 0x7351), b = __byte_perm(h[2], h[3], 0x7351);
      *reinterpret_cast<uint2*>(p + n * x_piece_bytes(nt)) =
          make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = sub_f16x2(h[q], h[q] & 0xff00ff00u);
    }
    const unsigned half = 0xffffu << (tid & 16);
    for (int o = 1; o < group / 8; o <<= 1) sum += __shfl_xor_sync(half, sum, o);
    if (c8 % (group / 8) == 0)
      sums[static_cast<size_t>(blk) * lay.per_block + c8 / (group / 8) * nt + t] = 0x1p-9f * sum;
  }
}

enum W4Mode { kMatvec, kGateUp, kDown };
struct W4Job {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  int scale_bf16;
  int whole_stages;  // K % kStepK == 0 and aligned tensors: a stage's scales in one load
  int mode, K;
  int n_rows;    // rows of the result: N, I or H
  int n_blocks;  // blocks of tokens (an upper bound for the layer)
  const uint8_t* xq;        // x (down: h), split: an XLayout for each block of tokens
  const __nv_bfloat16* x;   // tokens (down: h by pair)
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
};

template <int PG, int NT>
struct W4Shape {
  static constexpr int kN = NT < 16 ? 16 : NT;  // MMA N (16 at least with 128 rows)
  static constexpr int kPerSm = NT == 8 ? 4 : NT == 16 ? 3 : 2;
  static constexpr int kTmem = NT <= 16 ? 128 : 256;  // columns of tensor memory
  // Columns of a unit, what is multiplied at a time: as many as leave room for
  // two buffers of A and two sets of accumulators (one is read during the next
  // unit's MMAs).
  static constexpr bool fits(int unit) { return unit / 2 + 2 * kN * (unit / (32 * PG)) <= kTmem; }
  static constexpr int kUnitK = fits(128) ? 128 : 64;
  static_assert(fits(kUnitK) && kUnitK >= 32 * PG, "a unit holds whole groups");
  static constexpr int kUnits = kBlockK / kUnitK;  // of a block of columns
  static constexpr int kSub = kUnitK / (32 * PG);  // groups, so accumulators, of a unit
  static constexpr int kACols = kUnitK / 4;
  static constexpr int kStages = NT == 8 ? 2 : 3;
  static constexpr int kXBytes = kPieces * x_piece_bytes(NT);
  static constexpr int kSumSlots = kStages + 1;              // stages' sums of x
  static constexpr int kSumBytes = 2 * (4 / PG) * NT * 4;    // of the two blocks of a stage
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes +
                                  kXSlots * kXBytes + kSumSlots * kSumBytes;
};

// sum_k x[k] (code[k] - zero) * scale over columns k0 .. k1 of a weight row,
// column by column: what a token with infinities or NaN gets.
__device__ __noinline__ float w4_row_plain(const W4Job& j, int group, size_t grow,
                                           const __nv_bfloat16* x, int k0, int k1) {
  const size_t g0 = grow * ((j.K + group - 1) / group);
  float sum = 0.f;
  for (int k = k0; k < k1;) {
    const int g = k / group, end = min(k1, (g + 1) * group);
    const float zero = j.zeros ? static_cast<float>(j.zeros[g0 + g]) : 8.f;
    const float scale = j.scale_bf16
                            ? __bfloat162float(static_cast<const __nv_bfloat16*>(j.scales)[g0 + g])
                            : static_cast<const float*>(j.scales)[g0 + g];
    float part = 0.f;
    for (; k < end; ++k) {
      const int code = j.codes[grow * (j.K / 2) + k / 2] >> (k % 2 * 4) & 15;
      part = fmaf(__bfloat162float(x[k]), static_cast<float>(code) - zero, part);
    }
    sum = fmaf(scale, part, sum);
  }
  return sum;
}

// PG: 32-column pieces of a group (1, 2, 4).  NT: tokens of a block at most.
template <int PG, bool ZP, int NT>
__global__ void __launch_bounds__(kThreads, (W4Shape<PG, NT>::kPerSm))
    w4_kernel(const __grid_constant__ CUtensorMap map, const W4Job j) {
  using S = W4Shape<PG, NT>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_codes[kStages];  // a stage's codes and sums of x are there
  __shared__ uint64_t s_x[kXSlots];      // a block of x is there
  __shared__ uint64_t s_done[2];         // even and odd units' MMAs are done
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* x_pieces = smem + kStages * kStageBytes;
  float* x_sums = reinterpret_cast<float*>(x_pieces + kXSlots * S::kXBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int CS = j.cluster;
  const int rank = CS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (tid == 0) {
    prefetch_tensormap(&map);
    for (int i = 0; i < kStages; ++i) mbar_init(&s_codes[i], 1);
    for (int i = 0; i < kXSlots; ++i) mbar_init(&s_x[i], 1);
    mbar_init(&s_done[0], 1);
    mbar_init(&s_done[1], 1);
    s_abort = 0;
    fence_mbarrier_init();
  }
  // Up to pdl_wait() nothing is read that the kernel before, which splits x, writes:
  // the weights and the lists of the alignment are older than it.

  // which rows and tokens; a block past the layer's last one leaves (all of its
  // cluster does)
  const int job = static_cast<int>(blockIdx.x) / CS;
  const int block = job % j.n_blocks;
  const int rows_out = j.mode == kGateUp ? kRows / 2 : kRows;  // rows of the result
  const int r0 = job / j.n_blocks * rows_out;
  int e = 0, valid;
  if (j.mode == kMatvec) {
    valid = min(NT, j.T - block * NT);
  } else {
    if (block * NT >= __ldg(j.num_padded)) return;
    e = __ldg(j.block_expert + block);
    const int32_t* ids = j.sorted_ids + static_cast<size_t>(block) * NT;
    valid = __popc(__ballot_sync(0xffffffffu, lane < NT && __ldg(ids + min(lane, NT - 1)) < j.P));
  }
  if (warp == 4) {
    tmem_alloc(&s_tmem, S::kTmem);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem, t_d = tmem + 2 * S::kACols;
  const size_t expert_row = static_cast<size_t>(e) * j.n_rows * (j.mode == kGateUp ? 2 : 1);

  // this block's slice of K, in stages and blocks of columns
  const int all_steps = (j.K + kStepK - 1) / kStepK;
  const int step0 = static_cast<int>(static_cast<long long>(rank) * all_steps / CS);
  const int step1 = static_cast<int>(static_cast<long long>(rank + 1) * all_steps / CS);
  const int n_steps = step1 - step0;
  const int k0 = step0 * kStepK, k1 = min(step1 * kStepK, j.K);
  const int n_blks = (k1 - k0 + kBlockK - 1) / kBlockK;
  // this thread's weight row (past the result's last one: that one)
  const int row = tid % kRows;
  const size_t grow = expert_row + min(r0 + row % rows_out, j.n_rows - 1) +
                      (j.mode == kGateUp && row >= rows_out ? j.n_rows : 0);

  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.f;
  bool ok = true;  // once a wait gives up, the loops run out without waits and MMAs

  if (warp == 4) {
    // ---------------------------------------------------------- copies and MMAs
    const XLayout lay(j.K, NT, 32 * PG);
    const uint8_t* xq = j.xq + block * lay.bytes();
    auto issue_codes = [&](int step) {
      uint64_t* bar = &s_codes[step % kStages];
      uint8_t* dst = smem + step % kStages * kStageBytes;
      mbar_arrive_expect_tx(bar, kStageBytes + S::kSumBytes);
      const int col = (step0 + step) * (kStepK / 2), row_a = static_cast<int>(expert_row) + r0;
      tma_load_2d(dst, &map, bar, col, row_a);
      tma_load_2d(dst + kStageBytes / 2, &map, bar, col,
                  row_a + (j.mode == kGateUp ? j.n_rows : kRows / 2));
    };
    auto issue_sums = [&](int step) {
      bulk_load(x_sums + step % S::kSumSlots * (S::kSumBytes / 4),
                xq + lay.sums() + static_cast<size_t>(step0 + step) * S::kSumBytes, S::kSumBytes,
                &s_codes[step % kStages]);
    };
    const int x_rows = (valid + 7) / 8 * 8;
    auto issue_x = [&](int blk) {
      uint64_t* bar = &s_x[blk % kXSlots];
      uint8_t* dst = x_pieces + blk % kXSlots * S::kXBytes;
      const uint8_t* src = xq + static_cast<size_t>(k0 / kBlockK + blk) * S::kXBytes;
      mbar_arrive_expect_tx(bar, kPieces * x_rows * 128);
      if (x_rows == NT) {
        bulk_load(dst, src, S::kXBytes, bar);
      } else {
        for (int n = 0; n < kPieces; ++n)
          bulk_load(dst + n * x_piece_bytes(NT), src + n * x_piece_bytes(NT), x_rows * 128, bar);
      }
    };
    int codes_issued = min(kStages, n_steps), x_issued = min(kXSlots, n_blks);
    if (elect_one())
      for (int i = 0; i < codes_issued; ++i) issue_codes(i);
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    if (elect_one()) {
      for (int i = 0; i < codes_issued; ++i) issue_sums(i);
      for (int i = 0; i < x_issued; ++i) issue_x(i);
    }
    __syncwarp();
    // N: the block's tokens, and eight stand for both eight-row halves of 16
    const uint32_t idesc = w4_idesc(max(16, (valid + 15) / 16 * 16));
    const uint64_t db0 = sdesc_kmajor_sw128(smem_addr(x_pieces)) -
                         (NT == 8 ? static_cast<uint64_t>(1024 >> 4) << 32 : 0);
    for (int blk = 0; blk < n_blks; ++blk) {
      ok = ok && warp_wait(&s_x[blk % kXSlots], blk / kXSlots & 1);
#pragma unroll
      for (int h = 0; h < S::kUnits; ++h) {
        const int u = blk * S::kUnits + h;
        named_barrier(1 + (u & 1), kThreads);  // A is in place
        if (ok && elect_one()) {
          tc_fence_after_sync();
          const uint64_t db = db0 + blk % kXSlots * (S::kXBytes / 16);
          const uint32_t a = tmem + (u & 1) * S::kACols;
          const uint32_t d = t_d + (u & 1) * (S::kN * S::kSub);
#pragma unroll
          for (int n = kPieces - 1; n >= 0; --n)  // small pieces first
#pragma unroll
            for (int i = 0; i < S::kUnitK / 32; ++i)
              umma_f8_ts(d + i / PG * S::kN, a + i * 8,
                         db + n * (x_piece_bytes(NT) / 16) + (h * (S::kUnitK / 32) + i) * 2, idesc,
                         n < kPieces - 1 || i % PG != 0);
          umma_commit(&s_done[u & 1]);
        }
        __syncwarp();
      }
      // Every warp has read the block's codes, and has added the sums of the block
      // before the last: a stage is free after its second block, and x's buffer of
      // two blocks ago too.
      if (ok && elect_one()) {
        if (blk % 2 == 1 && codes_issued < n_steps) {
          issue_codes(codes_issued);
          issue_sums(codes_issued);
        }
        if (blk >= 2 && x_issued < n_blks) issue_x(x_issued);
      }
      __syncwarp();
      if (blk % 2 == 1 && codes_issued < n_steps) ++codes_issued;
      if (blk >= 2 && x_issued < n_blks) ++x_issued;
    }
    if (!ok) {  // the copies in flight land before the block leaves
      for (int i = max(0, codes_issued - kStages); i < codes_issued; ++i)
        warp_wait(&s_codes[i % kStages], i / kStages & 1);
      for (int i = max(0, x_issued - kXSlots); i < x_issued; ++i)
        warp_wait(&s_x[i % kXSlots], i / kXSlots & 1);
    }
  } else {
    // ---------------------------------------------------------- codes and sums
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const int groups = (j.K + 32 * PG - 1) / (32 * PG);
    const size_t group0 = grow * groups + k0 / (32 * PG);
    // the row's scales and zero points of this slice on their way to L2
    {
      const int n = (k1 - k0 + 32 * PG - 1) / (32 * PG), lg = j.scale_bf16 ? 1 : 2;
      const uint8_t* p = static_cast<const uint8_t*>(j.scales) + (group0 << lg);
      for (int i = 0; i < n << lg; i += 128) prefetch_l2(p + i);
      prefetch_l2(p + ((n - 1) << lg));
      if (ZP) {
        for (int i = 0; i < n; i += 128) prefetch_l2(j.zeros + group0 + i);
        prefetch_l2(j.zeros + group0 + n - 1);
      }
    }
    // Scales and zero points of a stage's groups, as they lie in memory: one load
    // each when every row's stage starts on its size (K a multiple of the stage's
    // columns), else group by group.
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
#pragma unroll
    for (int i = 0; i < (kGroups + 3) / 4; ++i) z_raw[i] = 0;
    fetch_scales(0);
    constexpr int kBlkGroups = 4 / PG;
    float s_step[kGroups], s_old[S::kSub], z_old[S::kSub];
    uint32_t z_step[(kGroups + 3) / 4];
    const float* sums_old = x_sums;  // of the last unit's groups
    // adds unit u's sums, scaled
    auto flush = [&](int u) {
      float4 xs[NT <= 8 ? S::kSub : 1][2];
      if (NT <= 8) {
#pragma unroll
        for (int i = 0; i < S::kSub; ++i) {
          xs[i][0] = *reinterpret_cast<const float4*>(sums_old + i * NT);
          xs[i][1] = *reinterpret_cast<const float4*>(sums_old + i * NT + 4);
        }
      }
      ok = ok && warp_wait(&s_done[u & 1], u >> 1 & 1);
      tc_fence_after_sync();
      const uint32_t at = t_d + lanes + (u & 1) * (S::kN * S::kSub);
#pragma unroll
      for (int t0 = 0; t0 < NT; t0 += 8) {
        if (t0 > 0 && t0 >= valid) break;
        uint32_t d[S::kSub][8];
#pragma unroll
        for (int i = 0; i < S::kSub; ++i) tmem_ld8_async(at + i * S::kN + t0, d[i]);
#pragma unroll
        for (int i = 0; i < S::kSub; ++i) {
          tmem_wait_ld8(d[i]);
          const uint64_t zz = pack2(-z_old[i], -z_old[i]), ss = pack2(s_old[i], s_old[i]);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float4 xv = NT <= 8 ? xs[i][n / 2]
                                      : *reinterpret_cast<const float4*>(sums_old + i * NT + t0 +
                                                                         n / 2 * 4);
            const uint64_t x2 = n % 2 ? pack2(xv.z, xv.w) : pack2(xv.x, xv.y);
            const uint64_t d2 =
                pack2(__uint_as_float(d[i][2 * n]), __uint_as_float(d[i][2 * n + 1]));
            float& lo = acc[t0 + 2 * n];
            float& hi = acc[t0 + 2 * n + 1];
            unpack2(fma2(ss, fma2(zz, x2, d2), pack2(lo, hi)), lo, hi);
          }
        }
      }
    };
    // a block of 128 columns, the hb-th of its stage
    auto columns = [&](int blk, int slot, const float* sums, auto which) {
      constexpr int hb = decltype(which)::value;
      const uint8_t* codes = smem + slot * kStageBytes + tid * 128;
#pragma unroll
      for (int h = 0; h < S::kUnits; ++h) {
        const int u = blk * S::kUnits + h;
        uint32_t v[S::kACols];
#pragma unroll
        for (int c = 0; c < S::kUnitK / 32; ++c) {
          const uint4 q = *reinterpret_cast<const uint4*>(
              codes + ((hb * 4 + h * (S::kUnitK / 32) + c) ^ (tid & 7)) * 16);
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            v[c * 8 + 2 * n] = w[n] & 0x0f0f0f0fu;
            v[c * 8 + 2 * n + 1] = w[n] >> 4 & 0x0f0f0f0fu;
          }
        }
        // the MMAs that read this buffer of A were waited for when their sums were added
        const uint32_t a = tmem + (u & 1) * S::kACols + lanes;
#pragma unroll
        for (int n = 0; n < S::kACols; n += 16) tmem_st16(a + n, v + n);
        tmem_wait_st();
        tc_fence_before_sync();
        // A is in place, and the unit's codes are read.  (After a wait that gave up
        // nothing but this barrier keeps the warps together.)
        if (ok) named_barrier_arrive(1 + (u & 1), kThreads);
        else named_barrier(1 + (u & 1), kThreads);
        if (u > 0) flush(u - 1);
#pragma unroll
        for (int i = 0; i < S::kSub; ++i) {
          const int g = hb * kBlkGroups + h * S::kSub + i;
          s_old[i] = s_step[g];
          z_old[i] = ZP ? static_cast<float>(z_step[g / 4] >> (8 * (g % 4)) & 0xffu) : 8.f;
        }
        sums_old = sums + (hb * kBlkGroups + h * S::kSub) * NT;
      }
    };
    int slot = 0, phase = 0, sum_slot = 0;
    for (int step = 0; step < n_steps; ++step) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        s_step[i] = __uint_as_float(!j.scale_bf16 ? s_raw[i]
                                    : i % 2       ? s_raw[i / 2] & 0xffff0000u
                                                  : s_raw[i / 2] << 16);
#pragma unroll
      for (int i = 0; i < (kGroups + 3) / 4; ++i) z_step[i] = z_raw[i];
      fetch_scales(step + 1);
      ok = ok && warp_wait(&s_codes[slot], phase);
      const float* sums = x_sums + sum_slot * (S::kSumBytes / 4);
      columns(2 * step, slot, sums, std::integral_constant<int, 0>{});
      if (2 * step + 1 < n_blks)
        columns(2 * step + 1, slot, sums, std::integral_constant<int, 1>{});
      if (++slot == kStages) slot = 0, phase ^= 1;
      if (++sum_slot == S::kSumSlots) sum_slot = 0;
    }
    flush(n_blks * S::kUnits - 1);
    pdl_wait();  // (what follows reads what the kernel before wrote, without a barrier)
    {
      const XLayout lay(j.K, NT, 32 * PG);
      const float* factors = reinterpret_cast<const float*>(j.xq + block * lay.bytes() + lay.factors());
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t < valid) acc[t] *= __ldg(factors + t);
    }
    // a sum that is not a number: as the weights and tokens have it, column by column
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t < valid && isnan(acc[t])) {
        size_t at = static_cast<size_t>(block) * NT + t;
        if (j.mode != kMatvec) {
          const int pair = __ldg(j.sorted_ids + at);
          at = static_cast<size_t>(j.mode == kGateUp ? pair / j.k : pair);
        }
        acc[t] = w4_row_plain(j, 32 * PG, grow, j.x + at * j.K, k0, k1);
      }
    }
  }
  if (!ok) s_abort = 1;
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (s_abort) {
    if (tid == 0 && j.err != nullptr) atomicOr(j.err, kDevErrTimeout);
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = __int_as_float(0x7fc00000);  // a wrong sum shows
  }
  if (warp == 4) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, S::kTmem);
  }
  // the sums over the cluster's slices of K, in rank order, in the stages' space:
  // red[token][row]
  float* red = reinterpret_cast<float*>(smem);
  if (warp < 4) {
#pragma unroll
    for (int t = 0; t < NT; ++t) red[t * kRows + tid] = acc[t];
  }
  __syncwarp();
  if (CS > 1) cluster_sync();
  else __syncthreads();
  const uint32_t red_at = smem_addr(red);
  auto sum = [&](int t, int r) {
    if (CS == 1) return red[t * kRows + r];
    float v = 0.f;
    for (int i = 0; i < CS; ++i)
      v += ld_cluster_f32(mapa_shared(red_at + (t * kRows + r) * 4, i));
    return v;
  };
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
        const float gate = sum(t, r), up = sum(t, r + rows_out);
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
  if (e == cudaSuccess)
    e = checked(cudaFuncSetAttribute(w4_kernel<PG, ZP, NT>,
                                     cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared),
                "smem attribute");
  if (e != cudaSuccess) return e;
  W4Job j = job;
  j.whole_stages = j.K % kStepK == 0 && reinterpret_cast<uintptr_t>(j.scales) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(j.zeros) % 8 == 0;
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
  return launch<PG, ZP, 32>(map, j, num_sms, st);
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

void set_weight(W4Job& j, const W4View& w) {
  j.codes = w.codes;
  j.scales = w.scales;
  j.zeros = w.zeros;
  j.scale_bf16 = w.scale_bf16;
}

}  // namespace

int w4_block_rows(int T) { return T <= 8 ? 8 : T <= 16 ? 16 : 32; }

int w4_layer_block_rows(int T, int E, int k) {
  const long long P = static_cast<long long>(T) * k;
  return T <= 8 || P <= 4ll * E ? 8 : T <= 16 || P <= 8ll * E ? 16 : 32;
}

size_t w4_split_bytes(long long blocks, int nt, int K, int group) {
  return static_cast<size_t>(blocks) * XLayout(K, nt, group).bytes();
}

namespace {

cudaError_t launch_split(const __nv_bfloat16* x, int T, int K, int n_blocks, int nt, int group,
                         uint8_t* xq, const int32_t* sorted_ids, const int32_t* num_padded, int P,
                         int k, cudaStream_t st) {
  return launch_pdl(w4_split_kernel, dim3(static_cast<unsigned>(n_blocks) * nt), dim3(kSplitThreads),
                    0, st,
                    x, T, K, nt, group, xq, sorted_ids, num_padded, P, k);
}

}  // namespace

cudaError_t launch_w4_matvec(const CUtensorMap& map, const __nv_bfloat16* x, int T, int K, int N,
                             const W4View& w, void* out, bool out_fp32, uint8_t* scratch,
                             int num_sms, cudaStream_t st) {
  const int nt = w4_block_rows(T);
  W4Job j{};
  set_weight(j, w);
  j.mode = kMatvec;
  j.K = K;
  j.n_rows = N;
  j.n_blocks = (T + nt - 1) / nt;
  j.xq = scratch;
  j.x = x;
  j.T = T;
  j.out = out;
  j.out_fp32 = out_fp32 ? 1 : 0;
  const cudaError_t e =
      launch_split(x, T, K, j.n_blocks, nt, w.group, scratch, nullptr, nullptr, 0, 1, st);
  if (e != cudaSuccess) return e;
  return launch_job(map, w.group, j, nt, num_sms, st);
}

cudaError_t launch_w4_layer(const CUtensorMap& map13, const CUtensorMap& map2,
                            const W4LayerParams& p, int num_sms, cudaStream_t st) {
  const int nt = w4_layer_block_rows(p.T, p.E, p.k);
  const long long P = static_cast<long long>(p.T) * p.k;
  W4Job j{};
  set_weight(j, p.w13);
  j.mode = kGateUp;
  j.K = p.H;
  j.n_rows = p.I;
  j.n_blocks = static_cast<int>(std::min(P, (P + std::min<long long>(p.E, P) * (nt - 1)) / nt));
  j.xq = p.xq;
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
  cudaError_t e = launch_split(p.x, p.T, p.H, j.n_blocks, nt, p.w13.group, p.xq, p.sorted_ids,
                               p.num_padded, j.P, p.k, st);
  if (e == cudaSuccess) e = launch_job(map13, p.w13.group, j, nt, num_sms, st);
  if (e == cudaSuccess)
    e = launch_split(p.h, 0, p.I, j.n_blocks, nt, p.w2.group, p.hq, p.sorted_ids, p.num_padded,
                     j.P, 1, st);
  if (e != cudaSuccess) return e;
  set_weight(j, p.w2);
  j.mode = kDown;
  j.K = p.I;
  j.n_rows = p.H;
  j.xq = p.hq;
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
