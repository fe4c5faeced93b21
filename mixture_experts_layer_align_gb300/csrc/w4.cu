// 4-bit weights with group scales: matrix-vector products and the expert
// products of the MoE layer for a few tokens.
//
// y[t][r] = sum over groups of scale[r][group] * sum_k x[t][k] (code[r][k] - zero[r][group]).
// What bounds it at a few tokens is reading the codes once.  They go from
// global memory to a per-warp ring in shared memory (cp.async), become bf16
// (code - zero is a small integer: exact) in registers and are the A operand
// (16 weight rows) of mma.m16n8k16 with 8 tokens in N, so that the products
// cost the same for one token as for eight; a group's sum is scaled in fp32.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;   // K blocks of a warp in its ring
constexpr int kBlockK = 128; // columns of one K block: 16 bytes of a row for each of 4 lanes

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8 x 16-byte matrices: lane (g, i) gets 4-byte word i of row g of each;
// lane 8 j + r gives the shared-memory address of row r of matrix j.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// D = A B + C, 16 x 8 x 16, bf16 in, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

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
__device__ __forceinline__ void w4_pairs(uint32_t w, uint32_t nz, uint32_t (&v)[4]) {
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

// The weight rows of a warp's MR m-tiles: where row 0 of each lies (a row of a
// tile is a 32-bit offset away) and how many rows from there exist.
template <int MR>
struct W4Rows {
  const uint8_t* codes[MR];
  const uint8_t* scales[MR];  // bf16 or fp32
  const uint8_t* zeros[MR];
  int last[MR];  // index of the last row that exists, >= 0
};

template <int MR>
__device__ __forceinline__ void w4_rows(W4Rows<MR>& t, int m, const W4View& w, int K, int groups,
                                        size_t row, int last) {
  t.codes[m] = w.codes + row * (K / 2);
  t.scales[m] = static_cast<const uint8_t*>(w.scales) + row * groups * (w.scale_bf16 ? 2 : 4);
  t.zeros[m] = w.zeros ? w.zeros + row * groups : nullptr;
  t.last[m] = last;
}

// One warp: acc[m][n] += rows x tokens over the K blocks wk, wk + WK, ...
//   xp[n]: this lane's token (8 n + g, or any other where there is none: its
//   column of the result is not used); ring: this warp's kStages * MR * 1024 bytes
// A K block of 16 rows is 64 16-byte pieces: piece c of row g (columns 32 c ..)
// sits at 16-byte slot 4 g + (c ^ (g >> 1 & 3)), so that both the copies and
// ldmatrix are free of bank conflicts.  ldmatrix gives lane (g, i) word i of
// piece c (columns 32 c + 8 i ..), so every mma sums columns of one piece, hence
// of one group.  Inside a word the columns come in the codes' order ((0,4),
// (1,5), ...), and x is permuted to match.
template <int PG, int MR, int NT>  // PG: pieces of a group, 1, 2 or 4
__device__ __forceinline__ void w4_warp_tile(const W4Rows<MR>& t, bool scale_bf16, int K,
                                             const __nv_bfloat16* const (&xp)[NT], int wk, int WK,
                                             uint32_t ring, float (&acc)[MR][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int groups = (K + 32 * PG - 1) / (32 * PG);
  const int nb = (K + kBlockK - 1) / kBlockK;
  const int n_iter = nb > wk ? (nb - wk + WK - 1) / WK : 0;
  const bool zeros = t.zeros[0] != nullptr;
  const uint32_t put = ring + (g * 4 + (tig ^ ((g >> 1) & 3))) * 16;
  // ldmatrix: lane 8 c + r addresses piece c of row r
  const uint32_t get = ring + (lane & 7) * 64 + ((lane >> 3) ^ ((lane >> 1) & 3)) * 16;

  uint32_t code_at[MR][2], group_at[MR][2];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t row = min(g + 8 * r, t.last[m]);
      code_at[m][r] = row * (K / 2) + wk * 64 + tig * 16;
      group_at[m][r] = row * groups + (wk * 4 + tig) / PG;
    }
  auto issue = [&](int i) {
    if (i < n_iter && (wk + i * WK) * kBlockK + tig * 32 < K) {
      const uint32_t dst = put + (i % kStages) * (MR * 1024);
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          cp_async16(dst + m * 1024 + r * 512, t.codes[m] + (code_at[m][r] + i * WK * 64));
    }
    cp_async_commit();
  };
  uint32_t s_nx[MR][2] = {}, z_nx[MR][2] = {};
  // lane tig holds the scale of piece tig's group (all four lanes when the block
  // is one group)
  auto fetch_scales = [&](int i) {
    if (i < n_iter && (PG == 4 || (wk + i * WK) * kBlockK + tig * 32 < K)) {
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t at = group_at[m][r] + i * WK * (4 / PG);
          s_nx[m][r] = scale_bf16
                           ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(t.scales[m]) + at)) << 16
                           : __ldg(reinterpret_cast<const uint32_t*>(t.scales[m]) + at);
          if (zeros) z_nx[m][r] = __ldg(t.zeros[m] + at);
        }
    }
  };
  uint4 x_nx[NT];
  auto fetch_x = [&](int col) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      x_nx[n] = __ldg(reinterpret_cast<const uint4*>(xp[n] + col + tig * 8));
  };

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  if (n_iter > 0) {
    fetch_scales(0);
    fetch_x(wk * kBlockK);
  }
  float part[MR][NT][4];
  const float none[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int i = 0; i < n_iter; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();  // every lane's copies of stage i have landed, and stage i - 1 is read
    issue(i + kStages - 1);
    const int col0 = (wk + i * WK) * kBlockK;
    const int pieces = min(4, (K - col0) / 32);
    uint32_t q[MR][2][4];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        ldmatrix4(q[m][r], get + (i % kStages) * (MR * 1024) + m * 1024 + r * 512);
    float s[MR][2];
    uint32_t z[MR][2];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        s[m][r] = __uint_as_float(s_nx[m][r]);
        z[m][r] = zeros ? w4_neg_zero(z_nx[m][r]) : kNegEight;
      }
    fetch_scales(i + 1);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c < pieces) {
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          b[n][0] = __byte_perm(x_nx[n].x, x_nx[n].z, 0x5410);
          b[n][1] = __byte_perm(x_nx[n].x, x_nx[n].z, 0x7632);
          b[n][2] = __byte_perm(x_nx[n].y, x_nx[n].w, 0x5410);
          b[n][3] = __byte_perm(x_nx[n].y, x_nx[n].w, 0x7632);
        }
        if (c + 1 < pieces) fetch_x(col0 + (c + 1) * 32);
        else if (i + 1 < n_iter) fetch_x(col0 + WK * kBlockK);
        const int from = (lane & ~3) | c;  // the lane that holds this piece's scale
#pragma unroll
        for (int m = 0; m < MR; ++m) {
          uint32_t z0 = z[m][0], z1 = z[m][1];
          if (PG < 4 && zeros) {
            z0 = __shfl_sync(0xffffffffu, z0, from);
            z1 = __shfl_sync(0xffffffffu, z1, from);
          }
          uint32_t v0[4], v1[4];
          w4_pairs(q[m][0][c], z0, v0);
          w4_pairs(q[m][1][c], z1, v1);
          const uint32_t a0[4] = {v0[0], v1[0], v0[1], v1[1]}, a1[4] = {v0[2], v1[2], v0[3], v1[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (c % PG == 0) mma_bf16(part[m][n], a0, b[n][0], b[n][1], none);
            else mma_bf16(part[m][n], a0, b[n][0], b[n][1], part[m][n]);
            mma_bf16(part[m][n], a1, b[n][2], b[n][3], part[m][n]);
          }
          if (c % PG == PG - 1 || c + 1 == pieces) {
            const float s0 = PG < 4 ? __shfl_sync(0xffffffffu, s[m][0], from) : s[m][0];
            const float s1 = PG < 4 ? __shfl_sync(0xffffffffu, s[m][1], from) : s[m][1];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[m][n][0] = fmaf(s0, part[m][n][0], acc[m][n][0]);
              acc[m][n][1] = fmaf(s0, part[m][n][1], acc[m][n][1]);
              acc[m][n][2] = fmaf(s1, part[m][n][2], acc[m][n][2]);
              acc[m][n][3] = fmaf(s1, part[m][n][3], acc[m][n][3]);
            }
          }
        }
      }
    }
  }
  cp_async_wait<0>();
}

// Sums the warps' accumulators over the WK warps that share rows, in shared
// memory: red[wk][(wr * MR + m) * 16 + row][8 NT] (the rings' space).
template <int MR, int NT>
__device__ __forceinline__ void w4_store_partials(float* red, int wk, int wr, int WR,
                                                  const float (&acc)[MR][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    float* p = red + (static_cast<size_t>(wk) * WR * MR + wr * MR + m) * 16 * 8 * NT;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      p[g * 8 * NT + n * 8 + tig * 2] = 64.f * acc[m][n][0];
      p[g * 8 * NT + n * 8 + tig * 2 + 1] = 64.f * acc[m][n][1];
      p[(g + 8) * 8 * NT + n * 8 + tig * 2] = 64.f * acc[m][n][2];
      p[(g + 8) * 8 * NT + n * 8 + tig * 2 + 1] = 64.f * acc[m][n][3];
    }
  }
}
template <int MR, int NT>
__device__ __forceinline__ float w4_sum_partials(const float* red, int WK, int WR, int row,
                                                 int tok) {
  float v = 0.f;
  for (int i = 0; i < WK; ++i)
    v += red[(static_cast<size_t>(i) * WR * MR * 16 + row) * 8 * NT + tok];
  return v;
}

template <int MR>
constexpr size_t w4_smem() {
  return static_cast<size_t>(kWarps) * kStages * MR * 1024;
}
static_assert(w4_smem<1>() >= size_t(kWarps) * 16 * 32 * 4, "partials fit the rings");

// ---------------------------------------------------------------- matvec
template <int PG, int MR, int NT>
__global__ void __launch_bounds__(kThreads)
    w4_matvec_kernel(const __nv_bfloat16* __restrict__ x, int T, int K, int N, W4View w,
                     void* __restrict__ out, int out_fp32, int WK) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int WR = kWarps / WK, wk = warp % WK, wr = warp / WK;
  pdl_wait();
  pdl_trigger();
  const int rows = WR * MR * 16;
  const long long r0 = static_cast<long long>(blockIdx.x) * rows;
  const int t0 = blockIdx.y * 8 * NT;
  const int groups = (K + 32 * PG - 1) / (32 * PG);
  W4Rows<MR> t;
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    const long long row = min(r0 + (wr * MR + m) * 16, static_cast<long long>(N) - 1);
    w4_rows(t, m, w, K, groups, row, static_cast<int>(min(N - 1 - row, 15ll)));
  }
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xp[n] = x + static_cast<size_t>(min(t0 + n * 8 + g, T - 1)) * K;
  float acc[MR][NT][4] = {};
  w4_warp_tile<PG, MR, NT>(t, w.scale_bf16, K, xp, wk, WK,
                           smem_addr(smem) + warp * (kStages * MR * 1024), acc);
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  w4_store_partials<MR, NT>(red, wk, wr, WR, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < rows * 8 * NT; i += kThreads) {
    const int tok = i / rows, r = i - tok * rows;
    if (t0 + tok < T && r0 + r < N) {
      const float v = w4_sum_partials<MR, NT>(red, WK, WR, r, tok);
      const size_t o = static_cast<size_t>(t0 + tok) * N + r0 + r;
      if (out_fp32) static_cast<float*>(out)[o] = v;
      else static_cast<__nv_bfloat16*>(out)[o] = __float2bfloat16_rn(v);
    }
  }
}

// ---------------------------------------------------------------- layer
// Gate/up products of one alignment block (up to 8 NT pairs of one expert) and
// 16 WR rows of I: h[p][i] = SiLU(gate) * up, bf16 (the down product's operand).
template <int PG, int NT>
__global__ void __launch_bounds__(kThreads) w4_gate_up_kernel(W4LayerParams p, int WK) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int WR = kWarps / WK, wk = warp % WK, wr = warp / WK;
  pdl_wait();
  pdl_trigger();
  const int block = blockIdx.x;
  if (block * 8 * NT >= __ldg(p.num_padded)) return;
  const int e = __ldg(p.block_expert + block);
  const int32_t* pairs = p.sorted_ids + static_cast<size_t>(block) * 8 * NT;
  const int P = p.T * p.k;
  const int i0 = blockIdx.y * WR * 16;
  const int groups = (p.H + 32 * PG - 1) / (32 * PG);
  W4Rows<2> t;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int i = min(i0 + wr * 16, p.I - 1);
    w4_rows(t, m, p.w13, p.H, groups,
            static_cast<size_t>(e) * 2 * p.I + static_cast<size_t>(m) * p.I + i,
            min(p.I - 1 - i, 15));
  }
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int pair = min(__ldg(pairs + n * 8 + g), P - 1);
    xp[n] = p.x + static_cast<size_t>(pair / p.k) * p.H;
  }
  float acc[2][NT][4] = {};
  w4_warp_tile<PG, 2, NT>(t, p.w13.scale_bf16, p.H, xp, wk, WK,
                          smem_addr(smem) + warp * (kStages * 2 * 1024), acc);
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  w4_store_partials<2, NT>(red, wk, wr, WR, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < WR * 16 * 8 * NT; i += kThreads) {
    const int tok = i / (WR * 16), r = i - tok * (WR * 16);
    const int pair = __ldg(pairs + tok);
    if (pair < P && i0 + r < p.I) {
      const int rr = (r / 16) * 32 + r % 16;  // the row's gate m-tile
      const float gate = w4_sum_partials<2, NT>(red, WK, WR, rr, tok);
      const float up = w4_sum_partials<2, NT>(red, WK, WR, rr + 16, tok);
      p.h[static_cast<size_t>(pair) * p.I + i0 + r] =
          __float2bfloat16_rn(gate / (1.f + expf(-gate)) * up);
    }
  }
}

// Down products: y[p][r] = weight of pair p * (w2[e] h[p])[r], fp32.
template <int PG, int MR, int NT>
__global__ void __launch_bounds__(kThreads) w4_down_kernel(W4LayerParams p, int WK) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int WR = kWarps / WK, wk = warp % WK, wr = warp / WK;
  pdl_wait();
  pdl_trigger();
  const int block = blockIdx.x;
  if (block * 8 * NT >= __ldg(p.num_padded)) return;
  const int e = __ldg(p.block_expert + block);
  const int32_t* pairs = p.sorted_ids + static_cast<size_t>(block) * 8 * NT;
  const int P = p.T * p.k;
  const int rows = WR * MR * 16, r0 = blockIdx.y * rows;
  const int groups = (p.I + 32 * PG - 1) / (32 * PG);
  W4Rows<MR> t;
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    const int r = min(r0 + (wr * MR + m) * 16, p.H - 1);
    w4_rows(t, m, p.w2, p.I, groups, static_cast<size_t>(e) * p.H + r, min(p.H - 1 - r, 15));
  }
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    xp[n] = p.h + static_cast<size_t>(min(__ldg(pairs + n * 8 + g), P - 1)) * p.I;
  float acc[MR][NT][4] = {};
  w4_warp_tile<PG, MR, NT>(t, p.w2.scale_bf16, p.I, xp, wk, WK,
                           smem_addr(smem) + warp * (kStages * MR * 1024), acc);
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  w4_store_partials<MR, NT>(red, wk, wr, WR, acc);
  __syncthreads();
  for (int i = threadIdx.x; i < rows * 8 * NT; i += kThreads) {
    const int tok = i / rows, r = i - tok * rows;
    const int pair = __ldg(pairs + tok);
    if (pair < P && r0 + r < p.H)
      p.y[static_cast<size_t>(pair) * p.H + r0 + r] =
          __ldg(p.wts + pair) * w4_sum_partials<MR, NT>(red, WK, WR, r, tok);
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

// Warps that share a row tile, splitting K: as many as leave each two K blocks.
int warps_on_k(int K) {
  const int nb = (K + kBlockK - 1) / kBlockK;
  int wk = 1;
  while (wk < kWarps && nb >= 2 * wk * 2) wk *= 2;
  return wk;
}

template <typename K>
cudaError_t smem_limit(K kernel, size_t bytes) {
  return checked(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(bytes)),
                 "smem attribute");
}

template <int PG, int MR, int NT>
cudaError_t matvec(const __nv_bfloat16* x, int T, int K, int N, const W4View& w, void* out,
                   bool out_fp32, cudaStream_t st) {
  const int WK = warps_on_k(K), rows = kWarps / WK * MR * 16;
  cudaError_t e = smem_limit(w4_matvec_kernel<PG, MR, NT>, w4_smem<MR>());
  if (e != cudaSuccess) return e;
  return launch_pdl(w4_matvec_kernel<PG, MR, NT>,
                    dim3((N + rows - 1) / rows, (T + 8 * NT - 1) / (8 * NT)), dim3(kThreads),
                    w4_smem<MR>(), st, x, T, K, N, w, out, out_fp32 ? 1 : 0, WK);
}

template <int PG>
cudaError_t matvec_any(const __nv_bfloat16* x, int T, int K, int N, const W4View& w, void* out,
                       bool out_fp32, cudaStream_t st) {
  if (T <= 8) return matvec<PG, 2, 1>(x, T, K, N, w, out, out_fp32, st);
  if (T <= 16) return matvec<PG, 2, 2>(x, T, K, N, w, out, out_fp32, st);
  return matvec<PG, 2, 4>(x, T, K, N, w, out, out_fp32, st);
}

template <int PG, int NT>
cudaError_t gate_up(const W4LayerParams& p, int blocks, cudaStream_t st) {
  const int WK = warps_on_k(p.H), rows = kWarps / WK * 16;
  cudaError_t e = smem_limit(w4_gate_up_kernel<PG, NT>, w4_smem<2>());
  if (e != cudaSuccess) return e;
  return launch_pdl(w4_gate_up_kernel<PG, NT>, dim3(blocks, (p.I + rows - 1) / rows),
                    dim3(kThreads), w4_smem<2>(), st, p, WK);
}

template <int PG, int NT>
cudaError_t down(const W4LayerParams& p, int blocks, cudaStream_t st) {
  const int WK = warps_on_k(p.I), rows = kWarps / WK * 2 * 16;
  cudaError_t e = smem_limit(w4_down_kernel<PG, 2, NT>, w4_smem<2>());
  if (e != cudaSuccess) return e;
  return launch_pdl(w4_down_kernel<PG, 2, NT>, dim3(blocks, (p.H + rows - 1) / rows),
                    dim3(kThreads), w4_smem<2>(), st, p, WK);
}

template <int NT>
cudaError_t layer(const W4LayerParams& p, cudaStream_t st) {
  const long long P = static_cast<long long>(p.T) * p.k;
  const int blocks = static_cast<int>(
      std::min(P, (P + std::min<long long>(p.E, P) * (8 * NT - 1)) / (8 * NT)));
  cudaError_t e = p.w13.group == 32   ? gate_up<1, NT>(p, blocks, st)
                  : p.w13.group == 64 ? gate_up<2, NT>(p, blocks, st)
                                      : gate_up<4, NT>(p, blocks, st);
  if (e != cudaSuccess) return e;
  e = p.w2.group == 32   ? down<1, NT>(p, blocks, st)
      : p.w2.group == 64 ? down<2, NT>(p, blocks, st)
                         : down<4, NT>(p, blocks, st);
  if (e != cudaSuccess) return e;
  const long long n = static_cast<long long>(p.T) * (p.H / 4);
  return launch_pdl(w4_combine_kernel,
                    dim3(static_cast<int>(std::min<long long>((n + 255) / 256, 2048))), dim3(256),
                    0, st, static_cast<const float*>(p.y), p.T, p.k, p.H, p.out);
}

}  // namespace

cudaError_t launch_w4_matvec(const __nv_bfloat16* x, int T, int K, int N, const W4View& w,
                             void* out, bool out_fp32, cudaStream_t st) {
  if (w.group == 32) return matvec_any<1>(x, T, K, N, w, out, out_fp32, st);
  if (w.group == 64) return matvec_any<2>(x, T, K, N, w, out, out_fp32, st);
  return matvec_any<4>(x, T, K, N, w, out, out_fp32, st);
}

int w4_block_rows(int T) { return T <= 8 ? 8 : T <= 16 ? 16 : 32; }

cudaError_t launch_w4_layer(const W4LayerParams& p, cudaStream_t st) {
  switch (w4_block_rows(p.T)) {
    case 8: return layer<1>(p, st);
    case 16: return layer<2>(p, st);
    default: return layer<4>(p, st);
  }
}

}  // namespace moe
