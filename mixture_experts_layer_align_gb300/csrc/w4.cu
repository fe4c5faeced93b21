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

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// D += A B, 16 x 8 x 16, bf16 in, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes i and i + 4 (i = shift / 4) of a word as bf16 128 + code, less the
// bf16 128 + zero in both halves: exactly code - zero.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int shift, uint32_t z) {
  uint32_t v = ((w >> shift) & 0x000f000fu) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(z));
  return r;
}

__device__ __forceinline__ float w4_scale(const W4View& w, size_t i) {
  if (w.scale_bf16)
    return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(w.scales) + i))
                           << 16);
  return __ldg(static_cast<const float*>(w.scales) + i);
}
__device__ __forceinline__ uint32_t w4_zero(const W4View& w, size_t i) {
  return w.zeros ? (static_cast<uint32_t>(__ldg(w.zeros + i)) * 0x00010001u) | 0x43004300u
                 : 0x43084308u;
}

// One warp: acc[m][n] += rows x tokens over the K blocks wk, wk + WK, ...
//   row[m][0/1]: this lane's weight rows (g and g + 8 of m-tile m, g = lane / 4)
//   xp[n]: this lane's token (8 n + g) at its column, or null (zeros)
//   ring: this warp's kStages * MR * 1024 bytes of shared memory
// A K block of 16 rows is 64 lanes' 16-byte pieces: piece c of row g (columns
// 32 c ..) sits at 16-byte slot 4 g + (c ^ (g >> 1 & 3)), so that both the
// copies and the 4-byte reads (lane (g, i) reads word i of piece c: columns
// 32 c + 8 i ..) are free of bank conflicts.  Every mma then sums columns of
// one 32-column piece, hence of one group.  The order of the columns inside a
// piece is the codes' ((0,4), (1,5), ...), and x is permuted to match.
template <int MR, int NT>
__device__ __forceinline__ void w4_warp_tile(const W4View& w, int K, const size_t (&row)[MR][2],
                                             const __nv_bfloat16* const (&xp)[NT], int wk, int WK,
                                             uint32_t ring, float (&acc)[MR][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int groups = (K + w.group - 1) / w.group;
  const int nb = (K + kBlockK - 1) / kBlockK;
  const int n_iter = nb > wk ? (nb - wk + WK - 1) / WK : 0;
  const uint32_t put = ring + (g * 4 + (tig ^ ((g >> 1) & 3))) * 16;
  const uint32_t get = ring + g * 64 + tig * 4;
  const uint32_t gx = ((g >> 1) & 3) * 16;
  const int per_group = w.group / 32;  // pieces of a group: 1, 2 or 4

  auto issue = [&](int i) {
    const int col = (wk + i * WK) * kBlockK + tig * 32;
    if (i < n_iter && col < K) {
      const uint32_t dst = put + (i % kStages) * (MR * 1024);
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        cp_async16(dst + m * 1024, w.codes + row[m][0] * (K / 2) + col / 2);
        cp_async16(dst + m * 1024 + 512, w.codes + row[m][1] * (K / 2) + col / 2);
      }
    }
    cp_async_commit();
  };
  float s_nx[MR][2];
  uint32_t z_nx[MR][2];
  auto fetch_scales = [&](int i) {
    const int col = (wk + i * WK) * kBlockK + tig * 32;
    if (i < n_iter && col < K) {
      const int gi = col / w.group;
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s_nx[m][r] = w4_scale(w, row[m][r] * groups + gi);
          z_nx[m][r] = w4_zero(w, row[m][r] * groups + gi);
        }
    }
  };
  uint4 x_nx[NT];
  auto fetch_x = [&](int i, int c) {
    const int col = (wk + i * WK) * kBlockK + c * 32 + tig * 8;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      x_nx[n] = (i < n_iter && col < K && xp[n] != nullptr)
                    ? __ldg(reinterpret_cast<const uint4*>(xp[n] + col))
                    : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      s_nx[m][r] = 0.f;
      z_nx[m][r] = 0x43084308u;
    }

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  fetch_scales(0);
  fetch_x(0, 0);
  float part[MR][NT][4];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[m][n][j] = 0.f;

  for (int i = 0; i < n_iter; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();  // every lane's copies of stage i have landed, and stage i - 1 is read
    issue(i + kStages - 1);
    const uint32_t src = get + (i % kStages) * (MR * 1024);
    const int pieces = min(4, (K - (wk + i * WK) * kBlockK) / 32);
    float s[MR][2];
    uint32_t z[MR][2];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        s[m][r] = s_nx[m][r];
        z[m][r] = z_nx[m][r];
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
        fetch_x(c + 1 < pieces ? i : i + 1, c + 1 < pieces ? c + 1 : 0);
        const bool last = ((c + 1) & (per_group - 1)) == 0 || c + 1 == pieces;
#pragma unroll
        for (int m = 0; m < MR; ++m) {
          const uint32_t w0 = lds32(src + m * 1024 + ((c * 16) ^ gx));
          const uint32_t w1 = lds32(src + m * 1024 + 512 + ((c * 16) ^ gx));
          uint32_t z0 = z[m][0], z1 = z[m][1];
          if (w.zeros) {
            z0 = __shfl_sync(0xffffffffu, z0, (lane & ~3) | c);
            z1 = __shfl_sync(0xffffffffu, z1, (lane & ~3) | c);
          }
          const uint32_t a0[4] = {w4_pair(w0, 0, z0), w4_pair(w1, 0, z1), w4_pair(w0, 4, z0),
                                  w4_pair(w1, 4, z1)};
          const uint32_t a1[4] = {w4_pair(w0, 8, z0), w4_pair(w1, 8, z1), w4_pair(w0, 12, z0),
                                  w4_pair(w1, 12, z1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_bf16(part[m][n], a0, b[n][0], b[n][1]);
            mma_bf16(part[m][n], a1, b[n][2], b[n][3]);
          }
          if (last) {
            const float s0 = __shfl_sync(0xffffffffu, s[m][0], (lane & ~3) | c);
            const float s1 = __shfl_sync(0xffffffffu, s[m][1], (lane & ~3) | c);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[m][n][0] = fmaf(s0, part[m][n][0], acc[m][n][0]);
              acc[m][n][1] = fmaf(s0, part[m][n][1], acc[m][n][1]);
              acc[m][n][2] = fmaf(s1, part[m][n][2], acc[m][n][2]);
              acc[m][n][3] = fmaf(s1, part[m][n][3], acc[m][n][3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) part[m][n][j] = 0.f;
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
      p[g * 8 * NT + n * 8 + tig * 2] = acc[m][n][0];
      p[g * 8 * NT + n * 8 + tig * 2 + 1] = acc[m][n][1];
      p[(g + 8) * 8 * NT + n * 8 + tig * 2] = acc[m][n][2];
      p[(g + 8) * 8 * NT + n * 8 + tig * 2 + 1] = acc[m][n][3];
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
template <int MR, int NT>
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
  size_t row[MR][2];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      row[m][r] = static_cast<size_t>(
          min(r0 + (wr * MR + m) * 16 + g + 8 * r, static_cast<long long>(N) - 1));
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = t0 + n * 8 + g;
    xp[n] = t < T ? x + static_cast<size_t>(t) * K : nullptr;
  }
  float acc[MR][NT][4] = {};
  w4_warp_tile<MR, NT>(w, K, row, xp, wk, WK,
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
template <int NT>
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
  size_t row[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      row[m][r] = static_cast<size_t>(e) * 2 * p.I + static_cast<size_t>(m) * p.I +
                  min(i0 + wr * 16 + g + 8 * r, p.I - 1);
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int pair = __ldg(pairs + n * 8 + g);
    xp[n] = pair < P ? p.x + static_cast<size_t>(pair / p.k) * p.H : nullptr;
  }
  float acc[2][NT][4] = {};
  w4_warp_tile<2, NT>(p.w13, p.H, row, xp, wk, WK, smem_addr(smem) + warp * (kStages * 2 * 1024),
                      acc);
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
template <int MR, int NT>
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
  size_t row[MR][2];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      row[m][r] = static_cast<size_t>(e) * p.H + min(r0 + (wr * MR + m) * 16 + g + 8 * r, p.H - 1);
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int pair = __ldg(pairs + n * 8 + g);
    xp[n] = pair < P ? p.h + static_cast<size_t>(pair) * p.I : nullptr;
  }
  float acc[MR][NT][4] = {};
  w4_warp_tile<MR, NT>(p.w2, p.I, row, xp, wk, WK, smem_addr(smem) + warp * (kStages * MR * 1024),
                       acc);
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

template <int MR, int NT>
cudaError_t matvec(const __nv_bfloat16* x, int T, int K, int N, const W4View& w, void* out,
                   bool out_fp32, cudaStream_t st) {
  const int WK = warps_on_k(K), rows = kWarps / WK * MR * 16;
  cudaError_t e = smem_limit(w4_matvec_kernel<MR, NT>, w4_smem<MR>());
  if (e != cudaSuccess) return e;
  return launch_pdl(w4_matvec_kernel<MR, NT>, dim3((N + rows - 1) / rows, (T + 8 * NT - 1) / (8 * NT)),
                    dim3(kThreads), w4_smem<MR>(), st, x, T, K, N, w, out, out_fp32 ? 1 : 0, WK);
}

template <int NT>
cudaError_t layer(const W4LayerParams& p, cudaStream_t st) {
  const int P = p.T * p.k;
  const int blocks = static_cast<int>(
      std::min<long long>(P, (P + static_cast<long long>(std::min(p.E, P)) * (8 * NT - 1)) / (8 * NT)));
  int WK = warps_on_k(p.H), rows = kWarps / WK * 16;
  cudaError_t e = smem_limit(w4_gate_up_kernel<NT>, w4_smem<2>());
  if (e == cudaSuccess)
    e = launch_pdl(w4_gate_up_kernel<NT>, dim3(blocks, (p.I + rows - 1) / rows), dim3(kThreads),
                   w4_smem<2>(), st, p, WK);
  if (e != cudaSuccess) return e;
  WK = warps_on_k(p.I), rows = kWarps / WK * 2 * 16;
  e = smem_limit(w4_down_kernel<2, NT>, w4_smem<2>());
  if (e == cudaSuccess)
    e = launch_pdl(w4_down_kernel<2, NT>, dim3(blocks, (p.H + rows - 1) / rows), dim3(kThreads),
                   w4_smem<2>(), st, p, WK);
  if (e != cudaSuccess) return e;
  const long long n = static_cast<long long>(p.T) * (p.H / 4);
  return launch_pdl(w4_combine_kernel, dim3(static_cast<int>(std::min<long long>((n + 255) / 256, 2048))),
                    dim3(256), 0, st, static_cast<const float*>(p.y), p.T, p.k, p.H, p.out);
}

}  // namespace

cudaError_t launch_w4_matvec(const __nv_bfloat16* x, int T, int K, int N, const W4View& w,
                             void* out, bool out_fp32, cudaStream_t st) {
  if (T <= 8) return matvec<2, 1>(x, T, K, N, w, out, out_fp32, st);
  if (T <= 16) return matvec<2, 2>(x, T, K, N, w, out, out_fp32, st);
  return matvec<2, 4>(x, T, K, N, w, out, out_fp32, st);
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
