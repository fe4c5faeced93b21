// 4-bit weights with group scales: matrix-vector products and the expert
// products of the MoE layer for a few tokens.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kW4Tokens = 8;  // tokens one warp carries through a weight row

__device__ __forceinline__ float w4_scale(const W4View& w, long long i) {
  return w.scale_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w.scales)[i])
                      : static_cast<const float*>(w.scales)[i];
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// acc[t] = sum_k x[t][k] * value[row][k] for nt <= N rows of x, one warp; every
// lane returns the sums.  A lane takes 32 codes (16 bytes, one group) at a time.
template <int N, typename TX>
__device__ __forceinline__ void w4_row_dot(const W4View& w, long long row, int K, const TX* x,
                                           int nt, int lane, float (&acc)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t) acc[t] = 0.f;
  const int groups = (K + w.group - 1) / w.group;
  for (int c = lane; c < K / 32; c += 32) {
    const uint4 q4 = *reinterpret_cast<const uint4*>(w.codes + row * (K / 2) + c * 16);
    const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
    const long long gi = row * groups + (c * 32) / w.group;
    const float s = w4_scale(w, gi);
    const float z = w.zeros ? static_cast<float>(w.zeros[gi]) : 8.f;
    float part[N] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = static_cast<float>((q[j] >> (4 * i)) & 15u) - z;
#pragma unroll
      for (int t = 0; t < N; ++t) {
        if (t < nt) {
          float xv[8];
          load8(x + static_cast<size_t>(t) * K + c * 32 + j * 8, xv);
#pragma unroll
          for (int i = 0; i < 8; ++i) part[t] = fmaf(xv[i], v[i], part[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < N; ++t) acc[t] = fmaf(s, part[t], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < N; ++t)
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
}

__global__ void __launch_bounds__(256)
    w4_matvec_kernel(const __nv_bfloat16* __restrict__ x, int T, int K, int N, W4View w, void* out,
                     int out_fp32) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long n = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (n >= N) return;
  for (int t0 = 0; t0 < T; t0 += kW4Tokens) {
    float acc[kW4Tokens];
    w4_row_dot(w, n, K, x + static_cast<size_t>(t0) * K, min(kW4Tokens, T - t0), lane, acc);
#pragma unroll
    for (int t = 0; t < kW4Tokens; ++t) {
      if (lane == t && t0 + t < T) {
        const size_t o = static_cast<size_t>(t0 + t) * N + n;
        if (out_fp32) static_cast<float*>(out)[o] = acc[t];
        else static_cast<__nv_bfloat16*>(out)[o] = __float2bfloat16_rn(acc[t]);
      }
    }
  }
}

// h[p][i] = SiLU(gate) * up of pair p = t * k + j, a warp per (pair, i).
__global__ void __launch_bounds__(256)
    w4_gate_up_kernel(const __nv_bfloat16* __restrict__ x, int k, int H, int I,
                      const int32_t* __restrict__ ids, W4View w, float* __restrict__ h) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (i >= I) return;
  const long long p = blockIdx.x;
  const long long row = static_cast<long long>(ids[p]) * 2 * I + i;
  const __nv_bfloat16* xr = x + (p / k) * H;
  float g[1], u[1];
  w4_row_dot(w, row, H, xr, 1, lane, g);
  w4_row_dot(w, row + I, H, xr, 1, lane, u);
  if (lane == 0) h[p * I + i] = g[0] / (1.f + expf(-g[0])) * u[0];
}

// out[t][r] = sum_j w[t][j] * (w2[e_j] h_j)[r], a warp per (token, r).
__global__ void __launch_bounds__(256)
    w4_down_kernel(const float* __restrict__ h, int k, int H, int I,
                   const int32_t* __restrict__ ids, const float* __restrict__ wts, W4View w,
                   __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (r >= H) return;
  const long long t = blockIdx.x;
  float sum = 0.f;
  for (int j = 0; j < k; ++j) {
    const long long p = t * k + j;
    float y[1];
    w4_row_dot(w, static_cast<long long>(ids[p]) * H + r, I, h + p * I, 1, lane, y);
    sum = fmaf(wts[p], y[0], sum);
  }
  if (lane == 0) out[t * H + r] = __float2bfloat16_rn(sum);
}

}  // namespace

cudaError_t launch_w4_matvec(const __nv_bfloat16* x, int T, int K, int N, const W4View& w,
                             void* out, bool out_fp32, cudaStream_t st) {
  return launch_pdl(w4_matvec_kernel, dim3((N + 7) / 8), dim3(256), 0, st, x, T, K, N, w, out,
                    out_fp32 ? 1 : 0);
}

cudaError_t launch_w4_gate_up(const W4LayerParams& p, cudaStream_t st) {
  return launch_pdl(w4_gate_up_kernel, dim3(p.T * p.k, (p.I + 7) / 8), dim3(256), 0, st, p.x, p.k,
                    p.H, p.I, static_cast<const int32_t*>(p.ids), p.w13, p.h);
}

cudaError_t launch_w4_down(const W4LayerParams& p, cudaStream_t st) {
  return launch_pdl(w4_down_kernel, dim3(p.T, (p.H + 7) / 8), dim3(256), 0, st,
                    static_cast<const float*>(p.h), p.k, p.H, p.I,
                    static_cast<const int32_t*>(p.ids), static_cast<const float*>(p.wts), p.w2,
                    p.out);
}

}  // namespace moe
