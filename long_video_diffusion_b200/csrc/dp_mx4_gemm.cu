// y = a W^T + bias with both operands in microscaled 4-bit floating point.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dp_device.cuh"
#include "dp_internal.h"

namespace dp {

namespace {

constexpr int kTile = 64;

__device__ __forceinline__ float mx4_value(const uint8_t* codes, const uint8_t* scales, int64_t row, int col, int k, int tiles) {
  const uint32_t v = codes[(row * k + col) >> 1] >> (4 * (col & 1));
  const uint32_t s = scales[mx4_scale_at(row, col >> 5, tiles)], mag = v & 7u;
  const float scale = s == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(s ? s << 23 : 0x00400000u);
  const float a = mag < 2u ? 0.5f * static_cast<float>(mag) : __uint_as_float(((126u + (mag >> 1)) << 23) | ((mag & 1u) << 22));
  return ((v & 8u) ? -a : a) * scale;
}

// 64 x 64 outputs per block, 32 of k at a time, 4 x 4 outputs per thread.
__global__ void __launch_bounds__(256) mx4_linear_kernel(Mx4Args g) {
  __shared__ float sa[32][kTile + 1], sw[32][kTile + 1];
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int n0 = blockIdx.x * kTile, tiles = (g.k + 127) / 128;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.k; k0 += 32) {
    for (int i = threadIdx.x; i < 32 * kTile; i += 256) {
      const int kk = i & 31, r = i >> 5;
      sa[kk][r] = m0 + r < g.m ? mx4_value((const uint8_t*)g.a, (const uint8_t*)g.a_scales, m0 + r, k0 + kk, g.k, tiles) : 0.0f;
      sw[kk][r] = n0 + r < g.n ? mx4_value((const uint8_t*)g.w, (const uint8_t*)g.w_scales, n0 + r, k0 + kk, g.k, tiles) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 32; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty + 16 * i], sw[kk][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = m0 + ty + 16 * i;
      const int c = n0 + tx + 16 * j;
      if (r >= g.m || c >= g.n) continue;
      const float v = acc[i][j] + (g.bias ? g.bias[c] : 0.0f);
      const int64_t at = r * g.n + c;
      if (g.y_dt == DP_F32) static_cast<float*>(g.y)[at] = v;
      else if (g.y_dt == DP_BF16) static_cast<uint16_t*>(g.y)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
      else static_cast<uint16_t*>(g.y)[at] = static_cast<uint16_t>(pack_f16x2_sat(v, 0.0f));
    }
}

}  // namespace

cudaError_t launch_mx4_linear(const Mx4Args& g, cudaStream_t s) {
  if (g.m <= 0 || g.n <= 0 || g.n % 8 || g.k <= 0 || g.k % 32) return cudaErrorInvalidValue;
  const int64_t gy = (g.m + kTile - 1) / kTile;
  if (gy > 65535) return cudaErrorInvalidValue;
  mx4_linear_kernel<<<dim3((g.n + kTile - 1) / kTile, static_cast<unsigned>(gy)), 256, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace dp
