// Microscaled 4-bit floating point: quantisation and its inverse — HBM-bandwidth bound.
//
// For each block of 32 elements of a row (the OCP Microscaling Formats specification, FP4
// elements under a shared power of two), with m the block's largest magnitude:
//   e = max(floor(log2 m) - 2, -127),  code = e2m1(x * 2^-e),  scale byte = e + 127.
// floor(log2 m) is m's fp32 exponent field, 2^-e a normal number for every e, and the product
// exact, so the only rounding is the one to the code (nearest even, saturating at 6: m * 2^-e
// lies in [4, 8)).  A block with an infinity or NaN (exponent field 255) gets the scale byte
// 255, NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dp_device.cuh"
#include "dp_internal.h"

namespace dp {

namespace {

constexpr int kThreads = 256;

// Eight consecutive elements as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    const T* h = reinterpret_cast<const T*>(&x);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(h[e]);
  }
}

// Four e2m1 pairs, element 0 in the lowest bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// 16 threads per (row, 128 columns): 8 elements each, four threads per block.  The unit's four
// scale bytes are one aligned word of the scales' tile.  Units behind the last row or column
// exist as far as the tiles reach; they write zero scales.
template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const T* __restrict__ x, uint32_t* __restrict__ codes,
                                                                uint32_t* __restrict__ scales, int64_t n_rows, int k,
                                                                int tiles, int64_t n_units) {
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 4;
  if (unit >= n_units) return;  // whole groups of 16
  const int sub = threadIdx.x & 15;
  const uint32_t group = 0xffffu << (threadIdx.x & 16);
  const int64_t row = unit / tiles;
  const int tile = static_cast<int>(unit - row * tiles);
  const int col = tile * 128 + sub * 8;
  const bool in = row < n_rows && col < k;
  float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (in) load8(x + row * k + col, f);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(group, m, 1));
  m = max(m, __shfl_xor_sync(group, m, 2));
  const uint32_t ex = m >> 23;
  const uint32_t byte = ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
  const float inv = __uint_as_float((ex == 255u ? 127u : 254u - byte) << 23);
  if (in) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    codes[(row * k + col) >> 3] = pack_e2m1x8(f);
  }
  uint32_t word = byte << (8 * (sub >> 2));
  word |= __shfl_xor_sync(group, word, 4);
  word |= __shfl_xor_sync(group, word, 8);
  if (sub == 0) scales[mx4_scale_at(row, tile * 4, tiles) >> 2] = word;
}

// One thread per eight elements.
template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  T* __restrict__ y, int64_t n_vec, int k, int tiles) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n_vec) return;
  const int64_t row = i / (k >> 3);
  const int col = static_cast<int>(i - row * (k >> 3)) * 8;
  const uint32_t s = scales[mx4_scale_at(row, col >> 5, tiles)];
  const float scale = s == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(s ? s << 23 : 0x00400000u);
  const uint32_t c = codes[i];
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t v = c >> (4 * e);
    const uint32_t mag = v & 7u;
    // e2m1: 0, 0.5, then (1 + m / 2) 2^(e - 1)
    const float a = mag < 2u ? 0.5f * static_cast<float>(mag)
                             : __uint_as_float(((126u + (mag >> 1)) << 23) | ((mag & 1u) << 22));
    f[e] = ((v & 8u) ? -a : a) * scale;
  }
  if constexpr (sizeof(T) == 4) {
    float4* d = reinterpret_cast<float4*>(y + i * 8);
    d[0] = make_float4(f[0], f[1], f[2], f[3]);
    d[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    constexpr bool f16 = std::is_same<T, __half>::value;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = f16 ? pack_f16x2_sat(f[2 * e], f[2 * e + 1]) : pack_bf16x2(f[2 * e], f[2 * e + 1]);
    *reinterpret_cast<uint4*>(y + i * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename T>
cudaError_t quantize(const void* x, int64_t n_rows, int32_t k, void* codes, void* scales, cudaStream_t s) {
  const int tiles = (k + 127) / 128;
  const int64_t n_units = (n_rows + 127) / 128 * 128 * tiles;
  const int64_t grid = (n_units * 16 + kThreads - 1) / kThreads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  mx4_quantize_kernel<T><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(
      static_cast<const T*>(x), static_cast<uint32_t*>(codes), static_cast<uint32_t*>(scales), n_rows, k, tiles, n_units);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize(const void* codes, const void* scales, int64_t n_rows, int32_t k, void* y, cudaStream_t s) {
  const int64_t n_vec = n_rows * (k / 8);
  const int64_t grid = (n_vec + kThreads - 1) / kThreads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  mx4_dequantize_kernel<T><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(
      static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales), static_cast<T*>(y), n_vec, k,
      (k + 127) / 128);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, int64_t n_rows, int32_t k, dp_dtype x_dt, void* codes, void* scales,
                                cudaStream_t s) {
  if (n_rows <= 0 || k <= 0 || k % 32) return cudaErrorInvalidValue;
  if (x_dt == DP_BF16) return quantize<__nv_bfloat16>(x, n_rows, k, codes, scales, s);
  if (x_dt == DP_F16) return quantize<__half>(x, n_rows, k, codes, scales, s);
  return quantize<float>(x, n_rows, k, codes, scales, s);
}

cudaError_t launch_mx4_dequantize(const void* codes, const void* scales, int64_t n_rows, int32_t k, void* y,
                                  dp_dtype y_dt, cudaStream_t s) {
  if (n_rows <= 0 || k <= 0 || k % 32) return cudaErrorInvalidValue;
  if (y_dt == DP_BF16) return dequantize<__nv_bfloat16>(codes, scales, n_rows, k, y, s);
  if (y_dt == DP_F16) return dequantize<__half>(codes, scales, n_rows, k, y, s);
  return dequantize<float>(codes, scales, n_rows, k, y, s);
}

}  // namespace dp
