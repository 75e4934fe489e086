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

// The eight elements of a thread's row as fp32.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4* raw, float (&f)[8]) {
  const T* h = reinterpret_cast<const T*>(raw);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(h[e]);
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

// The eight elements of a code word as fp32.
__device__ __forceinline__ void unpack_e2m1x8(uint32_t c, float (&f)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
    f[2 * e] = t.x;
    f[2 * e + 1] = t.y;
  }
}

// Both kernels: 16 threads per unit of 128 columns by four rows 32 apart in a tile of 128 rows,
// eight elements of each row per thread (four threads per block of 32).  The four rows' scale
// words lie side by side in the tile: one 16-byte access; and a thread has four loads in flight.
// 49920 x 1536 bf16: 33 us quantising (5.8 TB/s, 0.89 of the measured HBM rate), 31 us back; with one
// row per thread 60 us.
// Tiles reach behind the last row and column; what is there is not read, its scales are written
// as zeros.
struct Unit {
  int64_t row0;  // of the four rows: row0 + 32 j
  int tile;      // of 128 columns
  int col;       // this thread's first
};

__device__ __forceinline__ Unit unit_of_thread(int tiles) {
  const uint32_t per_block = 2u * static_cast<uint32_t>(tiles);  // thread blocks per 128 rows
  const uint32_t rb = blockIdx.x / per_block;
  const uint32_t local = (blockIdx.x - rb * per_block) * (kThreads / 16) + (threadIdx.x >> 4);
  const uint32_t r = local / static_cast<uint32_t>(tiles);
  Unit u;
  u.tile = static_cast<int>(local - r * tiles);
  u.row0 = static_cast<int64_t>(rb) * 128 + r;
  u.col = u.tile * 128 + (threadIdx.x & 15) * 8;
  return u;
}

// The larger of two pairs of 16-bit magnitudes, given by their bits: those order like the values,
// infinities and NaN last.
__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const T* x, uint32_t* codes, uint32_t* scales,
                                                                int64_t n_rows, int k, int tiles) {
  constexpr bool kWide = sizeof(T) == 4;
  wait_for_earlier_kernels();
  let_next_kernel_start();
  const Unit u = unit_of_thread(tiles);
  const int sub = threadIdx.x & 15;
  // (bound by the issue slots as much as by the memory: one address, one row count, few selects)
  const int rows = u.col < k ? static_cast<int>(min(n_rows - u.row0, static_cast<int64_t>(128))) : 0;  // this thread's: j * 32 < rows
  const int64_t at = u.row0 * k + u.col;
  const int64_t step = 32ll * k;
  uint4 raw[4][kWide ? 2 : 1];
  const T* src = x + at;
#pragma unroll
  for (int j = 0; j < 4; ++j, src += step)
#pragma unroll
    for (int h = 0; h < (kWide ? 2 : 1); ++h)
      raw[j][h] = 32 * j < rows ? ld_once(reinterpret_cast<const uint4*>(src) + h) : make_uint4(0, 0, 0, 0);
  // each row's largest magnitude in its block of 32 (four threads), as fp32 bits
  uint32_t top[4];
  if constexpr (kWide) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m = max(m, max(raw[j][h].x & 0x7fffffffu, raw[j][h].y & 0x7fffffffu));
        m = max(m, max(raw[j][h].z & 0x7fffffffu, raw[j][h].w & 0x7fffffffu));
      }
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      top[j] = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    }
  } else {
    // two rows' 16-bit magnitudes in one word
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      uint32_t m[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 v = raw[j + r][0];
        m[r] = umax2(umax2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), umax2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
      }
      uint32_t both = umax2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
      both = umax2(both, __shfl_xor_sync(0xffffffffu, both, 1));
      both = umax2(both, __shfl_xor_sync(0xffffffffu, both, 2));
      if constexpr (std::is_same<T, __half>::value) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&both));
        top[j] = __float_as_uint(t.x);
        top[j + 1] = __float_as_uint(t.y);
      } else {
        top[j] = both << 16;
        top[j + 1] = both & 0xffff0000u;
      }
    }
  }
  uint32_t mine = 0;  // this block's four scale bytes, row j's at byte j
  uint32_t* dst = codes + (at >> 3);
#pragma unroll
  for (int j = 0; j < 4; ++j, dst += step >> 3) {
    const uint32_t ex = top[j] >> 23;  // no sign: at most 255
    const uint32_t least = max(ex, 2u);
    mine |= (ex == 255u ? 255u : least - 2u) << (8 * j);
    if (32 * j < rows) {
      const float inv = __uint_as_float((256u - least) << 23);  // 2^-e; with an infinity or NaN whatever
      float f[8];
      unpack8<T>(raw[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv;
      *dst = pack_e2m1x8(f);
    }
  }
  // 4 x 4 bytes turned between the four blocks' threads: block b's thread gets row b's word
  const int b = sub >> 2;
  uint32_t o = __shfl_xor_sync(0xffffffffu, mine, 4);
  mine = (b & 1) ? __byte_perm(mine, o, 0x3715) : __byte_perm(mine, o, 0x6240);
  o = __shfl_xor_sync(0xffffffffu, mine, 8);
  mine = (b & 2) ? __byte_perm(mine, o, 0x3276) : __byte_perm(mine, o, 0x5410);
  if ((sub & 3) == 0) scales[(mx4_scale_at(u.row0, u.tile * 4, tiles) >> 2) + b] = mine;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint32_t* codes, const uint32_t* scales, T* y,
                                                                  int64_t n_rows, int k, int tiles) {
  wait_for_earlier_kernels();
  let_next_kernel_start();
  const Unit u = unit_of_thread(tiles);
  if (u.row0 >= n_rows || u.col >= k) return;
  const int rows = static_cast<int>(min(n_rows - u.row0, static_cast<int64_t>(128)));
  const int64_t at = u.row0 * k + u.col;
  const int64_t step = 32ll * k;
  const uint4 s4 = *reinterpret_cast<const uint4*>(scales + (mx4_scale_at(u.row0, u.tile * 4, tiles) >> 2));
  const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w};
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = 32 * j < rows ? codes[(at >> 3) + j * (step >> 3)] : 0u;
  T* d = y + at;
#pragma unroll
  for (int j = 0; j < 4; ++j, d += step) {
    if (32 * j >= rows) break;
    const uint32_t s = (sw[j] >> (8 * ((threadIdx.x & 15) >> 2))) & 255u;
    const float scale = s == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(s ? s << 23 : 0x00400000u);
    float f[8];
    unpack_e2m1x8(c[j], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(d)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(d)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      constexpr bool f16 = std::is_same<T, __half>::value;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f16 ? pack_f16x2_sat(f[2 * e], f[2 * e + 1]) : pack_bf16x2(f[2 * e], f[2 * e + 1]);
      *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Thread blocks for `rows` x k: two per 128 x 128 tile.
int64_t mx4_grid(int64_t rows, int32_t k) { return (rows + 127) / 128 * 2 * ((static_cast<int64_t>(k) + 127) / 128); }

template <typename T>
cudaError_t quantize(const void* x, int64_t n_rows, int32_t k, void* codes, void* scales, cudaStream_t s) {
  const int64_t grid = mx4_grid(n_rows, k);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_early(mx4_quantize_kernel<T>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 1, s, static_cast<const T*>(x),
                      static_cast<uint32_t*>(codes), static_cast<uint32_t*>(scales), n_rows, static_cast<int>(k), (k + 127) / 128);
}

template <typename T>
cudaError_t dequantize(const void* codes, const void* scales, int64_t n_rows, int32_t k, void* y, cudaStream_t s) {
  const int64_t grid = mx4_grid(n_rows, k);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_early(mx4_dequantize_kernel<T>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 1, s,
                      static_cast<const uint32_t*>(codes), static_cast<const uint32_t*>(scales), static_cast<T*>(y), n_rows,
                      static_cast<int>(k), (k + 127) / 128);
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
