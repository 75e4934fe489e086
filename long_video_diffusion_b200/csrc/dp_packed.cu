// Attention over packed sequences of different lengths, grouped heads, causal or not: the host's
// plan for all types, and the fp32 kernel, on the CUDA cores (fp32 inputs ask for more than tf32's
// 10 bits of mantissa).
//
//   out_t,h = sum_j softmax_j(q_t,h . k_j,g * scale) v_j,g,  g = h / group,
//   j < k_len, causal j <= k_len - q_len + t;  lse_t,h = log sum_j exp(q_t,h . k_j,g * scale)
//
// One pass over the keys with a running maximum and sum; with few rows the keys are cut over the blocks
// of a cluster, which join their parts through distributed shared memory in a fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "dp_device.cuh"
#include "dp_packed.h"

namespace dp {

int64_t plan_packed(const PackedArgs& a, int64_t per_token, int rows, int32_t* n, int32_t* tile0, int32_t* first_q, int32_t* q_len,
                    int32_t* first_k, int32_t* k_len) {
  int32_t order[DP_MAX_SEQS];
  for (int i = 0; i < a.n_seqs; ++i) order[i] = i;
  std::sort(order, order + a.n_seqs, [&](int32_t x, int32_t y) {
    return a.k_len[x] != a.k_len[y] ? a.k_len[x] > a.k_len[y] : x < y;
  });
  int64_t tiles = 0;
  *n = a.n_seqs;
  for (int i = 0; i < a.n_seqs; ++i) {
    const int32_t o = order[i];
    tile0[i] = static_cast<int32_t>(tiles);
    first_q[i] = a.first_q[o];
    q_len[i] = a.q_len[o];
    first_k[i] = a.first_k[o];
    k_len[i] = a.k_len[o];
    if (a.q_len[o] * per_token > INT_MAX) return -1;
    tiles += (a.q_len[o] * per_token + rows - 1) / rows;
    if (tiles > INT_MAX) return -1;
  }
  tile0[a.n_seqs] = static_cast<int32_t>(tiles);
  return tiles;
}

bool encode_packed_kv(const PackedArgs& a, int box_rows, bool f16, CUtensorMap* tk, CUtensorMap* tv) {
  int64_t rows = 0;
  for (int i = 0; i < a.n_seqs; ++i) {
    const int64_t end = static_cast<int64_t>(a.first_k[i]) + a.k_len[i];
    if (a.k_len[i] > 0 && end > rows) rows = end;
  }
  const int cols = a.n_kv_heads * a.head_dim;
  // with no keys at all nothing is loaded: q's first row will do for the maps
  if (!rows) return encode_tmap_16_pitch(tk, a.q, 1, cols, a.ld_q, box_rows, f16) && encode_tmap_16_pitch(tv, a.q, 1, cols, a.ld_q, box_rows, f16);
  return encode_tmap_16_pitch(tk, a.k, rows, cols, a.ld_k, box_rows, f16) && encode_tmap_16_pitch(tv, a.v, rows, cols, a.ld_v, box_rows, f16);
}

cudaError_t device_and_sms(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= 64) return cudaErrorInvalidDevice;
  e = cudaSetDevice(*dev);
  if (e != cudaSuccess) return e;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
}

namespace {

constexpr int kKeys = 64;  // keys per tile: two per lane
// key tiles that a block's start and end cost, and those of a block that joins parts
constexpr int kF32Whole = 1, kF32Part = 2;

// RPW: query rows per warp.
template <int HD, int RPW>
struct F32Lay {
  static constexpr int kWarps = RPW == 8 ? 4 : 8;
  static constexpr int kRows = kWarps * RPW;  // per block
  static constexpr int KP = HD + 4;       // pitch of a key row: 16-byte reads of 32 rows without conflicts
  static constexpr int OFF_V = kKeys * KP;
  static constexpr int OFF_Q = OFF_V + kKeys * HD;
  static constexpr int OFF_P = OFF_Q + kRows * HD;
  static constexpr int FLOATS = OFF_P + kRows * kKeys;  // weights: [two rows][key][row]
};

struct Strides {
  int64_t q, k, v, out;
};

// Items, (row tile, k/v head), whose keys a cluster's blocks share: the first n_cut.
struct F32Items {
  FastDiv by_kv;
  int32_t n_kv, log_cluster, n_cut, n_items;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// 16 bytes of block `rank`'s shared memory.
__device__ __forceinline__ float4 ld_peer4(const float* at, int rank) {
  uint32_t a;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// A warp's RPW rows against a tile of 64 keys: a lane holds two keys' scores of each row, then, with
// the weights in shared memory, HD / 32 columns of each row's output.  Bound by the reads from shared
// memory: at eight rows a 16-byte read feeds 6 (scores) to 11 (outputs) multiply-adds per lane, which go
// in pairs (even and odd columns of a score, two rows of an output).  2048 causal tokens of 16 heads of
// 128: 475 us, 36 TFLOP/s (about half of what the multiply-adds alone allow).
template <int HD, int RPW, int N>
__global__ void __launch_bounds__(32 * F32Lay<HD, RPW>::kWarps) packed_f32_kernel(const float* q, const float* k,
                                                                 const float* v, float* out, float* lse, Strides ld,
                                                                 const __grid_constant__ PackedSeqs<N> seqs, int n_heads,
                                                                 int group, float scale, int causal, F32Items items) {
  using L = F32Lay<HD, RPW>;
  const ItemPart ip = item_part(items.log_cluster, items.n_cut);
  if (ip.item >= items.n_items) return;  // behind the last item: its cluster never joins
  const int parts = 1 << ip.log_parts;
  wait_for_earlier_kernels();
  constexpr int kRows = L::kRows, kWarps = L::kWarps;
  extern __shared__ __align__(16) float smem[];
  constexpr int C = HD / 32;  // output columns per lane
  float* sk = smem;           // [kKeys][KP]
  float* sv = smem + L::OFF_V;
  float* sq = smem + L::OFF_Q;  // [kRows][HD], scaled
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* sp = smem + L::OFF_P + warp * RPW * kKeys;
  const int tile = items.by_kv.div(ip.item), kv = ip.item - tile * items.n_kv;
  const int s = seq_of_tile(seqs, tile);
  const int q_len = seqs.q_len[s], k_len = seqs.k_len[s];
  const int rows = q_len * group;
  const int row0 = (seqs.tile0[s + 1] - 1 - tile) * kRows;
  const int n_rows = min(kRows, rows - row0);
  const int seen = min(k_len, keys_seen((row0 + n_rows - 1) / group, q_len, k_len, causal));  // by the tile's last row

  for (int i = threadIdx.x; i < kRows * (HD / 4); i += 32 * kWarps) {
    const int r = i / (HD / 4), c = (i % (HD / 4)) * 4;
    float4 x = make_float4(0, 0, 0, 0);
    if (r < n_rows) {
      const int tok = (row0 + r) / group, h = kv * group + (row0 + r) % group;
      x = *reinterpret_cast<const float4*>(q + (seqs.first_q[s] + static_cast<int64_t>(tok)) * ld.q + h * HD + c);
    }
    *reinterpret_cast<float4*>(sq + r * HD + c) = make_float4(x.x * scale, x.y * scale, x.z * scale, x.w * scale);
  }
  int lim[RPW];
  float m[RPW], l[RPW];      // l: this lane's keys
  uint64_t acc[RPW / 2][C];  // of two rows each
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    const int row = row0 + warp * RPW + r;
    lim[r] = row < rows ? min(k_len, keys_seen(row / group, q_len, k_len, causal)) : 0;
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[r / 2][c] = 0;
  }
  // 64 rows of k (or v) into shared memory; rows behind the sequence count as zeros, whatever they hold
  auto load = [&](const float* src, int64_t pitch, float* dst, int dst_pitch, int j0) {
    constexpr int kStep = 32 * kWarps / (HD / 4);
    const int c = (threadIdx.x % (HD / 4)) * 4;
    int j = threadIdx.x / (HD / 4);
    const float* p = src + (seqs.first_k[s] + static_cast<int64_t>(j0 + j)) * pitch + kv * HD + c;
#pragma unroll
    for (; j < kKeys; j += kStep, p += kStep * pitch) copy16(dst + j * dst_pitch + c, j0 + j < k_len ? p : src, j0 + j < k_len);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // V comes while the scores are taken, the next K while the products with V are
  const int per = ((seen + kKeys - 1) / kKeys + parts - 1) >> ip.log_parts;  // key tiles of a part
  const int begin = ip.rank * per * kKeys, end = min(seen, begin + per * kKeys);
  if (begin < end) load(k, ld.k, sk, L::KP, begin);
  for (int j0 = begin; j0 < end; j0 += kKeys) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    load(v, ld.v, sv, HD, j0);
    if (warp * RPW < n_rows) {
      uint64_t dot[RPW][2];  // sums over the even and over the odd columns
#pragma unroll
      for (int r = 0; r < RPW; ++r) dot[r][0] = dot[r][1] = 0;
      const float* k0 = sk + lane * L::KP;
      const float* qr = sq + warp * RPW * HD;
#pragma unroll 2
      for (int c = 0; c < HD; c += 4) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(k0 + c);
        const ulonglong2 z = *reinterpret_cast<const ulonglong2*>(k0 + 32 * L::KP + c);
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
          const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(qr + r * HD + c);
          dot[r][0] = ffma2(x.x, y.x, ffma2(x.y, y.y, dot[r][0]));
          dot[r][1] = ffma2(z.x, y.x, ffma2(z.y, y.y, dot[r][1]));
        }
      }
#pragma unroll
      for (int r = 0; r < RPW; r += 2) {
        float p0[2], p1[2], f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float d0, d1, d2, d3;
          f32x2_split(dot[r + h][0], d0, d1);
          f32x2_split(dot[r + h][1], d2, d3);
          const float x0 = j0 + lane < lim[r + h] ? d0 + d1 : -INFINITY;
          const float x1 = j0 + 32 + lane < lim[r + h] ? d2 + d3 : -INFINITY;
          float t = fmaxf(x0, x1);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
          const float mn = fmaxf(m[r + h], t);
          const float ref = mn == -INFINITY ? 0.0f : mn;  // a row that has seen no key: weights 0
          f[h] = expf(m[r + h] - ref);
          p0[h] = expf(x0 - ref);
          p1[h] = expf(x1 - ref);
          m[r + h] = mn;
          l[r + h] = l[r + h] * f[h] + (p0[h] + p1[h]);
        }
        const uint64_t f2 = f32x2(f[0], f[1]);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r / 2][c] = ffma2(acc[r / 2][c], f2, 0);
        *reinterpret_cast<float2*>(sp + (r * kKeys + 2 * lane)) = make_float2(p0[0], p0[1]);
        *reinterpret_cast<float2*>(sp + (r * kKeys + 2 * lane + 64)) = make_float2(p1[0], p1[1]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (j0 + kKeys < end) load(k, ld.k, sk, L::KP, j0 + kKeys);
    if (warp * RPW >= n_rows) continue;
    const int n_keys = min(kKeys, seen - j0);
#pragma unroll 1
    for (int j = 0; j < n_keys; j += 4) {  // (rows behind the sequence are zeros, weights behind `seen` too)
      uint64_t y[4][C];  // each value twice
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* at = sv + (j + e) * HD + lane * C;
        if constexpr (C == 4) {
          const float4 t = *reinterpret_cast<const float4*>(at);
          y[e][0] = f32x2(t.x, t.x);
          y[e][1] = f32x2(t.y, t.y);
          y[e][2] = f32x2(t.z, t.z);
          y[e][3] = f32x2(t.w, t.w);
        } else {
          const float2 t = *reinterpret_cast<const float2*>(at);
          y[e][0] = f32x2(t.x, t.x);
          y[e][1] = f32x2(t.y, t.y);
        }
      }
#pragma unroll
      for (int r = 0; r < RPW; r += 2) {
        const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(sp + r * kKeys + 2 * j);
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(sp + r * kKeys + 2 * j + 4);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r / 2][c] = ffma2(p.x, y[0][c], ffma2(p.y, y[1][c], ffma2(w.x, y[2][c], ffma2(w.y, y[3][c], acc[r / 2][c]))));
      }
    }
  }
  auto store = [&](int row, int c, float4 a, float top, float sum, bool sees) {
    const int64_t tok = seqs.first_q[s] + static_cast<int64_t>(row / group);
    const int h = kv * group + row % group;
    const float inv = 1.0f / sum;
    *reinterpret_cast<float4*>(out + tok * ld.out + h * HD + c) =
        sees ? make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv) : make_float4(0, 0, 0, 0);
    if (lse && c == 0) lse[tok * n_heads + h] = sees ? top + logf(sum) : -INFINITY;
  };
  // the rows' results through shared memory (over K: every warp has left the scores): [row][HD], then
  // (maximum, sum)
  float* sums = sk;
  float* sml = sk + kRows * HD;
  static_assert(kRows * (HD + 4) <= kKeys * L::KP, "the results fit over K");
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    float sum = l[r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int row = warp * RPW + r;
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      float x[2], z[2];
      f32x2_split(acc[r / 2][c], x[0], x[1]);
      f32x2_split(acc[r / 2][c + 1], z[0], z[1]);
      *reinterpret_cast<float2*>(sums + row * HD + lane * C + c) = make_float2(x[r & 1], z[r & 1]);
    }
    if (lane == 0) *reinterpret_cast<float4*>(sml + row * 4) = make_float4(m[r], sum, 0.0f, 0.0f);
  }
  __syncthreads();
  if (parts > 1) cluster_sync();
  // block `rank` joins the rows rank, rank + parts, ...
  for (int i = threadIdx.x; i < ((n_rows - ip.rank + parts - 1) >> ip.log_parts) * (HD / 4); i += 32 * kWarps) {
    const int row = ip.rank + (i / (HD / 4)) * parts, c = (i % (HD / 4)) * 4;
    const bool sees = min(k_len, keys_seen((row0 + row) / group, q_len, k_len, causal)) > 0;
    if (parts == 1) {
      store(row0 + row, c, *reinterpret_cast<const float4*>(sums + row * HD + c), sml[row * 4], sml[row * 4 + 1], sees);
    } else {
      float top = -INFINITY, sum = 0.0f;
      for (int t = 0; t < parts; ++t) top = fmaxf(top, ld_peer4(sml + row * 4, t).x);
      float4 a = make_float4(0, 0, 0, 0);
      for (int t = 0; t < parts; ++t) {
        const float4 ml = ld_peer4(sml + row * 4, t), x = ld_peer4(sums + row * HD + c, t);
        const float w = ml.x == -INFINITY ? 0.0f : expf(ml.x - top);
        sum = fmaf(w, ml.y, sum);
        a.x = fmaf(w, x.x, a.x);
        a.y = fmaf(w, x.y, a.y);
        a.z = fmaf(w, x.z, a.z);
        a.w = fmaf(w, x.w, a.w);
      }
      store(row0 + row, c, a, top, sum, sees);
    }
  }
  if (parts > 1) cluster_sync();  // no block leaves while another reads its shared memory
}

template <int HD, int RPW, int N>
cudaError_t launch_rows(const PackedArgs& a, int sms, cudaStream_t st) {
  PackedSeqs<N> s;
  const int64_t tiles = plan_packed(a, a.n_heads / a.n_kv_heads, F32Lay<HD, RPW>::kRows, s);
  if (tiles < 0 || tiles * a.n_kv_heads > INT_MAX) return cudaErrorInvalidValue;
  constexpr int bytes = F32Lay<HD, RPW>::FLOATS * 4;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> attr_set[64];
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(packed_f32_kernel<HD, RPW, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const int64_t n_items = tiles * a.n_kv_heads;
  const Cut cut = choose_cut(a.causal, s, a.n_kv_heads, kKeys, (HD == 64 ? 4 : 2) * sms, kF32Whole, kF32Part, kMaxCluster);
  const F32Items items = {fast_div(a.n_kv_heads), a.n_kv_heads, cut.log_cluster(), static_cast<int32_t>(cut.items), static_cast<int32_t>(n_items)};
  return launch_items(packed_f32_kernel<HD, RPW, N>, cut, n_items, 32 * F32Lay<HD, RPW>::kWarps, bytes, st, static_cast<const float*>(a.q),
                      static_cast<const float*>(a.k), static_cast<const float*>(a.v), static_cast<float*>(a.out), a.lse,
                      Strides{a.ld_q, a.ld_k, a.ld_v, a.ld_out}, s, static_cast<int>(a.n_heads),
                      static_cast<int>(a.n_heads / a.n_kv_heads), a.softmax_scale, static_cast<int>(a.causal), items);
}

// 32 rows per block: four warps of eight rows, the fewest reads from shared memory; while such blocks
// do not fill half the SMs (single tokens, short prompts) eight warps of two, whose blocks of 16 rows
// are twice as many and each warp's chain shorter.  Measured, us, two | eight rows: one head over 512
// tokens (16 blocks of 32 rows) 12.7 | 18.8, four single tokens over 100 to 4000 keys, 8 k/v heads
// (32) 31 | 46, 8 heads on 4 over 512 (128) 23.5 | 20.4, 40 heads on 8 over 540 (680) 80 | 64, 2048
// tokens x 16 heads (1024) 772 | 475.  Four rows in eight warps: 16.8, 39, 23.7, 69, 533.
template <int HD, int N>
cudaError_t launch_n(const PackedArgs& a, cudaStream_t st) {
  int dev = 0, sms = 148;
  const cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  int64_t blocks = 0;
  for (int i = 0; i < a.n_seqs; ++i)
    blocks += (static_cast<int64_t>(a.q_len[i]) * (a.n_heads / a.n_kv_heads) + 31) / 32 * a.n_kv_heads;
  return 2 * blocks >= sms ? launch_rows<HD, 8, N>(a, sms, st) : launch_rows<HD, 2, N>(a, sms, st);
}

cudaError_t launch_f32(const PackedArgs& a, cudaStream_t st) {
  if (a.n_seqs <= kFewSeqs) return a.head_dim == 64 ? launch_n<64, kFewSeqs>(a, st) : launch_n<128, kFewSeqs>(a, st);
  return a.head_dim == 64 ? launch_n<64, DP_MAX_SEQS>(a, st) : launch_n<128, DP_MAX_SEQS>(a, st);
}

}  // namespace

cudaError_t launch_packed(const PackedArgs& a, cudaStream_t s) {
  if (a.n_seqs < 1 || a.n_seqs > DP_MAX_SEQS || (a.head_dim != 64 && a.head_dim != 128)) return cudaErrorInvalidValue;
  if (a.dt == DP_F32) return launch_f32(a, s);
  // Sequences with few rows go to the kernel for few rows, which reads their keys at twice the rate
  // (eight tokens over 1 to 8191 keys: 27 us, 66 with the other).  Beside longer ones a launch of
  // their own has to pay: it does from about 40 tiles of 64 keys per SM on.  Measured, us, one launch
  // | two, 32 heads on 8 k/v heads of 128, a chunk of 512 tokens and single tokens: 8 over 4000 keys
  // (27 tiles per SM) 36.6 | 40.1; 64 over 1000 (55) 68 | 60; 31 over 4000 (105) 163 | 123; 200 over
  // 2000 (346) 325 | 274; 16 k/v heads of 64, 8 over 4000 (54) 44.7 | 35.3, 64 over 1000 (110) 115 | 57.
  const int group = a.n_heads / a.n_kv_heads;
  auto is_few = [&](int i) { return static_cast<int64_t>(a.q_len[i]) * group <= kFewRows; };
  int n_few = 0;
  int64_t tiles = 0;  // of the keys of the sequences with few rows
  for (int i = 0; i < a.n_seqs; ++i)
    if (is_few(i)) {
      ++n_few;
      tiles += (static_cast<int64_t>(a.k_len[i]) + 63) / 64;
    }
  if (n_few == a.n_seqs) return launch_packed_few(a, s);
  int dev = 0, sms = 148;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (tiles * a.n_kv_heads < 40 * static_cast<int64_t>(sms)) return launch_packed_tc(a, s);
  int32_t first_q[DP_MAX_SEQS], q_len[DP_MAX_SEQS], first_k[DP_MAX_SEQS], k_len[DP_MAX_SEQS];
  for (int few = 0; few < 2; ++few) {
    PackedArgs part = a;
    part.n_seqs = 0;
    for (int i = 0; i < a.n_seqs; ++i)
      if (is_few(i) == (few == 1)) {
        first_q[part.n_seqs] = a.first_q[i];
        q_len[part.n_seqs] = a.q_len[i];
        first_k[part.n_seqs] = a.first_k[i];
        k_len[part.n_seqs++] = a.k_len[i];
      }
    part.first_q = first_q;
    part.q_len = q_len;
    part.first_k = first_k;
    part.k_len = k_len;
    e = few ? launch_packed_few(part, s) : launch_packed_tc(part, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dp
