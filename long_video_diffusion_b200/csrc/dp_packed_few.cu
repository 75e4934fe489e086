// Attention over packed sequences with few query rows (bf16 or f16): single tokens over a cache,
// short drafts, very short prompts.  Formulas in dp_packed.cu.
//
// All of a sequence's query rows under one k/v head, (token, head of the group) pairs, fit in 16;
// the work is reading K and V once, so the kernel is built around that: TMA brings tiles of 64
// keys into a ring of stages, two blocks per SM keep 2 x 96 KB (head_dim 128) in flight, and each
// of a block's four warps takes 16 keys of a tile by itself, with a running maximum and sum of its
// own, so that no warp waits for another before the end.  The products are warp-wide m16n8k16
// (mma.sync): a tcgen05 tile has 128 rows, of which these would fill an eighth or less, and its
// softmax one thread per row.  Eight tokens over 1 to 8191 keys, 32 heads on 8 k/v heads of 128:
// 27.3 us (0.78 of the measured HBM rate), 66 with the kernel for many rows; 32 tokens over 2000
// keys each: 6.4 TB/s.
// The keys of the long sequences are cut over the blocks of a cluster; each block sends its part
// of the columns to the block that joins them (distributed shared memory), in a fixed order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "dp_device.cuh"
#include "dp_packed.h"

namespace dp {

namespace {

// f16 weights are taken 2^15 times as large, so that those under 2^-14 of the largest keep their
// bits; sums and outputs carry the factor, which cancels.
template <bool F16>
constexpr float kWeightLog2 = F16 ? 15.0f : 0.0f;
constexpr int kRows = 16;
constexpr int kKeys = 64;     // per tile
constexpr int kWarps = 4;     // of 16 keys each; one more loads
constexpr int kThreads = 32 * (kWarps + 1);

template <int HD>
struct Few {
  static constexpr int CHUNKS = HD / 64;           // of 128 bytes of a row
  static constexpr int CHUNK = kKeys * 128;
  static constexpr int STAGE = 2 * CHUNKS * CHUNK;  // K, then V
  static constexpr int STAGES = HD == 128 ? 3 : 5;
  static constexpr int OFF_JOIN = STAGES * STAGE;   // what the cluster's blocks send: [part][row][HD / parts], then (m, l)
  static constexpr int OFF_ML = OFF_JOIN + kRows * HD * 4;
  static constexpr int OFF_WML = OFF_ML + kFewCluster * kRows * 8;  // the warps' (m, l)
  static constexpr int OFF_BAR = OFF_WML + kWarps * kRows * 8;
  static constexpr int OFF_MISC = OFF_BAR + 2 * STAGES * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert(kWarps * kRows * HD * 4 <= STAGES * STAGE, "the warps' sums fit over the stages");
  static_assert(2 * (ALLOC + 1024) <= 228 * 1024, "two blocks per SM");
};

struct FewParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t ld_q, ld_out;
  int32_t n_heads, n_kv, group;
  FastDiv by_kv, by_group;
  int32_t log_cluster, n_cut, n_items;
  int32_t causal;
  float scale_log2;
  uint32_t* status;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two softmax weights.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint32_t peer_smem(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

template <int HD, bool F16, int N>
__global__ void __launch_bounds__(kThreads, 2)
    packed_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const FewParams p,
                      const __grid_constant__ PackedSeqs<N> seqs) {
  using L = Few<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const ItemPart ip = item_part(p.log_cluster, p.n_cut);
  if (ip.item >= p.n_items) return;  // behind the last item: its cluster never joins
  const int parts = 1 << ip.log_parts;
  auto full = [&](int s) { return sb + L::OFF_BAR + 8u * s; };
  auto empty = [&](int s) { return sb + L::OFF_BAR + 8u * (L::STAGES + s); };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::OFF_MISC);
  if (warp == kWarps && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);
    }
    *abort = 0;
    fence_mbar_init();
  }
  // the cluster's blocks have started before one writes into another
  if (parts > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");

  const int seq = p.by_kv.div(ip.item);  // one tile of rows per sequence
  const int kv = ip.item - seq * p.n_kv;
  const int q_len = seqs.q_len[seq], k_len = seqs.k_len[seq];
  const int first_q = seqs.first_q[seq], first_k = seqs.first_k[seq];
  const int rows = q_len * p.group;
  const int seen = min(k_len, keys_seen(q_len - 1, q_len, k_len, p.causal));
  const int tiles = (seen + kKeys - 1) / kKeys;
  const int per = (tiles + parts - 1) >> ip.log_parts;
  const int t_begin = ip.rank * per;
  const int n_loc = max(0, min(tiles - t_begin, per));

  // Key tile t of the part into its stage.
  auto load_tile = [&](int t) {
    const int s = t % L::STAGES;
    mbar_arrive_expect_tx(full(s), L::STAGE);
    const int row = first_k + (t_begin + t) * kKeys;
#pragma unroll
    for (int c = 0; c < L::CHUNKS; ++c) {
      tma_load_2d(sb + s * L::STAGE + c * L::CHUNK, &tm_k, kv * HD + c * 64, row, full(s));
      tma_load_2d(sb + s * L::STAGE + (L::CHUNKS + c) * L::CHUNK, &tm_v, kv * HD + c * 64, row, full(s));
    }
  };
  wait_for_earlier_kernels();
  // the first stages' loads, before the others are up
  int issued = 0;
  if (warp == kWarps && lane == 0)
    for (; issued < min(n_loc, L::STAGES); ++issued) load_tile(issued);
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      for (; issued < n_loc; ++issued) {
        if (!mbar_wait(empty(issued % L::STAGES), (issued / L::STAGES - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_EMPTY)) break;
        load_tile(issued);
      }
      for (int t = max(0, issued - L::STAGES); t < issued; ++t) mbar_drain_wait(full(t % L::STAGES), (t / L::STAGES) & 1, p.status);
    }
  } else {
    // ------------------------------------------------------------ 16 keys of each tile
    // fragment rows of this lane: r0 = lane / 4 and r0 + 8
    const int pair = (lane & 3) * 2;
    int lim[2];
    uint32_t qf[HD / 16][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = lane / 4 + 8 * h;
      const int tok = p.by_group.div(row);
      lim[h] = row < rows ? min(k_len, keys_seen(tok, q_len, k_len, p.causal)) : 0;
      const uint16_t* src = p.q + (first_q + static_cast<int64_t>(tok)) * p.ld_q + (kv * p.group + row - tok * p.group) * HD + pair;
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        qf[c][h] = row < rows ? *reinterpret_cast<const uint32_t*>(src + c * 16) : 0u;
        qf[c][h + 2] = row < rows ? *reinterpret_cast<const uint32_t*>(src + c * 16 + 8) : 0u;
      }
    }
    float o[HD / 8][4];
#pragma unroll
    for (int c = 0; c < HD / 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    // ldmatrix rows of this lane: K pieces (keys 0-7 | 8-15) x (two neighbouring pieces), V the same, turned
    const int krow = warp * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, kpiece = (lane >> 3) & 1;
    const int vrow = warp * 16 + (lane & 15), vpiece = lane >> 4;
    bool ok = true;
    for (int t = 0; t < n_loc; ++t) {
      const int s = t % L::STAGES;
      ok = mbar_wait(full(s), (t / L::STAGES) & 1, abort, p.status, DEV_ERR_TIMEOUT_KV);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t ks = sb + s * L::STAGE, vs = ks + L::CHUNKS * L::CHUNK;
      float sc[2][4] = {};
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        uint32_t b[4];
        const int pc = 2 * c + kpiece;
        ldsm4(ks + (pc >> 3) * L::CHUNK + krow * 128 + (((pc & 7) ^ (krow & 7)) << 4), b);
        mma16816<F16>(sc[0], qf[c], b[0], b[1]);
        mma16816<F16>(sc[1], qf[c], b[2], b[3]);
      }
      const int key0 = (t_begin + t) * kKeys + warp * 16;
      float f[2];
      uint32_t pf[4];
      bool move = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + (e >> 1) * 8 + pair + (e & 1);
          x[e] = key < lim[h] ? sc[e >> 1][2 * h + (e & 1)] * p.scale_log2 : -INFINITY;
        }
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[h], top);
        const float ref = mn == -INFINITY ? 0.0f : mn;  // a row that has seen no key: weights 0
        f[h] = ex2_approx(m[h] - ref);
        move |= mn != m[h];
        m[h] = mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = ex2_approx(x[e] - (ref - kWeightLog2<F16>));
        l[h] = l[h] * f[h] + (x[0] + x[1]) + (x[2] + x[3]);
        pf[h] = pack2<F16>(x[0], x[1]);
        pf[h + 2] = pack2<F16>(x[2], x[3]);
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int c = 0; c < HD / 8; ++c) {
          o[c][0] *= f[0];
          o[c][1] *= f[0];
          o[c][2] *= f[1];
          o[c][3] *= f[1];
        }
      }
      // rows behind the sequence's end hold what they hold: as zeros they meet their zero weights
      const bool cut = key0 + 16 > k_len;
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
      if (cut) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = key0 + 8 * h + pair;
          keep[h] = key + 1 < k_len ? 0xffffffffu : key < k_len ? 0xffffu : 0u;
        }
      }
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        uint32_t b[4];
        const int pc = 2 * c + vpiece;
        ldsm4_t(vs + (pc >> 3) * L::CHUNK + vrow * 128 + (((pc & 7) ^ (vrow & 7)) << 4), b);
        mma16816<F16>(o[2 * c], pf, b[0] & keep[0], b[1] & keep[1]);
        mma16816<F16>(o[2 * c + 1], pf, b[2] & keep[0], b[3] & keep[1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    // the warps' results over the stages, once all have read them
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    float* sums = reinterpret_cast<float*>(smem) + warp * kRows * HD;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = lane / 4 + 8 * h;
      if (row < rows) {
#pragma unroll
        for (int c = 0; c < HD / 8; ++c)
          *reinterpret_cast<float2*>(sums + row * HD + c * 8 + pair) = make_float2(o[c][2 * h], o[c][2 * h + 1]);
        if ((lane & 3) == 0) reinterpret_cast<float2*>(smem + L::OFF_WML)[warp * kRows + row] = make_float2(m[h], l[h]);
      }
    }
  }
  __syncthreads();
  // ------------------------------------------------------------ the warps' results joined
  if (parts > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  const float2* wml = reinterpret_cast<const float2*>(smem + L::OFF_WML);
  const int width = HD >> ip.log_parts;  // columns that each of the cluster's blocks joins
  auto finish = [&](int row, int c, float4 a, float top, float l) {
    const int tok = p.by_group.div(row);
    const int head = kv * p.group + row - tok * p.group;
    const bool sees = min(k_len, keys_seen(tok, q_len, k_len, p.causal)) > 0;
    const float inv = 1.0f / l;
    const int64_t at = first_q + static_cast<int64_t>(tok);
    // a row that sees nothing: zeros, not 0 times what the weights of 0 made of hidden values
    *reinterpret_cast<uint2*>(p.out + at * p.ld_out + head * HD + c) =
        sees ? make_uint2(pack_out<F16>(a.x * inv, a.y * inv), pack_out<F16>(a.z * inv, a.w * inv)) : make_uint2(0, 0);
    if (p.lse && c == 0) p.lse[at * p.n_heads + head] = sees ? (top + (log2f(l) - kWeightLog2<F16>)) * 0.6931471805599453f : -INFINITY;
  };
  for (int i = threadIdx.x; i < rows * (HD / 4); i += kThreads) {
    const int row = i / (HD / 4), c = (i % (HD / 4)) * 4;
    float2 ml[kWarps];
    float top = -INFINITY, l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ml[w] = wml[w * kRows + row];
      top = fmaxf(top, ml[w].x);
    }
    float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float g = ml[w].x == -INFINITY ? 0.0f : ex2_approx(ml[w].x - top);
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + (w * kRows + row) * HD + c);
      l = fmaf(g, ml[w].y, l);
      a.x = fmaf(g, x.x, a.x);
      a.y = fmaf(g, x.y, a.y);
      a.z = fmaf(g, x.z, a.z);
      a.w = fmaf(g, x.w, a.w);
    }
    if (parts == 1) {
      finish(row, c, a, top, l);
    } else {
      const int to = c / width;
      const uint32_t dst = peer_smem(sb + L::OFF_JOIN + ((ip.rank * kRows + row) * width + c - to * width) * 4, to);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(a.x), "f"(a.y), "f"(a.z), "f"(a.w) : "memory");
      if (c % width == 0) {
        const uint32_t mdst = peer_smem(sb + L::OFF_ML + (ip.rank * kRows + row) * 8, to);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mdst), "f"(top), "f"(l) : "memory");
      }
    }
  }
  if (parts > 1) {
    // ---------------------------------------------------------- the parts joined, this block's columns
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    const float2* pml = reinterpret_cast<const float2*>(smem + L::OFF_ML);
    const float* join = reinterpret_cast<const float*>(smem + L::OFF_JOIN);
    for (int i = threadIdx.x; i < rows * (width / 4); i += kThreads) {
      const int row = i / (width / 4), c = (i % (width / 4)) * 4;
      float top = -INFINITY, l = 0.0f;
      for (int s = 0; s < parts; ++s) top = fmaxf(top, pml[s * kRows + row].x);
      float4 a = make_float4(0, 0, 0, 0);
      for (int s = 0; s < parts; ++s) {
        const float2 ml = pml[s * kRows + row];
        const float g = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - top);
        const float4 x = *reinterpret_cast<const float4*>(join + (s * kRows + row) * width + c);
        l = fmaf(g, ml.y, l);
        a.x = fmaf(g, x.x, a.x);
        a.y = fmaf(g, x.y, a.y);
        a.z = fmaf(g, x.z, a.z);
        a.w = fmaf(g, x.w, a.w);
      }
      finish(row, ip.rank * width + c, a, top, l);
    }
  }
}

template <int HD, bool F16, int N>
cudaError_t launch_n(const PackedArgs& a, cudaStream_t s) {
  using L = Few<HD>;
  PackedSeqs<N> seqs;
  const int64_t tiles = plan_packed(a, a.n_heads / a.n_kv_heads, kRows, seqs);
  if (tiles != a.n_seqs || tiles * a.n_kv_heads > INT_MAX) return cudaErrorInvalidValue;
  int dev = 0, sms = 148;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  CUtensorMap tk, tv;
  if (!encode_packed_kv(a, kKeys, F16, &tk, &tv)) return cudaErrorInvalidValue;
  auto kernel = packed_few_kernel<HD, F16, N>;
  static std::atomic<bool> attr_set[64];
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const int64_t items = tiles * a.n_kv_heads;
  const Cut cut = choose_cut(a.causal, seqs, a.n_kv_heads, kKeys, 2 * sms, kFewOverhead, kFewOverhead, kFewCluster);
  FewParams p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.ld_q = a.ld_q;
  p.ld_out = a.ld_out;
  p.n_heads = a.n_heads;
  p.n_kv = a.n_kv_heads;
  p.group = a.n_heads / a.n_kv_heads;
  p.by_kv = fast_div(p.n_kv);
  p.by_group = fast_div(p.group);
  p.log_cluster = cut.log_cluster();
  p.n_cut = static_cast<int32_t>(cut.items);
  p.n_items = static_cast<int32_t>(items);
  p.causal = a.causal;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.status = a.status;
  return launch_items(kernel, cut, items, kThreads, L::ALLOC, s, tk, tv, p, seqs);
}

template <int HD, bool F16>
cudaError_t launch_hd(const PackedArgs& a, cudaStream_t s) {
  return a.n_seqs <= kFewSeqs ? launch_n<HD, F16, kFewSeqs>(a, s) : launch_n<HD, F16, DP_MAX_SEQS>(a, s);
}

}  // namespace

cudaError_t launch_packed_few(const PackedArgs& a, cudaStream_t s) {
  if (a.head_dim == 64) return a.dt == DP_F16 ? launch_hd<64, true>(a, s) : launch_hd<64, false>(a, s);
  return a.dt == DP_F16 ? launch_hd<128, true>(a, s) : launch_hd<128, false>(a, s);
}

}  // namespace dp
