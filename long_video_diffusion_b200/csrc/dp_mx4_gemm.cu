// y = a W^T + bias with both operands in microscaled 4-bit floating point, on the sm_100a tensor
// cores: tcgen05.mma kind::mxf4 takes the e2m1 codes from shared memory (packed, two to a byte,
// 256 of a row in one 128-byte swizzle row) and one power-of-two scale per 32 of them from
// tensor memory, and sums exact products in fp32.
//
// A step is 256 of k: TMA brings the codes' tiles and the scales' (whose layout in memory, tiles
// of 128 rows by 128 columns in 512 bytes, is the one tcgen05.cp spreads over tensor memory);
// what lies behind k or behind the last row arrives as zeros.  Scales go round several column
// ranges of tensor memory, so that a step's copy never meets an earlier step's products.
//
// Few rows of a (mx4_narrow_kernel): bound by reading W once.  W's rows are the tile's M (128
// features per block), the tokens its N, and k is cut into as many parts as a cluster has blocks,
// so that all SMs read W at once; the parts are summed through distributed shared memory in a
// fixed order.  One row by W of 4096 x 4096 (8.9 MB): 4.9 us, where reading W alone takes 1.4 us: the
// launch, the first bytes' way from memory and the join are the rest.
//
// Many rows (mx4_wide_kernel).  A persistent kernel of block pairs,
// each pair one output tile of 256 x 256 (tcgen05 cta_group::2: a block holds 128 rows of a and
// 128 of W, and its half of the sums): at 4 bits a product of 64 of k takes 128 clocks and 8 KB
// of a block's shared memory, half of what it can read and be filled with in that time, where a
// block by itself would need 12 KB.  The tensor pipe is busy 62 % of the time; whether the fill from L2
// (35840 bytes per 512 clocks and block) or the six scale copies ahead of a step's products hold the rest
// is not told apart.  8192 x 8192 x 8192: 202 us, 5.4 PFLOP/s (3.3 times the measured bf16 rate), and 231
// in a loop, where the power limit lowers the clock to 1440 of 1965 MHz.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>

#include "dp_device.cuh"
#include "dp_internal.h"

namespace dp {

namespace {

constexpr int kStepK = 256;        // of k per step: 128 bytes of codes
constexpr int kScaleTile = 512;    // bytes: 128 rows x 128 of k
constexpr int kMaxSplits = 8;      // portable cluster size

// Instruction descriptor of kind::mxf4: e2m1 operands (bits 7, 10), e8m0 scales (bit 23), N / 8
// at 17, M / 128 at 27; which two bytes of a scale word hold this product's scales: a at 29, b
// at 4.
__host__ __device__ constexpr uint32_t idesc_mx4(int M, int N, uint32_t sf_id) {
  return (1u << 7) | (1u << 10) | (1u << 23) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 7) << 27) | (sf_id << 29) | (sf_id << 4);
}

// Descriptor of a scale tile for tcgen05.cp: 32 rows of 16 bytes, no swizzle, 128 bytes from one
// eight rows to the next.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float4 ld_peer4(uint32_t a, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 p;\n\t"
      "mapa.shared::cluster.u32 p, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(a), "r"(rank)
      : "memory");
  return v;
}

struct Mx4Params {
  const float* bias;
  void* y;
  int64_t m;
  int32_t n, k;
  int32_t log_splits;  // log2 of the blocks per cluster: parts of k
  int32_t y_dt;
  uint32_t* status;
};

// Four consecutive outputs of a row.
__device__ __forceinline__ void store4(const Mx4Params& p, int64_t at, float4 v) {
  if (p.y_dt == DP_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
        p.y_dt == DP_BF16 ? make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w))
                          : make_uint2(pack_f16x2_sat(v.x, v.y), pack_f16x2_sat(v.z, v.w));
}

// ------------------------------------------------------------------ few rows of a

template <int NT>  // tokens per tile
struct Narrow {
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int A_BYTES = NT * 128;
  static constexpr int OFF_A = W_BYTES;
  static constexpr int OFF_SW = OFF_A + A_BYTES;
  static constexpr int OFF_SA = OFF_SW + 2 * kScaleTile;
  static constexpr int STAGE = OFF_SA + 2 * kScaleTile;
  static constexpr int STAGES = 4;
  static constexpr int PITCH = 128 + 4;  // floats between two tokens of the sums in shared memory
  static constexpr int SUMS = NT * PITCH * 4;
  static constexpr int OFF_BAR = STAGES * STAGE > SUMS ? STAGES * STAGE : (SUMS + 15) / 16 * 16;
  static constexpr int N_BAR = 2 * STAGES + 1;
  static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static constexpr int SF_COLS = 16;  // columns of a step's scales: W's, then the tokens'
  static constexpr int COL_SF = NT < 32 ? 32 : NT;
  static constexpr int COLS = COL_SF + STAGES * SF_COLS;  // a range of scales per stage
  static constexpr int TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int kThreads = 192;
  static_assert(ALLOC <= 227 * 1024, "shared memory budget");
};

template <int NT>
__global__ void __launch_bounds__(Narrow<NT>::kThreads)
    mx4_narrow_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                      const __grid_constant__ CUtensorMap tm_sw, const __grid_constant__ CUtensorMap tm_sa, const Mx4Params p) {
  using L = Narrow<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = 1 << p.log_splits;  // blocks of the cluster
  const int rank = blockIdx.x & (splits - 1);
  const int n_tile = blockIdx.x >> p.log_splits, m_tile = blockIdx.y;
  const int steps = (p.k + kStepK - 1) / kStepK;
  const int per = (steps + splits - 1) >> p.log_splits;
  const int first = rank * per;
  const int n_loc = max(0, min(per, steps - first));

  const uint32_t bar0 = sb + L::OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (L::STAGES + s); };
  const uint32_t acc_full = bar0 + 8u * (2 * L::STAGES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  auto load_step = [&](int i) {
    const int s = i % L::STAGES;
    const uint32_t st = sb + s * L::STAGE;
    const int kb = first + i;
    mbar_arrive_expect_tx(full(s), L::STAGE);
    tma_load_2d(st, &tm_w, kb * 128, n_tile * 128, full(s));
    tma_load_3d(st + L::OFF_SW, &tm_sw, 0, kb * 2, n_tile, full(s));
    tma_load_2d(st + L::OFF_A, &tm_a, kb * 128, m_tile * NT, full(s));
    tma_load_3d(st + L::OFF_SA, &tm_sa, 0, kb * 2, m_tile * NT / 128, full(s));
  };
  int issued = 0;
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    *abort = 0;
    fence_mbar_init();
    // the first stages' loads, before the other warps are up
    wait_for_earlier_kernels();
    for (; issued < min(n_loc, L::STAGES); ++issued) load_step(issued);
  }
  if (warp == 1) {
    wait_for_earlier_kernels();
    tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      for (; issued < n_loc; ++issued) {
        if (!mbar_wait(empty(issued % L::STAGES), (issued / L::STAGES - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_EMPTY)) break;
        load_step(issued);
      }
      const int from = issued > L::STAGES ? issued - L::STAGES : 0;
      for (int i = from; i < issued; ++i) mbar_drain_wait(full(i % L::STAGES), (i / L::STAGES) & 1, p.status);
    }
  } else if (warp == 1) {
    // the whole warp, one lane elected for the tensor-core instructions (see mx4_wide_kernel)
    const uint64_t dw = sdesc_sw128(sb, 16, 1024);
    const uint64_t da = sdesc_sw128(sb + L::OFF_A, 16, 1024);
    const uint64_t dsw = sdesc_scales(sb + L::OFF_SW);
    const uint64_t dsa = sdesc_scales(sb + L::OFF_SA);
    for (int i = 0; i < n_loc; ++i) {
      const int s = i % L::STAGES;
      const bool ok = mbar_wait(full(s), (i / L::STAGES) & 1, abort, p.status, DEV_ERR_TIMEOUT_KV);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t sw = tmem + L::COL_SF + s * L::SF_COLS;
      // a scale tile is of 128 rows, 32 to a column: the second 64 tokens' start two columns on
      const uint32_t sa = sw + 8;
      const uint32_t sa_mine = sa + (NT == 64 ? (m_tile & 1) * 2 : 0);
      const uint32_t so = (s * L::STAGE) >> 4;
      const int chunks = min(4, (p.k - (first + i) * kStepK + 63) / 64);  // of 64: those behind k are zeros
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          cp_scales(sw + c * 4, sdesc_add(dsw, so + c * (kScaleTile >> 4)));
          cp_scales(sa + c * 4, sdesc_add(dsa, so + c * (kScaleTile >> 4)));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks)
            mma_mx4(tmem, sdesc_add(dw, so + c * 2), sdesc_add(da, so + c * 2), idesc_mx4(128, NT, (c & 1) * 2), sw + (c >> 1) * 4,
                    sa_mine + (c >> 1) * 4, (i > 0 || c > 0) ? 1u : 0u);
        mma_commit(empty(s));
      }
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(acc_full);
      mbar_drain_wait(acc_full, 0, p.status);
    }
    __syncwarp();
  } else {
    // one thread per feature: its sums, over the stages, as [token][feature]
    const int quarter = warp & 3;
    bool ok = mbar_wait(acc_full, 0, abort, p.status, DEV_ERR_TIMEOUT_O);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      float* dst = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
      const uint32_t src = tmem + ((static_cast<uint32_t>(quarter) * 32u) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < NT; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(src + c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c0 + c < NT) dst[(c0 + c) * L::PITCH] = n_loc > 0 ? __uint_as_float(r[c]) : 0.0f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
  if (splits > 1) cluster_sync();
  wait_for_earlier_kernels();
  // this block's share of the tile's tokens x 32 groups of four features
  const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), p.m - static_cast<int64_t>(m_tile) * NT));
  const int share = (tokens * 32 + splits - 1) >> p.log_splits;
  const int end = min(tokens * 32, (rank + 1) * share);
  for (int i = rank * share + threadIdx.x; i < end; i += L::kThreads) {
    const int f = (i & 31) * 4, col = n_tile * 128 + f, t = i >> 5;
    if (col >= p.n) continue;
    float4 v = p.bias ? *reinterpret_cast<const float4*>(p.bias + col) : make_float4(0, 0, 0, 0);
    const uint32_t at = (t * L::PITCH + f) * 4;
    if (splits == 1) {
      const float4 x = *reinterpret_cast<const float4*>(smem + at);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    } else {
      float4 x[kMaxSplits];
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s)
        if (s < splits) x[s] = ld_peer4(sb + at, s);
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s)
        if (s < splits) v.x += x[s].x, v.y += x[s].y, v.z += x[s].z, v.w += x[s].w;
    }
    store4(p, (static_cast<int64_t>(m_tile) * NT + t) * p.n + col, v);
  }
  if (splits > 1) cluster_sync();  // no block leaves while another reads its shared memory
}

// ------------------------------------------------------------------ many rows of a

// The forms of the instructions above for a pair of blocks, issued by its first.
__device__ __forceinline__ void mma_mx4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Arrives on `bar` in both blocks once all that this thread issued has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"(static_cast<uint16_t>(3))
               : "memory");
}

// Loads into this block's shared memory that signal a barrier of either block of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Shared address `a` of this block in the pair's first block.
__device__ __forceinline__ uint32_t in_first(uint32_t a) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0));
  return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tensor memory: two accumulators of 256 columns do not fit beside the scales, so they overlap
// by half (0-255 and 128-383).  A tile's epilogue reads the shared columns first, which is all
// that the next tile's products wait for.  Every stage has a range of columns for its scales.
struct Wide {
  static constexpr int BN = 256;
  static constexpr int CODES = 128 * 128;  // bytes of a block's rows of a, or of W, per step
  static constexpr int OFF_B = CODES;
  static constexpr int OFF_SA = 2 * CODES;
  static constexpr int OFF_SB = OFF_SA + 2 * kScaleTile;
  static constexpr int STAGE = OFF_SB + 4 * kScaleTile;
  static constexpr int STAGES = 5;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 32 * (2 + kEpiWarps);
  static constexpr int OUT_BYTES = 32 * 128;  // an epilogue warp's 32 rows of 128 bytes of output
  static constexpr int OFF_OUT = STAGES * STAGE;
  static constexpr int OFF_BAR = OFF_OUT + kEpiWarps * OUT_BYTES;
  static constexpr int N_BAR = 2 * STAGES + 5;
  static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static constexpr int COL_ACC1 = 128;
  static constexpr int COL_SF = 384;
  static constexpr int SF_COLS = 24;  // a's 8, then W's 16
  static_assert(COL_ACC1 + BN <= COL_SF && COL_SF + STAGES * SF_COLS <= 512, "tensor memory budget");
  static_assert(COL_ACC1 >= 128, "the shared columns lie in the two groups of 64 read first");
  static_assert(ALLOC <= 227 * 1024, "shared memory budget");
};

struct WideParams {
  Mx4Params p;
  int32_t m_tiles, n_tiles, tiles;
  int32_t group_m;
};

// Tile t -> (m tile, n tile): groups of group_m m tiles, m fastest inside a group.
__device__ __forceinline__ void wide_coords(const WideParams& w, int t, int& m_tile, int& n_tile) {
  const int per_group = w.group_m * w.n_tiles;
  const int group = t / per_group;
  const int first_m = group * w.group_m;
  const int gm = min(w.group_m, w.m_tiles - first_m);
  const int within = t - group * per_group;
  m_tile = first_m + within % gm;
  n_tile = within / gm;
}

__global__ void __launch_bounds__(Wide::kThreads, 1)
    mx4_wide_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sw,
                    const __grid_constant__ CUtensorMap tm_y, const WideParams w) {
  using L = Wide;
  const Mx4Params& p = w.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;  // in the pair
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int steps = (p.k + kStepK - 1) / kStepK;
  const int n_mine = w.tiles > pair ? (w.tiles - pair + pairs - 1) / pairs : 0;

  const uint32_t bar0 = sb + L::OFF_BAR;
  auto full = [&](int s) { return bar0 + 8u * s; };  // used in the first block only
  auto empty = [&](int s) { return bar0 + 8u * (L::STAGES + s); };
  auto acc_full = [&](int b) { return bar0 + 8u * (2 * L::STAGES + b); };
  auto shared_read = [&](int b) { return bar0 + 8u * (2 * L::STAGES + 2 + b); };  // in the first block only
  const uint32_t fin = bar0 + 8u * (2 * L::STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(shared_read(b), 2 * L::kEpiWarps);
    }
    mbar_init(fin, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    wait_for_earlier_kernels();
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_sa);
    tma_prefetch_desc(&tm_sw);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are there
  wait_for_earlier_kernels();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int g = 0;
      bool ok = true;
      for (int i = 0; ok && i < n_mine; ++i) {
        int m_tile, n_tile;
        wide_coords(w, pair + i * pairs, m_tile, n_tile);
        for (int kt = 0; kt < steps; ++kt, ++g) {
          const int s = g % L::STAGES;
          if (g >= L::STAGES && !mbar_wait(empty(s), ((g / L::STAGES) - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t st = sb + s * L::STAGE;
          const uint32_t bar = in_first(full(s));
          if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * L::STAGE);
          tma_load_2d_pair(st, &tm_a, kt * 128, m_tile * 256 + rank * 128, bar);
          tma_load_2d_pair(st + L::OFF_B, &tm_w, kt * 128, n_tile * 256 + rank * 128, bar);
          tma_load_3d_pair(st + L::OFF_SA, &tm_sa, 0, kt * 2, m_tile * 2 + rank, bar);
          tma_load_3d_pair(st + L::OFF_SB, &tm_sw, 0, kt * 2, n_tile * 2, bar);
        }
      }
      // both blocks' copies land before either's shared memory is released (the second waits for
      // the first at the end)
      if (rank == 0)
        for (int i = max(0, g - L::STAGES); i < g; ++i) mbar_drain_wait(full(i % L::STAGES), (i / L::STAGES) & 1, p.status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer of the pair
    // The warp's own instructions have to stay ahead of the tensor cores' 512 clocks per step: it
    // runs the loop as a whole (uniform control flow and operands) and elects one lane for the
    // tensor-core instructions; the ring is unrolled, so that addresses are constants off a base.
    if (rank == 0 && n_mine > 0) {
      const uint64_t da = sdesc_sw128(sb, 16, 1024);
      const uint64_t db = sdesc_sw128(sb + L::OFF_B, 16, 1024);
      const uint64_t dsa = sdesc_scales(sb + L::OFF_SA);
      const uint64_t dsb = sdesc_scales(sb + L::OFF_SB);
      const int last_chunks = (p.k - (steps - 1) * kStepK + 63) / 64;  // of 64, in a tile's last step
      uint32_t parity = 0;
      int i = 0, kt = 0;
      bool more = true;
      while (more) {
#pragma unroll
        for (int s = 0; s < L::STAGES; ++s) {
          if (!more) break;
          bool ok = true;
          // the tile before has left the shared columns (and the one before that its own)
          if (kt == 0 && i >= 1) ok = mbar_wait(shared_read((i - 1) & 1), ((i - 1) >> 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_O);
          ok = ok && mbar_wait(full(s), parity, abort, p.status, DEV_ERR_TIMEOUT_KV);
          if (!__all_sync(0xffffffffu, ok)) {
            more = false;
            break;
          }
          tc_fence_after();
          constexpr uint32_t kStage16 = L::STAGE >> 4;
          const uint32_t d = tmem + (i & 1) * L::COL_ACC1;
          const uint32_t sa = tmem + L::COL_SF + s * L::SF_COLS;
          const uint32_t sw = sa + 8;
          const int chunks = kt == steps - 1 ? last_chunks : 4;
          const uint32_t go_on = kt > 0 ? 1u : 0u;
          const bool tile_done = kt == steps - 1;
          if (elect_one()) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 128 of k: its scales
              if (2 * h >= chunks) break;
              cp_scales_pair(sa + h * 4, sdesc_add(dsa, s * kStage16 + h * (kScaleTile >> 4)));
              cp_scales_pair(sw + h * 8, sdesc_add(dsb, s * kStage16 + h * (kScaleTile >> 4)));
              cp_scales_pair(sw + h * 8 + 4, sdesc_add(dsb, s * kStage16 + (2 + h) * (kScaleTile >> 4)));
            }
            mma_mx4_pair(d, sdesc_add(da, s * kStage16), sdesc_add(db, s * kStage16), idesc_mx4(256, L::BN, 0), sa, sw, go_on);
            if (chunks > 1) mma_mx4_pair(d, sdesc_add(da, s * kStage16 + 2), sdesc_add(db, s * kStage16 + 2), idesc_mx4(256, L::BN, 2), sa, sw, 1u);
            if (chunks > 2) mma_mx4_pair(d, sdesc_add(da, s * kStage16 + 4), sdesc_add(db, s * kStage16 + 4), idesc_mx4(256, L::BN, 0), sa + 4, sw + 8, 1u);
            if (chunks > 3) mma_mx4_pair(d, sdesc_add(da, s * kStage16 + 6), sdesc_add(db, s * kStage16 + 6), idesc_mx4(256, L::BN, 2), sa + 4, sw + 8, 1u);
            commit_pair(empty(s));
            if (tile_done) commit_pair(acc_full(i & 1));
          }
          __syncwarp();
          ++kt;
          if (tile_done) {
            kt = 0;
            more = ++i < n_mine;
          }
        }
        parity ^= 1;
      }
      if (elect_one()) {
        commit_pair(fin);
        mbar_drain_wait(fin, 0, p.status);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue: one thread per row
    // A warp's 32 rows by 128 bytes go through shared memory (128-byte swizzle) to a TMA store,
    // which writes whole lines and leaves out what lies behind m or n.
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t tlane = (static_cast<uint32_t>(quarter) * 32u) << 16;
    const uint32_t read0 = in_first(shared_read(0)), read1 = in_first(shared_read(1));
    uint8_t* stage = smem + L::OFF_OUT + (warp - 2) * L::OUT_BYTES;
    auto put = [&](const uint32_t (&wd)[32], int64_t row0, int col) {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the store before has read it
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(wd[4 * c], wd[4 * c + 1], wd[4 * c + 2], wd[4 * c + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && row0 < p.m && col < p.n) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(&tm_y)),
                     "r"(smem_u32(stage)), "r"(col), "r"(static_cast<int32_t>(row0))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    };
    for (int i = 0; i < n_mine; ++i) {
      const int b = i & 1;
      bool ok = mbar_wait(acc_full(b), (i >> 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_O);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      int m_tile, n_tile;
      wide_coords(w, pair + i * pairs, m_tile, n_tile);
      const int64_t row0 = static_cast<int64_t>(m_tile) * 256 + rank * 128 + quarter * 32;
#pragma unroll 1
      for (int j = 0; j < 2; ++j) {
        // groups of 64 columns, those with shared columns first: 3 and 2 of accumulator 0, 0 and 1 of 1
        const int c0 = (b ? 2 * j + half : 3 - 2 * j - half) * 64;
        uint32_t r[2][32];
        tmem_ld32(tmem + tlane + b * L::COL_ACC1 + c0, r[0]);
        tmem_ld32(tmem + tlane + b * L::COL_ACC1 + c0 + 32, r[1]);
        tmem_wait_ld();
        if (j == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(b ? read1 : read0);
        }
        const int col = n_tile * L::BN + c0;
        if (p.bias) {
#pragma unroll
          for (int c = 0; c < 64; c += 4)
            if (col + c < p.n) {
              const float4 x = *reinterpret_cast<const float4*>(p.bias + col + c);
              uint32_t* v = &r[c >> 5][c & 31];
              v[0] = __float_as_uint(__uint_as_float(v[0]) + x.x);
              v[1] = __float_as_uint(__uint_as_float(v[1]) + x.y);
              v[2] = __float_as_uint(__uint_as_float(v[2]) + x.z);
              v[3] = __float_as_uint(__uint_as_float(v[3]) + x.w);
            }
        }
        if (p.y_dt == DP_F32) {
          put(r[0], row0, col);
          put(r[1], row0, col + 32);
        } else {
          uint32_t wd[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float lo = __uint_as_float(r[c >> 4][(2 * c) & 31]), hi = __uint_as_float(r[c >> 4][(2 * c + 1) & 31]);
            wd[c] = p.y_dt == DP_BF16 ? pack_bf16x2(lo, hi) : pack_f16x2_sat(lo, hi);
          }
          put(wd, row0, col);
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of the pair is in flight
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  cluster_sync();
}

// ------------------------------------------------------------------ host

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

// Codes [rows][k / 2] bytes, boxes of 128 bytes by box_rows.
bool encode_codes(EncodeFn fn, CUtensorMap* t, const void* base, int64_t rows, int32_t k, int box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(k / 2), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(k / 2)};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t one[2] = {1, 1};
  return fn(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles [rows / 128][k / 128][128 words], boxes of two tiles along k by box_rows / 128.
bool encode_scales(EncodeFn fn, CUtensorMap* t, const void* base, int64_t rows, int32_t k, int box_rows) {
  const cuuint64_t tiles = static_cast<cuuint64_t>((k + 127) / 128);
  cuuint64_t dims[3] = {kScaleTile / 4, tiles, static_cast<cuuint64_t>((rows + 127) / 128)};
  cuuint64_t strides[2] = {kScaleTile, tiles * kScaleTile};
  cuuint32_t box[3] = {kScaleTile / 4, 2, static_cast<cuuint32_t>(box_rows > 128 ? box_rows / 128 : 1)};
  cuuint32_t one[3] = {1, 1, 1};
  return fn(t, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y [m][n], boxes of 32 rows by 128 bytes.
bool encode_out(EncodeFn fn, CUtensorMap* t, void* y, int64_t m, int32_t n, dp_dtype dt) {
  const int eb = dt == DP_F32 ? 4 : 2;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(m)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(n) * eb};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / eb), 32};
  cuuint32_t one[2] = {1, 1};
  const CUtensorMapDataType type = dt == DP_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dt == DP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(t, type, 2, y, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
cudaError_t launch_narrow(const Mx4Args& g, cudaStream_t s) {
  using L = Narrow<NT>;
  int dev = 0, sms = 148;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  EncodeFn fn = tensor_map_encoder();
  CUtensorMap tw, ta, tsw, tsa;
  if (!fn || !encode_codes(fn, &tw, g.w, g.n, g.k, 128) || !encode_codes(fn, &ta, g.a, g.m, g.k, NT) ||
      !encode_scales(fn, &tsw, g.w_scales, g.n, g.k, 128) || !encode_scales(fn, &tsa, g.a_scales, g.m, g.k, NT))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(mx4_narrow_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  Mx4Params p;
  p.bias = g.bias;
  p.y = g.y;
  p.m = g.m;
  p.n = g.n;
  p.k = g.k;
  p.y_dt = g.y_dt;
  p.status = g.status;
  const int64_t m_tiles = (g.m + NT - 1) / NT, n_tiles = (static_cast<int64_t>(g.n) + 127) / 128;
  const int steps = (g.k + kStepK - 1) / kStepK;
  // as many parts of k as the SMs take at once, each of a step at least
  int splits = 1;
  p.log_splits = 0;
  while (splits < kMaxSplits && m_tiles * n_tiles * splits * 2 <= sms && steps >= splits * 2) splits *= 2, ++p.log_splits;
  if (m_tiles > 65535 || n_tiles * splits > INT_MAX) return cudaErrorInvalidValue;
  return launch_early(mx4_narrow_kernel<NT>, dim3(static_cast<unsigned>(n_tiles * splits), static_cast<unsigned>(m_tiles)),
                      L::kThreads, L::ALLOC, splits, s, tw, ta, tsw, tsa, p);
}

cudaError_t launch_wide(const Mx4Args& g, cudaStream_t s) {
  using L = Wide;
  int dev = 0, sms = 148;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  EncodeFn fn = tensor_map_encoder();
  CUtensorMap ta, tw, tsa, tsw, ty;
  if (!fn || !encode_out(fn, &ty, g.y, g.m, g.n, g.y_dt) || !encode_codes(fn, &ta, g.a, g.m, g.k, 128) || !encode_codes(fn, &tw, g.w, g.n, g.k, 128) ||
      !encode_scales(fn, &tsa, g.a_scales, g.m, g.k, 128) || !encode_scales(fn, &tsw, g.w_scales, g.n, g.k, 256))
    return cudaErrorInvalidValue;
  static std::atomic<int> pairs_of[64];  // pairs that fit on the device at once
  int most = pairs_of[dev].load(std::memory_order_acquire);
  if (!most) {
    e = cudaFuncSetAttribute(mx4_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::ALLOC;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&most, mx4_wide_kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (most < 1) return cudaErrorInvalidConfiguration;
    pairs_of[dev].store(most, std::memory_order_release);
  }
  WideParams w;
  w.p.bias = g.bias;
  w.p.y = g.y;
  w.p.m = g.m;
  w.p.n = g.n;
  w.p.k = g.k;
  w.p.log_splits = 0;
  w.p.y_dt = g.y_dt;
  w.p.status = g.status;
  const int64_t m_tiles = (g.m + 255) / 256, n_tiles = (g.n + 255) / 256;
  if (m_tiles * n_tiles > INT_MAX) return cudaErrorInvalidValue;
  w.m_tiles = static_cast<int32_t>(m_tiles);
  w.n_tiles = static_cast<int32_t>(n_tiles);
  w.tiles = w.m_tiles * w.n_tiles;
  w.group_m = 8;  // a wave of 74 pairs takes 8 tiles of a by 9 or 10 of W: the fewest rows to read
  const int pairs = w.tiles < most ? w.tiles : most;
  return launch_early(mx4_wide_kernel, dim3(2 * pairs), L::kThreads, L::ALLOC, 2, s, ta, tw, tsa, tsw, ty, w);
}

}  // namespace

cudaError_t launch_mx4_linear(const Mx4Args& g, cudaStream_t s) {
  if (g.m <= 0 || g.n <= 0 || g.n % 8 || g.k <= 0 || g.k % 32) return cudaErrorInvalidValue;
  // Few tokens: one tile of them.  More: tiles of 64, as long as their blocks fit on the SMs at once
  // (two on each); then block pairs.  Measured with n x k = 4608 x 1536 and 4096 x 4096, us, tiles of
  // 64 | pairs: m = 64 7.0 | 7.9, 7.0 | 10.8; m = 512 (288 and 256 blocks) 8.2 | 8.6, 11.4 | 11.7;
  // m = 768 12.9 | 8.8, 18.5 | 11.8.  Tiles of 128 or 256 tokens were nowhere faster.
  if (g.m <= 16) return launch_narrow<16>(g, s);
  if (g.m <= 32) return launch_narrow<32>(g, s);
  int dev = 0, sms = 148;
  const cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (g.m + 63) / 64 * ((static_cast<int64_t>(g.n) + 127) / 128);
  return blocks <= 2 * sms ? launch_narrow<64>(g, s) : launch_wide(g, s);
}

}  // namespace dp
