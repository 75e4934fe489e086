// Attention over packed sequences on the sm_100a tensor cores (bf16 or f16; the fp32 form is in
// dp_packed.cu, which also states the formulas).
//
// An item = two query tiles of one sequence under one k/v head; a tile is as many whole
// tokens as their rows, one for each head of the group, fit in 128 (groups of more than 128 heads
// are cut), so that its keys are read once for all the heads that share them, and one TMA box
// {64 columns, heads, tokens} brings 64 columns of it.  (256 threads with 16 loads each took 5 us
// to bring 256 rows of 128 under load.)  Keys go by in
// tiles of BN rows (128 at head_dim 64, 64 at head_dim 128) up to the last one that a row of the
// tile sees; only tiles that the mask cuts pay for it (warp-uniform test).
//   warps 0-3  softmax of query tile 0, one thread per row
//   warps 4-7  softmax of query tile 1
//   warp 8     TMA producer: K and V tiles into a ring of shared-memory stages
//   warps 9-11 issue S_g = Q_g K^T and O_g += P_g V, the same number of products each
//              (head_dim 64: S of both tiles, PV_0, PV_1; head_dim 128: S_0, S_1, PV of both)
// Tensor memory holds S (fp32), P (16 bits, the A operand of PV) and O of both tiles.  The
// softmax runs in fp32 in units of log2 with a running maximum that O is rescaled for only when
// it grows by more than 2^8; P is rounded to the operands' 16-bit type (the tensor cores take
// nothing wider beside 16-bit V), the row sum takes it unrounded.
//
// Few rows and many keys (single tokens over a cache): the keys are cut into as many parts as a
// thread-block cluster has blocks, each block keeps its part's O, maximum and sum, and at the
// end the blocks join them through distributed shared memory, in a fixed order, with no
// workspace and no second launch.  Only the sequences with many keys are cut (they come first);
// the blocks of the clusters behind them take one whole item each.
//
// Where no keys are cut, a block goes on with the items of blocks that have not started (cluster
// launch control hands them over): the producer warp asks, decodes the item for the other warps and
// loads its queries and first keys while the item before is finished and written.
//
// A tile of keys that ends behind its sequence holds other rows: their scores are masked, and
// the producer warp writes zeros over their V rows before the product reads them (0 * NaN).
// Every wait is bounded (dp_device.cuh).
//
// Bound by the softmax's issue slots and exponentials at head_dim 64.  At 128 no one unit is full (tensor
// pipe 49 % of the active cycles of 4096 causal tokens, 74 % on the busiest SM; issue slots 43 %): a query
// tile's softmax and products wait for each other, and two tiles do not quite cover it; long runs meet the
// power limit besides.  Causal 16384 tokens of 16 heads on 4: head_dim 128 930 to 970 us in short bursts
// (1.18 PFLOP/s), 1075 in a loop, at 1640 of 1965 MHz; head_dim 64 715, and 755 at 1865 MHz; nine prompts
// of 1 to 2048 tokens, 32 heads on 8 of 128: 111 us, 124 in a loop at 1765 MHz.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>

#include "dp_device.cuh"
#include "dp_packed.h"

namespace dp {

namespace {

constexpr int BM = 128;
constexpr float kRescaleLog2 = 8.0f;

// 2^x on the FMA pipe for some columns (the MUFU unit gives 16 exponentials per clock and SM, as
// many as the tensor cores need at head_dim 128): n = round(x), 2^n p(x - n), p the degree-4
// minimax polynomial of 2^f on [-1/2, 1/2] (csrc/fit_exp2_poly.py 4; relative error
// 2.7e-6, so that the row sum and the log-sum-exp keep fp32's use).
constexpr float kC0 = 0.9999992847442627f, kC1 = 0.6931217908859253f, kC2 = 0.240247443318367f;
constexpr float kC3 = 0.05591785907745361f, kC4 = 0.009570102207362652f;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
constexpr float kMinX = -125.0f;
constexpr float kLost = 1e30f;  // no row sum reaches this
// f16 weights are taken 2^7 times as large (at most 2^15: the running maximum may lag by 2^8), so that
// those under 2^-14 of the largest keep their bits; sum and O carry the factor, which cancels.
template <bool F16>
constexpr float kWeightLog2 = F16 ? 7.0f : 0.0f;
constexpr uint32_t kPolyMask = 0x1111u;  // column pairs of each 16 that use it

constexpr int NQ = 2;            // query tiles per block
constexpr int kTmemCols = 512;

template <int HD>
struct Lay {
  static constexpr int BN = HD == 64 ? 128 : 64;
  static constexpr int W_PROD = 4 * NQ;
  static constexpr int W_ISS = W_PROD + 1;
  static constexpr int kThreads = 32 * (W_PROD + 4);
  static constexpr int kLaunchRegs = (65536 / kThreads) & ~7;
  static constexpr int kLowRegs = 72, kHighRegs = 216;
  static_assert(NQ * 128 * kHighRegs + 128 * kLowRegs <= kThreads * kLaunchRegs, "register split exceeds the launch");
  static constexpr int KCH = HD / 64;
  static constexpr int STAGES = 4;
  static constexpr int Q_CHUNK = BM * 128;
  static constexpr int KV_CHUNK = BN * 128;
  static constexpr int Q_BYTES = BM * HD * 2;
  static constexpr int KV_BYTES = BN * HD * 2;
  // key tiles that a block's start and end cost, and those of a block that joins parts
  static constexpr int kWhole = HD == 64 ? 4 : 5, kPart = kWhole + 4;
  static constexpr bool S_PER_TILE = HD > BN;  // the issuers' split (see above)
  static constexpr int kPvIssuers = S_PER_TILE ? 1 : NQ;
  // Whether a block goes on with further items.  At head_dim 64 a row's 128 scores leave the softmax
  // no registers for that: 100 of them spilled, and a 16384-token prompt took 1094 us, not 676.
  static constexpr bool KEEP_ON = HD == 128;
  static constexpr int COL_S = HD >= BN ? NQ * HD : 0;
  static constexpr int COL_P = COL_S + NQ * BN;
  static constexpr int COL_O = HD >= BN ? 0 : COL_P + NQ * (BN / 2);
  static_assert(NQ * (BN + BN / 2 + HD) <= kTmemCols, "tensor memory budget");
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = NQ * Q_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * KV_BYTES;
  static constexpr int OFF_OUT = OFF_V + STAGES * KV_BYTES;  // 64 columns of each query tile's output
  static constexpr int OFF_BAR = OFF_OUT + NQ * Q_CHUNK;
  static constexpr int N_BAR = 3 * STAGES + 6 * NQ + 8;
  static constexpr int OFF_WORK = (OFF_BAR + N_BAR * 8 + 15) / 16 * 16;  // two items
  static constexpr int OFF_NEXT = OFF_WORK + 2 * 64;                     // the hardware's answer
  static constexpr int OFF_MISC = OFF_NEXT + 16;
  static constexpr int BYTES = OFF_MISC + 32;
  static constexpr int ALLOC = BYTES + 1024;
  // a part's result for the join, over Q, K and V: O rows (a pitch that spreads the banks), then
  // (maximum, sum) per row
  static constexpr int O_PITCH = HD + 4;
  static constexpr int OFF_ML = NQ * BM * O_PITCH * 4;
  static_assert(OFF_ML + NQ * BM * 8 <= OFF_OUT, "the join's rows fit");
  static_assert(ALLOC <= 227 * 1024, "shared memory budget");
};

// An item (or this block's part of one), as the producer decodes it for the other warps.
struct Work {
  int32_t some;            // 0: none, the block is done
  int32_t kv, head0, heads;
  int32_t q_len, k_len, first_q, first_k;
  int32_t tok0;            // the first query tile's first token
  int32_t t_begin, n_loc;  // key tiles of the part
  int32_t nt[NQ];          // of them, those that each query tile sees (its first ones)
  int32_t tail_rows;       // rows of the part's last key tile that are the sequence's (BN: all)
  int32_t pad[2];
};
static_assert(sizeof(Work) == 64, "two of them in shared memory");

struct PackedParams {
  uint16_t* out;
  float* lse;
  int64_t ld_out;
  int32_t n_heads, n_kv, group;  // n_kv: k/v heads times the cuts of a group
  int32_t cuts, cut_heads;       // of a group of more than 128 heads (else 1, group)
  int32_t tokens;                // of a query tile
  FastDiv by_kv, by_cut_heads;
  int32_t log_cluster;  // of the blocks per cluster
  int32_t n_cut;    // items whose keys a cluster's blocks share; n_items: all
  int32_t n_items;
  int32_t causal;
  float scale_log2;
  uint32_t* status;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Shared address `a` of this block in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_smem(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

__device__ __forceinline__ float4 ld_peer4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float2 ld_peer2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// Two softmax weights.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// The larger, NaN if either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <int BN, int N>
__device__ __forceinline__ Work decode(const PackedSeqs<N>& seqs, const PackedParams& p, int item, int rank, int log_parts) {
  Work w;
  w.some = 1;
  const int tile = p.by_kv.div(item);
  const int kvc = item - tile * p.n_kv;
  w.kv = p.cuts == 1 ? kvc : kvc / p.cuts;
  w.head0 = w.kv * p.group + (kvc - w.kv * p.cuts) * p.cut_heads;
  w.heads = min(p.cut_heads, (w.kv + 1) * p.group - w.head0);
  const int seq = seq_of_tile(seqs, tile);
  w.q_len = seqs.q_len[seq];
  w.k_len = seqs.k_len[seq];
  w.first_q = seqs.first_q[seq];
  w.first_k = seqs.first_k[seq];
  w.tok0 = (seqs.tile0[seq + 1] - 1 - tile) * (NQ * p.tokens);
#pragma unroll
  for (int g = 0; g < NQ; ++g) {
    const int end = min(w.q_len, w.tok0 + (g + 1) * p.tokens);  // behind the query tile's last token
    const int seen = end > w.tok0 + g * p.tokens ? min(w.k_len, keys_seen(end - 1, w.q_len, w.k_len, p.causal)) : 0;
    w.nt[g] = (seen + BN - 1) / BN;
  }
  const int per = (max(w.nt[0], w.nt[1]) + (1 << log_parts) - 1) >> log_parts;
  w.t_begin = rank * per;
#pragma unroll
  for (int g = 0; g < NQ; ++g) w.nt[g] = max(0, min(w.nt[g] - w.t_begin, per));
  w.n_loc = max(w.nt[0], w.nt[1]);
  const int rows = w.n_loc > 0 ? w.k_len - (w.t_begin + w.n_loc - 1) * BN : BN;
  w.tail_rows = min(rows, BN);
  return w;
}

// Asks for a block of the grid that has not started: the answer (16 bytes) comes to `to`, its
// arrival to `bar`.
__device__ __forceinline__ void ask_next(uint32_t to, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to), "r"(bar)
               : "memory");
}

// The index of the block that the answer at `at` hands over, or -1.
__device__ __forceinline__ int next_item(uint32_t at) {
  uint32_t yes, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(yes), "=r"(x)
      : "r"(at)
      : "memory");
  return yes ? static_cast<int>(x) : -1;
}

template <int HD, bool F16, int N>
__global__ void __launch_bounds__(Lay<HD>::kThreads, 1)
    packed_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const PackedParams p,
                          const __grid_constant__ PackedSeqs<N> seqs) {
  using L = Lay<HD>;
  constexpr int BN = L::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const ItemPart ip = item_part(p.log_cluster, p.n_cut);
  const int splits = 1 << ip.log_parts;
  if (ip.item >= p.n_items) return;  // behind the last item: its cluster never joins
  const bool keep_on = L::KEEP_ON && p.log_cluster == 0;  // this block takes over blocks that have not started

  const uint32_t bar0 = sb + L::OFF_BAR;
  auto k_full = [&](int s) { return bar0 + 8u * s; };
  auto v_full = [&](int s) { return bar0 + 8u * (L::STAGES + s); };
  auto kv_empty = [&](int s) { return bar0 + 8u * (2 * L::STAGES + s); };
  constexpr uint32_t kPer = 3 * L::STAGES;
  auto q_full = [&](int g) { return bar0 + 8u * (kPer + g); };
  auto q_free = [&](int g) { return bar0 + 8u * (kPer + NQ + g); };   // the item's last S has read Q
  auto s_full = [&](int g) { return bar0 + 8u * (kPer + 2 * NQ + g); };
  auto s_free = [&](int g) { return bar0 + 8u * (kPer + 3 * NQ + g); };
  auto p_full = [&](int g) { return bar0 + 8u * (kPer + 4 * NQ + g); };
  auto o_done = [&](int g) { return bar0 + 8u * (kPer + 5 * NQ + g); };
  const uint32_t fin = bar0 + 8u * (kPer + 6 * NQ);
  const uint32_t v_fixed = fin + 8u;     // the last key tile's rows behind the sequence are zeros
  const uint32_t v_seen = fin + 16u;     // the PV issuers have waited for that
  const uint32_t next_full = fin + 24u;  // the answer about the next item is there
  auto work_full = [&](int b) { return fin + 32u + 8u * b; };  // item of parity b is decoded
  auto work_read = [&](int b) { return fin + 48u + 8u * b; };  // the other warps are done with it
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::OFF_MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC + 4);
  // what a warpgroup goes by at an item's end, [warpgroup][parity of the item]: 1 leave, 2 whole tile
  volatile int* verdict = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 8);
  auto work_at = [&](int b) { return reinterpret_cast<volatile Work*>(smem + L::OFF_WORK + 64 * b); };

  if (warp == L::W_PROD && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(kv_empty(s), L::kPvIssuers);
    }
    for (int g = 0; g < NQ; ++g) {
      mbar_init(q_full(g), 1);
      mbar_init(q_free(g), 1);
      mbar_init(s_full(g), 1);
      mbar_init(s_free(g), 128);
      mbar_init(p_full(g), 128);
      mbar_init(o_done(g), 1);
    }
    mbar_init(fin, 3);
    mbar_init(v_fixed, 1);
    mbar_init(v_seen, L::kPvIssuers);
    mbar_init(next_full, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(work_full(b), 1);
      mbar_init(work_read(b), L::kThreads / 32 - 1);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == L::W_ISS) {
    wait_for_earlier_kernels();
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }

  // ------------------------------------------------------------ producer's state
  Work w;               // the producer's item, then each issuer's
  int ring = 0;         // key tiles issued (producer) or of the items before (issuers)
  int loads[NQ] = {0, 0};  // items so far with key tiles of each query tile
  auto load_q = [&](int g) {
    mbar_arrive_expect_tx(q_full(g), L::KCH * 128 * p.cut_heads * p.tokens);
#pragma unroll
    for (int c = 0; c < L::KCH; ++c)
      tma_load_3d(sb + L::OFF_Q + g * L::Q_BYTES + c * L::Q_CHUNK, &tm_q, c * 64, w.head0, w.first_q + w.tok0 + g * p.tokens, q_full(g));
  };
  auto load_tile = [&](int j) {  // key tile j of the part
    const int st = ring % L::STAGES;
    const int row = w.first_k + (w.t_begin + j) * BN;
    mbar_arrive_expect_tx(k_full(st), L::KV_BYTES);
#pragma unroll
    for (int c = 0; c < L::KCH; ++c)
      tma_load_2d(sb + L::OFF_K + st * L::KV_BYTES + c * L::KV_CHUNK, &tm_k, w.kv * HD + c * 64, row, k_full(st));
    mbar_arrive_expect_tx(v_full(st), L::KV_BYTES);
#pragma unroll
    for (int c = 0; c < L::KCH; ++c)
      tma_load_2d(sb + L::OFF_V + st * L::KV_BYTES + c * L::KV_CHUNK, &tm_v, w.kv * HD + c * 64, row, v_full(st));
    ++ring;
  };
  auto publish = [&](int b) {  // the producer's item to the other warps
    if (lane == 0) {
      volatile Work* to = work_at(b);
      to->some = w.some;
      to->kv = w.kv;
      to->head0 = w.head0;
      to->heads = w.heads;
      to->q_len = w.q_len;
      to->k_len = w.k_len;
      to->first_q = w.first_q;
      to->first_k = w.first_k;
      to->tok0 = w.tok0;
      to->t_begin = w.t_begin;
      to->n_loc = w.n_loc;
      to->nt[0] = w.nt[0];
      to->nt[1] = w.nt[1];
      to->tail_rows = w.tail_rows;
      mbar_arrive(work_full(b));
    }
    __syncwarp();
  };
  wait_for_earlier_kernels();
  if (warp == L::W_PROD) {
    // the first item and its first loads, before the other warps are up
    w = decode<BN>(seqs, p, ip.item, ip.rank, ip.log_parts);
    __syncwarp();
    publish(0);
    if (lane == 0) {
#pragma unroll
      for (int g = 0; g < NQ; ++g)
        if (w.nt[g] > 0) load_q(g);
      for (int j = 0; j < min(w.n_loc, L::STAGES); ++j) load_tile(j);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= L::W_PROD) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kLowRegs));
    if (warp == L::W_PROD) {
      // ------------------------------------------------------------ TMA producer
      int fixes = 0;
      for (int it = 0;; ++it) {
        bool ok = true;
        if (lane == 0) {
          if (keep_on) {
            mbar_arrive_expect_tx(next_full, 16);
            ask_next(sb + L::OFF_NEXT, next_full);
          }
          int done = it == 0 ? ring : 0;  // of this item's tiles
          if (it > 0) {
#pragma unroll
            for (int g = 0; g < NQ; ++g)
              if (ok && w.nt[g] > 0) {
                ok = loads[g] == 0 || mbar_wait(q_free(g), (loads[g] - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_EMPTY);
                if (ok) load_q(g);
              }
          }
          for (; ok && done < w.n_loc; ++done) {
            ok = ring < L::STAGES ||
                 mbar_wait(kv_empty(ring % L::STAGES), (ring / L::STAGES - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_EMPTY);
            if (ok) load_tile(done);
          }
        }
        ring = __shfl_sync(0xffffffffu, ring, 0);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
#pragma unroll
        for (int g = 0; g < NQ; ++g) loads[g] += w.nt[g] > 0 ? 1 : 0;
        if (w.tail_rows < BN) {
          const int g = ring - 1, st = g % L::STAGES;
          ok = mbar_wait(v_full(st), (g / L::STAGES) & 1, abort, p.status, DEV_ERR_TIMEOUT_KV) &&
               (fixes == 0 || mbar_wait(v_seen, (fixes - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_KV));
          if (!__all_sync(0xffffffffu, ok)) break;
          for (int i = w.tail_rows * 8 + lane; i < BN * 8; i += 32)
#pragma unroll
            for (int c = 0; c < L::KCH; ++c)
              *reinterpret_cast<uint4*>(smem + L::OFF_V + st * L::KV_BYTES + c * L::KV_CHUNK + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_fixed);
          ++fixes;
        }
        // the next item
        int item = -1;
        if (keep_on) {
          ok = mbar_wait(next_full, it & 1, abort, p.status, DEV_ERR_TIMEOUT_Q);
          if (!__all_sync(0xffffffffu, ok)) break;
          item = next_item(sb + L::OFF_NEXT);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (item >= 0)
          w = decode<BN>(seqs, p, item, 0, 0);
        else
          w.some = 0;
        const int b = (it + 1) & 1;
        ok = it == 0 || mbar_wait(work_read(b), ((it - 1) >> 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_Q);
        if (!__all_sync(0xffffffffu, ok)) break;
        publish(b);
        if (!L::KEEP_ON || item < 0) break;
      }
      if (lane == 0) {
        // every copy this block issued lands before its shared memory is released
#pragma unroll
        for (int g = 0; g < NQ; ++g)
          if (loads[g] > 0) mbar_drain_wait(q_full(g), (loads[g] - 1) & 1, p.status);
        for (int g = max(0, ring - L::STAGES); g < ring; ++g) {
          mbar_drain_wait(k_full(g % L::STAGES), (g / L::STAGES) & 1, p.status);
          mbar_drain_wait(v_full(g % L::STAGES), (g / L::STAGES) & 1, p.status);
        }
      }
    } else {
      // ------------------------------------------------------------ MMA issuers
      // Each warp runs its loop as a whole and elects one lane for the tensor-core instructions:
      // with uniform operands the issue stays ahead of the products.
      constexpr uint32_t idS = idesc_f32acc(Operand<F16>::kFmt, BM, BN, false);
      constexpr uint32_t idPV = idesc_f32acc(Operand<F16>::kFmt, BM, HD, true);
      auto wait = [&](uint32_t bar, uint32_t parity, uint32_t code) {
        return mbar_wait(bar, parity, abort, p.status, code);
      };
      const uint64_t dq0 = sdesc_sw128(sb + L::OFF_Q, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sb + L::OFF_K, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sb + L::OFF_V, L::KV_CHUNK, 1024);
      int tiles[NQ] = {0, 0};  // each query tile's key tiles of the items before
      int fixes = 0;
      int nt[NQ] = {0, 0}, n_loc = 0;
      bool tail = false, ok = true;
      // S_g of tile t, once K_t is there and S_g of the tile before is in the softmax's registers
      auto do_s = [&](int t, int g) {
        const int st = (ring + t) % L::STAGES;
        const int n = tiles[g] + t;
        ok = (t > 0 || wait(q_full(g), loads[g] & 1, DEV_ERR_TIMEOUT_Q)) && (n == 0 || wait(s_free(g), (n - 1) & 1, DEV_ERR_TIMEOUT_S)) &&
             wait(k_full(st), ((ring + t) / L::STAGES) & 1, DEV_ERR_TIMEOUT_KV);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dq = sdesc_add(dq0, (g * L::Q_BYTES) >> 4);
        const uint64_t dk = sdesc_add(dk0, (st * L::KV_BYTES) >> 4);
        const uint32_t d = tmem + L::COL_S + g * BN;
        const bool last = t == nt[g] - 1;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_ss(d, sdesc_add(dq, ((kk >> 2) * L::Q_CHUNK + (kk & 3) * 32) >> 4),
                   sdesc_add(dk, ((kk >> 2) * L::KV_CHUNK + (kk & 3) * 32) >> 4), idS, kk > 0);
          mma_commit(s_full(g));
          if (last) mma_commit(q_free(g));
        }
        __syncwarp();
      };
      // before a part's last tile is multiplied, its rows behind the sequence have to be zeros
      auto fixed = [&](int t) { return !tail || t != n_loc - 1 || wait(v_fixed, fixes & 1, DEV_ERR_TIMEOUT_KV); };
      auto saw_fixed = [&](int t) {
        if (tail && t == n_loc - 1 && elect_one()) mbar_arrive(v_seen);
        __syncwarp();
      };
      // O_g += P_g V of tile t; `done`: the tile's last product, which frees the stage
      auto do_pv = [&](int t, int g, bool done) {
        const int st = (ring + t) % L::STAGES;
        ok = wait(p_full(g), (tiles[g] + t) & 1, DEV_ERR_TIMEOUT_P) && wait(v_full(st), ((ring + t) / L::STAGES) & 1, DEV_ERR_TIMEOUT_KV) &&
             fixed(t);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dv = sdesc_add(dv0, (st * L::KV_BYTES) >> 4);
        const uint32_t pa = tmem + L::COL_P + g * (BN / 2);
        const uint32_t d = tmem + L::COL_O + g * HD;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(d, pa + kk * 8, sdesc_add(dv, (kk * 2048) >> 4), idPV, (t > 0 || kk > 0) ? 1u : 0u);
          mma_commit(o_done(g));
          if (done) mma_commit(kv_empty(st));
        }
        __syncwarp();
        if (done) saw_fixed(t);
      };
      const int iw = warp - L::W_ISS;
      for (int it = 0;; ++it) {
        const int b = it & 1;
        ok = wait(work_full(b), (it >> 1) & 1, DEV_ERR_TIMEOUT_Q);
        if (!__all_sync(0xffffffffu, ok)) break;
        const bool some = work_at(b)->some != 0;
        nt[0] = work_at(b)->nt[0];
        nt[1] = work_at(b)->nt[1];
        n_loc = work_at(b)->n_loc;
        tail = work_at(b)->tail_rows < BN;
        __syncwarp();
        if (lane == 0) mbar_arrive(work_read(b));
        if (!some) break;
        if constexpr (L::S_PER_TILE) {
          if (iw < NQ) {
            const int n = iw == 0 ? nt[0] : nt[1];
            for (int t = 0; ok && t < n; ++t) do_s(t, iw);
          } else {
            for (int t = 0; ok && t < n_loc; ++t) {
              if (t < nt[0]) do_pv(t, 0, t >= nt[1]);
              if (ok && t < nt[1]) do_pv(t, 1, true);
            }
          }
        } else {
          if (iw == 0) {
            for (int t = 0; ok && t < n_loc; ++t) {
              if (t < nt[0]) do_s(t, 0);
              if (ok && t < nt[1]) do_s(t, 1);
            }
          } else {
            const int g = iw - 1;
            const int n = g == 0 ? nt[0] : nt[1];
            for (int t = 0; ok && t < n_loc; ++t) {
              const int st = (ring + t) % L::STAGES;
              if (t < n) {
                do_pv(t, g, true);
              } else {
                // not this query tile's: its arrival for the stage, once per fill
                ok = wait(v_full(st), ((ring + t) / L::STAGES) & 1, DEV_ERR_TIMEOUT_KV) && fixed(t);
                ok = __all_sync(0xffffffffu, ok);
                if (ok && elect_one()) mbar_arrive(kv_empty(st));
                __syncwarp();
                if (ok) saw_fixed(t);
              }
            }
          }
        }
        if (!ok) break;
        ring += n_loc;
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          tiles[g] += nt[g];
          loads[g] += nt[g] > 0 ? 1 : 0;
        }
        fixes += tail ? 1 : 0;
        if (!L::KEEP_ON) break;
      }
      // every product this warp issued completes before tensor memory is released
      if (elect_one()) {
        mma_commit(fin);
        mbar_drain_wait(fin, 0, p.status);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kHighRegs));
    // ------------------------------------------------------------ softmax
    const int g = warp >> 2;
    const int t = threadIdx.x & 127;
    const uint32_t trow = tmem + ((static_cast<uint32_t>(warp & 3) * 32u) << 16);
    const uint32_t s_col = trow + L::COL_S + g * BN;
    const uint32_t p_col = trow + L::COL_P + g * (BN / 2);
    const uint32_t o_col = trow + L::COL_O + g * HD;
    constexpr int NCH = BN / 32;
    constexpr int NG = BN / 16;
    const uint64_t sl2 = f32x2(p.scale_log2, p.scale_log2);
    // 16-byte piece c of row r of the 64 output columns under way
    uint8_t* so = smem + L::OFF_OUT + g * L::Q_CHUNK;
    auto piece = [&](int r, int c) { return reinterpret_cast<uint4*>(so + r * 128 + ((c ^ (r & 7)) << 4)); };
    auto warpgroup_sync = [&]() {
      if (g == 0)
        asm volatile("bar.sync 1, 128;" ::: "memory");
      else
        asm volatile("bar.sync 2, 128;" ::: "memory");
    };
    int tiles = 0;  // this query tile's key tiles of the items before
    for (int it = 0;; ++it) {
      const int b = it & 1;
      volatile Work* wk = work_at(b);
      bool ok = mbar_wait(work_full(b), (it >> 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_Q);
      ok = __all_sync(0xffffffffu, ok);
      // Without an item (there is none left, or the block gives up) a warp does nothing until the
      // warpgroup leaves together.
      const bool some = ok && wk->some != 0;
      const int my_nt = some ? wk->nt[g] : 0;
      // keys that this thread's row sees (a row that does not exist needs no mask: nothing of it is stored)
      auto row_of = [&](int r, int& tok, int& head) {
        const int of_tok = p.by_cut_heads.div(r);
        tok = wk->tok0 + g * p.tokens + of_tok;
        head = wk->head0 + r - of_tok * p.cut_heads;
        return some && of_tok < p.tokens && tok < wk->q_len && r - of_tok * p.cut_heads < wk->heads;
      };
      auto keys_of = [&](bool row_ok, int tok) {
        return row_ok ? min(wk->k_len, keys_seen(tok, wk->q_len, wk->k_len, p.causal)) : INT_MAX;
      };
      int lim;  // of this part's keys
      bool live;
      {
        int tok, head;
        const bool row_ok = row_of(t, tok, head);
        lim = keys_of(row_ok, tok) - wk->t_begin * BN;
        live = __any_sync(0xffffffffu, row_ok);
      }
      // tiles of this part that every row of the warp sees whole
      const int n_whole = __reduce_min_sync(0xffffffffu, lim) / BN;
      float m_ref = -INFINITY;
      float l_sum = 0.0f;

      for (int j = 0; ok && j < my_nt; ++j) {
        ok = mbar_wait(s_full(g), (tiles + j) & 1, abort, p.status, DEV_ERR_TIMEOUT_S);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (!live) {  // no rows: keep the barriers going, P's no sooner than the others may
          mbar_arrive(s_free(g));
          if (j > 0) {
            ok = mbar_wait(o_done(g), (tiles + j - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_O);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          mbar_arrive(p_full(g));
          continue;
        }
        tc_fence_after();
        uint32_t sr[NCH][32];
#pragma unroll
        for (int i = 0; i < NCH; ++i) tmem_ld32(s_col + i * 32, sr[i]);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(s_free(g));
        const bool cut = j >= n_whole;
        const int valid = lim - j * BN;  // columns of this tile that the row sees
        if (cut) {
#pragma unroll
          for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (i * 32 + c >= valid) sr[i][c] = 0xff800000u;
        }
        float mc[NG];
#pragma unroll
        for (int h = 0; h < NG; ++h) {
          const uint32_t* r = &sr[h >> 1][(h & 1) * 16];
          float m = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[15]));
#pragma unroll
          for (int c = 1; c < 15; c += 2) m = fmax3(m, __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
          mc[h] = m;
        }
        float mx;
        if constexpr (NG == 8)
          mx = fmax3(fmax3(mc[0], mc[1], mc[2]), fmax3(mc[3], mc[4], mc[5]), fmaxf(mc[6], mc[7]));
        else
          mx = fmaxf(fmax3(mc[0], mc[1], mc[2]), mc[3]);
        const float m_new = fmaxf(m_ref, mx * p.scale_log2);
        if (j == 0) {
          m_ref = m_new;
        } else {
          const bool need = m_new > m_ref + kRescaleLog2;
          if (__any_sync(0xffffffffu, need)) {
            ok = mbar_wait(o_done(g), (tiles + j - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_O);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float f = need ? ex2_approx(m_ref - m_new) : 1.0f;
#pragma unroll
            for (int c0 = 0; c0 < HD; c0 += 32) {
              uint32_t orr[32];
              tmem_ld32(o_col + c0, orr);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) orr[c] = __float_as_uint(__uint_as_float(orr[c]) * f);
              tmem_st32(o_col + c0, orr);
            }
            tmem_wait_st();
            if (need) {
              l_sum *= f;
              m_ref = m_new;
            }
          }
        }
        // a row that has seen no key yet has no maximum: all its scores are -inf, all its weights 0
        const float ref = m_ref == -INFINITY ? 0.0f : m_ref;
        const float nm = kWeightLog2<F16> - ref;
        const uint64_t nm2 = f32x2(nm, nm);
        const uint64_t magic2 = f32x2(kMagic, kMagic), nmagic2 = f32x2(-kMagic, -kMagic), neg1_2 = f32x2(-1.0f, -1.0f);
        const uint64_t c0_2 = f32x2(kC0, kC0), c1_2 = f32x2(kC1, kC1), c2_2 = f32x2(kC2, kC2);
        const uint64_t c3_2 = f32x2(kC3, kC3), c4_2 = f32x2(kC4, kC4);
        uint64_t acc0 = f32x2(0.0f, 0.0f), acc1 = acc0;
        uint32_t pk[NCH][16];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint64_t x = ffma2(f32x2(__uint_as_float(sr[i][2 * c]), __uint_as_float(sr[i][2 * c + 1])), sl2, nm2);
            float x0, x1, a, b;
            f32x2_split(x, x0, x1);
            if ((kPolyMask >> c) & 1u) {
              const uint64_t xc = f32x2(max_nan(x0, kMinX), max_nan(x1, kMinX));
              const uint64_t r = fadd2(xc, magic2);
              const uint64_t f = ffma2(fadd2(r, nmagic2), neg1_2, xc);
              uint64_t q = ffma2(c4_2, f, c3_2);
              q = ffma2(q, f, c2_2);
              q = ffma2(q, f, c1_2);
              q = ffma2(q, f, c0_2);
              float q0, q1, r0, r1;
              f32x2_split(q, q0, q1);
              f32x2_split(r, r0, r1);
              a = __int_as_float(__float_as_int(q0) + (__float_as_int(r0) << 23));
              b = __int_as_float(__float_as_int(q1) + (__float_as_int(r1) << 23));
            } else {
              a = ex2_approx(x0);
              b = ex2_approx(x1);
            }
            const uint64_t ab = f32x2(a, b);
            if (c & 1)
              acc1 = fadd2(acc1, ab);
            else
              acc0 = fadd2(acc0, ab);
            pk[i][c] = pack2<F16>(a, b);
          }
        }
        if (cut) {
          // the polynomial gives 2^-125, not 0, for a masked column: nothing in the sum, but no
          // weight may be left on the V rows behind it
#pragma unroll
          for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if ((kPolyMask >> c) & 1u) {
                if (i * 32 + 2 * c >= valid) pk[i][c] &= 0xffff0000u;
                if (i * 32 + 2 * c + 1 >= valid) pk[i][c] &= 0xffffu;
              }
        }
        if (j > 0) {
          // P of tile j - 1 has been read
          ok = mbar_wait(o_done(g), (tiles + j - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_O);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int i = 0; i < NCH; ++i) tmem_st16(p_col + i * 16, pk[i]);
        float a0, a1;
        f32x2_split(fadd2(acc0, acc1), a0, a1);
        l_sum += a0 + a1;
        // A NaN score (or infinity - infinity) is a weight of NaN, or 3.4e38 by the polynomial's integer
        // addition; true weights stay below 2^8 (in f16 2^15), true sums below 2^31 of them.  From here on
        // the row is NaN.
        if (!(l_sum < kLost)) l_sum = NAN;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(g));
      }

      if (ok && my_nt > 0) {
        ok = mbar_wait(o_done(g), (tiles + my_nt - 1) & 1, abort, p.status, DEV_ERR_TIMEOUT_O);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      tiles += my_nt;
      // (worked out again: registers are short over the tiles)
      int again = t, tok, head;
      asm volatile("" : "+r"(again));
      const bool row_ok = row_of(again, tok, head);
      const bool sees = keys_of(row_ok, tok) > 0;
      const int64_t q_row = wk->first_q + static_cast<int64_t>(tok);
      if (splits == 1) {
        // The tile's output goes out 64 columns at a time, through shared memory, as the queries
        // came; where rows of the box are not this tile's (the sequence's last tokens, a cut
        // group's last heads) the lanes of a row store it themselves.
        // The warpgroup goes by one thread's view, so that it leaves together if the block gives up.
        int what = 0;
        const float inv_l = !sees ? 0.0f : m_ref == -INFINITY ? NAN : 1.0f / l_sum;  // (all its scores -inf: NaN)
        if (ok && p.lse && row_ok) p.lse[q_row * p.n_heads + head] = sees ? (m_ref + (log2f(l_sum) - kWeightLog2<F16>)) * 0.6931471805599453f : -INFINITY;
#pragma unroll 1
        for (int c = 0; c < L::KCH; ++c) {
          if (t == 0) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the store before has read it
            if (c == 0)
              verdict[2 * g + b] = (*abort || !some ? 1 : 0) |
                                   (wk->tok0 + (g + 1) * p.tokens <= wk->q_len && wk->heads == p.cut_heads ? 2 : 0);
          }
          warpgroup_sync();
          if (c == 0) what = verdict[2 * g + b];
          if (what & 1) break;
          if (ok && some && live) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r[32];
              if (my_nt > 0) {
                tmem_ld32(o_col + c * 64 + h * 32, r);
                tmem_wait_ld();
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  x[e] = pack_out<F16>(__uint_as_float(r[q * 8 + 2 * e]) * inv_l, __uint_as_float(r[q * 8 + 2 * e + 1]) * inv_l);
                *piece(t, h * 4 + q) = sees ? make_uint4(x[0], x[1], x[2], x[3]) : make_uint4(0, 0, 0, 0);
              }
            }
          }
          if (what & 2) {
            fence_proxy_async_smem();
            warpgroup_sync();
            if (t == 0 && ok && some) {
              asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                               reinterpret_cast<uint64_t>(&tm_o)),
                           "r"(smem_u32(so)), "r"(c * 64), "r"(wk->head0), "r"(wk->first_q + wk->tok0 + g * p.tokens)
                           : "memory");
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          } else if (ok && some && live) {
            __syncwarp();
            const int64_t at = row_ok ? q_row * p.ld_out + head * HD + c * 64 : -1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t to = __shfl_sync(0xffffffffu, at, i * 4 + lane / 8);
              if (to >= 0) reinterpret_cast<uint4*>(p.out + to)[lane % 8] = *piece((warp & 3) * 32 + i * 4 + lane / 8, lane % 8);
            }
          }
        }
        if (what & 1) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(work_read(b));
        if (!L::KEEP_ON || !keep_on) break;
      } else {
        // the part's result where the join finds it; Q, K and V have been read once all the
        // softmax warps are here
        asm volatile("bar.sync 3, %0;" ::"n"(NQ * 128) : "memory");
        if (ok && live) {
          float* od = reinterpret_cast<float*>(smem) + (g * BM + t) * L::O_PITCH;
          if (my_nt > 0) {
#pragma unroll
            for (int c0 = 0; c0 < HD; c0 += 32) {
              uint32_t r[32];
              tmem_ld32(o_col + c0, r);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; c += 4)
                *reinterpret_cast<uint4*>(od + c0 + c) = make_uint4(r[c], r[c + 1], r[c + 2], r[c + 3]);
            }
          }
          // a part in which the row saw nothing: weight 0, its O (unwritten, or a product of zeros) unread
          reinterpret_cast<float2*>(smem + L::OFF_ML)[g * BM + t] = make_float2(my_nt > 0 ? (l_sum < kLost ? m_ref : NAN) : -INFINITY, l_sum);
        }
        break;
      }
    }
    if (t == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::W_ISS) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (splits > 1) {
    cluster_sync();
    // block `rank` joins the rows r = rank, rank + splits, ...: four columns per thread
    volatile Work* wk = work_at(0);
    const int tok0 = wk->tok0, head0 = wk->head0, heads = wk->heads, q_len = wk->q_len, k_len = wk->k_len, first_q = wk->first_q;
    const int n_rows = tok0 + p.tokens < q_len ? NQ * BM : BM;
    const int n_mine = (n_rows - ip.rank + splits - 1) >> ip.log_parts;
    for (int i = threadIdx.x; i < n_mine * (HD / 4); i += L::kThreads) {
      const int r = ip.rank + (i / (HD / 4)) * splits;
      const int c = (i % (HD / 4)) * 4;
      const int rg = r & (BM - 1);
      const int of_tok = p.by_cut_heads.div(rg);
      const int tok = tok0 + (r / BM) * p.tokens + of_tok;
      const int head = head0 + rg - of_tok * p.cut_heads;
      if (of_tok >= p.tokens || tok >= q_len || head >= head0 + heads) continue;
      float2 ml[kMaxCluster];
      float4 o[kMaxCluster];
      float top = -INFINITY;
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s)
        if (s < splits) {
          ml[s] = ld_peer2(peer_smem(sb + L::OFF_ML + r * 8, s));
          o[s] = ld_peer4(peer_smem(sb + (r * L::O_PITCH + c) * 4, s));
          top = fmaxf(top, ml[s].x);
        }
      float4 a = make_float4(0, 0, 0, 0);
      float l = 0.0f;
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s)
        if (s < splits && ml[s].x != -INFINITY) {
          const float w = ex2_approx(ml[s].x - top);
          l = fmaf(w, ml[s].y, l);
          a.x = fmaf(w, o[s].x, a.x);
          a.y = fmaf(w, o[s].y, a.y);
          a.z = fmaf(w, o[s].z, a.z);
          a.w = fmaf(w, o[s].w, a.w);
        }
      const bool sees = min(k_len, keys_seen(tok, q_len, k_len, p.causal)) > 0;
      const float inv = sees ? 1.0f / l : 0.0f;
      const int64_t at = first_q + static_cast<int64_t>(tok);
      *reinterpret_cast<uint2*>(p.out + at * p.ld_out + head * HD + c) =
          make_uint2(pack_out<F16>(a.x * inv, a.y * inv), pack_out<F16>(a.z * inv, a.w * inv));
      if (p.lse && c == 0) p.lse[at * p.n_heads + head] = sees ? (top + (log2f(l) - kWeightLog2<F16>)) * 0.6931471805599453f : -INFINITY;
    }
    cluster_sync();  // no block leaves while another reads its shared memory
  }
}

template <int HD, bool F16, int N>
cudaError_t launch_n(const PackedArgs& a, cudaStream_t s) {
  using L = Lay<HD>;
  const int group = a.n_heads / a.n_kv_heads;
  PackedParams p;
  p.cuts = (group + BM - 1) / BM;
  p.cut_heads = (group + p.cuts - 1) / p.cuts;
  p.tokens = BM / p.cut_heads;
  p.n_kv = a.n_kv_heads * p.cuts;
  PackedSeqs<N> seqs;
  const int64_t tiles = plan_packed(a, 1, NQ * p.tokens, seqs);
  if (tiles < 0 || tiles * p.n_kv > INT_MAX) return cudaErrorInvalidValue;
  int dev = 0, sms = 148;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv, to;
  int64_t q_rows = 0;
  for (int i = 0; i < a.n_seqs; ++i) {
    const int64_t end = static_cast<int64_t>(a.first_q[i]) + a.q_len[i];
    q_rows = end > q_rows ? end : q_rows;
  }
  if (!encode_packed_kv(a, L::BN, F16, &tk, &tv) || !encode_tmap_16_heads(&tq, a.q, q_rows, a.n_heads, HD, a.ld_q, p.cut_heads, p.tokens, F16) ||
      !encode_tmap_16_heads(&to, a.out, q_rows, a.n_heads, HD, a.ld_out, p.cut_heads, p.tokens, F16))
    return cudaErrorInvalidValue;
  auto kernel = packed_attn_tc_kernel<HD, F16, N>;
  static std::atomic<bool> attr_set[64];
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < L::kLaunchRegs) return cudaErrorInvalidConfiguration;  // setmaxnreg.inc would wait for good
    attr_set[dev].store(true, std::memory_order_release);
  }
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.ld_out = a.ld_out;
  p.n_heads = a.n_heads;
  p.group = group;
  const Cut cut = choose_cut(a.causal, seqs, p.n_kv, L::BN, sms, L::kWhole, L::kPart, kMaxCluster);
  p.by_kv = fast_div(p.n_kv);
  p.by_cut_heads = fast_div(p.cut_heads);
  p.log_cluster = cut.log_cluster();
  p.n_cut = static_cast<int32_t>(cut.items);
  p.causal = a.causal;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.status = a.status;
  const int64_t items = tiles * p.n_kv;
  p.n_items = static_cast<int32_t>(items);
  return launch_items(kernel, cut, items, L::kThreads, L::ALLOC, s, tq, tk, tv, to, p, seqs);
}

template <int HD, bool F16>
cudaError_t launch_hd(const PackedArgs& a, cudaStream_t s) {
  return a.n_seqs <= kFewSeqs ? launch_n<HD, F16, kFewSeqs>(a, s) : launch_n<HD, F16, DP_MAX_SEQS>(a, s);
}

}  // namespace

cudaError_t launch_packed_tc(const PackedArgs& a, cudaStream_t s) {
  if (a.head_dim == 64) return a.dt == DP_F16 ? launch_hd<64, true>(a, s) : launch_hd<64, false>(a, s);
  return a.dt == DP_F16 ? launch_hd<128, true>(a, s) : launch_hd<128, false>(a, s);
}

}  // namespace dp
