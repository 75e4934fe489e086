// What the packed-attention kernels share: the sequences as a kernel argument, the tiles.
#pragma once

#include "dp_device.cuh"
#include "dp_internal.h"

namespace dp {

// The query rows of a sequence under one k/v head are its tokens' rows of the `group` query
// heads that share it: row r is token r / group, head r % group of the group.  They are cut
// into a kernel's tiles; tile0[i] is sequence i's first tile.  The host puts the
// sequences with the most keys first, and a sequence's last tile (causal: the one with the
// most keys) is its first, so that the longest work starts first.
template <int N>
struct PackedSeqs {
  int32_t n;
  int32_t tile0[N + 1];
  int32_t first_q[N];
  int32_t q_len[N];
  int32_t first_k[N];
  int32_t k_len[N];
};

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (umulhi(n, m) + n) >> s.  The divisors of a launch are
// known to the host, and a block's start is a chain of these: five divisions took it 0.5 us.
struct FastDiv {
  uint32_t m, s;
  __device__ __forceinline__ int div(int n) const { return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s); }
};

inline FastDiv fast_div(uint32_t d) {
  FastDiv f = {0, 0};
  while ((1ull << f.s) < d) ++f.s;
  f.m = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.s) - d)) / d + 1);
  return f;
}

// The sequence of tile t: the last i with tile0[i] <= t.
template <int N>
__device__ __forceinline__ int seq_of_tile(const PackedSeqs<N>& s, int t) {
  int lo = 0, hi = s.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.tile0[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Two outputs.  The weights that meet the values are rounded, those in the row sum are not, so an
// output can pass the largest value by half a step of a weight, 2^-11 of it in f16; behind f16's end
// it saturates (NaN stays NaN).
template <bool F16>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  return F16 ? pack_f16x2_sat(lo, hi) : pack_bf16x2(lo, hi);
}

// Keys that token `tok` of a sequence sees.
__host__ __device__ __forceinline__ int keys_seen(int tok, int q_len, int k_len, bool causal) {
  const int n = causal ? k_len - q_len + tok + 1 : k_len;
  return n < 0 ? 0 : n;
}

// Fills s for tiles that hold `rows` of the q_len * per_token rows of a sequence; returns the number
// of tiles, or -1 if it passes 2^31 - 1.
int64_t plan_packed(const PackedArgs& a, int64_t per_token, int rows, int32_t* n, int32_t* tile0, int32_t* first_q, int32_t* q_len,
                    int32_t* first_k, int32_t* k_len);

template <int N>
int64_t plan_packed(const PackedArgs& a, int64_t per_token, int rows, PackedSeqs<N>& s) {
  return plan_packed(a, per_token, rows, &s.n, s.tile0, s.first_q, s.q_len, s.first_k, s.k_len);
}

constexpr int kFewSeqs = 32;  // launches of up to this many sequences carry a small argument (0.7 KB, not 20)

// An item is a tile of rows under one k/v head, k/v heads fastest.  The keys of the first
// n_cut items are cut into as many parts as a cluster has blocks; the clusters behind theirs
// take one whole item per block.
constexpr int kMaxCluster = 8;   // portable cluster size
constexpr int kFewCluster = 16;  // the largest there is, for the kernel for few rows

struct Cut {
  int cluster;  // a power of two
  int64_t items;
  int log_cluster() const { return cluster == 16 ? 4 : cluster == 8 ? 3 : cluster == 4 ? 2 : cluster == 2 ? 1 : 0; }
};

struct ItemPart {
  int item, rank, log_parts;
};

// log_cluster: log2 of the cluster size.  The parts' number is a power of two too.
__device__ __forceinline__ ItemPart item_part(int log_cluster, int n_cut) {
  const int c = blockIdx.x >> log_cluster, r = blockIdx.x & ((1 << log_cluster) - 1);
  if (c < n_cut) return ItemPart{c, r, log_cluster};
  return ItemPart{n_cut + ((c - n_cut) << log_cluster) + r, 0, 0};
}

// The cluster size, and with it which sequences' keys are cut, that promises the earliest end:
// an even share of all key tiles, with `whole` tiles for the start and end of a block with an item
// of its own and `part` for those of a block with a part of one, over `slots` blocks at a time; or
// the longest block, whichever is later.  per_tile: items per row tile.  Measured against every fixed
// size, 16 cases a kernel: the chosen one is within 6 % of the fastest in 13 for few rows (at worst 14 %
// behind, sizes up to 16), in 13 for many (11 %, up to 8) and in all 16 in fp32 (4 %, up to 8).
template <int N>
Cut choose_cut(bool causal, const PackedSeqs<N>& s, int64_t per_tile, int bn, int slots, int whole, int part, int most_parts) {
  auto key_tiles = [&](int i) { return (static_cast<int64_t>(s.k_len[i]) + bn - 1) / bn; };
  int64_t total = 0;
  for (int i = 0; i < s.n; ++i) {
    // causal: a sequence's row tiles see from k_len - q_len to k_len keys
    const int64_t fewest = !causal ? s.k_len[i] : s.k_len[i] > s.q_len[i] ? s.k_len[i] - s.q_len[i] : 0;
    total += (s.tile0[i + 1] - s.tile0[i]) * (((fewest + s.k_len[i]) / 2 + bn - 1) / bn);
  }
  total *= per_tile;
  const int64_t items = static_cast<int64_t>(s.tile0[s.n]) * per_tile;
  const int64_t most = key_tiles(0);
  Cut best = {1, 0};
  int64_t best_end = -1;
  for (int c = 1; c <= most_parts && (c == 1 || most >= 2 * c); c *= 2) {
    const int64_t longest = (most + c - 1) / c;
    Cut now = {c, 0};
    if (c > 1)
      for (int i = 0; i < s.n && key_tiles(i) > longest; ++i) now.items = static_cast<int64_t>(s.tile0[i + 1]) * per_tile;
    const int64_t blocks = items + now.items * (c - 1);
    int64_t share = (total + whole * (items - now.items) + part * now.items * c) / slots;
    if (blocks > slots) share = share * (8 + c) / 9;  // a cluster waits for all its blocks' places
    const int64_t last = longest + (c > 1 ? part : whole);
    const int64_t end = share > last ? share : last;
    if (best_end < 0 || end < best_end) {
      best = now;
      best_end = end;
    }
  }
  return best;
}

// Tensor maps of k and v with boxes of `box_rows` keys by 64 columns.
bool encode_packed_kv(const PackedArgs& a, int box_rows, bool f16, CUtensorMap* tk, CUtensorMap* tv);

// One block per item or part of one.
template <typename K, typename... A>
cudaError_t launch_items(K kernel, const Cut& cut, int64_t items, int threads, int smem, cudaStream_t s, const A&... args) {
  const int64_t grid = (cut.items + (items - cut.items + cut.cluster - 1) / cut.cluster) * cut.cluster;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_early(kernel, dim3(static_cast<unsigned>(grid)), threads, smem, cut.cluster, s, args...);
}

// The kernels for bf16 and f16: few rows (at most kFewRows of a sequence under one k/v head,
// dp_packed_few.cu) or many (dp_packed_tc.cu).
constexpr int kFewRows = 16;
constexpr int kFewOverhead = 6;  // key tiles that a block's start and end cost in dp_packed_few.cu
cudaError_t launch_packed_few(const PackedArgs& a, cudaStream_t s);
cudaError_t launch_packed_tc(const PackedArgs& a, cudaStream_t s);

}  // namespace dp
