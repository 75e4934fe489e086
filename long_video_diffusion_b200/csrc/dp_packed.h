// What the packed-attention kernels share: the sequences as a kernel argument, the tiles.
#pragma once

#include "dp_internal.h"

namespace dp {

// The query rows of a sequence under one k/v head are its tokens' rows of the `group` query
// heads that share it: row r is token r / group, head r % group of the group.  They are cut
// into tiles of a kernel's row count; tile0[i] is sequence i's first tile.  The host puts the
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

// Keys that token `tok` of a sequence sees.
__host__ __device__ __forceinline__ int keys_seen(int tok, int q_len, int k_len, bool causal) {
  const int n = causal ? k_len - q_len + tok + 1 : k_len;
  return n < 0 ? 0 : n;
}

// Fills s for tiles of `rows` rows; returns the number of tiles, or -1 if it passes 2^31 - 1.
int64_t plan_packed(const PackedArgs& a, int rows, int32_t* n, int32_t* tile0, int32_t* first_q, int32_t* q_len,
                    int32_t* first_k, int32_t* k_len);

template <int N>
int64_t plan_packed(const PackedArgs& a, int rows, PackedSeqs<N>& s) {
  return plan_packed(a, rows, &s.n, s.tile0, s.first_q, s.q_len, s.first_k, s.k_len);
}

constexpr int kFewSeqs = 32;  // launches of up to this many sequences carry a small argument (0.7 KB, not 20)

}  // namespace dp
