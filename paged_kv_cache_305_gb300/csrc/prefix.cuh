// Which tokens of a sequence its group's shared prefix covers.
#pragma once

#include "stream.h"

namespace pa {

// Start of group g's members, kept inside [0, num_seqs] whatever group_start holds.
__device__ __forceinline__ int group_begin(const PrefixArgs& x, int g) {
  return min(max(x.group_start[g], 0), x.num_seqs);
}

// Length of group g's prefix: what is asked for, kept inside [0, max_prefix_len]
// and the table.
__device__ __forceinline__ int group_prefix(const PrefixArgs& x, int g, int Lmax) {
  return min(min(max(x.prefix_lens[g], 0), x.max_prefix_len), Lmax);
}

// The group of sequence s: the last one that starts at or before s.
__device__ __forceinline__ int group_of(const PrefixArgs& x, int s) {
  int lo = 0, hi = x.num_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (x.group_start[mid] <= s) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Pieces that the prefix pass, where there is one, leaves for a sequence with
// `shared` tokens of prefix.
__device__ __forceinline__ int prefix_pieces(const PrefixArgs& x, int shared) {
  return x.max_chunks == 0 ? 0 : static_cast<int>((static_cast<unsigned>(shared) + x.piece_tokens - 1) / x.piece_tokens);
}

// Counts the groups whose start, size or prefix is out of range (one thread a
// group; called by one CTA).
__device__ __forceinline__ void count_bad_groups(const PrefixArgs& x, int tid, int threads,
                                                 unsigned long long* bad) {
  for (int g = tid; g < x.num_groups; g += threads) {
    const int b = x.group_start[g], e = x.group_start[g + 1], n = x.prefix_lens[g];
    if (b < 0 || e < b || e > x.num_seqs || (g == 0 && b != 0) ||
        (g == x.num_groups - 1 && e != x.num_seqs) || e - b > x.max_group_size || n < 0 ||
        n > x.max_prefix_len)
      atomicAdd(bad, 1ull);
  }
}

// Tokens of sequence s (length L) that are read through its group's table: the
// group's prefix, or 0 for a sequence that is computed alone (shorter than the
// prefix, beyond max_group_size members, or outside its group). *lead is the
// sequence whose table the prefix is read through.
__device__ __forceinline__ int prefix_of(const PrefixArgs& x, int s, int L, int Lmax, int* lead) {
  const int g = group_of(x, s);
  const int b = group_begin(x, g), e = group_begin(x, g + 1);
  *lead = s;
  if (s < b || s >= e || s - b >= x.max_group_size) return 0;
  const int n = group_prefix(x, g, Lmax);
  if (L < n) return 0;
  *lead = b;
  return n;
}

}  // namespace pa
