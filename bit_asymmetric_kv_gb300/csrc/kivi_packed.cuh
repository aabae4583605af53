// kivi_packed.cuh -- prompts packed into one token axis: which rows a CTA takes.
//
// Sequence s is rows start_s .. start_s + len_s - 1 of the token axis, read from the
// bounds cu[s], cu[s + 1] on the device.  The host does not see them, so they are
// clamped here: start into [0, T], end into [start, T].
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kivi {

constexpr int kPackedMaxSeqs = 512;

struct PackedBlock {
  int seq;      // sequence
  int start;    // its first row in the token axis
  int len;      // its rows
  int level;    // which block of the sequence
};

__device__ __forceinline__ void packed_bounds(const int32_t *cu, int s, int T, int *start, int *len) {
  const int a = min(max(__ldg(cu + s), 0), T);
  *start = a;
  *len = min(max(__ldg(cu + s + 1), a), T) - a;
}

// Block `idx` of all sequences' blocks of `bt` rows, longest first: the blocks of
// level L (the L-th of their sequence, whose causal rows see L + 1 blocks of keys) come
// before those of level L - 1, and within a level in the order of the sequences.
// f(L) = sum_s max(0, blocks_s - L) blocks have level L or more, so the level of `idx`
// is the largest L with f(L) > idx: a binary search, each step one sum over the warp.
// Every lane of a warp calls it; false when there is no such block (or the bounds
// overlap so that the sums overflow: nothing outside a sequence is ever returned).
__device__ __forceinline__ bool packed_block(const int32_t *cu, int n_seqs, int T, int bt, unsigned idx,
                                             PackedBlock *out) {
  const int lane = threadIdx.x & 31;
  int nb[kPackedMaxSeqs / 32];
  int most = 0;
#pragma unroll
  for (int k = 0; k < kPackedMaxSeqs / 32; ++k) {
    nb[k] = 0;
    if (32 * k < n_seqs) {
      const int s = 32 * k + lane;
      if (s < n_seqs) {
        int start, len;
        packed_bounds(cu, s, T, &start, &len);
        nb[k] = len / bt + (len % bt != 0);
        most = max(most, nb[k]);
      }
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  auto f = [&](int L) {
    unsigned c = 0;
#pragma unroll
    for (int k = 0; k < kPackedMaxSeqs / 32; ++k)
      if (32 * k < n_seqs) c += (unsigned)max(nb[k] - L, 0);
    return __reduce_add_sync(0xffffffffu, c);
  };
  if (most == 0 || f(0) <= idx) return false;
  int lo = 0, hi = most;  // f(lo) > idx >= f(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (f(mid) > idx)
      lo = mid;
    else
      hi = mid;
  }
  unsigned rank = idx - f(lo + 1);  // among the sequences with more than lo blocks
  int found = -1;
#pragma unroll
  for (int k = 0; k < kPackedMaxSeqs / 32; ++k) {
    if (32 * k < n_seqs) {
      const uint32_t m = __ballot_sync(0xffffffffu, nb[k] > lo);
      const unsigned c = __popc(m);
      if (found < 0) {
        if (rank < c)
          found = 32 * k + (int)__fns(m, 0, (int)rank + 1);
        else
          rank -= c;
      }
    }
  }
  if (found < 0 || found >= n_seqs) return false;
  out->seq = found;
  packed_bounds(cu, found, T, &out->start, &out->len);
  out->level = lo;
  return (int64_t)lo * bt < out->len;
}

}  // namespace kivi
