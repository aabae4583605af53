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

// All sequences' blocks of `bt` rows, longest first: the blocks of level L (the L-th of
// their sequence, whose causal rows see L + 1 blocks of keys) come before those of level
// L - 1.  With the sequences sorted by their number of blocks, nb_1 >= nb_2 >= ..., the
// levels from nb_{j+1} to nb_j - 1 have one block of each of the first j sequences, and
//   C_j = sum_{i <= j} (nb_i - nb_j)
// blocks come before them, so that block `item` is found by a binary search in C and one
// division.  Kept in shared memory, built once by a CTA.
struct PackedList {
  int nb[kPackedMaxSeqs];             // blocks of the j-th longest sequence
  int before[kPackedMaxSeqs];         // C_j
  int start[kPackedMaxSeqs], len[kPackedMaxSeqs];  // by sequence, as given
  int work[kPackedMaxSeqs];           // blocks by sequence, as given
  uint16_t order[kPackedMaxSeqs];     // sequence of rank j
  int n, total;

  // Every thread of the CTA calls it; synchronises.
  __device__ __forceinline__ void build(const int32_t *cu, int n_seqs, int T, int bt) {
    const int tid = threadIdx.x;
    for (int s = tid; s < n_seqs; s += blockDim.x) {
      int a, m;
      packed_bounds(cu, s, T, &a, &m);
      start[s] = a;
      len[s] = m;
      work[s] = m / bt + (m % bt != 0);
    }
    __syncthreads();
    for (int s = tid; s < n_seqs; s += blockDim.x) {
      const int mine = work[s];
      int rank = 0;
#pragma unroll 8
      for (int o = 0; o < n_seqs; ++o) {
        const int other = work[o];
        rank += other > mine || (other == mine && o < s);
      }
      nb[rank] = mine;
      order[rank] = (uint16_t)s;
    }
    __syncthreads();
    if (tid < 32) {
      // sums up to each rank, 32 at a time; bounds that overlap may pass any count: cut at
      // what lengths that do not overlap can reach
      const int64_t most = (int64_t)T / bt + n_seqs;
      int64_t carry = 0;
      for (int j0 = 0; j0 < n_seqs; j0 += 32) {
        const int j = j0 + tid, mine = j < n_seqs ? nb[j] : 0;
        int64_t sum = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t o = __shfl_up_sync(0xffffffffu, sum, off);
          if (tid >= off) sum += o;
        }
        sum += carry;
        if (j < n_seqs) before[j] = (int)min(most, sum - (int64_t)(j + 1) * mine);
        carry = __shfl_sync(0xffffffffu, sum, 31);
      }
      if (tid == 0) {
        n = n_seqs;
        total = (int)min(most, carry);
      }
    }
    __syncthreads();
  }

  // Block `item` < total.
  __device__ __forceinline__ PackedBlock find(unsigned item) const {
    int lo = 0, hi = n;  // before[lo] <= item < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((unsigned)before[mid] <= item)
        lo = mid;
      else
        hi = mid;
    }
    const unsigned rest = item - before[lo], width = lo + 1, down = rest / width;
    PackedBlock b;
    b.seq = order[rest - down * width];
    b.start = start[b.seq];
    b.len = len[b.seq];
    b.level = max(nb[lo] - 1 - (int)down, 0);
    return b;
  }
};

}  // namespace kivi
