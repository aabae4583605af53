// kivi_packed_attention.cu -- causal attention over prompts of different lengths packed
// into one token axis (sm_103a).
//
// For row i of a sequence (rows counted from its start) and query head h, reading KV
// head h / (Hq / Hkv):
//   out_i = sum_{j <= i} softmax_j(sigma q_i . k_j) v_j,   j over the same sequence.
// One CTA takes 16 query rows of one head and walks the sequence's keys in tiles of 32
// with a running maximum and sum (fp32 throughout, the output rounded once to fp16).
#include <math.h>

#include "kivi_device.cuh"
#include "kivi_internal.h"
#include "kivi_packed.cuh"

namespace kivi {

namespace {

constexpr int kARows = 16, kAKeys = 32, kAThreads = 256;

__global__ void __launch_bounds__(kAThreads) packed_attention_kernel(const PackedAttentionArgs a) {
  __shared__ float sq[kARows][kD], sk[kAKeys][kD + 1], sv[kAKeys][kD], sp[kARows][kAKeys];
  const int tid = threadIdx.x;
  const int h = (int)(blockIdx.x % (unsigned)a.Hq);
  PackedBlock blk;
  if (!packed_block(a.cu, a.n_seqs, a.T, kARows, blockIdx.x / (unsigned)a.Hq, &blk)) return;
  const int kvh = h / (a.Hq / a.Hkv);
  const int r0 = blk.level * kARows;
  const int rows = min(kARows, blk.len - r0);
  auto at = [](const PackedRows &x, int64_t tok, int head) { return x.p + tok * x.ts + head * x.hs; };
  for (int i = tid; i < kARows * kD; i += kAThreads) {
    const int r = i / kD, c = i % kD;
    sq[r][c] = r < rows ? h2f(at(a.q, blk.start + r0 + r, h)[c]) : 0.f;
  }
  const int row = tid >> 4, c0 = (tid & 15) * 8;
  float o[8] = {}, m = -INFINITY, l = 0.f;
  for (int k0 = 0; k0 < r0 + rows; k0 += kAKeys) {
    __syncthreads();
    for (int i = tid; i < kAKeys * kD; i += kAThreads) {
      const int r = i / kD, c = i % kD;
      const bool ok = k0 + r < r0 + rows;
      sk[r][c] = ok ? h2f(at(a.k, blk.start + k0 + r, kvh)[c]) : 0.f;
      sv[r][c] = ok ? h2f(at(a.v, blk.start + k0 + r, kvh)[c]) : 0.f;
    }
    __syncthreads();
    // thread (row, t): keys t and t + 16
    float s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int key = (tid & 15) + 16 * e;
      float acc = 0.f;
      for (int c = 0; c < kD; ++c) acc += sq[row][c] * sk[key][c];
      s[e] = k0 + key > r0 + row ? -INFINITY : acc * a.softmax_scale;
    }
    float mx = fmaxf(s[0], s[1]);
    for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float mn = fmaxf(m, mx);  // finite: key 0 is in the first tile of every row
    const float al = expf(m - mn);
    m = mn;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float p = expf(s[e] - m);
      sp[row][(tid & 15) + 16 * e] = p;
      sum += p;
    }
    for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    l = l * al + sum;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] *= al;
    for (int key = 0; key < kAKeys; ++key) {
      const float p = sp[row][key];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += p * sv[key][c0 + j];
    }
  }
  if (row < rows) {
    uint16_t *dst = a.out.p + (int64_t)(blk.start + r0 + row) * a.out.ts + (int64_t)h * a.out.hs + c0;
    const float inv = 1.f / l;
#pragma unroll
    for (int j = 0; j < 8; ++j) dst[j] = f2h(o[j] * inv);
  }
}

}  // namespace

static int64_t grid_of(const PackedAttentionArgs &a) { return ((int64_t)a.T / kARows + a.n_seqs) * a.Hq; }

bool packed_attention_fits(const PackedAttentionArgs &a) { return grid_of(a) <= 0x7fffffff; }

cudaError_t launch_packed_attention(const PackedAttentionArgs &a, cudaStream_t st) {
  packed_attention_kernel<<<(unsigned)grid_of(a), kAThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kivi
