// kivi_packed_quant.cu -- prompts packed into one token axis, quantized into the pages
// of their sequences in one launch (sm_103a).
//
// The method is kivi_paged_prefill's (KIVI page, headline paragraph and section "Iddia
// ve Gerceklik", paragraphs 2-3): keys per channel in G-token groups, the rest of a
// sequence's last group kept in fp16, values per token.  One CTA of 4 warps takes 64
// tokens of one (sequence, KV head), which lie in one page and hold whole key groups.
// Thread (rh, cp) holds channels 2cp, 2cp + 1 of token rows 32 rh .. 32 rh + 31, so a
// channel's min and max need no shuffle (G = 64 merges two threads); a row of values is
// held by 4 lanes.
#include "kivi_device.cuh"
#include "kivi_internal.h"
#include "kivi_packed.cuh"

namespace kivi {

namespace {

constexpr int kQUnit = 64, kQThreads = 128;

// Unit `idx` (kQUnit tokens) of the sequences' units in order, sequences cut to `cap`
// tokens: lane i sums the units of 16 consecutive sequences, a warp scan finds the
// lane, its own sequences the unit.  Every lane of a warp calls it.
__device__ __forceinline__ bool packed_unit(const int32_t *cu, int n_seqs, int T, int cap, unsigned idx,
                                            PackedBlock *out) {
  constexpr int kPer = kPackedMaxSeqs / 32;
  const int lane = threadIdx.x & 31;
  const int per = (n_seqs + 31) / 32;
  int nu[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    nu[k] = 0;
    if (k < per) {
      const int s = lane * per + k;
      if (s < n_seqs) {
        int start, len;
        packed_bounds(cu, s, T, &start, &len);
        nu[k] = (min(len, cap) + kQUnit - 1) / kQUnit;
        sum += nu[k];
      }
    }
  }
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  const uint32_t past = __ballot_sync(0xffffffffu, (unsigned)incl > idx);
  if (past == 0) return false;
  const int owner = __ffs(past) - 1;
  int rest = (int)idx - (incl - sum), seq = 0;
  bool found = false;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (k < per && !found) {
      if (rest < nu[k]) {
        found = true;
        seq = lane * per + k;
      } else {
        rest -= nu[k];
      }
    }
  }
  seq = __shfl_sync(0xffffffffu, seq, owner);
  rest = __shfl_sync(0xffffffffu, rest, owner);
  if (seq >= n_seqs || rest < 0) return false;
  out->seq = seq;
  packed_bounds(cu, seq, T, &out->start, &out->len);
  out->len = min(out->len, cap);
  out->level = rest;
  return (int64_t)rest * kQUnit < out->len;
}

template <int BITS>
__global__ void __launch_bounds__(kQThreads) packed_quantize_kernel(const PackedQuantArgs a) {
  constexpr int WPR = words_per_row<BITS>();
  constexpr int LPW = 16 / BITS;  // channel pairs per packed word
  __shared__ uint2 s_mm[kQThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, G = a.G;
  PackedBlock blk;
  if (!packed_unit(a.cu, a.B, a.T, a.max_pages << a.shift, blockIdx.x, &blk)) return;
  const int b = blk.seq, n = blk.len, t0 = blk.level * kQUnit;
  const int nq = n / G * G, rows = min(kQUnit, n - t0);
  const int nv = a.v_res ? nq : n;  // values quantized token by token
  if (t0 == 0 && h == 0 && tid == 0) a.seq_lens[b] = n;
  const uint16_t *ks = a.k.p + (int64_t)(blk.start + t0) * a.k.ts + (int64_t)h * a.k.hs;
  const uint16_t *vs = a.v.p + (int64_t)(blk.start + t0) * a.v.ts + (int64_t)h * a.v.hs;
  const int64_t page = a.bt[(int64_t)b * a.max_pages + (t0 >> a.shift)];
  const bool paged = page >= 0 && page < a.num_pages;
  // first row of the unit in the pool (the first page when the table gives none: not written)
  const int64_t row0 = (((paged ? page : 0) * a.Hkv + h) << a.shift) + (t0 & ((1 << a.shift) - 1));

  // ---- all loads of the unit: keys by column pair, values by row
  const int cp = tid & 63, rh = tid >> 6;
  uint32_t x[32];
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    const int row = 32 * rh + r;
    x[r] = row < rows ? __ldg(reinterpret_cast<const uint32_t *>(ks + (int64_t)row * a.k.ts) + cp) : 0u;
  }
  const int q = lane & 3;
  uint4 y[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 32 * i + 8 * warp + (lane >> 2);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[i][k] = row < rows ? __ldg(reinterpret_cast<const uint4 *>(vs + (int64_t)row * a.v.ts) + q + 4 * k)
                           : make_uint4(0u, 0u, 0u, 0u);
  }
  // ---- key groups
  __half2 mn = u2h2(x[0]), mx = mn;
#pragma unroll
  for (int r = 1; r < 32; ++r) {
    mn = __hmin2(mn, u2h2(x[r]));
    mx = __hmax2(mx, u2h2(x[r]));
  }
  if (G == 64) {  // uniform over the CTA
    s_mm[tid] = make_uint2(h22u(mn), h22u(mx));
    __syncthreads();
    const uint2 o = s_mm[tid ^ 64];
    mn = __hmin2(mn, u2h2(o.x));
    mx = __hmax2(mx, u2h2(o.y));
  }
  const int g0 = G == 32 ? 32 * rh : 0;               // first row of this thread's group in the unit
  const bool whole = paged && t0 + g0 + G <= nq;      // a quantized group (not the residual)
  key_pair_codes<BITS>(x, mn, mx, lane, whole, G == 32 || rh == 0, a.k_meta + ((row0 + g0) / G) * kD + 2 * cp,
                       a.k_codes + (row0 + 32 * rh) * WPR + cp / LPW);
  // ---- the residual: rows nq .. n - 1 that lie in this unit
  for (int it = tid; it < kQUnit * (kD / 8); it += kQThreads) {
    const int r = it / (kD / 8), ch = it % (kD / 8);
    if (t0 + r < nq || r >= rows) continue;
    const int64_t dst = (((int64_t)b * a.Hkv + h) * G + (t0 + r - nq)) * kD + 8 * ch;
    *reinterpret_cast<uint4 *>(a.k_res + dst) = __ldg(reinterpret_cast<const uint4 *>(ks + (int64_t)r * a.k.ts) + ch);
    if (a.v_res)
      *reinterpret_cast<uint4 *>(a.v_res + dst) = __ldg(reinterpret_cast<const uint4 *>(vs + (int64_t)r * a.v.ts) + ch);
  }
  // ---- value rows: lane q of a row holds chunks q + 4k (8 channels each)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 32 * i + 8 * warp + (lane >> 2);
    const bool ok_row = paged && t0 + r < nv;
    __half2 vmn = u2h2(y[i][0].x), vmx = vmn;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w[4] = {y[i][k].x, y[i][k].y, y[i][k].z, y[i][k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        vmn = __hmin2(vmn, u2h2(w[j]));
        vmx = __hmax2(vmx, u2h2(w[j]));
      }
    }
    // (min, -max) so that one __hmin2 reduces both over the row's 4 lanes
    __half2 red = __halves2half2(__hmin(__low2half(vmn), __high2half(vmn)),
                                 __hneg(__hmax(__low2half(vmx), __high2half(vmx))));
    red = __hmin2(red, u2h2(__shfl_xor_sync(0xffffffffu, h22u(red), 1)));
    red = __hmin2(red, u2h2(__shfl_xor_sync(0xffffffffu, h22u(red), 2)));
    const QParams p = make_qparams<BITS>(__low2float(red), -__high2float(red));
    uint32_t *codes_row = a.v_codes + (row0 + r) * WPR;
    if constexpr (BITS == 4) {
      if (ok_row) {
#pragma unroll
        for (int k = 0; k < 4; ++k) codes_row[q + 4 * k] = qchunk8<4>(y[i][k], p);
      }
    } else {
      // lane q < 3 proves threshold q + 1 of the row (the second is the strict one)
      bool ok = true;
      uint32_t xq = 0x7c00u;
      if (p.s != 0.f && q < 3) xq = fp16_threshold(p.mn, q == 0 ? p.t1 : (q == 1 ? p.t2 : p.t3), q == 1, ok);
      const int base = lane & ~3;
      const uint32_t x1 = __shfl_sync(0xffffffffu, xq, base), x2 = __shfl_sync(0xffffffffu, xq, base + 1),
                     x3 = __shfl_sync(0xffffffffu, xq, base + 2);
      uint32_t c[4];
      if (__all_sync(0xffffffffu, ok)) {
        const uint32_t p1 = x1 | (x1 << 16), p2 = x2 | (x2 << 16), p3 = x3 | (x3 << 16);
        const uint32_t X1[4] = {p1, p1, p1, p1}, X2[4] = {p2, p2, p2, p2}, X3[4] = {p3, p3, p3, p3};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w[4] = {y[i][k].x, y[i][k].y, y[i][k].z, y[i][k].w};
          c[k] = codes2_chunk8(w, X1, X2, X3);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = quant_chunk8<2>(y[i][k], p);
      }
      // word w = chunk 2w | chunk 2w + 1 << 16: lanes q, q ^ 1 hold the halves of words
      // q / 2 + 2k; the even lane stores k = 0, 1, the odd one k = 2, 3
      const uint32_t A = __byte_perm(c[0], c[1], 0x5410), B = __byte_perm(c[2], c[3], 0x5410);
      const uint32_t recv = __shfl_xor_sync(0xffffffffu, (q & 1) ? A : B, 1);
      const uint32_t lo = (q & 1) ? recv : A, hi = (q & 1) ? B : recv;
      if (ok_row) {
        const int w = (q >> 1) + ((q & 1) ? 4 : 0);
        codes_row[w] = __byte_perm(lo, hi, 0x5410);
        codes_row[w + 2] = __byte_perm(lo, hi, 0x7632);
      }
    }
    if (ok_row && q == 0) a.v_meta[row0 + r] = p.meta;
  }
}

}  // namespace

cudaError_t launch_packed_quantize(const PackedQuantArgs &a, cudaStream_t st) {
  const dim3 grid((unsigned)(a.T / kQUnit + a.B), (unsigned)a.Hkv);
  if (a.bits == 2)
    packed_quantize_kernel<2><<<grid, kQThreads, 0, st>>>(a);
  else
    packed_quantize_kernel<4><<<grid, kQThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kivi
