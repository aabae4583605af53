// kivi_packed_quant.cu -- prompts packed into one token axis, quantized into the pages
// of their sequences in one launch (sm_103a).
//
// The method is kivi_paged_prefill's (KIVI page, headline paragraph and section "Iddia
// ve Gerceklik", paragraphs 2-3): keys per channel in G-token groups, the rest of a
// sequence's last group kept in fp16, values per token.  The work is dealt out in units of
// 64 tokens of one (sequence, KV head), which lie in one page and hold whole key groups;
// a CTA of 4 warps takes a run of neighbouring units (heads of the same tokens first), so
// that the device's lengths are searched once a CTA.  Keys and values of a unit are two
// passes.  Keys: warp w takes rows 32 (w / 2) .. + 31 and channels 64 (w % 2) .. + 63; lane
// (t4, c8) holds the 16-byte chunk c8 (8 channels) of rows t4, t4 + 4, .., so that a
// channel's min and max are two shuffle rounds (G = 64 merges two warps through shared
// memory), and derives the parameters of channel pair t4 of its chunk.  Values: a row is
// held by 4 lanes.
//
// Measured on 16 prompts of up to 8192 tokens, 8 KV heads, G = 64: 43 us, 0.55 of the measured
// copy bandwidth.  No unit is full: the integer and comparison unit is busy for 53% of the
// cycles, as is the scheduler; waits for a unit's loads, which go out when the unit before is
// stored, and for code that every warp reads anew take the rest.  Units found one by one by a CTA each took 58 us, keys held as
// column pairs of 32 rows (packed by a transpose across lanes) too; keys and values of a unit in
// one pass at five CTAs an SM 45 us; codes put together by logic instead of sums (below) 46 us;
// five to nine CTAs an SM 44 to 49 us.
#include "kivi_device.cuh"
#include "kivi_internal.h"
#include "kivi_packed.cuh"

namespace kivi {

namespace {

constexpr int kQUnit = 64, kQThreads = 128;

static_assert(kPackedMaxSeqs == kPagedMaxBatch, "a packed batch is a paged batch");
constexpr int kQCtas = 7;  // CTAs that fit on an SM (registers): a launch is one wave of them

// Where a run of units stands.
struct UnitWalk {
  const int32_t *cu;
  int n_seqs, T, cap;
  int seq, start, len, t0;  // sequence, its first row, its tokens (cut to the capacity), the unit's first

  __device__ __forceinline__ void at(int s) {
    seq = s;
    packed_bounds(cu, s, T, &start, &len);
    len = min(len, cap);
    t0 = 0;
  }
  // The next unit; there is one.
  __device__ __forceinline__ void next() {
    t0 += kQUnit;
    while (t0 >= len && seq + 1 < n_seqs) at(seq + 1);
  }
  // Every lane of a warp calls it: the units of all sequences.  Lane i sums those of `per`
  // neighbouring sequences.
  __device__ __forceinline__ int64_t begin(int *incl, int *mine) {
    const int lane = threadIdx.x & 31, per = (n_seqs + 31) / 32;
    int sum = 0;
    for (int k = 0; k < per; ++k) {
      const int s = lane * per + k;
      if (s < n_seqs) {
        int a, m;
        packed_bounds(cu, s, T, &a, &m);
        sum += (min(m, cap) + kQUnit - 1) / kQUnit;
      }
    }
    *mine = sum;
    int in = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, in, off);
      if (lane >= off) in += o;
    }
    *incl = in;
    // bounds that overlap can pass any count: cut at what lengths that do not overlap can reach
    return min((int64_t)T / kQUnit + n_seqs, (int64_t)max(__shfl_sync(0xffffffffu, in, 31), 0));
  }
  // To unit `idx` < begin(): a scan over the warp finds the lane, its sequences the unit.
  __device__ __forceinline__ void find(int64_t idx, int incl, int mine) {
    const int per = (n_seqs + 31) / 32;
    const uint32_t past = __ballot_sync(0xffffffffu, (int64_t)incl > idx);
    const int owner = past ? __ffs(past) - 1 : 31;
    int rest = (int)(idx - __shfl_sync(0xffffffffu, incl - mine, owner));
    int s = owner * per;
    at(min(s, n_seqs - 1));
    while (rest >= (len + kQUnit - 1) / kQUnit && seq + 1 < n_seqs) {
      rest -= (len + kQUnit - 1) / kQUnit;
      at(seq + 1);
    }
    t0 = rest * kQUnit;
  }
};

// The 2-bit codes of a 16-byte chunk as codes2_chunk8 gives them (channel i at bits 2i, 2i + 1 of
// 16), with the counting done in fp16: every comparison is 1 or 0, the codes of channels i and
// i + 2 are summed to 1024 + c_i + 16 c_{i+2}, an integer that fp16 holds exactly, and the low
// byte of its pattern is the two codes.  The sums run beside the comparisons and logic, whose unit is
// what bounds this kernel.
__device__ __forceinline__ uint32_t codes2_counted(const uint32_t x[4], const uint32_t X1[4], const uint32_t X2[4],
                                                   const uint32_t X3[4]) {
  const __half2 sixteen = __float2half2_rn(16.f), base = __float2half2_rn(1024.f);
  __half2 c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 v = u2h2(x[j]);
    c[j] = __hadd2(__hadd2(__hgt2(v, u2h2(X1[j])), __hgt2(v, u2h2(X2[j]))), __hgt2(v, u2h2(X3[j])));
  }
  const uint32_t a = h22u(__hfma2(c[1], sixteen, __hadd2(c[0], base)));  // channels 0, 2 | 1, 3
  const uint32_t b = h22u(__hfma2(c[3], sixteen, __hadd2(c[2], base)));  // channels 4, 6 | 5, 7
  const uint32_t w = prmt(a, b, 0x6240);                                 // even channels | odd channels
  return (w & 0x3333u) | ((w >> 14) & 0xccccu);
}

template <int BITS>
__global__ void __launch_bounds__(kQThreads, kQCtas) packed_quantize_kernel(const PackedQuantArgs a) {
  constexpr int WPR = words_per_row<BITS>();
  __shared__ uint2 s_mm[kQThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.G;
  UnitWalk u = {a.cu, a.B, a.T, a.max_pages << a.shift, 0, 0, 0, 0};
  int incl, mine;
  const int64_t items = u.begin(&incl, &mine) * a.Hkv * 2;  // keys and values of a unit apart
  const int64_t first = items * blockIdx.x / gridDim.x, end = items * (blockIdx.x + 1) / gridDim.x;
  if (first >= end) return;
  u.find(first / 2 / a.Hkv, incl, mine);
  int h = (int)(first / 2 % a.Hkv);
  for (int64_t item = first; item < end; ++item) {
    const bool keys = (item & 1) == 0;
    if (item > first && keys) ++h;
    if (h == a.Hkv) {
      h = 0;
      u.next();
    }
    const int b = u.seq, n = u.len, t0 = u.t0;
    if ((unsigned)t0 >= (unsigned)n) return;  // only where bounds overlap
    const int nq = n / G * G, rows = min(kQUnit, n - t0);
    const int nv = a.v_res ? nq : n;  // values quantized token by token
    if (keys && t0 == 0 && h == 0 && tid == 0) a.seq_lens[b] = n;
    const uint16_t *ks = a.k.p + (int64_t)(u.start + t0) * a.k.ts + (int64_t)h * a.k.hs;
    const uint16_t *vs = a.v.p + (int64_t)(u.start + t0) * a.v.ts + (int64_t)h * a.v.hs;
    const int64_t page = a.bt[(int64_t)b * a.max_pages + (t0 >> a.shift)];
    const bool paged = page >= 0 && page < a.num_pages;
    // first row of the unit in the pool (the first page when the table gives none: not written)
    const int64_t row0 = (((paged ? page : 0) * a.Hkv + h) << a.shift) + (t0 & ((1 << a.shift) - 1));

    // What fills no group stays in fp16: rows nq .. n - 1 that lie in this unit.
    auto keep = [&](const uint16_t *src, int64_t ts, uint16_t *dst) {
      for (int it = tid; it < kQUnit * (kD / 8); it += kQThreads) {
        const int r = it / (kD / 8), c = it % (kD / 8);
        if (t0 + r < nq || r >= rows) continue;
        *reinterpret_cast<uint4 *>(dst + (((int64_t)b * a.Hkv + h) * G + (t0 + r - nq)) * kD + 8 * c) =
            __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)r * ts) + c);
      }
    };
    if (keys) {
      const int rh = warp >> 1, ch = warp & 1, t4 = lane >> 3, c8 = lane & 7;
      uint32_t x[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int row = 32 * rh + t4 + 4 * k;
        const uint4 c = row < rows ? __ldg(reinterpret_cast<const uint4 *>(ks + (int64_t)row * a.k.ts) + 8 * ch + c8)
                                   : make_uint4(0u, 0u, 0u, 0u);
        x[k][0] = c.x;
        x[k][1] = c.y;
        x[k][2] = c.z;
        x[k][3] = c.w;
      }
      // ---- key groups
      __half2 mn[4], mx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mn[j] = mx[j] = u2h2(x[0][j]);
#pragma unroll
        for (int k = 1; k < 8; ++k) {
          mn[j] = __hmin2(mn[j], u2h2(x[k][j]));
          mx[j] = __hmax2(mx[j], u2h2(x[k][j]));
        }
#pragma unroll
        for (int off = 8; off < 32; off <<= 1) {
          mn[j] = __hmin2(mn[j], u2h2(__shfl_xor_sync(0xffffffffu, h22u(mn[j]), off)));
          mx[j] = __hmax2(mx[j], u2h2(__shfl_xor_sync(0xffffffffu, h22u(mx[j]), off)));
        }
      }
      // this lane's channel pair: t4 of the chunk (channels 8 c8 + 2 t4, + 1)
      __half2 pmn = mn[0], pmx = mx[0];
#pragma unroll
      for (int j = 1; j < 4; ++j)
        if (t4 == j) {
          pmn = mn[j];
          pmx = mx[j];
        }
      if (G == 64) {  // uniform over the CTA
        __syncthreads();  // the unit before has read its own
        s_mm[tid] = make_uint2(h22u(pmn), h22u(pmx));
        __syncthreads();
        const uint2 o = s_mm[tid ^ 64];
        pmn = __hmin2(pmn, u2h2(o.x));
        pmx = __hmax2(pmx, u2h2(o.y));
      }
      const int g0 = G == 32 ? 32 * rh : 0;           // first row of the warp's group in the unit
      if (paged && t0 + g0 + G <= nq) {               // a quantized group (not the residual)
        const QParams p0 = make_qparams<BITS>(__low2float(pmn), __low2float(pmx));
        const QParams p1 = make_qparams<BITS>(__high2float(pmn), __high2float(pmx));
        if (G == 32 || rh == 0)
          *reinterpret_cast<uint2 *>(a.k_meta + ((row0 + g0) / G) * kD + 64 * ch + 8 * c8 + 2 * t4) =
              make_uint2(p0.meta, p1.meta);
        uint32_t *codes = a.k_codes + (row0 + 32 * rh + t4) * WPR;
        if constexpr (BITS == 4) {
          // every channel of the chunk: pair j from lane 8 j + c8 (1/s, 0 where s = 0)
          const float rs0 = p0.s == 0.f ? 0.f : __frcp_rn(p0.s), rs1 = p1.s == 0.f ? 0.f : __frcp_rn(p1.s);
          float2 cmn[4], cs[4], crs[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int sl = 8 * j + c8;
            cmn[j] = make_float2(__shfl_sync(0xffffffffu, p0.mn, sl), __shfl_sync(0xffffffffu, p1.mn, sl));
            cs[j] = make_float2(__shfl_sync(0xffffffffu, p0.s, sl), __shfl_sync(0xffffffffu, p1.s, sl));
            crs[j] = make_float2(__shfl_sync(0xffffffffu, rs0, sl), __shfl_sync(0xffffffffu, rs1, sl));
          }
          // chunk c8 of channel half ch is word 8 ch + c8 of a token row
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) word |= code4x2(__half22float2(u2h2(x[k][j])), cmn[j], cs[j], crs[j]) << (8 * j);
            codes[4 * k * WPR + 8 * ch + c8] = word;
          }
        } else {
          uint32_t a1, a2, a3, b1, b2, b3;
          bool oa, ob;
          fp16_thresholds(p0, a1, a2, a3, oa);
          fp16_thresholds(p1, b1, b2, b3, ob);
          uint32_t r[8];
          if (__all_sync(0xffffffffu, oa && ob)) {
            const uint32_t P1 = a1 | (b1 << 16), P2 = a2 | (b2 << 16), P3 = a3 | (b3 << 16);
            uint32_t T1[4], T2[4], T3[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // pair j of the chunk lives in lane 8 j + c8
              T1[j] = __shfl_sync(0xffffffffu, P1, 8 * j + c8);
              T2[j] = __shfl_sync(0xffffffffu, P2, 8 * j + c8);
              T3[j] = __shfl_sync(0xffffffffu, P3, 8 * j + c8);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = codes2_counted(x[k], T1, T2, T3);
          } else {
            // the fp32 comparison form with every channel's parameters of the chunk
            float qm[8], q1[8], q2[8], q3[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int sl = 8 * (j / 2) + c8;
              const QParams &p = j & 1 ? p1 : p0;
              qm[j] = __shfl_sync(0xffffffffu, p.mn, sl);
              q1[j] = __shfl_sync(0xffffffffu, p.t1, sl);
              q2[j] = __shfl_sync(0xffffffffu, p.t2, sl);
              q3[j] = __shfl_sync(0xffffffffu, p.t3, sl);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              r[k] = 0;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float d = __fsub_rn(h2f((uint16_t)(x[k][j / 2] >> (16 * (j & 1)))), qm[j]);
                r[k] |= ((uint32_t)(d > q1[j]) + (uint32_t)(d >= q2[j]) + (uint32_t)(d > q3[j])) << (2 * j);
              }
            }
          }
          // chunks 2m and 2m + 1 (lanes c8, c8 ^ 1) are the halves of word 4 ch + m of a token
          // row: the even lane stores rows t4 + 8 i, the odd one rows t4 + 8 i + 4
          const bool odd = c8 & 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? r[2 * i] : r[2 * i + 1], 1);
            const uint32_t lo = odd ? got : r[2 * i], hi = odd ? r[2 * i + 1] : got;
            codes[(8 * i + (odd ? 4 : 0)) * WPR + 4 * ch + (c8 >> 1)] = __byte_perm(lo, hi, 0x5410);
          }
        }
      }
      if (t0 + rows > nq) keep(ks, a.k.ts, a.k_res);
    } else {
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
              c[k] = codes2_counted(w, X1, X2, X3);
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
      if (a.v_res && t0 + rows > nq) keep(vs, a.v.ts, a.v_res);
    }
  }
}

}  // namespace

cudaError_t launch_packed_quantize(const PackedQuantArgs &a, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int64_t items = ((int64_t)a.T / kQUnit + a.B) * a.Hkv * 2, wave = (int64_t)sms * kQCtas;
  const unsigned grid = (unsigned)(items < wave ? items : wave);
  if (a.bits == 2)
    packed_quantize_kernel<2><<<grid, kQThreads, 0, st>>>(a);
  else
    packed_quantize_kernel<4><<<grid, kQThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kivi
