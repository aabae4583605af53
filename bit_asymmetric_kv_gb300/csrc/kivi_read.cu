// kivi_read.cu -- tokens of a paged cache read back as fp16 rows of a token axis (sm_103a).
//
// Of sequence b's n tokens, c are taken: the first f = min(first, c), then the newest c - f, into the
// rows of the sequence one after the other.  A quantized element is z + code * s, the exact product and
// one rounding to fp16 (a half-precision fused multiply-add); beyond fp16's largest finite value it is that
// value, so that the rows can be attended to.  Residual tokens are copied.
//
// What bounds it: 512 bytes are written for every token and KV head, and 64 to 136 read, and this GPU writes
// alone at 3.6 to 4.0 TB/s (cudaMemset's rate too; a copy moves 6.8, half of it reads).  32 sequences' 4099
// tokens and 8 KV heads, 2-bit codes: 290 MB written in 68 us, 4.3 TB/s with what stays in L2.  The work is
// dealt out in items of 32 positions of one KV head, keys and values, one warp each: a warp writes two
// whole rows (512 bytes) at once, lane (t, c) chunk c of 8 channels of row t, so that the scales of a
// key group's channels are read once an item and stay in registers.  The warps of a CTA take heads side by
// side, so that the heads of a token, neighbours in memory, are written at about the same time (each warp a
// run of its own: 80 us; four warps a CTA: 74).  More of an item's loads in flight, at fewer CTAs, were
// slower (79 us).
#include "kivi_device.cuh"
#include "kivi_internal.h"
#include "kivi_packed.cuh"

namespace kivi {

namespace {

constexpr int kBlock = 32, kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtas = 4;  // CTAs of an SM in one wave (registers)

// What is read of one sequence: positions 0 .. f - 1, then from .. n - 1, to rows row, row + 1, ..
struct Piece {
  int row, f, from, n;
  __device__ __forceinline__ int head_blocks() const { return (f + kBlock - 1) / kBlock; }
  __device__ __forceinline__ int blocks() const {
    return head_blocks() + (n > from ? (n + kBlock - 1) / kBlock - from / kBlock : 0);
  }
};

__device__ __forceinline__ Piece piece_of(const ReadArgs &a, int b) {
  Piece p;
  int room;
  packed_bounds(a.cu, b, a.T, &p.row, &room);
  p.n = min(max(a.seq_lens[b], 0), a.max_pages << a.shift);
  const int c = min(min(room, p.n), a.take ? max(a.take[b], 0) : room);
  p.f = min(a.first, c);
  p.from = p.n - (c - p.f);
  return p;
}

// The 8 elements of a chunk from its codes (element i at bits BITS * i): z + code * s, of scale and zero
// pairs s[j], z[j], at most the largest fp16 (the smallest is z: scales are not negative).
// A code is masked into the mantissa of 1024, at bit 0, 4 or 8: 1024 + 16^i code, which one
// multiply-add brings to the code, exactly.
template <int BITS>
__device__ __forceinline__ uint4 widen(uint32_t w, const __half2 s[4], const __half2 z[4]) {
  const uint32_t b = 0x64006400u;
  const __half2 m1024 = u2h2(0xe400e400u), m64 = u2h2(0xd400d400u), m4 = u2h2(0xc400c400u);  // -1024 / 16^i
  const __half2 i16 = u2h2(0x2c002c00u), i256 = u2h2(0x1c001c00u);                           // 1 / 16, 1 / 256
  __half2 c[4];
  if constexpr (BITS == 2) {
    // codes 2 j (low half) and 2 j + 1 (high half) at bits 4 j; bits 14 and 15 of the low half are mixed up
    const uint32_t y = w | (w << 14), y3 = y >> 8;
    c[0] = __hadd2(u2h2((y & 0x00030003u) | b), m1024);
    c[1] = __hfma2(u2h2((y & 0x00300030u) | b), i16, m64);
    c[2] = __hfma2(u2h2((y & 0x03000300u) | b), i256, m4);
    c[3] = __hfma2(u2h2((y3 & 0x00300030u) | b), i16, m64);
  } else {
    // codes j and j + 4, brought beside their neighbours below
    const uint32_t y = w >> 8;
    c[0] = __hadd2(u2h2((w & 0x000f000fu) | b), m1024);
    c[1] = __hfma2(u2h2((w & 0x00f000f0u) | b), i16, m64);
    c[2] = __hadd2(u2h2((y & 0x000f000fu) | b), m1024);
    c[3] = __hfma2(u2h2((y & 0x00f000f0u) | b), i16, m64);
    const uint32_t a = h22u(c[0]), d = h22u(c[1]), e = h22u(c[2]), f = h22u(c[3]);
    c[0] = u2h2(prmt(a, d, 0x5410u));
    c[1] = u2h2(prmt(e, f, 0x5410u));
    c[2] = u2h2(prmt(a, d, 0x7632u));
    c[3] = u2h2(prmt(e, f, 0x7632u));
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[j] = h22u(__hmin2(__hfma2(c[j], s[j], z[j]), u2h2(0x7bff7bffu)));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, kCtas) paged_read_kernel(const ReadArgs a) {
  constexpr int WPR = words_per_row<BITS>();
  const int lane = threadIdx.x & 31, t = lane >> 4, c = lane & 15;
  const int per = (a.B + 31) / 32, P = 1 << a.shift;
  // blocks of all sequences; lane i sums those of `per` neighbouring ones
  int mine = 0;
  for (int k = 0; k < per; ++k)
    if (lane * per + k < a.B) mine += piece_of(a, lane * per + k).blocks();
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  // bounds that overlap can pass any count: cut at what lengths that do not overlap can reach
  const int64_t most = (int64_t)a.T / kBlock + 4 * a.B;
  const int64_t blocks = min(most, (int64_t)max(__shfl_sync(0xffffffffu, incl, 31), 0));
  const int64_t items = blocks * a.Hkv;
  const int64_t first = items * blockIdx.x / gridDim.x + (threadIdx.x >> 5), end = items * (blockIdx.x + 1) / gridDim.x;
  if (first >= end) return;
  int64_t at = first / a.Hkv;
  int h = (int)(first - at * a.Hkv);
  const uint32_t past = __ballot_sync(0xffffffffu, (int64_t)incl > at);
  const int owner = past ? __ffs(past) - 1 : 31;
  int blk = (int)(at - __shfl_sync(0xffffffffu, incl - mine, owner));
  int b = min(owner * per, a.B - 1);
  Piece p = piece_of(a, b);
  for (int64_t item = first; item < end; item += kWarps, h += kWarps) {
    while (h >= a.Hkv) {
      h -= a.Hkv;
      ++blk;
    }
    while (blk >= p.blocks()) {
      if (b + 1 >= a.B) return;  // only where bounds overlap
      blk -= p.blocks();
      p = piece_of(a, ++b);
    }
    // positions lo .. hi - 1 of the block that starts at t0, to rows from `row` on
    const int hb = p.head_blocks();
    const bool head = blk < hb;
    const int t0 = head ? blk * kBlock : (p.from / kBlock + blk - hb) * kBlock;
    const int lo = head ? t0 : max(p.from, t0), hi = min(head ? p.f : p.n, t0 + kBlock);
    const int64_t row = (int64_t)p.row + (head ? lo : p.f + lo - p.from) - (lo - t0);  // of position t0
    const int nq = p.n / a.G * a.G;
    const bool late = t0 >= nq;  // in the residual
    const int64_t page = a.bt[(int64_t)b * a.max_pages + (t0 >> a.shift)];
    const bool paged = page >= 0 && page < a.num_pages;
    // first row of the block in the pool (the first page when the table gives none: zeros are written)
    const int64_t row0 = (((paged ? page : 0) * a.Hkv + h) << a.shift) + (t0 & (P - 1));
    const int64_t res0 = ((int64_t)b * a.Hkv + h) * a.G + (t0 - nq);
    uint16_t *ko = a.k.p + row * a.k.ts + (int64_t)h * a.k.hs + 8 * c, *vo = a.v.p + row * a.v.ts + (int64_t)h * a.v.hs + 8 * c;
    // positions t0 + 2 i + t, i = 0 .. 15
    auto copy = [&](const uint16_t *res, uint16_t *out, int64_t ts) {
      const uint4 *src = reinterpret_cast<const uint4 *>(res + res0 * kD) + c;
#pragma unroll 8
      for (int i = 0; i < kBlock / 2; ++i) {
        const int r = 2 * i + t;
        if (t0 + r >= lo && t0 + r < hi) *reinterpret_cast<uint4 *>(out + r * ts) = src[r * (kD / 8)];
      }
    };
    auto codes = [&](const uint32_t *pool, int r) -> uint32_t {
      const uint32_t *q = pool + (row0 + r) * WPR;
      if constexpr (BITS == 2)
        return __ldg(reinterpret_cast<const uint16_t *>(q) + c);
      else
        return __ldg(q + c);
    };
    if (late) {
      copy(a.k_res, ko, a.k.ts);
    } else {
      __half2 s[4], z[4];
      const uint4 *m = reinterpret_cast<const uint4 *>(a.k_meta + row0 / a.G * kD + 8 * c);
      const uint4 m0 = __ldg(m), m1 = __ldg(m + 1);
      const uint32_t mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = u2h2(paged ? prmt(mm[2 * j], mm[2 * j + 1], 0x5410u) : 0u);
        z[j] = u2h2(paged ? prmt(mm[2 * j], mm[2 * j + 1], 0x7632u) : 0u);
      }
#pragma unroll
      for (int i0 = 0; i0 < kBlock / 2; i0 += 8) {
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = codes(a.k_codes, 2 * (i0 + i) + t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 2 * (i0 + i) + t;
          const uint4 o = widen<BITS>(x[i], s, z);
          if (t0 + r >= lo && t0 + r < hi) *reinterpret_cast<uint4 *>(ko + r * a.k.ts) = o;
        }
      }
    }
    if (late && a.v_res) {
      copy(a.v_res, vo, a.v.ts);
    } else {
      const uint32_t vm = paged ? __ldg(a.v_meta + row0 + lane) : 0u;  // of the block's rows
#pragma unroll
      for (int i0 = 0; i0 < kBlock / 2; i0 += 8) {
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = codes(a.v_codes, 2 * (i0 + i) + t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 2 * (i0 + i) + t;
          const uint32_t mr = __shfl_sync(0xffffffffu, vm, r);
          const __half2 sr = u2h2(prmt(mr, mr, 0x1010u)), zr = u2h2(prmt(mr, mr, 0x3232u));
          const __half2 s[4] = {sr, sr, sr, sr}, z[4] = {zr, zr, zr, zr};
          const uint4 o = widen<BITS>(x[i], s, z);
          if (t0 + r >= lo && t0 + r < hi) *reinterpret_cast<uint4 *>(vo + r * a.v.ts) = o;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_read(const ReadArgs &a, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  // one wave of CTAs, or fewer where there is less work
  const int64_t items = ((int64_t)a.T / kBlock + 4 * a.B) * a.Hkv, wave = (int64_t)sms * kCtas;
  const int64_t want = (items + kWarps - 1) / kWarps;
  const unsigned grid = (unsigned)(want < wave ? want : wave);
  if (a.bits == 2)
    paged_read_kernel<2><<<grid, kThreads, 0, st>>>(a);
  else
    paged_read_kernel<4><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kivi
