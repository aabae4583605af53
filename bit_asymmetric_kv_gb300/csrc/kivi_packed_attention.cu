// kivi_packed_attention.cu -- causal attention over prompts of different lengths packed
// into one token axis (sm_103a, tensor memory and the tensor-map copy engine).
//
// For row i of a sequence (rows counted from its start) and query head h, reading KV
// head h / (Hq / Hkv):
//   out_i = sum_{j <= i} softmax_j(sigma q_i . k_j) v_j,   j over the same sequence.
//
// A block of work is two tiles, A and B, of 128 query rows, which walk the keys and
// values in tiles of 128 rows from the diagonal down to the sequence's first.  A query
// tile is 128 / P consecutive tokens of P query heads that read the same KV head, P the
// largest power of two (up to 16) that divides Hq / Hkv: the heads of a group share every
// key and value tile, and a short prompt wastes fewer rows of a tile.  One CTA per SM
// takes block after block, longest first, so that the next block's copies and first
// products run under the last one's output.
//
// Roles (12 warps, the last idle: registers go by four warps):
//   warps 0-3, 4-7  softmax of tile A, of tile B: a thread holds one row.  It reads the 128
//                   scores from tensor memory, keeps the running maximum and sum, and
//                   writes the probabilities over the scores, as fp16; at the end of a
//                   block it divides the output by the sum and stores it.
//   warp 8          one lane issues the MMAs: S = Q K^T (both operands in shared memory) and
//                   O += P V (P in tensor memory), tile A and B in turn, so that one
//                   tile's softmax runs under the other's MMAs.
//   warp 9          finds the CTA's next block, one ahead.
//   warp 10         one lane issues the tensor-map copies: Q, and K and V tiles through a
//                   ring of stages.
// Tensor memory: S/P of A and B (128 columns each), O of A and B (128 each): all 512.
//
// The maximum that the probabilities are relative to may lag behind the true one by 2^11:
// only beyond that are the sums and the output in tensor memory rescaled, which
// happens in the first tiles of a row and then hardly ever.  The probabilities are scaled by
// 2^4 on top, so that they use fp16's range (at most 2^15; the smallest lie 2^28 below)
// and their rounding, 2^-11 of each, is the only one below fp32 before the output's.
//
// Rows behind a sequence's end share its last tiles.  As query rows they are computed and
// not stored, and have no vote in what a warp does for its rows together (a new reference,
// the form for scores far from zero), so that a prompt's bits are those that it has alone;
// as keys they are masked by causality; as values they would meet probability 0, and a NaN
// there would spread, so the MMA warp overwrites them with zeros first.
//
// Measured with inputs that L2 does not hold (two prompts of 16384 and 8200 tokens, 32 query
// heads on 8): 2.04 ms, 1.35 PFLOP/s of causal work, 0.72 of the measured bf16 peak; eight ragged
// prompts of up to 4113 tokens with 32 KV heads: 0.49 ms, 0.57 of it; 128 prompts of up to 512
// tokens: 70 us.
// What bounds it: per pass, a tile's softmax (about 1300 cycles, of which the exponential
// unit needs 512) and its P.V and next scores (1024 of MMAs and about 400 of waits for
// barriers) come one after the other, and the two tiles overlap only in part.  Tried and
// slower on the long prompts: probabilities handed over in halves (1.05x), the maximum checked
// beside the exponentials instead of before them (1.08x), two threads a row in 16 softmax
// warps (1.3x), tiles of 80 keys with P in columns of its own, so that the next scores go out
// before P.V (1.13x), turns on the exponential unit (1.15x), MMAs issued by a softmax warp
// (1.6x: it stands still until they are taken).  An MMA warp for each tile is level there and
// 10% slower on short prompts.  Short prompts are bound by the length of one block's chain:
// copies, scores, softmax, P.V and output.
//
// Every wait is bounded: one that runs out (a copy that never completes) ends all roles
// of the CTA; the rows of its block are NaN, those of its later blocks not written.
#include <algorithm>
#include <atomic>

#include "kivi_packed.cuh"
#include "kivi_tcgen05.cuh"

namespace kivi {

namespace {

constexpr int kThreads = 384;               // three warpgroups
constexpr int kMmaWarp = 8, kBlockWarp = 9, kLoadWarp = 10;
// Registers a thread: the CTA's share at launch, and how the warpgroups split it (a
// softmax thread holds a row of 128 scores).
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "more registers than the CTA was launched with");
constexpr int kStages = 4;                  // K and V tiles in flight

// One block of work.
struct __align__(16) Block {
  int start, len;         // the sequence
  int head0, kvh;
  int base0, base1;       // first token of A, of B
  int nt0, nt1;           // key tiles of each, the last one on the diagonal (B: 0 when it has no row)
  int n;                  // passes: pass i works on key tile n - 1 - i
  int tail;               // rows of the last key tile inside the sequence (more than a tile: all)
  int there;              // 0: no block, and none after it
};

struct __align__(16) Bars {
  uint64_t q[2];            // Q tile landed
  uint64_t q_free[2];       // the block's last scores of it are done
  uint64_t full[kStages];   // K or V tile landed
  uint64_t empty[kStages];  // the MMAs that read it are done
  uint64_t s[2];            // scores of a tile written
  uint64_t p[2];            // its probabilities written
  uint64_t o[2];            // their P.V done
  uint64_t block[2];        // block k written to slot k % 2
  uint64_t block_read[2];   // by every warp that works on it
  Block slot[2];
  uint32_t tmem;
  int abort;
  PackedList list;
};
constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + (int)sizeof(Bars);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

struct Maps {
  CUtensorMap q, k, v;
};

// What the roles of a CTA share.
struct Cta {
  unsigned char *tiles;   // Q of A, Q of B, the stages
  uint32_t sQ, sKV;
  uint32_t tmem;
  int tpt;                // tokens of a query tile
  unsigned hgroups;       // head groups that share a tile
  unsigned sets;          // of head groups, one after the other
  int heads_per_kv, pack;
  int64_t items;          // blocks of all sequences and head groups
};

// ---------------------------------------------------------------------------- blocks
constexpr int kReaders = 10;  // warps that work on a block

// Block k of this CTA into slot k % 2, for the warps that work on it.  The list is dealt out
// back and forth, so that the first CTAs do not get the longer block of every round.  Where K
// and V of all heads are more than L2 holds, the head groups are taken in sets that fit, one
// set's blocks after the other's, every other set shortest first (the last one longest first):
// the blocks' lengths then rise and fall without a jump, which back and forth deals evenly.
__device__ __forceinline__ void block_role(const Cta &c, Bars &sh, int lane) {
  const int64_t G = gridDim.x;
  for (int k = 0;; ++k) {
    const int64_t at = k * G + ((k & 1) ? G - 1 - blockIdx.x : blockIdx.x);
    Block w = {};
    w.there = at < c.items;
    if (w.there) {
      // which set of head groups (the first `more` sets have one more), which block, which group
      const unsigned total = (unsigned)sh.list.total, size = c.hgroups / c.sets, more = c.hgroups % c.sets;
      unsigned rest = (unsigned)at, set, width = size + 1, group;
      if (rest < more * width * total) {
        set = rest / (width * total);
        rest -= set * width * total;
        group = set * width;
      } else {
        rest -= more * width * total;
        group = more * width;
        width = size;
        set = rest / (width * total);
        rest -= set * width * total;
        group += set * width;
        set += more;
      }
      unsigned item = rest / width;
      const unsigned hg = group + rest - item * width;
      if ((c.sets - 1 - set) & 1) item = total - 1 - item;
      const PackedBlock b = sh.list.find(item);
      w.start = b.start;
      w.len = b.len;
      w.head0 = (int)hg * c.pack;
      w.kvh = w.head0 / c.heads_per_kv;
      w.base0 = b.level * 2 * c.tpt;
      w.base1 = w.base0 + c.tpt;
      w.nt0 = w.base0 / kRows + 1;
      w.nt1 = w.base1 < w.len ? w.base1 / kRows + 1 : 0;
      w.n = max(w.nt0, w.nt1);
      w.tail = w.len - (w.n - 1) * kRows;
    }
    if (k >= 2 && !__all_sync(0xffffffffu, bar_wait(&sh.block_read[k & 1], (k / 2 - 1) & 1, &sh.abort))) return;
    if (lane == 0) {
      sh.slot[k & 1] = w;
      bar_arrive(&sh.block[k & 1]);
    }
    __syncwarp();
    if (!w.there) return;
  }
}

// A warp's next block; false after the last one (or an abort).
__device__ __forceinline__ bool next_block(Bars &sh, int k, int lane, Block *w) {
  if (!__all_sync(0xffffffffu, bar_wait(&sh.block[k & 1], (k >> 1) & 1, &sh.abort))) return false;
  *w = sh.slot[k & 1];
  __syncwarp();
  if (lane == 0) bar_arrive(&sh.block_read[k & 1]);
  return w->there != 0;
}

// ---------------------------------------------------------------------------- copies
// The CTA's copies are counted through all its blocks: copy number c goes to stage
// c % kStages.  Pass i of a block takes K from the block's copy 2 i and V from 2 i + 1.
__device__ __forceinline__ void load_role(const Maps &maps, const Cta &cta, Bars &sh, int lane) {
  bool ok = true;
  int c = 0, loads[2] = {0, 0};
  Block w;
  for (int k = 0; ok && next_block(sh, k, lane, &w); ++k) {
    for (int i = 0; i < 2 * w.n && ok; ++i) {
      const int st = c % kStages;
      if (c >= kStages) ok = __all_sync(0xffffffffu, bar_wait(&sh.empty[st], (c / kStages - 1) & 1, &sh.abort));
      if (!ok) break;
      if (lane == 0) {
        bar_expect(&sh.full[st], kTileBytes);
        for (int half = 0; half < 2; ++half)
          tma_3d(cta.sKV + st * kTileBytes + half * kHalfBytes, i & 1 ? &maps.v : &maps.k, 64 * half,
                 w.start + (w.n - 1 - i / 2) * kRows, w.kvh, &sh.full[st]);
      }
      ++c;
      if (i == 0) {  // Q behind the first K, which never waits for the block before
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x && !w.nt1) break;
          if (loads[x]) ok = __all_sync(0xffffffffu, bar_wait(&sh.q_free[x], (loads[x] - 1) & 1, &sh.abort));
          if (!ok) break;
          if (lane == 0) {
            bar_expect(&sh.q[x], kTileBytes);
            for (int half = 0; half < 2; ++half)
              tma_3d(cta.sQ + x * kTileBytes + half * kHalfBytes, &maps.q, 64 * half, w.start + (x ? w.base1 : w.base0),
                     w.head0, &sh.q[x]);
          }
          ++loads[x];
        }
      }
    }
  }
  // The CTA ends when nothing is under way any more: every copy has landed, and every
  // arrival that the MMAs still owe has come.
  int never = 0;
  for (int x = 0; x < 2 && !never; ++x)
    if (loads[x]) bar_wait(&sh.q[x], (loads[x] - 1) & 1, &never);
  for (int j = max(0, c - kStages); j < c && !never; ++j) bar_wait(&sh.full[j % kStages], (j / kStages) & 1, &never);
  for (int x = 0; x < 2 && ok; ++x)
    if (loads[x]) ok = bar_wait(&sh.q_free[x], (loads[x] - 1) & 1, &sh.abort);
  for (int j = max(0, c - kStages); j < c && ok; ++j) ok = bar_wait(&sh.empty[j % kStages], (j / kStages) & 1, &sh.abort);
  __syncwarp();
}

// The rows of a value tile from `tail` on.
__device__ __forceinline__ void zero_rows(unsigned char *v, int tail, int lane) {
  for (int r = tail * 8 + lane; r < kRows * 8; r += 32)
    for (int half = 0; half < 2; ++half)
      *reinterpret_cast<uint4 *>(v + half * kHalfBytes + r * 16) = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  __syncwarp();
}

// -------------------------------------------------------------------------- products
// Tile A and B in turn: a tile's P.V and its next scores go out together, and run while the
// other tile's softmax does.
__device__ __forceinline__ void mma_role(const Cta &cta, Bars &sh, int lane) {
  const uint32_t one = elect_one();
  const uint32_t q0 = desc_lo(cta.sQ, 16), k0 = desc_lo(cta.sKV, 16), v0 = desc_lo(cta.sKV, kHalfBytes);
  constexpr uint32_t kTile16 = kTileBytes >> 4;
  auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(b, parity, &sh.abort)) != 0; };
  auto landed = [&](int c) { return wait(&sh.full[c % kStages], (c / kStages) & 1); };
  auto give = [&](int c) { tc_commit(&sh.empty[c % kStages], one); };
  int c = 0, t[2] = {0, 0}, tiles[2] = {0, 0};  // copies, passes and Q tiles before
  Block w;
  auto qk = [&](int x, int c) {  // scores of tile x with the K tile of copy c
    mma_qk(cta.tmem + x * kRows, q0 + x * kTile16, k0 + (c % kStages) * kTile16, kIdescQK, 0, one);
    tc_commit(&sh.s[x], one);
  };
  for (int k = 0; next_block(sh, k, lane, &w); ++k) {
    if (!landed(c)) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!(x ? w.nt1 : w.nt0)) continue;
      if (!wait(&sh.q[x], tiles[x] & 1)) return;
      ++tiles[x];
      tc_fence_after();
      if ((x ? w.nt1 : w.nt0) == w.n) {
        qk(x, c);
        if (w.n == 1) tc_commit(&sh.q_free[x], one);
      }
    }
    give(c);
    if (!landed(c + 1)) return;
    if (w.tail < kRows) zero_rows(cta.tiles + (2 + (c + 1) % kStages) * kTileBytes, w.tail, lane);
    for (int i = 0; i < w.n; ++i, c += 2) {
      const int left = w.n - 1 - i;  // key tile of this pass
      if (i && !landed(c + 1)) return;
      if (left && !landed(c + 2)) return;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int nt = x ? w.nt1 : w.nt0;
        if (left < nt) {
          if (!wait(&sh.p[x], t[x] & 1)) return;
          tc_fence_after();
          const uint32_t d = cta.tmem + 2 * kRows + x * kD, a = cta.tmem + x * kRows, v = v0 + ((c + 1) % kStages) * kTile16;
          mma_pv(d, a, v, kIdescPV, left < nt - 1, one);
          mma_pv(d, a + 32, v + 512, kIdescPV, 1, one);
          tc_commit(&sh.o[x], one);
          ++t[x];
        }
        if (left && left - 1 < nt) {
          qk(x, c + 2);
          if (left == 1) tc_commit(&sh.q_free[x], one);
        }
      }
      give(c + 1);
      if (left) give(c + 2);
    }
  }
}

// --------------------------------------------------------------------------- softmax
__device__ __forceinline__ void softmax_role(const PackedAttentionArgs &a, const Cta &cta, Bars &sh, int x, int warp,
                                             int lane) {
  const int r = 32 * warp + lane;  // row of tile x
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t tS = cta.tmem + x * kRows + lanes, tO = cta.tmem + 2 * kRows + x * kD + lanes;
  const float c0 = a.softmax_scale * kLog2eP;
  // whole 32-byte sectors where the output's rows allow it
  const bool wide = ((reinterpret_cast<uintptr_t>(a.out.p) | (uintptr_t)(a.out.ts * 2) | (uintptr_t)(a.out.hs * 2)) & 31) == 0;
  auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(b, parity, &sh.abort)) != 0; };
  bool ok = true;
  int t0 = 0;  // passes of this tile in the blocks before
  Block w;
  for (int k = 0; next_block(sh, k, lane, &w); ++k) {
    const int base = x ? w.base1 : w.base0, nt = x ? w.nt1 : w.nt0;
    if (nt == 0) continue;
    const int token = base + r % cta.tpt;
    float m = 0.f, off = 0.f;  // the reference maximum, and the exponents' offset with it
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;  // the sum, in four parts
    bool far = false;          // far from zero that offset has no digits: subtract the maximum first
    const int last = token - (nt - 1) * kRows;  // the row's own key in the tile on the diagonal
    const bool mine = token < w.len;            // the sequence's own row
    for (int t = t0; t < t0 + nt && ok; ++t) {
      ok = wait(&sh.s[x], t & 1);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[kRows];
#pragma unroll
      for (int j = 0; j < 4; ++j) tmem_ld32(tS + 32 * j, s + 32 * j);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 4; ++j) landed32(s + 32 * j);
      if (t == t0) {  // the tile on the diagonal
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (j > last) s[j] = 0xff800000u;
      }
      const float mx = fmaxf(max64(s), max64(s + 64));
      const bool first = t == t0;
      if (first || __any_sync(0xffffffffu, mine && (mx - m) * c0 > kLag)) {  // a new reference
        const float mn = first ? mx : fmaxf(m, mx);
        const bool far_now = __any_sync(0xffffffffu, mine && fabsf(mn * c0) > kFar);
        const float off_now = far_now ? kShift : kShift - mn * c0;
        if (!first) {
          // What lies between the weights before, 2^(c0 (s - [far] m) + off), and those from now on.
          // It takes both offsets as they were rounded (by up to 2^-9 below kFar): from the maxima
          // alone old and new weights would be as far apart as the two roundings, 0.27% at most.
          const float al = ex2(fmaf((far ? m : 0.f) - (far_now ? mn : 0.f), c0, off_now - off));
          sum0 = __fmul2_rn(sum0, make_float2(al, al));
          sum1 = __fmul2_rn(sum1, make_float2(al, al));
          ok = wait(&sh.o[x], (t - 1) & 1);  // the last product into the output
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * j, o);
            tc_wait_ld();
            landed32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            tmem_st32(tO + 32 * j, o);
          }
        }
        m = mn;
        far = far_now;
        off = off_now;
      }
      if (__builtin_expect(far, 0)) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) - m);
      }
      const float2 c2 = make_float2(c0, c0), b2 = make_float2(off, off);
#pragma unroll
      for (int j = 0; j < kRows / 2; ++j) {
        const float2 e = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, b2);
        const float2 v = make_float2(ex2(e.x), ex2(e.y));
        if (j & 1)
          sum1 = __fadd2_rn(sum1, v);
        else
          sum0 = __fadd2_rn(sum0, v);
        s[j] = h22u(__floats2half2_rn(v.x, v.y));
      }
      tmem_st32(tS, s);
      tmem_st32(tS + 32, s + 32);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.p[x]);
    }
    t0 += nt;
    ok = ok && wait(&sh.o[x], (t0 - 1) & 1);
    tc_fence_after();
    // ---- the tile's rows
    const float2 sum = __fadd2_rn(sum0, sum1);
    const float inv = ok ? 1.f / (sum.x + sum.y) : __int_as_float(0x7fc00000);
    uint16_t *dst = a.out.p + (int64_t)(w.start + token) * a.out.ts + (int64_t)(w.head0 + r / cta.tpt) * a.out.hs;
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
      uint32_t o[64];
      tmem_ld32(tO + 64 * j, o);
      tmem_ld32(tO + 64 * j + 32, o + 32);
      tc_wait_ld();
      landed32(o);
      landed32(o + 32);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        o[i] = h22u(__floats2half2_rn(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv));
      if (mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint16_t *d = dst + 64 * j + 16 * i;
          const uint32_t *v = o + 8 * i;
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(d), "r"(v[0]), "r"(v[1]),
                         "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                         : "memory");
          } else {
            *reinterpret_cast<uint4 *>(d) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4 *>(d + 8) = make_uint4(v[4], v[5], v[6], v[7]);
          }
        }
      }
    }
    tc_fence_before();  // the output is read: the next block's probabilities say so
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    packed_attention_kernel(const __grid_constant__ PackedAttentionArgs a, const __grid_constant__ Maps maps, int pack,
                            unsigned sets) {
  extern __shared__ unsigned char raw[];
  Cta cta;
  // tiles start at a multiple of the swizzle's 1024-byte pattern
  cta.tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Bars &sh = *reinterpret_cast<Bars *>(cta.tiles + (2 + kStages) * kTileBytes);
  cta.sQ = smem_u32(cta.tiles);
  cta.sKV = cta.sQ + 2 * kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cta.tpt = kRows / pack;
  cta.pack = pack;
  cta.heads_per_kv = a.Hq / a.Hkv;
  cta.hgroups = (unsigned)(a.Hq / pack);
  cta.sets = sets;

  if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int x = 0; x < 2; ++x) {
        bar_init(&sh.q[x], 1);
        bar_init(&sh.q_free[x], 1);
        bar_init(&sh.s[x], 1);
        bar_init(&sh.p[x], 4);
        bar_init(&sh.o[x], 1);
      }
      for (int i = 0; i < kStages; ++i) {
        bar_init(&sh.full[i], 1);
        bar_init(&sh.empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        bar_init(&sh.block[i], 1);
        bar_init(&sh.block_read[i], kReaders);
      }
      sh.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  sh.list.build(a.cu, a.n_seqs, a.T, 2 * cta.tpt);  // the CTA's threads together
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cta.tmem = sh.tmem;
  cta.items = (int64_t)sh.list.total * cta.hgroups;
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kLoadWarp)
      load_role(maps, cta, sh, lane);
    else if (warp == kMmaWarp)
      mma_role(cta, sh, lane);
    else if (warp == kBlockWarp)
      block_role(cta, sh, lane);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
    softmax_role(a, cta, sh, warp >> 2, warp & 3, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(cta.tmem), "r"(kTmemCols) : "memory");
}

bool encode_all(Maps *m, const PackedAttentionArgs &a, int pack) {
  return encode(&m->q, a.q, a.T, a.Hq, kRows / pack, pack) && encode(&m->k, a.k, a.T, a.Hkv, kRows, 1) &&
         encode(&m->v, a.v, a.T, a.Hkv, kRows, 1);
}

int pack_of(const PackedAttentionArgs &a) {
  const int R = a.Hq / a.Hkv;
  int p = 1;
  while (p < kMaxPack && R % (2 * p) == 0) p *= 2;
  return p;
}

// Sets of head groups whose K and V fit in 96 MB of the 129 MB of L2.  Eight ragged prompts of 18
// thousand tokens together with 32 KV heads (300 MB of K and V), inputs cold: 487 us and 0.70 GB
// read from memory in four sets, 514 us and 1.86 GB in one; with sets of half the heads and no
// turning of the order, 506 to 488 us against 469 with inputs that L2 had held.  Two prompts of 25
// thousand tokens with 8 KV heads lie just above the bound: 2035 us and 0.33 GB in two sets, 2050 us
// and 0.55 GB in one.  Where one set holds all, nothing changes.
unsigned sets_of(const PackedAttentionArgs &a, int pack) {
  const int64_t per_head = (int64_t)a.T * kD * 2 * 2;
  const int64_t heads = std::max<int64_t>(1, (96ll << 20) / per_head);  // KV heads of a set
  const int64_t groups = a.Hq / pack, width = std::min(groups, heads * (groups / a.Hkv));
  return (unsigned)((groups + width - 1) / width);
}

// Most blocks there can be: what the lengths allow.
int64_t blocks_of(const PackedAttentionArgs &a) {
  const int pack = pack_of(a);
  return ((int64_t)a.T / (2 * kRows / pack) + a.n_seqs) * (a.Hq / pack);
}

// The current device.  Once per device: the shared memory's limit, and that the kernel has the
// registers that the warpgroups' split of them rests on.
cudaError_t prepare_kernel(int *device) {
  static std::atomic<bool> ready[64];
  cudaError_t e = cudaGetDevice(device);
  if (e != cudaSuccess) return e;
  const int dev = *device;
  if (dev < 64 && ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaFuncAttributes f;
  if ((e = cudaFuncGetAttributes(&f, packed_attention_kernel)) != cudaSuccess) return e;
  if (f.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(packed_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess && dev < 64) ready[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace

bool packed_attention_fits(const PackedAttentionArgs &a) { return blocks_of(a) <= 0x7fffffff; }

cudaError_t launch_packed_attention(const PackedAttentionArgs &a, cudaStream_t st) {
  const int pack = pack_of(a);
  int dev = 0, sms = 0;
  cudaError_t e = prepare_kernel(&dev);
  if (e == cudaSuccess) e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  Maps maps;
  if (!encode_all(&maps, a, pack)) {
    // The encoder is a driver call and wants a context.  A host thread that has not called the
    // runtime yet has none, and cudaSetDevice gives it the device's; any other thread keeps the
    // context that it has, since the maps are made at once.
    if ((e = cudaSetDevice(dev)) != cudaSuccess) return e;
    if (!encode_all(&maps, a, pack)) return cudaErrorInvalidValue;
  }
  packed_attention_kernel<<<(unsigned)std::min<int64_t>(blocks_of(a), sms), kThreads, kSmem, st>>>(a, maps, pack, sets_of(a, pack));
  return cudaGetLastError();
}

}  // namespace kivi
