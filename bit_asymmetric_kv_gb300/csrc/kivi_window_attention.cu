// kivi_window_attention.cu -- attention with a sliding window and sinks over prompts, or chunks
// behind earlier tokens, packed into one token axis (sm_103a, tensor memory and the tensor-map
// copy engine).
//
// A sequence has n query rows and m key rows; its queries are its last tokens, row i at position
// p = i + m - n.  For query head h, reading KV head h / (Hq / Hkv):
//   out_i = sum_j softmax_j(sigma q_i . k_j) v_j   over  p - window < j <= p  and  j < min(sinks, p + 1);
// a row that sees nothing (p < 0) is zero.
//
// A block of work is two tiles, A and B, of 128 query rows (128 / P consecutive tokens of P query
// heads of one KV head, P the largest power of two up to 16 that divides Hq / Hkv), as in the attention
// over whole prompts.  They walk the keys in tiles of 128 that end where the block's last position does,
// so that every row's own key lies in its tile's first pass and the running maximum is finite from then
// on: pass i takes positions end - 128 (i + 1) .. end - 128 i - 1, down to the first that a row of the
// tile sees.  A tile takes only the passes that hold a key for it (A's first may be B's second, B's last
// A's last but one).  The sinks are passes of their own behind, from position 0 up, unless the whole of
// the keys below is not more passes than that.  Masks cost only where a pass is not seen whole by every
// row of the tile: at the diagonal, at the window's end and in the last tile of the sinks.  There a row's
// visible columns are built as four words of bits.
//
// Keys and values that no row of a block sees (other sequences' rows before and behind, rows outside
// the window) may be anything: their scores are replaced, and their values, which meet probability 0,
// are overwritten with zeros by the MMA warp, so that a NaN does not spread.
//
// Roles, tensor memory, the softmax's arithmetic and its rounding are those of the attention over
// whole prompts (kivi_packed_attention.cu).
//
// Measured: two prompts of 16384 and 8200 tokens, window 4096, 32 query heads on 8: 1.12 ms a call,
// 1.07 of them the kernel, 1.29 PFLOP/s of visible work in it, 0.66 of the measured bf16 peak
// (tensor pipe 56%); 16 chunks of 200 to 512 tokens behind up to 4099 earlier ones, the same heads:
// 0.17 ms, 0.44; eight ragged prompts of up to 4113 tokens, window 1024 and 4 sinks, 32 heads: 0.37
// ms, 0.42.  What bounds it: a tile's pass is a chain (scores, softmax, P.V) of about 3300 cycles,
// of which its own MMAs are 1024, and the two tiles overlap only in part, as over whole prompts.  A
// window of w tiles costs a tile w + 1 passes, half of the first and of the last masked, and one
// more for the sinks: 10 where 8 would hold the visible keys, in the third case.  Tried and not
// faster there: a sinks' pass of 32 columns (a second form of the softmax costs every pass 2%, as
// much as it saves), the passes of all blocks as one stream (the next block's first scores beside a
// block's last product: level; with the choices made at each product, 11% slower).  Sorting blocks
// by the level in their own sequence, as the attention over whole prompts does, made the chunks
// behind earlier tokens 1.25 times slower.
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

// All sequences' blocks, those whose last row stands at the highest position first: a block's passes
// never grow as its position falls, so that long and short blocks are dealt out evenly whatever the
// sequences' queries and keys.  Block L of sequence s has the order lead_s + L, in blocks of
// positions; block `item` is found by a binary search for its order and a count over the sequences.
// Kept in shared memory, built once by a CTA.
struct WindowList {
  int qrow[kPackedMaxSeqs], len[kPackedMaxSeqs], krow[kPackedMaxSeqs], keys[kPackedMaxSeqs];
  int lead[kPackedMaxSeqs], nb[kPackedMaxSeqs];
  int n, lo, hi;  // sequences; the lowest and highest order
  int total;

  // Every thread of the CTA calls it; synchronises.
  __device__ __forceinline__ void build(const WindowAttentionArgs &a, int bt) {
    for (int s = threadIdx.x; s < a.n_seqs; s += blockDim.x) {
      int r, m, kr, km;
      packed_bounds(a.cu, s, a.T, &r, &m);
      packed_bounds(a.cu_kv, s, a.Tk, &kr, &km);
      qrow[s] = r;
      len[s] = m;
      krow[s] = kr;
      keys[s] = km;
      nb[s] = m / bt + (m % bt != 0);
      lead[s] = km > m ? (km - m) / bt : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      int64_t sum = 0;
      int x = 0x7fffffff, y = 0;
      for (int s = threadIdx.x; s < a.n_seqs; s += 32)
        if (nb[s]) {
          sum += nb[s];
          x = min(x, lead[s]);
          y = max(y, lead[s] + nb[s] - 1);
        }
#pragma unroll
      for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      x = __reduce_min_sync(0xffffffffu, x);
      y = __reduce_max_sync(0xffffffffu, y);
      if (threadIdx.x == 0) {
        n = a.n_seqs;
        lo = x;
        hi = y;
        // bounds that overlap may pass any count: cut at what lengths that do not overlap can reach
        total = (int)min((int64_t)a.T / bt + a.n_seqs, sum);
      }
    }
    __syncthreads();
  }

  // Sequence and level of block `item` < total; every lane of a warp calls it.
  __device__ __forceinline__ void find(unsigned item, int lane, int *seq, int *level) const {
    auto from = [&](int order) {  // blocks of that order and higher
      unsigned c = 0;
      for (int s = lane; s < n; s += 32) c += (unsigned)min(nb[s], max(0, lead[s] + nb[s] - order));
      return __reduce_add_sync(0xffffffffu, c);
    };
    int a = lo, b = hi;  // the highest order with more than `item` blocks from it on
    while (a < b) {
      const int mid = a + (b - a + 1) / 2;
      if (from(mid) > item)
        a = mid;
      else
        b = mid - 1;
    }
    unsigned rest = item - from(a + 1);
    *seq = 0;
    *level = 0;
    for (int s0 = 0; s0 < n; s0 += 32) {
      const int s = s0 + lane;
      const uint32_t has = __ballot_sync(0xffffffffu, s < n && nb[s] && a >= lead[s] && a < lead[s] + nb[s]);
      if (rest < (unsigned)__popc(has)) {
        *seq = s0 + (int)__fns(has, 0, (int)rest + 1);
        *level = a - lead[*seq];
        return;
      }
      rest -= __popc(has);
    }
  }
};

// One block of work.
struct __align__(16) Block {
  int qrow, len;          // the sequence's first query row, its queries
  int krow, keys;         // its first key row, its keys
  int head0, kvh;
  int base[2];            // first query of A, of B
  int from[2], to[2];     // passes of the window that each takes
  int nt[2];              // and all its passes (0: it has no row, or its rows see nothing)
  int end;                // the window's passes end at this position
  int low;                // first position in the window of a row of the block
  int nw, n;              // passes of the window, of window and sinks
  int split;              // first position of the window's passes that counts (the sinks, where they have passes of their own)
  int there;              // 0: no block, and none after it

  // First position of pass i.
  __device__ __forceinline__ int at(int i) const { return i < nw ? end - kRows * (i + 1) : kRows * (i - nw); }
  __device__ __forceinline__ bool takes(int x, int i) const {
    return nt[x] && ((i >= from[x] && i < to[x]) || i >= nw);
  }
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
  WindowList list;
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

__device__ __forceinline__ int tiles_of(int positions) { return positions > 0 ? (positions - 1) / kRows + 1 : 0; }

// Passes of a block whose sequence, queries and base are known.
__device__ __forceinline__ void plan_passes(const WindowAttentionArgs &a, int tpt, Block *w) {
  if (w->base[0] >= w->len) return;  // only where bounds overlap: no pass
  const int off = w->keys - w->len;
  const bool two = w->base[1] < w->len;
  w->end = (two ? w->base[1] : w->base[0]) + tpt + off;
  w->low = w->base[0] + off - a.window + 1;
  const int whole = tiles_of(w->end), sinks = tiles_of(min(a.sinks, w->keys));
  w->from[0] = two && tpt == kRows ? 1 : 0;  // A's positions end one tile before B's
  w->from[1] = 0;
  w->to[0] = tiles_of(w->end - max(w->low, 0));
  w->to[1] = tiles_of(w->end - max(w->low + tpt, 0));
  // Sinks by passes of their own: fewer passes, and every row's own key is behind them.
  const bool own = a.sinks > 0 && w->base[0] + off >= a.sinks && w->to[0] + sinks < whole;
  w->split = own ? a.sinks : 0;
  if (a.sinks > 0 && !own) w->to[0] = w->to[1] = whole;
  w->nw = w->to[0];
  w->n = w->nw + (own ? sinks : 0);
  w->nt[0] = max(w->to[0] - w->from[0], 0) + (own ? sinks : 0);
  w->nt[1] = two ? w->to[1] + (own ? sinks : 0) : 0;
}

// Block k of this CTA into slot k % 2, for the warps that work on it.  The list is dealt out back and
// forth, so that the first CTAs do not get the longer block of every round.  Where K and V of all heads are more than L2 holds, the
// head groups are taken in sets that fit, one set's blocks after the other's, every other set in reverse.
__device__ __forceinline__ void block_role(const WindowAttentionArgs &a, const Cta &c, Bars &sh, int lane) {
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
      int seq, level;
      sh.list.find(item, lane, &seq, &level);
      w.qrow = sh.list.qrow[seq];
      w.len = sh.list.len[seq];
      w.krow = sh.list.krow[seq];
      w.keys = sh.list.keys[seq];
      w.head0 = (int)hg * c.pack;
      w.kvh = w.head0 / c.heads_per_kv;
      w.base[0] = level * 2 * c.tpt;
      w.base[1] = w.base[0] + c.tpt;
      plan_passes(a, c.tpt, &w);
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
        for (int half = 0; half < 2; ++half)  // rows before and behind the tensor are filled with zeros
          tma_3d(cta.sKV + st * kTileBytes + half * kHalfBytes, i & 1 ? &maps.v : &maps.k, 64 * half,
                 w.krow + w.at(i / 2), w.kvh, &sh.full[st]);
      }
      ++c;
      if (i == 0) {  // Q behind the first K, which never waits for the block before
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!w.nt[x]) continue;
          if (loads[x]) ok = ok && __all_sync(0xffffffffu, bar_wait(&sh.q_free[x], (loads[x] - 1) & 1, &sh.abort));
          if (!ok) break;
          if (lane == 0) {
            bar_expect(&sh.q[x], kTileBytes);
            for (int half = 0; half < 2; ++half)
              tma_3d(cta.sQ + x * kTileBytes + half * kHalfBytes, &maps.q, 64 * half, w.qrow + w.base[x], w.head0,
                     &sh.q[x]);
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

// Rows [from, to) of a value tile; a warp.
__device__ __forceinline__ void zero_rows(unsigned char *v, int from, int to, int lane) {
  for (int r = from * 8 + lane; r < to * 8; r += 32)
    for (int half = 0; half < 2; ++half)
      *reinterpret_cast<uint4 *>(v + half * kHalfBytes + r * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// The rows of pass i's value tile that no row of the block sees.
__device__ __forceinline__ void zero_unseen(const WindowAttentionArgs &a, const Block &w, int i, unsigned char *v,
                                            int lane) {
  const int at = w.at(i);
  auto row = [&](int p) { return min(max(p - at, 0), kRows); };
  // [0, f) and [t, 128) are not seen, nor [g0, g1)
  int f = 0, t = kRows, g0 = 0, g1 = 0;
  if (i >= w.nw) {
    t = row(a.sinks);
  } else {
    t = row(w.keys);
    if (a.sinks > 0 && !w.split) {
      f = row(0);
      g0 = row(a.sinks);
      g1 = row(w.low);
    } else {
      f = row(max(max(w.low, w.split), 0));
    }
  }
  if (f > 0 || t < kRows || g0 < g1) {
    zero_rows(v, 0, f, lane);
    zero_rows(v, g0, g1, lane);
    zero_rows(v, t, kRows, lane);
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    __syncwarp();
  }
}

// -------------------------------------------------------------------------- products
// Tile A and B in turn: a tile's P.V and its next scores go out together, and run while the
// other tile's softmax does.
__device__ __forceinline__ void mma_role(const WindowAttentionArgs &a, const Cta &cta, Bars &sh, int lane) {
  const uint32_t one = elect_one();
  const uint32_t q0 = desc_lo(cta.sQ, 16), k0 = desc_lo(cta.sKV, 16), v0 = desc_lo(cta.sKV, kHalfBytes);
  constexpr uint32_t kTile16 = kTileBytes >> 4;
  auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(b, parity, &sh.abort)) != 0; };
  auto landed = [&](int c) { return wait(&sh.full[c % kStages], (c / kStages) & 1); };
  auto give = [&](int c) { tc_commit(&sh.empty[c % kStages], one); };
  int c = 0, t[2] = {0, 0}, tiles[2] = {0, 0};  // copies, passes and Q tiles before
  Block w;
  for (int k = 0; next_block(sh, k, lane, &w); ++k) {
    if (w.n == 0) continue;
    int asked[2] = {0, 0};  // scores asked for in this block
    auto qk = [&](int x, int c) {  // scores of tile x with the K tile of copy c
      mma_qk(cta.tmem + x * kRows, q0 + x * kTile16, k0 + (c % kStages) * kTile16, kIdescQK, 0, one);
      tc_commit(&sh.s[x], one);
      if (++asked[x] == w.nt[x]) tc_commit(&sh.q_free[x], one);
    };
    if (!landed(c)) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!w.nt[x]) continue;
      if (!wait(&sh.q[x], tiles[x] & 1)) return;
      ++tiles[x];
      tc_fence_after();
      if (w.takes(x, 0)) qk(x, c);
    }
    give(c);
    int done[2] = {0, 0};
    for (int i = 0; i < w.n; ++i, c += 2) {
      const bool more = i + 1 < w.n;
      if (!landed(c + 1)) return;
      zero_unseen(a, w, i, cta.tiles + (2 + (c + 1) % kStages) * kTileBytes, lane);
      if (more && !landed(c + 2)) return;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (w.takes(x, i)) {
          if (!wait(&sh.p[x], t[x] & 1)) return;
          tc_fence_after();
          const uint32_t d = cta.tmem + 2 * kRows + x * kD, p = cta.tmem + x * kRows, v = v0 + ((c + 1) % kStages) * kTile16;
          mma_pv(d, p, v, kIdescPV, done[x] > 0, one);
          mma_pv(d, p + 32, v + 512, kIdescPV, 1, one);
          tc_commit(&sh.o[x], one);
          ++t[x];
          ++done[x];
        }
        if (more && w.takes(x, i + 1)) qk(x, c + 2);
      }
      give(c + 1);
      if (more) give(c + 2);
    }
  }
}

// --------------------------------------------------------------------------- softmax
// Bits [a, b) of word w of a row of columns.
__device__ __forceinline__ uint32_t columns(int a, int b, int w) {
  a = min(max(a - 32 * w, 0), 32);
  b = min(max(b - 32 * w, 0), 32);
  const uint64_t lo = (1ull << a) - 1, hi = (1ull << b) - 1;
  return (uint32_t)(hi & ~lo);
}

__device__ __forceinline__ void softmax_role(const WindowAttentionArgs &a, const Cta &cta, Bars &sh, int x, int warp,
                                             int lane) {
  const int r = 32 * warp + lane;  // row of tile x
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t tS = cta.tmem + x * kRows + lanes, tO = cta.tmem + 2 * kRows + x * kD + lanes;
  const float c0 = a.softmax_scale * kLog2eP;
  // whole 32-byte sectors where the output's rows allow it
  const bool wide = ((reinterpret_cast<uintptr_t>(a.out.p) | (uintptr_t)(a.out.ts * 2) | (uintptr_t)(a.out.hs * 2)) & 31) == 0;
  auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(b, parity, &sh.abort)) != 0; };
  bool ok = true;
  int t = 0;  // passes of this tile before
  Block w;
  for (int k = 0; next_block(sh, k, lane, &w); ++k) {
    const int base = x ? w.base[1] : w.base[0], from = x ? w.from[1] : w.from[0], to = x ? w.to[1] : w.to[0];
    if (base >= w.len) continue;
    const int token = base + r % cta.tpt, off_p = w.keys - w.len;
    const int pos = token + off_p;              // the row's position, its last key
    const int first_p = base + off_p, last_p = base + cta.tpt - 1 + off_p;  // of the tile's rows
    const bool mine = token < w.len;            // the sequence's own row
    const bool sees = pos >= 0;                 // and it has a key
    const bool votes = mine && sees;
    uint16_t *dst = a.out.p + (int64_t)(w.qrow + token) * a.out.ts + (int64_t)(w.head0 + r / cta.tpt) * a.out.hs;
    if (!(x ? w.nt[1] : w.nt[0])) {  // no row sees anything, and nothing is asked of the tensor cores
      if (mine)
        for (int i = 0; i < kD; i += 8) *reinterpret_cast<uint4 *>(dst + i) = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    float m = 0.f, off = 0.f;  // the reference maximum, and the exponents' offset with it
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;  // the sum, in four parts
    bool far = false;          // far from zero that offset has no digits: subtract the maximum first
    bool first = true;
    for (int i = from < to ? from : w.nw; i < w.n && ok; i = i + 1 == to ? w.nw : i + 1) {
      ok = wait(&sh.s[x], t & 1);
      if (!ok) break;
      tc_fence_after();
      const int at = w.at(i);
      // seen whole by every row of the tile: inside the window (or the sinks) of all
      const bool clean = i < w.nw ? at + kRows - 1 <= first_p && ((at >= w.split && at > last_p - a.window) ||
                                                                  (at >= 0 && !w.split && at + kRows <= a.sinks))
                                  : at + kRows <= a.sinks;
      uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
      if (!clean) {
        // columns [l, e) of the window, [z, f) of the sinks
        int l = 0, e = 0, z = 0, f;
        if (i < w.nw) {
          l = max(pos - a.window + 1, w.split) - at;
          e = pos + 1 - at;
          z = -at;
          f = w.split ? 0 : min(a.sinks, pos + 1) - at;
        } else {
          f = a.sinks - at;
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) seen[v] = columns(l, max(l, e), v) | columns(z, max(z, f), v);
      }
      uint32_t s[kRows];
#pragma unroll
      for (int j = 0; j < 4; ++j) tmem_ld32(tS + 32 * j, s + 32 * j);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 4; ++j) landed32(s + 32 * j);
      if (!clean) {
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (!(seen[j / 32] >> (j % 32) & 1)) s[j] = 0xff800000u;
      }
      const float mx = fmaxf(max64(s), max64(s + 64));
      if (first || __any_sync(0xffffffffu, votes && (mx - m) * c0 > kLag)) {  // a new reference
        const float mn = first ? mx : fmaxf(m, mx);
        const bool far_now = __any_sync(0xffffffffu, votes && fabsf(mn * c0) > kFar);
        const float off_now = far_now ? kShift : kShift - mn * c0;
        if (!first) {
          // What lies between the weights before, 2^(c0 (s - [far] m) + off), and those from now on,
          // with both offsets as they were rounded.
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
      first = false;
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
      ++t;
    }
    // ---- the tile's rows
    ok = ok && wait(&sh.o[x], (t - 1) & 1);
    tc_fence_after();
    const float2 sum = __fadd2_rn(sum0, sum1);
    const float inv = ok ? 1.f / (sum.x + sum.y) : __int_as_float(0x7fc00000);
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
        o[i] = sees ? h22u(__floats2half2_rn(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv))
                           : 0u;
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
    window_attention_kernel(const __grid_constant__ WindowAttentionArgs a, const __grid_constant__ Maps maps, int pack,
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
  sh.list.build(a, 2 * cta.tpt);  // the CTA's threads together
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
      mma_role(a, cta, sh, lane);
    else if (warp == kBlockWarp)
      block_role(a, cta, sh, lane);
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

bool encode_all(Maps *m, const WindowAttentionArgs &a, int pack) {
  if (!encode(&m->q, a.q, a.T, a.Hq, kRows / pack, pack)) return false;
  if (a.Tk == 0) {  // no key in the call: no copy of one
    m->k = m->v = m->q;
    return true;
  }
  return encode(&m->k, a.k, a.Tk, a.Hkv, kRows, 1) && encode(&m->v, a.v, a.Tk, a.Hkv, kRows, 1);
}

int pack_of(const WindowAttentionArgs &a) {
  const int R = a.Hq / a.Hkv;
  int p = 1;
  while (p < kMaxPack && R % (2 * p) == 0) p *= 2;
  return p;
}

// Sets of head groups whose K and V fit in 96 MB of the 129 MB of L2, as in the attention over whole
// prompts.
unsigned sets_of(const WindowAttentionArgs &a, int pack) {
  const int64_t per_head = std::max<int64_t>(1, (int64_t)a.Tk * kD * 2 * 2);
  const int64_t heads = std::max<int64_t>(1, (96ll << 20) / per_head);  // KV heads of a set
  const int64_t groups = a.Hq / pack, width = std::min(groups, heads * (groups / a.Hkv));
  return (unsigned)((groups + width - 1) / width);
}

// Most blocks there can be: what the lengths allow.
int64_t blocks_of(const WindowAttentionArgs &a) {
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
  if ((e = cudaFuncGetAttributes(&f, window_attention_kernel)) != cudaSuccess) return e;
  if (f.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(window_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess && dev < 64) ready[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace

bool window_attention_fits(const WindowAttentionArgs &a) { return blocks_of(a) <= 0x7fffffff; }

cudaError_t launch_window_attention(const WindowAttentionArgs &a, cudaStream_t st) {
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
  window_attention_kernel<<<(unsigned)std::min<int64_t>(blocks_of(a), sms), kThreads, kSmem, st>>>(a, maps, pack, sets_of(a, pack));
  return cudaGetLastError();
}

}  // namespace kivi
