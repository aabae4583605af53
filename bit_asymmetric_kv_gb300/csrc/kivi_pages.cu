// kivi_pages.cu -- pages of a paged cache handed out, shared, copied, given back and
// moved (sm_103a).
//
// The state is the block table and one reference count per page: a page is free when
// its count is not positive, and holds no other mark, so nothing can disagree with it.
// Every call works on the lowest free pages, in the order of the sequences, so its
// result does not depend on timing.
//
// Each call is one planning kernel, a cluster of 8 CTAs that share the counts out
// between them (counts per CTA are exchanged through distributed shared memory, then
// every CTA lists its own slice), and, where data moves, kernels that copy it, launched so
// that they start as the one before ends.
//
// Measured: reserve with a reorder before it, 512 sequences and 53 thousand pages, 31 us (8
// sequences: 18); a beam step of 256 sequences of up to 4096 tokens, 21 us (one beam search of
// 4: 14); a pool of 11 thousand pages compacted, 117 MB moved, 41 us, of which the copy is 18
// (0.94 of the measured copy bandwidth).  Small calls are bound by latency: a launch, a few
// cluster barriers and dependent reads of the counts.
#include <cooperative_groups.h>

#include "kivi_internal.h"

namespace cg = cooperative_groups;

namespace kivi {

namespace {

constexpr int kPoolCtas = 8, kPoolThreads = 1024, kPoolWarps = kPoolThreads / 32;
constexpr int kTile = 4 * kPoolThreads;  // counts a CTA reads at once
constexpr int kD = 128;

// Workspace, all of it written before it is read:
//   list  [num_pages]         free pages in order (reserve, reorder); pages to fill (compact)
//   from  [num_pages]         compact: pages to move
//   table [B][max_pages]      reorder: the new rows
//   plan  [6][B]              reorder: Plan below
//   count [4]                 compact: pages to move
//   snap  [B][Hkv][G][128] fp16, twice with a value residual: residuals about to be overwritten
struct Ws {
  int32_t *list, *from, *table, *plan, *count;
  uint16_t *k_snap, *v_snap;
};
struct Plan {        // of sequence b
  int src;           // sequence it becomes a copy of, -1: nothing to copy
  int from, to;      // page to copy, -1: none
  int n;             // its tokens
  int snap;          // 1: its residual is needed by another sequence, copied aside first
  int old_n;         // tokens before the call
};

size_t round16(size_t x) { return (x + 15) / 16 * 16; }

size_t layout(int B, int Hkv, int G, int max_pages, int64_t num_pages, bool v_res, void *base, Ws *w) {
  char *p = static_cast<char *>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char *r = p + at;
    at += round16(bytes);
    return r;
  };
  char *list = take((size_t)num_pages * 4), *from = take((size_t)num_pages * 4);
  char *table = take((size_t)B * max_pages * 4), *plan = take((size_t)B * 24), *count = take(16);
  const size_t res = (size_t)B * Hkv * G * kD * 2;
  char *ks = take(res), *vs = v_res ? take(res) : nullptr;
  if (w) {
    w->list = reinterpret_cast<int32_t *>(list);
    w->from = reinterpret_cast<int32_t *>(from);
    w->table = reinterpret_cast<int32_t *>(table);
    w->plan = reinterpret_cast<int32_t *>(plan);
    w->count = reinterpret_cast<int32_t *>(count);
    w->k_snap = reinterpret_cast<uint16_t *>(ks);
    w->v_snap = reinterpret_cast<uint16_t *>(vs);
  }
  return at;
}

struct Shared {
  int warp[kPoolWarps];
  int total;
  int share[2][kPoolCtas];
};

// Exclusive prefix of v over the CTA's threads; *total gets the sum.
__device__ int block_scan(int v, Shared &sh, int *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  __syncthreads();  // the last scan's sums have been read
  if (lane == 31) sh.warp[w] = incl;
  __syncthreads();
  const int x = sh.warp[lane];
  int before = __reduce_add_sync(0xffffffffu, lane < w ? x : 0);
  *total = __reduce_add_sync(0xffffffffu, x);
  return before + incl - v;
}

// Gives every CTA the counts of all (two of them at once): the sums over the CTAs
// before this one, and over all.  It writes into the other CTAs' shared memory, so a cluster
// barrier has to come before it: until then one of them may not have started.  A kernel that
// has none by then arrives at one on entry and waits for it here, behind its counting pass.
struct Spread {
  int before, all;
};
__device__ void exchange(cg::cluster_group &cl, Shared &sh, int a, int b, Spread *x, Spread *y) {
  const int r = (int)cl.block_rank();
  if (threadIdx.x < kPoolCtas) {
    Shared *o = cl.map_shared_rank(&sh, threadIdx.x);
    o->share[0][r] = a;
    o->share[1][r] = b;
  }
  cl.sync();
  *x = *y = Spread{0, 0};
  for (int i = 0; i < kPoolCtas; ++i) {
    const int u = sh.share[0][i], v = sh.share[1][i];
    x->all += u;
    y->all += v;
    if (i < r) {
      x->before += u;
      y->before += v;
    }
  }
}

// This CTA's slice [lo, hi) of the counts: whole tiles, so that reads stay aligned.
__device__ void slice(int rank, int n, int *lo, int *hi) {
  const int64_t tiles = ((int64_t)n + kTile - 1) / kTile, per = (tiles + kPoolCtas - 1) / kPoolCtas;
  *lo = (int)min((int64_t)n, per * rank * kTile);
  *hi = (int)min((int64_t)n, per * (rank + 1) * kTile);
}

// Four counts from i, 1 where none (past the end).  Other CTAs may have changed them
// in this kernel: read at L2.
__device__ int4 counts4(const int32_t *refs, int i, int hi, int none) {
  if (i + 3 < hi) return __ldcg(reinterpret_cast<const int4 *>(refs + i));
  int4 c = make_int4(none, none, none, none);
  if (i < hi) c.x = __ldcg(refs + i);
  if (i + 1 < hi) c.y = __ldcg(refs + i + 1);
  if (i + 2 < hi) c.z = __ldcg(refs + i + 2);
  return c;
}

// Pages of the slice with pred(count, id).
template <class Pred>
__device__ int count_slice(const int32_t *refs, int lo, int hi, int none, Shared &sh, Pred pred) {
  int c = 0;
  for (int i = lo + 4 * threadIdx.x; i < hi; i += kTile) {
    const int4 x = counts4(refs, i, hi, none);
    c += (int)pred(x.x, i) + (int)pred(x.y, i + 1) + (int)pred(x.z, i + 2) + (int)pred(x.w, i + 3);
  }
  int total;
  block_scan(c, sh, &total);
  return total;
}

// Calls emit(rank, id) for every such page, ranks in order of the ids from `rank0`, while
// ranks stay below `limit`.
template <class Pred, class Emit>
__device__ void list_slice(const int32_t *refs, int lo, int hi, int none, Shared &sh, int rank0, int limit, Pred pred,
                           Emit emit) {
  for (int base = lo; base < hi && rank0 < limit; base += kTile) {
    const int i = base + 4 * threadIdx.x;
    const int4 x = counts4(refs, i, hi, none);
    const bool p0 = pred(x.x, i), p1 = pred(x.y, i + 1), p2 = pred(x.z, i + 2), p3 = pred(x.w, i + 3);
    int total;
    int k = rank0 + block_scan((int)p0 + (int)p1 + (int)p2 + (int)p3, sh, &total);
    if (p0) {
      if (k < limit) emit(k, i);
      ++k;
    }
    if (p1) {
      if (k < limit) emit(k, i + 1);
      ++k;
    }
    if (p2) {
      if (k < limit) emit(k, i + 2);
      ++k;
    }
    if (p3 && k < limit) emit(k, i + 3);
    rank0 += total;
  }
}

__device__ __forceinline__ bool in_pool(const PoolArgs &a, int page) { return page >= 0 && page < a.num_pages; }

// Tokens of a length, clamped to what the table can hold.
__device__ __forceinline__ int clamp_len(const PoolArgs &a, int n) { return min(max(n, 0), a.max_pages << a.shift); }

// ------------------------------------------------------------------------- reserve
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads)
    pool_reserve_kernel(const PoolArgs a, const Ws ws) {
  __shared__ Shared sh;
  __shared__ int s_rank[64];  // missing entries of this CTA's rows, then the rank of each row's first
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();  // this CTA runs: see exchange()
  const int r = (int)cl.block_rank(), lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int per = (a.B + kPoolCtas - 1) / kPoolCtas;  // <= 64
  const int b0 = min(a.B, per * r), rows = min(a.B, b0 + per) - b0;
  auto entries = [&](int b) {  // table entries that sequence b is to have
    const int extra = a.arg[b];
    if (extra <= 0) return 0;
    const int64_t cap = (int64_t)a.max_pages << a.shift;
    const int64_t want = min(cap, (int64_t)max(a.seq_lens[b], 0) + extra);
    return (int)((want + (1 << a.shift) - 1) >> a.shift);
  };
  for (int i = w; i < rows; i += kPoolWarps) {
    const int m = entries(b0 + i);
    const int32_t *row = a.bt + (int64_t)(b0 + i) * a.max_pages;
    int c = 0;
#pragma unroll 4
    for (int j = lane; j < m; j += 32) c += !in_pool(a, row[j]);
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) s_rank[i] = c;
  }
  int lo, hi;
  slice(r, a.num_pages, &lo, &hi);
  auto is_free = [](int c, int) { return c <= 0; };
  const int nfree = count_slice(a.refs, lo, hi, 1, sh, is_free);  // synchronises: s_rank is complete
  int missing;
  const int before = block_scan((int)threadIdx.x < rows ? s_rank[threadIdx.x] : 0, sh, &missing);
  Spread fr, ms;
  cl.barrier_wait();  // every CTA runs
  exchange(cl, sh, nfree, missing, &fr, &ms);
  if ((int)threadIdx.x < rows) s_rank[threadIdx.x] = ms.before + before;
  const int got = min(fr.all, ms.all);
  list_slice(a.refs, lo, hi, 1, sh, fr.before, got, is_free, [&](int k, int id) {
    ws.list[k] = id;
    a.refs[id] = 1;
  });
  cl.sync();  // the list is complete
  for (int i = w; i < rows; i += kPoolWarps) {
    const int m = entries(b0 + i);
    int32_t *row = a.bt + (int64_t)(b0 + i) * a.max_pages;
    int k = s_rank[i];
    for (int j0 = 0; j0 < m; j0 += 128) {  // four loads in flight
      int page[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) page[u] = j0 + 32 * u + lane < m ? row[j0 + 32 * u + lane] : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool want = !in_pool(a, page[u]);  // page 0 past the end is one
        const uint32_t mask = __ballot_sync(0xffffffffu, want);
        const int mine = k + __popc(mask & ((1u << lane) - 1u));
        if (want) row[j0 + 32 * u + lane] = mine < got ? __ldcg(ws.list + mine) : -1;
        k += __popc(mask);
      }
    }
  }
  if (r == 0 && threadIdx.x == 0) {
    a.info[0] = got;
    a.info[1] = ms.all - got;
    a.info[2] = a.num_pages - fr.all + got;
    a.info[3] = 0;
  }
}

// ------------------------------------------------------------------------- reorder
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads)
    pool_reorder_kernel(const PoolArgs a, const Ws ws) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __shared__ Shared sh;
  __shared__ int s_parent[kPagedMaxBatch], s_first[kPagedMaxBatch], s_len[kPagedMaxBatch];
  __shared__ int s_rank[kPagedMaxBatch], s_from[kPagedMaxBatch];
  cg::cluster_group cl = cg::this_cluster();
  const int r = (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int B = a.B, P = 1 << a.shift;
  for (int b = tid; b < B; b += kPoolThreads) {
    const int p = a.arg[b];
    s_parent[b] = p >= 0 && p < B ? p : -1;
    s_first[b] = B;
    s_len[b] = clamp_len(a, a.seq_lens[b]);
  }
  __syncthreads();
  // s_first[s]: the lowest other sequence that becomes a copy of s (B: none)
  for (int b = tid; b < B; b += kPoolThreads)
    if (s_parent[b] >= 0 && s_parent[b] != b) atomicMin(&s_first[s_parent[b]], b);
  __syncthreads();
  // the heir of s keeps its pages: s itself, else the lowest of its copies
  auto heir = [&](int s) { return s_parent[s] == s ? s : s_first[s]; };
  int want = 0;
  if (tid < B) {
    const int s = s_parent[tid];
    s_from[tid] = -1;
    if (s >= 0 && heir(s) != tid && s_len[s] % P != 0) {
      const int page = a.bt[(int64_t)s * a.max_pages + s_len[s] / P];
      if (in_pool(a, page)) {
        s_from[tid] = page;
        want = 1;
      }
    }
  }
  int wanted;
  const int rank = block_scan(want, sh, &wanted);
  if (tid < B) s_rank[tid] = rank;
  __syncthreads();
  int lo, hi;
  slice(r, a.num_pages, &lo, &hi);
  auto is_free = [](int c, int) { return c <= 0; };
  const int before = count_slice(a.refs, lo, hi, 1, sh, is_free);
  cl.sync();  // every count has been read
  // ---- the new rows, staged, and the counts of the pages that rows lose and gain
  const int per = (B + kPoolCtas - 1) / kPoolCtas;
  const int b0 = min(B, per * r), b1 = min(B, b0 + per);
  for (int b = b0 + w; b < b1; b += kPoolWarps) {
    const int s = s_parent[b];
    if (s == b) continue;
    const int32_t *old = a.bt + (int64_t)b * a.max_pages;
    const int32_t *src = s >= 0 ? a.bt + (int64_t)s * a.max_pages : old;
    const int shared = s < 0 ? 0 : (heir(s) == b ? a.max_pages : s_len[s] / P);
    for (int j0 = lane; j0 < a.max_pages; j0 += 128) {  // four loads of each in flight
      int o[4], n[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + 32 * u;
        o[u] = j < a.max_pages ? old[j] : -1;
        n[u] = j < shared ? src[j] : -1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + 32 * u;
        if (j >= a.max_pages) break;
        if (!in_pool(a, o[u])) o[u] = -1;
        if (!in_pool(a, n[u])) n[u] = -1;
        if (o[u] != n[u]) {
          if (o[u] >= 0) atomicAdd(a.refs + o[u], -1);
          if (n[u] >= 0) atomicAdd(a.refs + n[u], 1);
        }
        ws.table[(int64_t)b * a.max_pages + j] = n[u];
      }
    }
  }
  cl.sync();  // all old rows read, all counts changed
  const int nfree = count_slice(a.refs, lo, hi, 1, sh, is_free);
  Spread fr, gone;
  exchange(cl, sh, nfree, nfree - before, &fr, &gone);
  const int got = min(fr.all, wanted);
  list_slice(a.refs, lo, hi, 1, sh, fr.before, got, is_free, [&](int k, int id) {
    ws.list[k] = id;
    a.refs[id] = 1;
  });
  cl.sync();  // the list is complete
  for (int b = b0 + w; b < b1; b += kPoolWarps) {
    const int s = s_parent[b];
    Plan p = {-1, -1, -1, s_len[b], s_first[b] < B && s != b, s_len[b]};
    if (s != b) {
      p.src = s;
      p.n = s >= 0 ? s_len[s] : 0;
      const int at = p.n / P;
      if (s_from[b] >= 0) {
        if (s_rank[b] < got) {
          p.from = s_from[b];
          p.to = __ldcg(ws.list + s_rank[b]);
        } else {
          p.n = at * P;  // no page for the last tokens: the sequence ends before them
        }
      }
      int32_t *row = a.bt + (int64_t)b * a.max_pages;
      for (int j = lane; j < a.max_pages; j += 32)
        row[j] = p.to >= 0 && j == at ? p.to : ws.table[(int64_t)b * a.max_pages + j];
      if (lane == 0) a.seq_lens[b] = p.n;
    }
    if (lane == 0) {
      int32_t *x = ws.plan + 6 * b;
      x[0] = p.src;
      x[1] = p.from;
      x[2] = p.to;
      x[3] = p.n;
      x[4] = p.snap;
      x[5] = p.old_n;
    }
  }
  if (r == 0 && tid == 0) {
    a.info[0] = got;
    a.info[1] = wanted - got;
    a.info[2] = a.num_pages - fr.all + got;
    a.info[3] = gone.all;
  }
}

__device__ void copy16(void *dst, const void *src, int64_t bytes) {
  const uint4 *s = static_cast<const uint4 *>(src);
  uint4 *d = static_cast<uint4 *>(dst);
  const int64_t n = bytes / 16;
  for (int64_t i = threadIdx.x; i < n; i += 4 * blockDim.x) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * blockDim.x < n) x[j] = s[i + j * blockDim.x];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * blockDim.x < n) d[i + j * blockDim.x] = x[j];
  }
}

__device__ Plan plan_of(const Ws &ws, int b) {
  const int32_t *x = ws.plan + 6 * b;
  return Plan{x[0], x[1], x[2], x[3], x[4], x[5]};
}

// One CTA per (KV head, sequence).  Pass 0 copies the used rows of the page that the
// sequence does not share, and its residual rows where neither end is overwritten or
// needed elsewhere; residuals that others need are copied aside.  Pass 1 copies the rest.
__global__ void __launch_bounds__(128) pool_copy_kernel(const PoolArgs a, const Ws ws, int pass) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int h = blockIdx.x, b = blockIdx.y, P = 1 << a.shift, G = a.G;
  const Plan p = plan_of(ws, b);
  const int64_t head = ((int64_t)b * a.Hkv + h) * G * kD;
  const bool aside = p.src >= 0 && ws.plan[6 * p.src + 4] != 0;  // the source's residual was copied aside
  if (pass == 0) {
    if (p.to >= 0) {
      const int r = p.n % P, rg = r / G * G, rv = a.v_res ? rg : r;
      const int W = 4 * a.bits;  // words of a token row
      const int64_t f = ((int64_t)p.from * a.Hkv + h) << a.shift, t = ((int64_t)p.to * a.Hkv + h) << a.shift;
      copy16(a.k_codes + t * W, a.k_codes + f * W, (int64_t)rg * W * 4);
      copy16(a.k_meta + t / G * kD, a.k_meta + f / G * kD, (int64_t)rg / G * kD * 4);
      copy16(a.v_codes + t * W, a.v_codes + f * W, (int64_t)rv * W * 4);
      for (int i = threadIdx.x; i < rv; i += blockDim.x) a.v_meta[t + i] = a.v_meta[f + i];
    }
    if (p.snap) {
      const int64_t bytes = (int64_t)(p.old_n % G) * kD * 2;
      copy16(ws.k_snap + head, a.k_res + head, bytes);
      if (a.v_res) copy16(ws.v_snap + head, a.v_res + head, bytes);
    }
  }
  if (p.src < 0 || (p.snap || aside) != (pass == 1)) return;
  const int64_t from = ((int64_t)p.src * a.Hkv + h) * G * kD;
  const int64_t bytes = (int64_t)(p.n % G) * kD * 2;
  copy16(a.k_res + head, (aside ? ws.k_snap : a.k_res) + from, bytes);
  if (a.v_res) copy16(a.v_res + head, (aside ? ws.v_snap : a.v_res) + from, bytes);
}

// ------------------------------------------------------------------------- compact
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads)
    pool_compact_kernel(const PoolArgs a, const Ws ws) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();  // this CTA runs: see exchange()
  const int r = (int)cl.block_rank();
  int lo, hi;
  slice(r, a.num_pages, &lo, &hi);
  Spread live, movers, holes, unused;
  const int nlive = count_slice(a.refs, lo, hi, 0, sh, [](int c, int) { return c > 0; });
  cl.barrier_wait();  // every CTA runs
  exchange(cl, sh, nlive, 0, &live, &unused);
  const int L = live.all;
  auto moves = [L](int c, int id) { return c > 0 && id >= L; };
  auto hole = [L](int c, int id) { return c <= 0 && id < L; };
  const int nm = count_slice(a.refs, lo, hi, 0, sh, moves);
  const int nh = count_slice(a.refs, lo, hi, 1, sh, hole);
  cl.sync();  // the first exchange has been read everywhere
  exchange(cl, sh, nm, nh, &movers, &holes);
  list_slice(a.refs, lo, hi, 0, sh, movers.before, movers.all, moves, [&](int k, int id) { ws.from[k] = id; });
  list_slice(a.refs, lo, hi, 1, sh, holes.before, holes.all, hole, [&](int k, int id) { ws.list[k] = id; });
  cl.sync();  // both lists are complete
  for (int i = lo + threadIdx.x; i < hi; i += kPoolThreads)
    a.new_ids[i] = i < L && a.refs[i] > 0 ? i : -1;
  cl.sync();  // before the moved pages get theirs
  for (int k = r * kPoolThreads + threadIdx.x; k < movers.all; k += kPoolCtas * kPoolThreads) {
    const int f = __ldcg(ws.from + k), t = __ldcg(ws.list + k);
    a.new_ids[f] = t;
    a.refs[t] = __ldcg(a.refs + f);
  }
  cl.sync();  // the moved counts are read
  for (int i = max(lo, L) + (int)threadIdx.x; i < hi; i += kPoolThreads) a.refs[i] = 0;
  if (r == 0 && threadIdx.x == 0) {
    ws.count[0] = movers.all;
    a.info[0] = movers.all;
    a.info[1] = 0;
    a.info[2] = L;
    a.info[3] = 0;
  }
}

// Moved pages, and the table's entries.  A warp copies pieces of 4 KB (8 x 16 bytes a lane in
// flight: with 16 warps an SM, more than the memory's latency needs), so that pages of any
// size keep every SM busy.
constexpr int kMoveThreads = 256, kMoveCtas = 4, kPiece = 4096;  // CTAs an SM

__global__ void __launch_bounds__(kMoveThreads) pool_move_kernel(const PoolArgs a, const Ws ws) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int n = ws.count[0], lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.Hkv << a.shift;  // of a page, all heads
  const int64_t codes = rows * 4 * a.bits * 4, meta = rows / a.G * kD * 4, vmeta = rows * 4;
  const int64_t pc = (codes + kPiece - 1) / kPiece, pm = (meta + kPiece - 1) / kPiece, pv = (vmeta + kPiece - 1) / kPiece;
  const int64_t pieces = 2 * pc + pm + pv;
  const int64_t warps = (int64_t)gridDim.x * (kMoveThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < n * pieces; i += warps) {
    const int64_t k = i / pieces;
    int64_t piece = i - k * pieces, bytes = codes;
    char *base = reinterpret_cast<char *>(a.k_codes);
    if (piece >= 2 * pc + pm) {
      piece -= 2 * pc + pm;
      base = reinterpret_cast<char *>(a.v_meta);
      bytes = vmeta;
    } else if (piece >= 2 * pc) {
      piece -= 2 * pc;
      base = reinterpret_cast<char *>(a.k_meta);
      bytes = meta;
    } else if (piece >= pc) {
      piece -= pc;
      base = reinterpret_cast<char *>(a.v_codes);
    }
    const uint4 *from = reinterpret_cast<const uint4 *>(base + ws.from[k] * bytes + piece * kPiece) + lane;
    uint4 *to = reinterpret_cast<uint4 *>(base + ws.list[k] * bytes + piece * kPiece) + lane;
    const int left = (int)min((int64_t)kPiece, bytes - piece * kPiece) / 16 - lane;  // 16-byte words from this lane's on
    uint4 x[kPiece / 512];
#pragma unroll
    for (int j = 0; j < kPiece / 512; ++j)
      if (32 * j < left) x[j] = __ldcs(from + 32 * j);
#pragma unroll
    for (int j = 0; j < kPiece / 512; ++j)
      if (32 * j < left) __stcs(to + 32 * j, x[j]);
  }
  const int64_t entries = (int64_t)a.B * a.max_pages;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < entries; i += (int64_t)gridDim.x * blockDim.x) {
    const int page = a.bt[i];
    a.bt[i] = in_pool(a, page) ? a.new_ids[page] : -1;
  }
}

// A launch that may start while the kernel before it on the stream still runs; the kernel
// waits for that one's end (griddepcontrol.wait) before it reads anything.
template <class... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

Ws workspace_of(const PoolArgs &a) {
  Ws w;
  layout(a.B, a.Hkv, a.G, a.max_pages, a.num_pages, a.v_res != nullptr, a.ws, &w);
  return w;
}

}  // namespace

size_t pool_workspace_bytes(int B, int Hkv, int G, int max_pages, int64_t num_pages, bool value_residual) {
  return layout(B, Hkv, G, max_pages, num_pages, value_residual, nullptr, nullptr);
}

cudaError_t launch_pool_reserve(const PoolArgs &a, cudaStream_t st) {
  pool_reserve_kernel<<<kPoolCtas, kPoolThreads, 0, st>>>(a, workspace_of(a));
  return cudaGetLastError();
}

cudaError_t launch_pool_reorder(const PoolArgs &a, cudaStream_t st) {
  const Ws ws = workspace_of(a);
  pool_reorder_kernel<<<kPoolCtas, kPoolThreads, 0, st>>>(a, ws);
  cudaError_t e = cudaGetLastError();
  const dim3 grid((unsigned)a.Hkv, (unsigned)a.B);
  for (int pass = 0; pass < 2 && e == cudaSuccess; ++pass) e = launch_behind(pool_copy_kernel, grid, 128, st, a, ws, pass);
  return e;
}

cudaError_t launch_pool_compact(const PoolArgs &a, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const Ws ws = workspace_of(a);
  pool_compact_kernel<<<kPoolCtas, kPoolThreads, 0, st>>>(a, ws);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_behind(pool_move_kernel, dim3((unsigned)(sms * kMoveCtas)), kMoveThreads, st, a, ws);
}

}  // namespace kivi
