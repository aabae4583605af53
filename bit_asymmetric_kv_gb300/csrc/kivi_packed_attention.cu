// kivi_packed_attention.cu -- causal attention over prompts of different lengths packed
// into one token axis (sm_103a, tensor memory and the tensor-map copy engine).
//
// For row i of a sequence (rows counted from its start) and query head h, reading KV
// head h / (Hq / Hkv):
//   out_i = sum_{j <= i} softmax_j(sigma q_i . k_j) v_j,   j over the same sequence.
//
// One CTA takes two tiles, A and B, of 128 query rows, and walks the keys and values
// in tiles of 128 rows from the diagonal down to the sequence's first.  A query tile is
// 128 / P consecutive tokens of P query heads that read the same KV head, P the
// largest power of two (up to 16) that divides Hq / Hkv: the heads of a group share every
// key and value tile, and a short prompt wastes fewer rows of a tile.
//
// Roles (12 warps, the last two idle):
//   warps 0-3, 4-7  softmax of tile A, of tile B: a thread holds one row.  It reads the 128
//                   scores from tensor memory, keeps the running maximum and sum, and
//                   writes the probabilities over the scores, as fp16.
//   warp 8          one lane issues the MMAs: S = Q K^T (both operands in shared memory) and
//                   O += P V (P in tensor memory), tile A and B in turn, so that one
//                   tile's softmax runs under the other's MMAs.
//   warp 9          one lane issues the tensor-map copies: Q once, K and V tiles through a
//                   ring of stages.
// Tensor memory: S/P of A and B (128 columns each), O of A and B (128 each): all 512.
//
// The maximum that the probabilities are relative to may lag behind the true one by 2^8:
// only beyond that are the sums and the output in tensor memory rescaled, which
// happens in the first tiles of a row and then hardly ever.  The probabilities are scaled by
// 2^7 on top, so that they use fp16's range (at most 2^15; the smallest lie 2^31 below)
// and their rounding, 2^-11 of each, is the only one below fp32 before the output's.
//
// Rows behind a sequence's end share its last tiles.  As query rows they are computed and
// not stored; as keys they are masked by causality; as values they would meet
// probability 0, and a NaN there would spread, so warp 9 overwrites them with zeros.
//
// Every wait is bounded: one that runs out (a copy that never completes) ends all roles
// of the CTA, whose rows are then NaN.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "kivi_device.cuh"
#include "kivi_internal.h"
#include "kivi_packed.cuh"

namespace kivi {

namespace {

constexpr int kRows = 128;                  // query rows of a tile, keys of a tile
constexpr int kThreads = 384;               // three warpgroups
constexpr int kMmaWarp = 8, kLoadWarp = 9;
// Registers a thread: the CTA's share at launch, and how the warpgroups split it (a
// softmax thread holds a row of 128 scores).
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "more registers than the CTA was launched with");
constexpr int kTileBytes = kRows * kD * 2;  // 32 KB: two halves of 64 channels
constexpr int kHalfBytes = kTileBytes / 2;  // 128 rows of 128 bytes, 128-byte swizzle
constexpr int kStages = 5;                  // K and V tiles in flight
constexpr int kMaxPack = 16;
constexpr float kLag = 8.f;                 // log2 by which the reference maximum may lag
constexpr float kShift = 7.f;               // log2 of the probabilities' scale
constexpr float kLog2eP = 1.4426950408889634f;
constexpr int kPolls = 1 << 22;             // of a wait, each suspended by the hardware for a while
constexpr uint32_t kTmemCols = 512;

struct __align__(8) Bars {
  uint64_t q[2];           // Q tile landed
  uint64_t full[kStages];  // K or V tile landed
  uint64_t empty[kStages]; // the MMAs that read it are done
  uint64_t s[2];           // scores of a tile written
  uint64_t p[2];           // its probabilities written
  uint64_t o[2];           // its P.V done
  uint64_t zeroed;         // value rows behind the sequence overwritten
  uint32_t tmem;
  int abort;
  int found;
  PackedBlock blk;
};
constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + (int)sizeof(Bars);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

struct Maps {
  CUtensorMap q, k, v;
};

// What the roles of a CTA work on.
struct Work {
  unsigned char *tiles;  // Q of A, Q of B, the stages
  uint32_t sQ, sKV;
  uint32_t tmem;
  int start, len;        // the sequence
  int head0, kvh;
  int tpt;               // tokens of a query tile
  int base[2];           // first token of A, of B
  bool on[2];
  int nt[2];             // key tiles, the last one on the diagonal
  int n;                 // passes: pass i works on key tile n - 1 - i
  int tail;              // rows of the last key tile inside the sequence (more than a tile: all)
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint64_t *b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// False when the wait ran out, here or in another role.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, int *abort) {
  for (int i = 0; i < kPolls; ++i) {
    if (bar_try(b, parity)) return true;
    if ((i & 255) == 255 && *reinterpret_cast<volatile int *>(abort)) return false;
  }
  *reinterpret_cast<volatile int *>(abort) = 1;
  return false;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// ---- tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// The MMA warp runs converged, so that addresses and descriptors stay in uniform
// registers; only the instructions themselves are one lane's (`one` is 1 in it, else 0).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one;
}
// arrives on the barrier when every MMA issued so far by the lane is done
__device__ __forceinline__ void tc_commit(uint64_t *b, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n"
      " @p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(b)),
      "r"(one)
      : "memory");
}

// Shared-memory descriptor of a tile half, 128-byte swizzle: addresses in 16-byte units
// in the low word, lead at bits 16-29, stride (8 rows of 128 bytes: 1024 bytes) at 32-45,
// version and swizzle above.  With the contraction along the rows' bytes (Q, K) lead is
// not used; with it along the rows (V) lead is the distance between the two 64-channel halves.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
// Instruction descriptor: fp32 accumulators (bit 4), fp16 operands, B's major axis (bit
// 16: 1 when its rows are the contraction), N / 8 at 17, M / 16 at 24.
constexpr uint32_t kIdescQK = (1u << 4) | ((kRows / 8) << 17) | ((kRows / 16) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((kD / 8) << 17) | ((kRows / 16) << 24);

// The eight MMAs of a 128 x 128 x 128 product, 16 of the contraction each, by the lane with
// `one` set.  Both operands in shared memory, contraction along the rows' bytes: 32 bytes a
// step, then the other half.  acc: add to what the accumulators hold.
__device__ __forceinline__ void mma_qk(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n"
      " .reg .pred p, q, t;\n"
      " .reg .b32 x, y;\n"
      " .reg .b64 a, b;\n"
      " setp.ne.u32 p, %6, 0;\n"
      " setp.ne.u32 q, %5, 0;\n"
      " setp.eq.u32 t, 0, 0;\n"
      " add.u32 x, %1, 0;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 0;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n"
      " add.u32 x, %1, 2;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 2;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 4;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 4;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 6;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 6;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1024;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 1024;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1026;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 1026;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1028;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 1028;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.u32 x, %1, 1030;\n"
      " mov.b64 a, {x, %4};\n"
      " add.u32 y, %2, 1030;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"(acc), "r"(one)
      : "memory");
}
// A in tensor memory (16 fp16 are 8 columns), B's contraction along the rows: 16 rows a step.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n"
      " .reg .pred p, q, t;\n"
      " .reg .b32 x, y;\n"
      " .reg .b64 a, b;\n"
      " setp.ne.u32 p, %6, 0;\n"
      " setp.ne.u32 q, %5, 0;\n"
      " setp.eq.u32 t, 0, 0;\n"
      " add.u32 x, %1, 0;\n"
      " add.u32 y, %2, 0;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n"
      " add.u32 x, %1, 8;\n"
      " add.u32 y, %2, 128;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n"
      " add.u32 x, %1, 16;\n"
      " add.u32 y, %2, 256;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n"
      " add.u32 x, %1, 24;\n"
      " add.u32 y, %2, 384;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n"
      " add.u32 x, %1, 32;\n"
      " add.u32 y, %2, 512;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n"
      " add.u32 x, %1, 40;\n"
      " add.u32 y, %2, 640;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n"
      " add.u32 x, %1, 48;\n"
      " add.u32 y, %2, 768;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n"
      " add.u32 x, %1, 56;\n"
      " add.u32 y, %2, 896;\n"
      " mov.b64 b, {y, %4};\n"
      " @p tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"(acc), "r"(one)
      : "memory");
}

// 32 columns of this warp's 32 lanes, one row per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};\n" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// ---------------------------------------------------------------------------- copies
// Copy c brings K of pass c / 2 (even c) or its V (odd c) into stage c % kStages.
__device__ __forceinline__ void load_role(const Maps &maps, const Work &w, Bars &sh, int lane) {
  bool ok = true;
  int issued = 0;
  if (lane == 0) {
    for (int x = 0; x < 2; ++x)
      if (w.on[x]) {
        bar_expect(&sh.q[x], kTileBytes);
        for (int half = 0; half < 2; ++half)
          tma_3d(w.sQ + x * kTileBytes + half * kHalfBytes, &maps.q, 64 * half, w.start + w.base[x], w.head0, &sh.q[x]);
      }
  }
  for (int c = 0; c < 2 * w.n && ok; ++c) {
    const int st = c % kStages;
    if (c >= kStages) ok = __all_sync(0xffffffffu, bar_wait(&sh.empty[st], (c / kStages - 1) & 1, &sh.abort));
    if (ok && lane == 0) {
      bar_expect(&sh.full[st], kTileBytes);
      for (int half = 0; half < 2; ++half)
        tma_3d(w.sKV + st * kTileBytes + half * kHalfBytes, c & 1 ? &maps.v : &maps.k, 64 * half,
               w.start + (w.n - 1 - c / 2) * kRows, w.kvh, &sh.full[st]);
    }
    issued += ok;
    if (c == min(2 * w.n, kStages) - 1 && w.tail < kRows) {
      // the value rows behind the sequence, in copy 1: its first use waits for `zeroed`
      ok = __all_sync(0xffffffffu, bar_wait(&sh.full[1], 0, &sh.abort));
      unsigned char *v = w.tiles + (2 + 1) * kTileBytes;
      for (int r = w.tail * 8 + lane; r < kRows * 8; r += 32)
        for (int half = 0; half < 2; ++half)
          *reinterpret_cast<uint4 *>(v + half * kHalfBytes + r * 16) = make_uint4(0u, 0u, 0u, 0u);
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.zeroed);
    }
  }
  if (!ok && lane == 0) {  // the copies in flight land before the CTA ends
    int never = 0;
    for (int x = 0; x < 2 && !never; ++x)
      if (w.on[x]) bar_wait(&sh.q[x], 0, &never);
    for (int c = max(0, issued - kStages); c < issued && !never; ++c)
      bar_wait(&sh.full[c % kStages], (c / kStages) & 1, &never);
  }
  __syncwarp();
}

// -------------------------------------------------------------------------- products
__device__ __forceinline__ void mma_role(const Work &w, Bars &sh) {
  const uint32_t one = elect_one();
  bool ok = true;
  const uint32_t q0 = desc_lo(w.sQ, 16), k0 = desc_lo(w.sKV, 16), v0 = desc_lo(w.sKV, kHalfBytes);
  constexpr uint32_t kTile16 = kTileBytes >> 4;
  auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(b, parity, &sh.abort)) != 0; };
  auto qk = [&](int x, int st) {  // scores of tile x with the K tile in stage st
    mma_qk(w.tmem + x * kRows, q0 + x * kTile16, k0 + st * kTile16, kIdescQK, 0, one);
    tc_commit(&sh.s[x], one);
  };
  auto pv = [&](int x, int st, bool acc) {  // output of tile x with the V tile in stage st
    mma_pv(w.tmem + 2 * kRows + x * kD, w.tmem + x * kRows, v0 + st * kTile16, kIdescPV, acc, one);
    tc_commit(&sh.o[x], one);
  };
  // A stage is handed back only where a later copy waits for it: no arrival is left over
  // when the CTA ends.
  auto give = [&](int c, int st) {
    if (c + kStages < 2 * w.n) tc_commit(&sh.empty[st], one);
  };
  const int nt0 = w.nt[0], nt1 = w.nt[1];
  int done0 = 0, done1 = 0;  // P.V products of each tile
  ok = wait(&sh.q[0], 0);
  if (ok && nt1) ok = wait(&sh.q[1], 0);
  ok = ok && wait(&sh.full[0], 0);
  tc_fence_after();
  if (ok) {
    if (w.n <= nt0) qk(0, 0);
    if (w.n <= nt1) qk(1, 0);
    give(0, 0);
    if (w.tail < kRows) ok = wait(&sh.zeroed, 0);
  }
  int sv = 1, sk = 2, cv = 1;       // stages of V of pass i and K of pass i + 1; copy of the former
  uint32_t pv_par = 0, pk_par = 0;  // and their phases
  for (int i = 0; i < w.n && ok; ++i) {
    const int left = w.n - 1 - i;  // key tile of this pass
    const bool more = left > 0;
    ok = wait(&sh.full[sv], pv_par);
    if (ok && left < nt0) {
      ok = wait(&sh.p[0], done0 & 1);
      if (!ok) break;
      tc_fence_after();
      pv(0, sv, done0 > 0);
      ++done0;
    }
    if (ok && more) ok = wait(&sh.full[sk], pk_par);
    if (!ok) break;
    // the scores go where the probabilities were: MMAs run in the order of issue
    if (more && left - 1 < nt0) qk(0, sk);
    if (left < nt1) {
      ok = wait(&sh.p[1], done1 & 1);
      if (!ok) break;
      tc_fence_after();
      pv(1, sv, done1 > 0);
      ++done1;
    }
    give(cv, sv);
    if (more && left - 1 < nt1) qk(1, sk);
    give(cv + 1, sk);
    cv += 2;
    sv += 2;
    if (sv >= kStages) {
      sv -= kStages;
      pv_par ^= 1;
    }
    sk += 2;
    if (sk >= kStages) {
      sk -= kStages;
      pk_par ^= 1;
    }
  }
}

// --------------------------------------------------------------------------- softmax
__device__ __forceinline__ void softmax_role(const PackedAttentionArgs &a, const Work &w, Bars &sh, int x, int warp,
                                             int lane) {
  const int r = 32 * warp + lane;  // row of tile x
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t tS = w.tmem + x * kRows + lanes, tO = w.tmem + 2 * kRows + x * kD + lanes;
  const int base = x ? w.base[1] : w.base[0], nt = x ? w.nt[1] : w.nt[0];
  const int token = base + r % w.tpt;
  const float c0 = a.softmax_scale * kLog2eP;
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  for (int t = 0; t < nt; ++t) {
    ok = __all_sync(0xffffffffu, bar_wait(&sh.s[x], t & 1, &sh.abort));
    if (!ok) break;
    tc_fence_after();
    uint32_t s[kRows];
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_ld32(tS + 32 * k, s + 32 * k);
    tc_wait_ld();
    if (t == 0) {  // the tile on the diagonal
      const int last = token - (nt - 1) * kRows;  // the row's own key in it
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (k > last) s[k] = 0xff800000u;
    }
    float mx0 = __uint_as_float(s[0]), mx1 = __uint_as_float(s[1]);
#pragma unroll
    for (int k = 2; k + 3 < kRows; k += 4) {
      mx0 = max3(mx0, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
      mx1 = max3(mx1, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
    }
    mx0 = max3(mx0, __uint_as_float(s[kRows - 2]), __uint_as_float(s[kRows - 1]));
    const float mx = fmaxf(mx0, mx1);
    if (t == 0) {
      m = mx;
    } else if (__any_sync(0xffffffffu, (mx - m) * c0 > kLag)) {
      const float mn = fmaxf(m, mx);
      const float al = ex2((m - mn) * c0);
      m = mn;
      l *= al;
      ok = __all_sync(0xffffffffu, bar_wait(&sh.o[x], (t - 1) & 1, &sh.abort));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * k, o);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
        tmem_st32(tO + 32 * k, o);
      }
    }
    const float b = kShift - m * c0;
    const float2 c2 = make_float2(c0, c0), b2 = make_float2(b, b);
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
    for (int k = 0; k < kRows / 2; ++k) {
      const float2 e = __ffma2_rn(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), c2, b2);
      const float2 p = make_float2(ex2(e.x), ex2(e.y));
      if (k & 1)
        sum1 = __fadd2_rn(sum1, p);
      else
        sum0 = __fadd2_rn(sum0, p);
      s[k] = h22u(__floats2half2_rn(p.x, p.y));
    }
    sum0 = __fadd2_rn(sum0, sum1);
    l += sum0.x + sum0.y;
    tmem_st32(tS, s);
    tmem_st32(tS + 32, s + 32);
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.p[x]);
  }
  if (ok) ok = __all_sync(0xffffffffu, bar_wait(&sh.o[x], (nt - 1) & 1, &sh.abort));
  tc_fence_after();
  // ---- the tile's rows, through the shared memory of its Q tile (16-byte chunk c of row r
  // at chunk c ^ (r % 8)), then written row by row
  const float inv = ok ? 1.f / l : __int_as_float(0x7fc00000);
  unsigned char *so = w.tiles + x * kTileBytes;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t o[32];
    tmem_ld32(tO + 32 * k, o);
    tc_wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[j] = h22u(__floats2half2_rn(__uint_as_float(o[8 * c + 2 * j]) * inv,
                                      __uint_as_float(o[8 * c + 2 * j + 1]) * inv));
      *reinterpret_cast<uint4 *>(so + r * 256 + ((4 * k + c) ^ (r & 7)) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
  __syncwarp();
  for (int it = 0; it < 16; ++it) {
    const int rr = 32 * warp + 2 * it + (lane >> 4), c = lane & 15;
    const int tok = base + rr % w.tpt;
    if (tok < w.len) {
      uint16_t *dst = a.out.p + (int64_t)(w.start + tok) * a.out.ts + (int64_t)(w.head0 + rr / w.tpt) * a.out.hs + 8 * c;
      *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(so + rr * 256 + (c ^ (rr & 7)) * 16);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    packed_attention_kernel(const __grid_constant__ PackedAttentionArgs a, const __grid_constant__ Maps maps, int pack) {
  extern __shared__ unsigned char raw[];
  Work w;
  // tiles start at a multiple of the swizzle's 1024-byte pattern
  w.tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Bars &sh = *reinterpret_cast<Bars *>(w.tiles + (2 + kStages) * kTileBytes);
  w.sQ = smem_u32(w.tiles);
  w.sKV = w.sQ + 2 * kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  w.tpt = kRows / pack;
  const unsigned hgroups = (unsigned)(a.Hq / pack);  // head groups that share a tile
  w.head0 = (int)(blockIdx.x % hgroups) * pack;
  w.kvh = w.head0 / (a.Hq / a.Hkv);

  if (warp == 0) {
    PackedBlock blk = {};
    const bool found = packed_block(a.cu, a.n_seqs, a.T, 2 * w.tpt, blockIdx.x / hgroups, &blk);
    if (lane == 0) {
      sh.found = found;
      sh.blk = blk;
      sh.abort = 0;
    }
  }
  if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int x = 0; x < 2; ++x) {
        bar_init(&sh.q[x], 1);
        bar_init(&sh.s[x], 1);
        bar_init(&sh.p[x], 4);
        bar_init(&sh.o[x], 1);
      }
      for (int i = 0; i < kStages; ++i) {
        bar_init(&sh.full[i], 1);
        bar_init(&sh.empty[i], 1);
      }
      bar_init(&sh.zeroed, 1);
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  w.tmem = sh.tmem;
  if (sh.found) {
    w.start = sh.blk.start;
    w.len = sh.blk.len;
    w.base[0] = sh.blk.level * 2 * w.tpt;
    w.base[1] = w.base[0] + w.tpt;
    w.on[0] = true;
    w.on[1] = w.base[1] < w.len;
    w.nt[0] = w.base[0] / kRows + 1;
    w.nt[1] = w.on[1] ? w.base[1] / kRows + 1 : 0;
    w.n = max(w.nt[0], w.nt[1]);
    w.tail = w.len - (w.n - 1) * kRows;
    if (warp >= kMmaWarp) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
      if (warp == kLoadWarp) {
        load_role(maps, w, sh, lane);
      } else if (warp == kMmaWarp) {
        mma_role(w, sh);
      }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
      const int x = warp >> 2;
      if (x == 0 || w.on[1]) softmax_role(a, w, sh, x, warp & 3, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(w.tmem), "r"(kTmemCols) : "memory");
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Map of a [T][heads][128] tensor with boxes of 64 channels, `box_tokens` rows and
// `box_heads` heads, stored one 128-byte row after another with the 128-byte swizzle.
bool encode(CUtensorMap *m, const PackedRows &r, int T, int heads, int box_tokens, int box_heads) {
  const EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)T, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)r.ts * 2, (cuuint64_t)r.hs * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_tokens, (cuuint32_t)box_heads};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, r.p, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int pack_of(const PackedAttentionArgs &a) {
  const int R = a.Hq / a.Hkv;
  int p = 1;
  while (p < kMaxPack && R % (2 * p) == 0) p *= 2;
  return p;
}

int64_t grid_of(const PackedAttentionArgs &a) {
  const int pack = pack_of(a);
  return ((int64_t)a.T / (2 * kRows / pack) + a.n_seqs) * (a.Hq / pack);
}

// Once per device: the shared memory's limit, and that the kernel has the registers that the
// warpgroups' split of them rests on.
cudaError_t prepare_kernel() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes f;
  if ((e = cudaFuncGetAttributes(&f, packed_attention_kernel)) != cudaSuccess) return e;
  if (f.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(packed_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace

bool packed_attention_fits(const PackedAttentionArgs &a) { return grid_of(a) <= 0x7fffffff; }

cudaError_t launch_packed_attention(const PackedAttentionArgs &a, cudaStream_t st) {
  const int pack = pack_of(a);
  Maps maps;
  if (!encode(&maps.q, a.q, a.T, a.Hq, kRows / pack, pack) || !encode(&maps.k, a.k, a.T, a.Hkv, kRows, 1) ||
      !encode(&maps.v, a.v, a.T, a.Hkv, kRows, 1))
    return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel();
  if (e != cudaSuccess) return e;
  packed_attention_kernel<<<(unsigned)grid_of(a), kThreads, kSmem, st>>>(a, maps, pack);
  return cudaGetLastError();
}

}  // namespace kivi
