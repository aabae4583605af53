// kivi_tcgen05.cuh -- what the attention kernels over packed prompts share: barriers, tensor-map
// copies, the tensor-core products of 128 x 128 tiles in tensor memory (tcgen05), and the softmax's
// small pieces (sm_103a).
#pragma once

#include <cuda.h>
#include <math.h>

#include "kivi_device.cuh"
#include "kivi_internal.h"

namespace kivi {

namespace {

constexpr int kRows = 128;                  // query rows of a tile, keys of a tile
constexpr int kTileBytes = kRows * kD * 2;  // 32 KB: two halves of 64 channels
constexpr int kHalfBytes = kTileBytes / 2;  // 128 rows of 128 bytes, 128-byte swizzle
constexpr int kMaxPack = 16;
constexpr float kLag = 11.f;                // log2 by which the reference maximum may lag
constexpr float kShift = 4.f;               // log2 of the probabilities' scale
constexpr float kFar = 1 << 16;             // |log2 score| from which an offset in fp32 (2^-8 there) is not enough
constexpr float kLog2eP = 1.4426950408889634f;
constexpr int kPolls = 1 << 22;             // of a wait, each suspended by the hardware for a while
constexpr uint32_t kTmemCols = 512;

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
// Four MMAs of a 128 x 64 x 128 product: A in tensor memory (16 fp16 are 8 columns), B's
// contraction along the rows, 16 rows a step.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n"
      " .reg .pred p, q, t;\n"
      " .reg .b32 x, y;\n"
      " .reg .b64 b;\n"
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

// ---- softmax
// Marks 32 registers as written here: what reads them stays behind the wait before.
__device__ __forceinline__ void landed32(uint32_t *r) {
#pragma unroll
  for (int k = 0; k < 32; k += 8)
    asm volatile(""
                 : "+r"(r[k]), "+r"(r[k + 1]), "+r"(r[k + 2]), "+r"(r[k + 3]), "+r"(r[k + 4]), "+r"(r[k + 5]),
                   "+r"(r[k + 6]), "+r"(r[k + 7]));
}

__device__ __forceinline__ float max64(const uint32_t *s) {
  float mx[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) mx[j] = fmaxf(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
#pragma unroll
  for (int k = 8; k < 64; k += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) mx[j] = max3(mx[j], __uint_as_float(s[k + 2 * j]), __uint_as_float(s[k + 2 * j + 1]));
  return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
}

// ---- tensor maps
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

}  // namespace

}  // namespace kivi
