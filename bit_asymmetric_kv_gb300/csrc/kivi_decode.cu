// kivi_decode.cu -- the decode kernels over whole contexts (dense, paged, small contexts), instantiated
// from kivi_decode_body.cuh and chosen by shape.
#include "kivi_decode_body.cuh"

namespace kivi {

namespace {

template <int R, int G, bool PAGED, int BITS, int VG = kD>
__global__ void __launch_bounds__(kThreads, KIVI_DECODE_MIN_CTAS) decode_kernel(const DecodeArgs a) {
  decode_body<R, G, PAGED ? kModePaged : kModeDense, BITS, kWarps, VG>(a);
}

template <int R, int G, int BITS>
__global__ void __launch_bounds__(kSmallWarps * 32, 1) decode_small_kernel(const DecodeArgs a) {
  decode_body<R, G, kModeSmall, BITS, kSmallWarps>(a);
}

// The small path on clusters: CTAs CL * h .. CL * h + CL - 1 of NW warps each form the
// cluster of (batch, KV head) h.
template <int R, int G, int BITS, int CL, int NW>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(NW * 32, 1) decode_cluster_kernel(const DecodeArgs a) {
  decode_body<R, G, kModeSmall, BITS, NW, kD, CL>(a);
}

template <int R, int G, bool PAGED, int BITS>
const void *kernel_ptr() {
  return reinterpret_cast<const void *>(&decode_kernel<R, G, PAGED, BITS>);
}

// Dense 2-bit kernels with value channel groups of VG channels (persistent grid only).
template <int VG>
const void *select_vg_kernel(int R, int G) {
  if (G == 32)
    return R == 1   ? reinterpret_cast<const void *>(&decode_kernel<1, 32, false, 2, VG>)
           : R == 2 ? reinterpret_cast<const void *>(&decode_kernel<2, 32, false, 2, VG>)
                    : reinterpret_cast<const void *>(&decode_kernel<4, 32, false, 2, VG>);
  return R == 1   ? reinterpret_cast<const void *>(&decode_kernel<1, 64, false, 2, VG>)
         : R == 2 ? reinterpret_cast<const void *>(&decode_kernel<2, 64, false, 2, VG>)
                  : reinterpret_cast<const void *>(&decode_kernel<4, 64, false, 2, VG>);
}

template <int VG>
int vg_smem_bytes(int R, int G) {
  if (G == 32)
    return R == 1 ? Layout<1, 32, 2, VG>::kSmem : R == 2 ? Layout<2, 32, 2, VG>::kSmem : Layout<4, 32, 2, VG>::kSmem;
  return R == 1 ? Layout<1, 64, 2, VG>::kSmem : R == 2 ? Layout<2, 64, 2, VG>::kSmem : Layout<4, 64, 2, VG>::kSmem;
}

template <bool PAGED, int BITS>
const void *select_kernel(int R, int G) {
  if (G == 32)
    return R == 1   ? kernel_ptr<1, 32, PAGED, BITS>()
           : R == 2 ? kernel_ptr<2, 32, PAGED, BITS>()
                    : kernel_ptr<4, 32, PAGED, BITS>();
  return R == 1 ? kernel_ptr<1, 64, PAGED, BITS>() : R == 2 ? kernel_ptr<2, 64, PAGED, BITS>() : kernel_ptr<4, 64, PAGED, BITS>();
}

template <int R, int G, int BITS>
const void *small_ptr() {
  return reinterpret_cast<const void *>(&decode_small_kernel<R, G, BITS>);
}

template <int BITS>
const void *select_small(int R, int G) {
  if (G == 32) return R == 1 ? small_ptr<1, 32, BITS>() : R == 2 ? small_ptr<2, 32, BITS>() : small_ptr<4, 32, BITS>();
  return R == 1 ? small_ptr<1, 64, BITS>() : R == 2 ? small_ptr<2, 64, BITS>() : small_ptr<4, 64, BITS>();
}

template <int R, int G, int BITS, int CL, int NW>
const void *cluster_ptr() {
  return reinterpret_cast<const void *>(&decode_cluster_kernel<R, G, BITS, CL, NW>);
}

template <int BITS, int CL, int NW>
const void *select_cluster(int R, int G) {
  if (G == 32)
    return R == 1   ? cluster_ptr<1, 32, BITS, CL, NW>()
           : R == 2 ? cluster_ptr<2, 32, BITS, CL, NW>()
                    : cluster_ptr<4, 32, BITS, CL, NW>();
  return R == 1 ? cluster_ptr<1, 64, BITS, CL, NW>() : R == 2 ? cluster_ptr<2, 64, BITS, CL, NW>() : cluster_ptr<4, 64, BITS, CL, NW>();
}

// Shared memory of a cluster kernel's CTA: its warps' rings and partials.  A CTA of
// fewer than 8 warps claims more than half of an SM's 228 KB, so that every CTA of a
// cluster has an SM to itself (8 warps of two CTAs on one SM take each unit's compute
// longer).
constexpr int kOwnSmSmem = 116 * 1024;
template <int R, int G, int BITS, int CL, int NW>
constexpr int cluster_smem() {
  constexpr int b = NW * Layout<R, G, BITS>::kWarpBytes + small_part_bytes<R, NW>();
  return NW < 8 && b < kOwnSmSmem ? kOwnSmSmem : b;
}

template <int BITS, int CL, int NW>
int cluster_smem_bytes(int R, int G) {
  if (G == 32)
    return R == 1   ? cluster_smem<1, 32, BITS, CL, NW>()
           : R == 2 ? cluster_smem<2, 32, BITS, CL, NW>()
                    : cluster_smem<4, 32, BITS, CL, NW>();
  return R == 1 ? cluster_smem<1, 64, BITS, CL, NW>() : R == 2 ? cluster_smem<2, 64, BITS, CL, NW>() : cluster_smem<4, 64, BITS, CL, NW>();
}

template <int BITS>
int small_smem_bytes(int R, int G) {
  if (G == 32)
    return R == 1   ? kSmallWarps * Layout<1, 32, BITS>::kWarpBytes + small_part_bytes<1>()
           : R == 2 ? kSmallWarps * Layout<2, 32, BITS>::kWarpBytes + small_part_bytes<2>()
                    : kSmallWarps * Layout<4, 32, BITS>::kWarpBytes + small_part_bytes<4>();
  return R == 1   ? kSmallWarps * Layout<1, 64, BITS>::kWarpBytes + small_part_bytes<1>()
         : R == 2 ? kSmallWarps * Layout<2, 64, BITS>::kWarpBytes + small_part_bytes<2>()
                  : kSmallWarps * Layout<4, 64, BITS>::kWarpBytes + small_part_bytes<4>();
}

template <int BITS>
int smem_bytes(int R, int G) {
  if (G == 32)
    return R == 1 ? Layout<1, 32, BITS>::kSmem : R == 2 ? Layout<2, 32, BITS>::kSmem : Layout<4, 32, BITS>::kSmem;
  return R == 1 ? Layout<1, 64, BITS>::kSmem : R == 2 ? Layout<2, 64, BITS>::kSmem : Layout<4, 64, BITS>::kSmem;
}

}  // namespace

DecodeKernels decode_kernels(int R, int G, int bits, bool paged, int B, int vg) {
  DecodeKernels k;
  if (vg != kD) {  // value channel groups: dense 2-bit caches, persistent grid
    k.decode = vg == 64 ? select_vg_kernel<64>(R, G) : select_vg_kernel<32>(R, G);
    k.smem = k.smem_limit = vg == 64 ? vg_smem_bytes<64>(R, G) : vg_smem_bytes<32>(R, G);
    k.combine = reinterpret_cast<const void *>(&combine_kernel);
    k.small = k.pair = k.quad = nullptr;
    k.small_smem = k.pair_smem = k.quad_smem = 0;
    return k;
  }
  const int base = bits == 2 ? smem_bytes<2>(R, G) : smem_bytes<4>(R, G);
  if (paged) {
    k.decode = bits == 2 ? select_kernel<true, 2>(R, G) : select_kernel<true, 4>(R, G);
    k.smem = base + paged_extra(B);
    k.smem_limit = base + paged_extra(kPagedMaxBatch);
    k.combine = reinterpret_cast<const void *>(&paged_combine_kernel);
    k.small = k.pair = k.quad = nullptr;
    k.small_smem = k.pair_smem = k.quad_smem = 0;
  } else {
    k.decode = bits == 2 ? select_kernel<false, 2>(R, G) : select_kernel<false, 4>(R, G);
    k.smem = k.smem_limit = base;
    k.combine = reinterpret_cast<const void *>(&combine_kernel);
    k.small = bits == 2 ? select_small<2>(R, G) : select_small<4>(R, G);
    k.small_smem = bits == 2 ? small_smem_bytes<2>(R, G) : small_smem_bytes<4>(R, G);
    constexpr int PC = kDecodePairCtas, PW = kDecodePairWarps, QC = kDecodeQuadCtas, QW = kDecodeQuadWarps;
    k.pair = bits == 2 ? select_cluster<2, PC, PW>(R, G) : select_cluster<4, PC, PW>(R, G);
    k.pair_smem = bits == 2 ? cluster_smem_bytes<2, PC, PW>(R, G) : cluster_smem_bytes<4, PC, PW>(R, G);
    k.quad = bits == 2 ? select_cluster<2, QC, QW>(R, G) : select_cluster<4, QC, QW>(R, G);
    k.quad_smem = bits == 2 ? cluster_smem_bytes<2, QC, QW>(R, G) : cluster_smem_bytes<4, QC, QW>(R, G);
  }
  return k;
}

}  // namespace kivi
