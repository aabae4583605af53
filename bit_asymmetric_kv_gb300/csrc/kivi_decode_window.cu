// kivi_decode_window.cu -- decode attention over a paged cache of which a sequence's newest token sees a
// window and the first tokens (sinks), instantiated from kivi_decode_body.cuh.
//
// The work is dealt out in the same units of 64 tokens, of which only those that hold a visible token
// count: the sinks', and those from the window's first token on.  Pages that hold no such unit are
// neither looked up nor read, so their table entries may hold anything.  Masks cost only in the unit at
// each end.
#include "kivi_decode_body.cuh"

namespace kivi {

namespace {

template <int R, int G, int BITS>
__global__ void __launch_bounds__(kThreads, KIVI_DECODE_MIN_CTAS) window_decode_kernel(const DecodeArgs a) {
  decode_body<R, G, kModeWindow, BITS, kWarps>(a);
}

template <int R, int G, int BITS>
DecodeKernels kernels(int extra) {
  DecodeKernels k = {};
  k.decode = reinterpret_cast<const void *>(&window_decode_kernel<R, G, BITS>);
  k.smem = Layout<R, G, BITS>::kSmem + extra;
  k.smem_limit = Layout<R, G, BITS>::kSmem + paged_extra(kPagedMaxBatch);
  k.combine = reinterpret_cast<const void *>(&paged_combine_kernel);
  return k;
}

template <int R>
DecodeKernels of_shape(int G, int bits, int extra) {
  if (G == 32) return bits == 2 ? kernels<R, 32, 2>(extra) : kernels<R, 32, 4>(extra);
  return bits == 2 ? kernels<R, 64, 2>(extra) : kernels<R, 64, 4>(extra);
}

}  // namespace

DecodeKernels decode_window_kernels(int R, int G, int bits, int B) {
  const int extra = paged_extra(B);
  return R == 1 ? of_shape<1>(G, bits, extra) : R == 2 ? of_shape<2>(G, bits, extra) : of_shape<4>(G, bits, extra);
}

}  // namespace kivi
