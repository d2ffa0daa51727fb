// attn8_f16.cu -- the attention kernels of attention.cuh over 8-bit caches, for 16-bit IEEE queries.

#include "attention.cuh"

int svattn::launch8_f16(const AttnParams& A, const Prep8& P, Layout l, int device, int grid,
                        int ctas, cudaStream_t st) {
  return A.D > 64 ? launch_dp8<128, false>(A, P, l, device, grid, ctas, st)
                  : launch_dp8<64, false>(A, P, l, device, grid, ctas, st);
}
