// attn_f16.cu -- the attention kernels of attention.cuh for 16-bit IEEE storage.

#include "attention.cuh"

int svattn::launch_f16(const AttnParams& A, Layout l, int device, int grid, int ctas,
                         cudaStream_t st) {
  return A.D > 64 ? launch_dp<128, false>(A, l, device, grid, ctas, st)
                  : launch_dp<64, false>(A, l, device, grid, ctas, st);
}
