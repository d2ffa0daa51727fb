// attn_bf16.cu -- the attention kernels of attention.cuh for bfloat16 storage.

#include "attention.cuh"

int svattn::launch_bf16(const AttnParams& A, Layout l, int device, int grid, int ctas,
                         cudaStream_t st) {
  return A.D > 64 ? launch_dp<128, true>(A, l, device, grid, ctas, st)
                  : launch_dp<64, true>(A, l, device, grid, ctas, st);
}
