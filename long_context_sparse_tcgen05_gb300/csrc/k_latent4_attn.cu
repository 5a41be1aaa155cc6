// Sparse attention over selected rows of the paged 4-bit latent cache: the kernel of latent_attn.cuh with gather warps
// that expand the codes.  404 bytes a row instead of 644.  Measured: see there.
#include "latent_attn.cuh"

namespace dsa {
cudaError_t launch_latent4_attn(const LatentAttnLaunch& p, cudaStream_t st) { return launch_rows<true>(p, st); }
}  // namespace dsa
