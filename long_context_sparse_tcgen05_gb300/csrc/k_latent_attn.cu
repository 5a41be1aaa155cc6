// Sparse attention over selected rows of the paged FP8 latent cache: the kernel of latent_attn.cuh.
#include "latent_attn.cuh"

namespace dsa {
cudaError_t launch_latent_attn(const LatentAttnLaunch& p, cudaStream_t st) { return launch_rows<false>(p, st); }
}  // namespace dsa
