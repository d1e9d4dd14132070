// Latent decode over FP8 caches (e4m3 codes, a power-of-two scale a row).
#include "latent_launch.cuh"

namespace pda {

cudaError_t launch_latent_decode_fp8(const LatentCall& c, cudaStream_t stream) {
  const bool wide = c.p->latent_dim == 512;
  switch (c.nt) {
    case 16: return wide ? launch_latent<512, true, 16>(c, stream) : launch_latent<256, true, 16>(c, stream);
    case 32: return wide ? launch_latent<512, true, 32>(c, stream) : launch_latent<256, true, 32>(c, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace pda
