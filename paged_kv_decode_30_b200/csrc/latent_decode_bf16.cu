// Latent decode over bf16 caches.
#include "latent_launch.cuh"

namespace pda {

cudaError_t launch_latent_decode_bf16(const LatentCall& c, cudaStream_t stream) {
  const bool wide = c.p->latent_dim == 512;
  switch (c.nt) {
    case 16: return wide ? launch_latent<512, false, 16>(c, stream) : launch_latent<256, false, 16>(c, stream);
    case 32: return wide ? launch_latent<512, false, 32>(c, stream) : launch_latent<256, false, 32>(c, stream);
    case 64: return wide ? launch_latent<512, false, 64>(c, stream) : launch_latent<256, false, 64>(c, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace pda
