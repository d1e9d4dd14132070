// Between the latent decode entry point and its kernels' launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_decode_attn.h"

namespace pda {

struct LatentCall {
  const pda_latent_params* p;
  const void *q, *latent_pages, *rope_pages;
  const int32_t *page_table, *kv_lens;
  void* out;
  float* lse;
  int* err;
  float *o_part, *lse_part;
  void* cut;
  int nt, row_tiles, teams, sms;
};

cudaError_t launch_latent_decode_bf16(const LatentCall& c, cudaStream_t stream);
cudaError_t launch_latent_decode_fp8(const LatentCall& c, cudaStream_t stream);

}  // namespace pda
