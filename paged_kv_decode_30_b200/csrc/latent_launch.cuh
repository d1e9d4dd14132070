// Launch of one latent decode variant: tensor maps, the kernel, the merge.
#pragma once

#include <algorithm>

#include "latent_decode.cuh"
#include "latent_decode.h"
#include "tensor_map.cuh"

namespace pda {

template <int R, bool FP8, int NT>
cudaError_t launch_latent(const LatentCall& c, cudaStream_t stream) {
  using C = LatentCfg<R, FP8, NT>;
  const pda_latent_params& p = *c.p;
  LatentArgs a{};
  a.q = static_cast<const uint16_t*>(c.q);
  a.latent_pages = static_cast<const uint8_t*>(c.latent_pages);
  a.rope_pages = static_cast<const uint16_t*>(c.rope_pages);
  a.scales = static_cast<const uint8_t*>(p.latent_scales);
  a.page_table = c.page_table;
  a.kv_lens = c.kv_lens;
  a.out = static_cast<uint16_t*>(c.out);
  a.lse = c.lse;
  a.err = c.err;
  a.o_part = c.o_part;
  a.lse_part = c.lse_part;
  a.cut = static_cast<int2*>(c.cut);
  a.B = p.batch;
  a.Lq = p.q_len;
  a.H = p.num_heads;
  a.M = p.q_len * p.num_heads;
  a.rope_dim = p.rope_dim;
  a.page_size = p.page_size;
  while ((1 << a.log2_page) < p.page_size) ++a.log2_page;
  a.max_pages = p.max_pages_per_seq;
  a.num_pages = p.num_pages;
  a.causal_offset = p.causal_offset;
  a.window = p.window;
  a.teams = c.teams;
  a.row_tiles = c.row_tiles;
  a.item_cost = C::ITEM_COST;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  const long long rows = (long long)p.num_pages * p.page_size;
  const int box = p.page_size < kTile ? p.page_size : kTile;
  alignas(64) CUtensorMap mc, mr, mq;
  if (!make_tokens_map(&mc, c.latent_pages, R, rows, FP8 ? 1 : 2, box, C::COLS_U) ||
      !make_rows_map(&mr, c.rope_pages, p.rope_dim, rows, p.rope_dim, 2, box) ||
      !make_rows_map(&mq, c.q, R + p.rope_dim, (long long)a.B * a.M, R + p.rope_dim, 2, NT))
    return cudaErrorInvalidValue;
  auto kern = latent_decode_kernel<R, FP8, NT>;
  static unsigned long long attr_set = 0;  // bit d: opt-in set on device d (< 64)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit == 0 || !(__atomic_load_n(&attr_set, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&attr_set, bit, __ATOMIC_RELEASE);
  }
  kern<<<dim3((unsigned)(a.teams * a.row_tiles)), C::THREADS, C::SMEM_ALLOC, stream>>>(mc, mr, mq, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.teams == 1) return e;  // one team cuts no sequence
  cudaLaunchConfig_t cfg = {};
  // a block for each row of the sequences that can be cut, up to two an SM
  const long long cut_rows = (long long)std::min(a.B, a.teams - 1) * a.M;
  cfg.gridDim = dim3((unsigned)std::min(cut_rows, 2ll * c.sms));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (p.flags & PDA_FLAG_NO_PDL) ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<R>, a, NT == 16 ? 4 : NT == 32 ? 5 : 6);
}

}  // namespace pda
