// Attention over an expanded latent cache: validation and launch.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "latent_prefill.cuh"
#include "paged_decode_attn.h"
#include "tensor_map.cuh"

namespace pda {

int* device_error_word();  // paged_decode_attn.cu

namespace {

pda_status validate(const pda_latent_prefill_params* p) {
  if (p == nullptr) return PDA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->total_q < 0 || p->total_kv < 0 || p->max_q_len < 0 || p->num_heads < 1 ||
      p->head_dim < 1 || p->rope_dim < 1)
    return PDA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return PDA_ERR_INVALID_ARG;
  if (p->causal_offset < PDA_CAUSAL_BOTTOM_RIGHT) return PDA_ERR_INVALID_ARG;
  if (p->head_dim != 128 || (p->rope_dim != 32 && p->rope_dim != 64) || p->num_heads > 256 ||
      p->batch > 65535)
    return PDA_ERR_UNSUPPORTED;
  if (p->k_rope_stride < p->rope_dim) return PDA_ERR_INVALID_ARG;
  if (p->k_rope_stride % 8) return PDA_ERR_MISALIGNED;
  return PDA_OK;
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" pda_status latent_prefill_attn(const void* q, const void* kv, const void* k_rope,
                                          const int32_t* q_offsets, const int32_t* kv_offsets,
                                          const pda_latent_prefill_params* params, void* out,
                                          float* lse, pda_stream_t stream) {
  pda_status st = validate(params);
  if (st != PDA_OK) return st;
  const pda_latent_prefill_params& p = *params;
  if (p.batch == 0 || p.total_q == 0 || p.max_q_len == 0) return PDA_OK;
  if (!q || !q_offsets || !kv_offsets || !out || (p.total_kv > 0 && (!kv || !k_rope)))
    return PDA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(kv, 16) || !al(k_rope, 16) || !al(out, 16) || !al(q_offsets, 4) ||
      !al(kv_offsets, 4) || !al(lse, 4))
    return PDA_ERR_MISALIGNED;
  const int rows = p.max_q_len < p.total_q ? p.max_q_len : p.total_q;
  const long long tiles = (rows + 2ll * PrefillCfg::QT - 1) / (2 * PrefillCfg::QT);
  // Units of 256 query rows: `tiles` a sequence, or as many as the rows can need, where
  // that is fewer by a fourth (finding a unit's sequence takes a search then). Rows of
  // 30 sequences of up to 3000, 16 heads: 696 -> 564 us; 400 of up to 300, a fifth fewer:
  // 540 -> 555 us; 64 of 500 without a bound on their rows: 985 -> 284 us.
  const long long by_tiles = tiles * p.batch, by_rows = p.total_q / 256ll + p.batch;
  const bool rows_fit = 4 * by_rows <= 3 * by_tiles;
  const long long units = rows_fit ? by_rows : by_tiles;
  if (units * p.num_heads > INT_MAX) return PDA_ERR_UNSUPPORTED;
  PrefillArgs a{};
  a.q_offsets = q_offsets;
  a.kv_offsets = kv_offsets;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.err = device_error_word();
  if (a.err == nullptr) return PDA_ERR_CUDA;
  a.B = p.batch;
  a.H = p.num_heads;
  a.total_q = p.total_q;
  a.total_kv = p.total_kv;
  a.max_q = rows;
  a.tiles = (int)tiles;
  a.units = (int)units;
  a.by_rows = rows_fit;
  a.causal_offset = p.causal_offset;
  a.window = p.window;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  const int D = PrefillCfg::D;
  alignas(64) CUtensorMap mq, mkv, mr;
  // without keys nothing is loaded through the last two maps; a map has to have a row
  if (!make_heads_map(&mq, q, D + p.rope_dim, p.num_heads, p.total_q, 128) ||
      !make_heads_map(&mkv, p.total_kv ? kv : q, 2 * D, p.num_heads, p.total_kv ? p.total_kv : 1, 64) ||
      !make_rows_map(&mr, p.total_kv ? k_rope : q, p.rope_dim, p.total_kv ? p.total_kv : 1,
                     p.k_rope_stride, 2, 128))
    return PDA_ERR_CUDA;
  static unsigned long long attr_set = 0;  // bit d: opt-in set on device d (< 64)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PDA_ERR_CUDA;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit == 0 || !(__atomic_load_n(&attr_set, __ATOMIC_ACQUIRE) & bit)) {
    if (cudaFuncSetAttribute(latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PrefillCfg::SMEM_ALLOC) != cudaSuccess)
      return PDA_ERR_CUDA;
    __atomic_fetch_or(&attr_set, bit, __ATOMIC_RELEASE);
  }
  latent_prefill_kernel<<<dim3((unsigned)(units * p.num_heads)), PrefillCfg::THREADS,
                          PrefillCfg::SMEM_ALLOC, reinterpret_cast<cudaStream_t>(stream)>>>(mq, mkv, mr, a);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}
