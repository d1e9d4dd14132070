// Latent decode attention, absorbed form: validation and launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "latent_decode.h"
#include "paged_decode_attn.h"

namespace pda {

// paged_decode_attn.cu
int* device_error_word();
int device_sms();
pda_status latent_library_workspace(size_t bytes, cudaStream_t stream, void** out);

namespace {

pda_status validate(const pda_latent_params* p) {
  if (p == nullptr) return PDA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->q_len < 1 || p->num_heads < 1 || p->latent_dim < 1 || p->rope_dim < 1 ||
      p->page_size < 1 || p->max_pages_per_seq < 1 || p->num_pages < 1)
    return PDA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return PDA_ERR_INVALID_ARG;
  if (p->causal_offset < PDA_CAUSAL_BOTTOM_RIGHT) return PDA_ERR_INVALID_ARG;
  if (p->kv_dtype != PDA_KV_BF16 && p->kv_dtype != PDA_KV_FP8_E4M3 && p->kv_dtype != PDA_KV_NVFP4)
    return PDA_ERR_INVALID_ARG;
  // (a position and a tile more fit 32 bits)
  if ((long long)p->max_pages_per_seq * p->page_size > INT_MAX - 128 ||
      (long long)p->num_pages * p->page_size > INT_MAX)
    return PDA_ERR_INVALID_ARG;
  if (p->flags & ~PDA_FLAG_NO_PDL) return PDA_ERR_INVALID_ARG;
  if ((p->latent_dim != 256 && p->latent_dim != 512) || (p->rope_dim != 32 && p->rope_dim != 64) ||
      p->page_size < 8 || p->page_size > 256 || (p->page_size & (p->page_size - 1)) ||
      p->kv_dtype == PDA_KV_NVFP4 || p->q_len > 8 || p->num_heads > 256 || p->batch > 65535)
    return PDA_ERR_UNSUPPORTED;
  if (p->batch * (((long long)p->max_pages_per_seq * p->page_size + 127) / 128 + 16) > INT_MAX)
    return PDA_ERR_UNSUPPORTED;  // tiles, and a few more a sequence, are counted in 32 bits
  return PDA_OK;
}

// Launch shape and workspace of a call.
struct Plan {
  int nt, row_tiles, teams;
  size_t lse_off, cut_off, total;  // the partial outputs come first
};

Plan make_plan(const pda_latent_params& p, int sms) {
  Plan pl{};
  const int M = p.q_len * p.num_heads;
  const bool fp8 = p.kv_dtype == PDA_KV_FP8_E4M3;
  // As many packed rows per CTA as TMEM (FP8: two terms a row, 32) or shared
  // memory (bf16: 64) take, no more than there are.
  pl.nt = M <= 16 ? 16 : (M <= 32 || fp8) ? 32 : 64;
  pl.row_tiles = (M + pl.nt - 1) / pl.nt;
  // One CTA per SM; a team walks a range of tokens with a CTA per row tile.
  // Never more teams than tiles.
  const long long tiles = (long long)p.batch * (((long long)p.max_pages_per_seq * p.page_size + 127) / 128);
  const long long teams = std::min(sms, 256) / pl.row_tiles;  // 256: what the merge can list
  pl.teams = (int)(teams < 1 ? 1 : teams < tiles ? teams : tiles);
  const size_t slots = (size_t)pl.teams * pl.row_tiles * 2 * pl.nt;
  pl.lse_off = slots * p.latent_dim * sizeof(float);
  pl.cut_off = (pl.lse_off + slots * sizeof(float) + 255) / 256 * 256;
  pl.total = pl.cut_off + (size_t)pl.teams * 2 * sizeof(int);
  return pl;
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" {

size_t paged_latent_decode_workspace_bytes(const pda_latent_params* params) {
  if (validate(params) != PDA_OK) return SIZE_MAX;
  if (params->batch == 0) return 0;
  const int sms = device_sms();
  return make_plan(*params, sms > 0 ? sms : 148).total;
}

pda_status paged_latent_decode(const void* q, const void* latent_pages, const void* rope_pages,
                               const int32_t* page_table, const int32_t* kv_lens,
                               const pda_latent_params* params, void* out, float* lse,
                               pda_stream_t stream_) {
  pda_status st = validate(params);
  if (st != PDA_OK) return st;
  const pda_latent_params& p = *params;
  if (p.batch == 0) return PDA_OK;
  const bool fp8 = p.kv_dtype == PDA_KV_FP8_E4M3;
  if (!q || !latent_pages || !rope_pages || !page_table || !kv_lens || !out || (fp8 && !p.latent_scales))
    return PDA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(latent_pages, 16) || !al(rope_pages, 16) || !al(out, 16) ||
      !al(page_table, 4) || !al(kv_lens, 4) || !al(lse, 4) || !al(p.workspace, 256))
    return PDA_ERR_MISALIGNED;
  LatentCall c{};
  c.err = device_error_word();
  const int sms = device_sms();
  if (c.err == nullptr || sms < 1) return PDA_ERR_CUDA;
  const Plan pl = make_plan(p, sms);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  void* ws = p.workspace;
  if (ws == nullptr) {
    if ((st = latent_library_workspace(pl.total, stream, &ws)) != PDA_OK) return st;
  } else if (p.workspace_bytes < pl.total) {
    return PDA_ERR_WORKSPACE;
  }
  char* base = static_cast<char*>(ws);
  c.p = &p;
  c.q = q;
  c.latent_pages = latent_pages;
  c.rope_pages = rope_pages;
  c.page_table = page_table;
  c.kv_lens = kv_lens;
  c.out = out;
  c.lse = lse;
  c.o_part = reinterpret_cast<float*>(base);
  c.lse_part = reinterpret_cast<float*>(base + pl.lse_off);
  c.cut = base + pl.cut_off;
  c.nt = pl.nt;
  c.row_tiles = pl.row_tiles;
  c.teams = pl.teams;
  c.sms = sms;
  const cudaError_t e = fp8 ? launch_latent_decode_fp8(c, stream) : launch_latent_decode_bf16(c, stream);
  if (e == cudaErrorNotSupported) return PDA_ERR_UNSUPPORTED;
  return e == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

}  // extern "C"
