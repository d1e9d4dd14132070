// Latent decode attention, absorbed form: validation and launch.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "paged_decode_attn.h"
#include "pda_device.cuh"

namespace pda {

int* device_error_word();  // paged_decode_attn.cu

namespace {

struct LatentArgs {
  const uint16_t* q;  // bf16 [B, q_len, H, R + rope_dim]
  const uint8_t* latent_pages;
  const uint16_t* rope_pages;
  const uint8_t* scales;
  const int32_t* page_table;
  const int32_t* kv_lens;
  uint16_t* out;
  float* lse;
  int* err;
  int B, Lq, H, M, rope_dim, page_size, log2_page, max_pages, num_pages, causal_offset, window;
  float scale_log2;
};

// Keys [lo, hi) that query row i of a sequence of L keys sees.
__device__ __forceinline__ void visible(const LatentArgs& a, int L, int i, int& lo, int& hi) {
  long long pos = (long long)L - 1;
  if (a.causal_offset >= 0) pos = (long long)a.causal_offset + i;
  else if (a.causal_offset == -2) pos = (long long)L - a.Lq + i;
  long long h = a.causal_offset != -1 ? pos + 1 : (long long)L;
  long long l = a.window > 0 ? pos - a.window + 1 : 0;
  hi = (int)(h < 0 ? 0 : (h > L ? L : h));
  lo = (int)(l < 0 ? 0 : (l > L ? L : l));
}

// One warp per query row: walks the row's keys one by one, lanes over the
// elements, with a running maximum and sum.
template <int R, bool FP8>
__global__ void __launch_bounds__(256) latent_decode_simple(const LatentArgs a) {
  constexpr int C = R / 256;
  constexpr unsigned FULL = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.M) return;
  const int b = (int)(row / a.M), i = (int)(row % a.M) / a.H;
  int L = __ldg(a.kv_lens + b);
  const int Lmax = a.max_pages * a.page_size;
  if (L < 0 || L > Lmax) {
    if (lane == 0) record_error_at(a.err, kErrBadPage);
    L = L < 0 ? 0 : Lmax;
  }
  int lo, hi;
  visible(a, L, i, lo, hi);
  const uint16_t* qr = a.q + row * (R + a.rope_dim);
  const bool has_rope = lane * 8 < a.rope_dim;
  float q[C][8], qe[8] = {}, o[C][8] = {};
#pragma unroll
  for (int c = 0; c < C; ++c) bf16x8_to_f32(*reinterpret_cast<const uint4*>(qr + (lane + 32 * c) * 8), q[c]);
  if (has_rope) bf16x8_to_f32(*reinterpret_cast<const uint4*>(qr + R + lane * 8), qe);
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int page = __ldg(a.page_table + (long long)b * a.max_pages + (j >> a.log2_page));
    if ((unsigned)page >= (unsigned)a.num_pages) {
      if (lane == 0) record_error_at(a.err, kErrBadPage);
      continue;
    }
    const long long slot = (long long)page * a.page_size + (j & (a.page_size - 1));
    float v[C][8], s = 0.f;
    float sc = 1.f;
    if constexpr (FP8) sc = __int_as_float(min(max((int)a.scales[slot], 97), 157) << 23);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (FP8)
        e4m3x8_to_f32(*reinterpret_cast<const uint2*>(a.latent_pages + slot * R + (lane + 32 * c) * 8), v[c]);
      else
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(a.latent_pages + (slot * R + (lane + 32 * c) * 8) * 2), v[c]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[c][k] *= sc;
        s = fmaf(q[c][k], v[c][k], s);
      }
    }
    if (has_rope) {
      float e[8];
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(a.rope_pages + slot * a.rope_dim + lane * 8), e);
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(qe[k], e[k], s);
    }
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(FULL, s, x);
    s *= a.scale_log2;
    const float m_new = fmaxf(m, s);
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - m_new), p = s == -INFINITY ? 0.f : exp2f(s - m_new);
    m = m_new;
    l = l * alpha + p;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) o[c][k] = fmaf(o[c][k], alpha, p * v[c][k]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(o[c][2 * k] * inv, o[c][2 * k + 1] * inv);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(a.out + row * R + (lane + 32 * c) * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane == 0 && a.lse) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

pda_status validate(const pda_latent_params* p) {
  if (p == nullptr) return PDA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->q_len < 1 || p->num_heads < 1 || p->latent_dim < 1 || p->rope_dim < 1 ||
      p->page_size < 1 || p->max_pages_per_seq < 1 || p->num_pages < 1)
    return PDA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return PDA_ERR_INVALID_ARG;
  if (p->causal_offset < PDA_CAUSAL_BOTTOM_RIGHT) return PDA_ERR_INVALID_ARG;
  if (p->kv_dtype != PDA_KV_BF16 && p->kv_dtype != PDA_KV_FP8_E4M3 && p->kv_dtype != PDA_KV_NVFP4)
    return PDA_ERR_INVALID_ARG;
  if ((long long)p->max_pages_per_seq * p->page_size > INT_MAX ||
      (long long)p->num_pages * p->page_size > INT_MAX)
    return PDA_ERR_INVALID_ARG;
  if (p->flags & ~PDA_FLAG_NO_PDL) return PDA_ERR_INVALID_ARG;
  if ((p->latent_dim != 256 && p->latent_dim != 512) || (p->rope_dim != 32 && p->rope_dim != 64) ||
      p->page_size < 8 || p->page_size > 256 || (p->page_size & (p->page_size - 1)) ||
      p->kv_dtype == PDA_KV_NVFP4 || p->q_len > 8 || p->num_heads > 256 || p->batch > 65535)
    return PDA_ERR_UNSUPPORTED;
  return PDA_OK;
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" {

size_t paged_latent_decode_workspace_bytes(const pda_latent_params* params) {
  if (validate(params) != PDA_OK) return SIZE_MAX;
  return 0;
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
  LatentArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.latent_pages = static_cast<const uint8_t*>(latent_pages);
  a.rope_pages = static_cast<const uint16_t*>(rope_pages);
  a.scales = static_cast<const uint8_t*>(p.latent_scales);
  a.page_table = page_table;
  a.kv_lens = kv_lens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.err = device_error_word();
  if (a.err == nullptr) return PDA_ERR_CUDA;
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
  a.scale_log2 = p.scale * 1.4426950408889634f;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const unsigned grid = (unsigned)(((long long)a.B * a.M + 7) / 8);
  if (p.latent_dim == 512) {
    if (fp8) latent_decode_simple<512, true><<<grid, 256, 0, stream>>>(a);
    else latent_decode_simple<512, false><<<grid, 256, 0, stream>>>(a);
  } else {
    if (fp8) latent_decode_simple<256, true><<<grid, 256, 0, stream>>>(a);
    else latent_decode_simple<256, false><<<grid, 256, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

}  // extern "C"
