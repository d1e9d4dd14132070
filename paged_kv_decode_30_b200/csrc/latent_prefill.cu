// Attention over an expanded latent cache: validation and launch.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "paged_decode_attn.h"
#include "pda_device.cuh"

namespace pda {

int* device_error_word();  // paged_decode_attn.cu

namespace {

struct PrefillArgs {
  const uint16_t* q;       // bf16 [total_q, H, D + rope_dim]
  const uint16_t* kv;      // bf16 [total_kv, H, 2 D]
  const uint16_t* k_rope;  // bf16 [total_kv, rope_dim], strided
  const int32_t* q_offsets;
  const int32_t* kv_offsets;
  uint16_t* out;
  float* lse;
  int* err;
  long long k_rope_stride;
  int B, H, rope_dim, total_q, total_kv, causal_offset, window;
  float scale_log2;
};

// Keys [lo, hi) that query row i of a sequence of nq rows and nk keys sees.
__device__ __forceinline__ void visible(const PrefillArgs& a, int nq, int nk, int i, int& lo, int& hi) {
  long long pos = (long long)nk - 1;
  if (a.causal_offset >= 0) pos = (long long)a.causal_offset + i;
  else if (a.causal_offset == -2) pos = (long long)nk - nq + i;
  long long h = a.causal_offset != -1 ? pos + 1 : (long long)nk;
  long long l = a.window > 0 ? pos - a.window + 1 : 0;
  hi = (int)(h < 0 ? 0 : (h > nk ? nk : h));
  lo = (int)(l < 0 ? 0 : (l > nk ? nk : l));
}

// One warp per (query row, head): walks the row's keys one by one, lanes over
// the elements, with a running maximum and sum.
__global__ void __launch_bounds__(256) latent_prefill_simple(const PrefillArgs a, int max_q) {
  constexpr unsigned FULL = 0xFFFFFFFFu;
  constexpr int D = 128;
  const int lane = threadIdx.x & 31, b = blockIdx.z, h = blockIdx.y;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1);
  const int k0 = __ldg(a.kv_offsets + b), k1 = __ldg(a.kv_offsets + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_kv) {
    if (lane == 0) record_error_at(a.err, kErrBadPage);
    return;
  }
  if (i >= q1 - q0 || i >= max_q) return;
  int lo, hi;
  visible(a, q1 - q0, k1 - k0, i, lo, hi);
  const long long row = (long long)(q0 + i) * a.H + h;
  const uint16_t* qr = a.q + row * (D + a.rope_dim);
  const bool has_rope = lane * 2 < a.rope_dim;
  auto two = [](const uint16_t* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  };
  const float2 qa = two(qr + 2 * lane), qb = two(qr + 64 + 2 * lane);
  const float2 qe = has_rope ? two(qr + D + 2 * lane) : make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  float2 oa = make_float2(0.f, 0.f), ob = oa;
  for (int j = lo; j < hi; ++j) {
    const uint16_t* kr = a.kv + ((long long)(k0 + j) * a.H + h) * 2 * D;
    const float2 ka = two(kr + 2 * lane), kb = two(kr + 64 + 2 * lane);
    float s = qa.x * ka.x + qa.y * ka.y + qb.x * kb.x + qb.y * kb.y;
    if (has_rope) {
      const float2 ke = two(a.k_rope + (long long)(k0 + j) * a.k_rope_stride + 2 * lane);
      s += qe.x * ke.x + qe.y * ke.y;
    }
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(FULL, s, x);
    s *= a.scale_log2;
    const float m_new = fmaxf(m, s);
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - m_new), p = s == -INFINITY ? 0.f : exp2f(s - m_new);
    m = m_new;
    l = l * alpha + p;
    const float2 va = two(kr + D + 2 * lane), vb = two(kr + D + 64 + 2 * lane);
    oa.x = fmaf(oa.x, alpha, p * va.x);
    oa.y = fmaf(oa.y, alpha, p * va.y);
    ob.x = fmaf(ob.x, alpha, p * vb.x);
    ob.y = fmaf(ob.y, alpha, p * vb.y);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(a.out + row * D);
  o[lane] = __floats2bfloat162_rn(oa.x * inv, oa.y * inv);
  o[32 + lane] = __floats2bfloat162_rn(ob.x * inv, ob.y * inv);
  if (lane == 0 && a.lse) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

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
  PrefillArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.kv = static_cast<const uint16_t*>(kv);
  a.k_rope = static_cast<const uint16_t*>(k_rope);
  a.q_offsets = q_offsets;
  a.kv_offsets = kv_offsets;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.err = device_error_word();
  if (a.err == nullptr) return PDA_ERR_CUDA;
  a.k_rope_stride = p.k_rope_stride;
  a.B = p.batch;
  a.H = p.num_heads;
  a.rope_dim = p.rope_dim;
  a.total_q = p.total_q;
  a.total_kv = p.total_kv;
  a.causal_offset = p.causal_offset;
  a.window = p.window;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  const int rows = p.max_q_len < p.total_q ? p.max_q_len : p.total_q;
  latent_prefill_simple<<<dim3((rows + 7) / 8, p.num_heads, p.batch), 256, 0,
                          reinterpret_cast<cudaStream_t>(stream)>>>(a, rows);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}
