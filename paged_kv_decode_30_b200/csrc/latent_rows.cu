// Rows of a latent cache: written into the pages (bf16, or e4m3 codes with
// one power-of-two scale a row) and read back as bf16.
//
// Both directions move each row once and compute next to nothing, so they are
// bound by HBM for many rows and by latency for few. A warp owns RB
// consecutive ragged rows: it looks up their slots at the same time (the owner
// from row_offsets, then the page table; rows to be written are loaded beside
// that), then streams the rows through registers, 16 bytes a lane and access,
// with the loads of several rows in flight before the first store.
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_decode_attn.h"
#include "pda_device.cuh"

namespace pda {

// paged_decode_attn.cu
int* device_error_word();
int device_sms();

namespace {

struct RowsArgs {
  const int32_t* row_offsets;
  const int32_t* page_table;
  const int32_t* starts;  // first position of each sequence (null: 0)
  uint16_t* latent;       // ragged side, bf16
  uint16_t* rope;
  uint8_t* latent_pages;
  uint16_t* rope_pages;
  uint8_t* scales;
  int* err;
  long long latent_stride, rope_stride;  // elements
  int B, total, rope_dim, page_size, log2_page, max_pages, num_pages;
};

constexpr int kScaleBias = 127, kScaleMin = -30, kScaleMax = 30;

// The sequence of each of the warp's RB rows r0, r0 + 1, ...: lane u < RB gets
// row r0 + u's, the last b with row_offsets[b] <= row (-1: none; B: behind the
// last). Up to 1024 sequences the warp loads 32 offsets at a time and counts by
// votes, two loads deep; beyond, each lane searches by halving.
template <int RB>
__device__ __forceinline__ int find_owners(const RowsArgs& a, int r0, int lane) {
  constexpr unsigned FULL = 0xFFFFFFFFu;
  const int n = a.B + 1;
  int b = -1;
  if (n <= 32) {
    const int v = lane < n ? __ldg(a.row_offsets + lane) : 0x7FFFFFFF;
#pragma unroll
    for (int u = 0; u < RB; ++u) {
      const int c = __popc(__ballot_sync(FULL, lane < n && v <= r0 + u));
      if (lane == u) b = c - 1;
    }
  } else if (n <= 1024) {
    const int step = (n + 31) / 32, at = lane * step;
    const int v = at < n ? __ldg(a.row_offsets + at) : 0x7FFFFFFF;
    int k[RB], w[RB];
#pragma unroll
    for (int u = 0; u < RB; ++u) {
      k[u] = max(__popc(__ballot_sync(FULL, at < n && v <= r0 + u)) - 1, 0) * step;
      w[u] = lane < step && k[u] + lane < n ? __ldg(a.row_offsets + k[u] + lane) : 0x7FFFFFFF;
    }
#pragma unroll
    for (int u = 0; u < RB; ++u) {
      const int c = __popc(__ballot_sync(FULL, lane < step && k[u] + lane < n && w[u] <= r0 + u));
      if (lane == u) b = k[u] + c - 1;
    }
  } else if (lane < RB) {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.row_offsets + mid) <= r0 + lane) lo = mid + 1;
      else hi = mid;
    }
    b = lo - 1;
  }
  return b;
}

// Slot (row of the flattened pools) of ragged row `row` of sequence b; -1 if no
// sequence owns it or (recorded) its position or page is out of range.
__device__ __forceinline__ long long slot_of_row(const RowsArgs& a, long long row, int b) {
  if (row >= a.total || b < 0 || b >= a.B) return -1;
  const long long t = row - __ldg(a.row_offsets + b);
  const int start = a.starts ? __ldg(a.starts + b) : 0;
  const long long pos = start + t;
  int page = -1;
  if (start >= 0 && t >= 0 && pos < (long long)a.max_pages * a.page_size)
    page = __ldg(a.page_table + (long long)b * a.max_pages + (pos >> a.log2_page));
  if ((unsigned)page >= (unsigned)a.num_pages) {
    record_error_at(a.err, kErrBadPage);
    return -1;
  }
  return (long long)page * a.page_size + (pos & (a.page_size - 1));
}

// Largest |x| of eight bf16 in a uint4, as bf16 bits (they order as the
// values do); NaN counts as 0.
__device__ __forceinline__ uint32_t amax_bits(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = w[k] & 0x7FFF7FFFu;
    m = __vmaxu2(m, x & ~__vcmpgtu2(x, 0x7F807F80u));
  }
  return max(m & 0xFFFFu, m >> 16);
}

// The least e in [kScaleMin, kScaleMax] with a <= 448 * 2^e, from the bf16
// bits of a: 448 = 1.75 * 2^8, so a = 1.f * 2^k gives k - 8, or k - 7 where
// 1.f > 1.75 (the seven fraction bits above 96). Zero and subnormals land on
// kScaleMin, infinity on kScaleMax, through the clamp.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int k = (int)(bits >> 7) - 127;
  return min(max(k - 8 + ((bits & 127u) > 96u ? 1 : 0), kScaleMin), kScaleMax);
}

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Eight bf16 times `inv` -> eight e4m3 codes (nearest even, saturating).
__device__ __forceinline__ uint2 quantise8(const uint4& v, float inv) {
  float f[8];
  bf16x8_to_f32(v, f);
  uint16_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(c[k])
        : "f"(f[2 * k + 1] * inv), "f"(f[2 * k] * inv));
  return make_uint2(c[0] | ((uint32_t)c[1] << 16), c[2] | ((uint32_t)c[3] << 16));
}

// Eight e4m3 codes times `scale` -> eight bf16. Exact: four significant bits
// and an exponent well inside bf16's.
__device__ __forceinline__ uint4 dequantise8(const uint2& c, float scale) {
  float f[8];
  e4m3x8_to_f32(c, f);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k] * scale, f[2 * k + 1] * scale);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of large calls pass the caches by (each byte is used once): 77 k FP8 rows
// gathered in 24.3 us instead of 26.1.
template <bool STREAM, typename T>
__device__ __forceinline__ T get(const T* p) {
  if constexpr (STREAM) return __ldcs(p);
  else return *p;
}
template <bool STREAM, typename T>
__device__ __forceinline__ void put(T* p, const T& v) {
  if constexpr (STREAM) __stcs(p, v);
  else *p = v;
}

template <int R, bool FP8, bool WRITE, int RB>
__global__ void __launch_bounds__(256, 4) latent_rows_kernel(const RowsArgs a) {
  constexpr unsigned FULL = 0xFFFFFFFFu;
  constexpr int C = R / 256;           // 16-byte bf16 pieces of a row per lane
  constexpr int U = RB < 4 ? RB : 4;   // rows in flight
  const int lane = threadIdx.x & 31;
  const long long r0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * RB;
  if (r0 < a.total) {
    uint4 v[U][C];  // bf16 pieces of U rows
    auto load_rows = [&](int u0) {  // of the ragged side: needs no slot
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint4* src = reinterpret_cast<const uint4*>(a.latent + min(r0 + u0 + u, a.total - 1ll) * a.latent_stride);
#pragma unroll
        for (int c = 0; c < C; ++c) v[u][c] = get<(RB > 1)>(src + lane + 32 * c);
      }
    };
    if constexpr (WRITE) load_rows(0);  // beside the lookups
    const int owner = find_owners<RB>(a, (int)r0, lane);
    const long long mine = lane < RB ? slot_of_row(a, r0 + lane, owner) : -1;
    if (__ballot_sync(FULL, mine >= 0) == 0) return;
    // rope parts: (row, 16-byte piece) pairs over the lanes
    const int log2_pieces = a.rope_dim == 64 ? 3 : 2;
    constexpr int RP = (RB * 8 + 31) / 32;
    uint4 rv[RP];
    long long rs[RP];
#pragma unroll
    for (int k = 0; k < RP; ++k) {
      const int p = lane + 32 * k, row = p >> log2_pieces, c = p & ((1 << log2_pieces) - 1);
      const long long s = __shfl_sync(FULL, mine, row & 31);
      rs[k] = row < RB ? s : -1;
      if (rs[k] >= 0)
        rv[k] = *reinterpret_cast<const uint4*>(WRITE ? a.rope + (r0 + row) * a.rope_stride + c * 8
                                                      : a.rope_pages + rs[k] * a.rope_dim + c * 8);
    }
#pragma unroll
    for (int u0 = 0; u0 < RB; u0 += U) {
      long long slot[U];
      uint2 q[U][C];  // e4m3 pieces
      uint32_t sb[U];
      if (WRITE && u0 > 0) load_rows(u0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        slot[u] = __shfl_sync(FULL, mine, u0 + u);
        if (slot[u] < 0) continue;
        if constexpr (WRITE) {
          // loaded already
        } else if constexpr (FP8) {
          const uint2* src = reinterpret_cast<const uint2*>(a.latent_pages + slot[u] * R);
#pragma unroll
          for (int c = 0; c < C; ++c) q[u][c] = get<(RB > 1)>(src + lane + 32 * c);
          sb[u] = a.scales[slot[u]];
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(a.latent_pages + slot[u] * R * 2);
#pragma unroll
          for (int c = 0; c < C; ++c) v[u][c] = get<(RB > 1)>(src + lane + 32 * c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (slot[u] < 0) continue;  // the same for the whole warp
        if constexpr (WRITE && FP8) {
          uint32_t m = 0;
#pragma unroll
          for (int c = 0; c < C; ++c) m = max(m, amax_bits(v[u][c]));
          const int e = scale_exponent(__reduce_max_sync(FULL, m));
          const float inv = exp2_int(-e);
          uint2* dst = reinterpret_cast<uint2*>(a.latent_pages + slot[u] * R);
#pragma unroll
          for (int c = 0; c < C; ++c) put<(RB > 1)>(dst + lane + 32 * c, quantise8(v[u][c], inv));
          if (lane == 0) a.scales[slot[u]] = (uint8_t)(e + kScaleBias);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(
              WRITE ? reinterpret_cast<uint16_t*>(a.latent_pages) + slot[u] * R
                    : a.latent + (r0 + u0 + u) * a.latent_stride);
          if constexpr (FP8) {
            const float s = exp2_int(min(max((int)sb[u] - kScaleBias, kScaleMin), kScaleMax));
#pragma unroll
            for (int c = 0; c < C; ++c) put<(RB > 1)>(dst + lane + 32 * c, dequantise8(q[u][c], s));
          } else {
#pragma unroll
            for (int c = 0; c < C; ++c) put<(RB > 1)>(dst + lane + 32 * c, v[u][c]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < RP; ++k) {
      const int p = lane + 32 * k, row = p >> log2_pieces, c = p & ((1 << log2_pieces) - 1);
      if (rs[k] >= 0)
        *reinterpret_cast<uint4*>(WRITE ? a.rope_pages + rs[k] * a.rope_dim + c * 8
                                        : a.rope + (r0 + row) * a.rope_stride + c * 8) = rv[k];
    }
  }
}

template <int R, bool FP8, bool WRITE>
void launch_rows(const RowsArgs& a, int sms, cudaStream_t stream) {
  // Few rows: one a warp, so that the lookups of all rows run side by side.
  // Many: four a warp, so that a lookup's chain of dependent loads is paid once
  // for four rows, and 64 or 128 bytes a lane are in flight (77 k FP8 rows: 24.3 us;
  // eight a warp 25.0).
  if (a.total <= sms * 16) {
    latent_rows_kernel<R, FP8, WRITE, 1><<<(a.total + 7) / 8, 256, 0, stream>>>(a);
  } else {
    latent_rows_kernel<R, FP8, WRITE, 4><<<(unsigned)((a.total + 31ll) / 32), 256, 0, stream>>>(a);
  }
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

pda_status rows_call(const pda_latent_rows_params* p, bool write, void* latent, void* rope,
                     const int32_t* row_offsets, const int32_t* page_table, const int32_t* starts,
                     void* latent_pages, void* rope_pages, pda_stream_t stream_) {
  if (p == nullptr) return PDA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->total_rows < 0 || p->latent_dim < 1 || p->rope_dim < 1 ||
      p->page_size < 1 || p->max_pages_per_seq < 1 || p->num_pages < 1)
    return PDA_ERR_INVALID_ARG;
  if (p->kv_dtype != PDA_KV_BF16 && p->kv_dtype != PDA_KV_FP8_E4M3 && p->kv_dtype != PDA_KV_NVFP4)
    return PDA_ERR_INVALID_ARG;
  if ((long long)p->max_pages_per_seq * p->page_size > 0x7FFFFFFFll ||
      (long long)p->num_pages * p->page_size > 0x7FFFFFFFll)
    return PDA_ERR_INVALID_ARG;
  if ((p->latent_dim != 256 && p->latent_dim != 512) || (p->rope_dim != 32 && p->rope_dim != 64) ||
      p->page_size < 8 || p->page_size > 256 || (p->page_size & (p->page_size - 1)) ||
      p->kv_dtype == PDA_KV_NVFP4)
    return PDA_ERR_UNSUPPORTED;
  if (p->latent_stride < p->latent_dim || p->rope_stride < p->rope_dim)
    return PDA_ERR_INVALID_ARG;
  if (p->latent_stride % 8 || p->rope_stride % 8) return PDA_ERR_MISALIGNED;
  if (p->batch == 0 || p->total_rows == 0) return PDA_OK;
  const bool fp8 = p->kv_dtype == PDA_KV_FP8_E4M3;
  if (!latent || !rope || !row_offsets || !page_table || (write && !starts) || !latent_pages ||
      !rope_pages || (fp8 && !p->latent_scales))
    return PDA_ERR_INVALID_ARG;
  if (!al(latent, 16) || !al(rope, 16) || !al(latent_pages, 16) || !al(rope_pages, 16) ||
      !al(row_offsets, 4) || !al(page_table, 4) || !al(starts, 4))
    return PDA_ERR_MISALIGNED;
  const int sms = device_sms();
  if (sms < 1) return PDA_ERR_CUDA;
  RowsArgs a{};
  a.row_offsets = row_offsets;
  a.page_table = page_table;
  a.starts = starts;
  a.latent = static_cast<uint16_t*>(latent);
  a.rope = static_cast<uint16_t*>(rope);
  a.latent_pages = static_cast<uint8_t*>(latent_pages);
  a.rope_pages = static_cast<uint16_t*>(rope_pages);
  a.scales = static_cast<uint8_t*>(p->latent_scales);
  a.err = device_error_word();
  if (a.err == nullptr) return PDA_ERR_CUDA;
  a.latent_stride = p->latent_stride;
  a.rope_stride = p->rope_stride;
  a.B = p->batch;
  a.total = p->total_rows;
  a.rope_dim = p->rope_dim;
  a.page_size = p->page_size;
  while ((1 << a.log2_page) < p->page_size) ++a.log2_page;
  a.max_pages = p->max_pages_per_seq;
  a.num_pages = p->num_pages;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const bool wide = p->latent_dim == 512;
  if (write) {
    if (fp8) wide ? launch_rows<512, true, true>(a, sms, stream) : launch_rows<256, true, true>(a, sms, stream);
    else wide ? launch_rows<512, false, true>(a, sms, stream) : launch_rows<256, false, true>(a, sms, stream);
  } else {
    if (fp8) wide ? launch_rows<512, true, false>(a, sms, stream) : launch_rows<256, true, false>(a, sms, stream);
    else wide ? launch_rows<512, false, false>(a, sms, stream) : launch_rows<256, false, false>(a, sms, stream);
  }
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

}  // namespace
}  // namespace pda

extern "C" {

pda_status paged_latent_append(const void* latent, const void* rope, const int32_t* row_offsets,
                               const int32_t* page_table, const int32_t* kv_lens,
                               const pda_latent_rows_params* params, void* latent_pages,
                               void* rope_pages, pda_stream_t stream) {
  return pda::rows_call(params, true, const_cast<void*>(latent), const_cast<void*>(rope),
                        row_offsets, page_table, kv_lens, latent_pages, rope_pages, stream);
}

pda_status paged_latent_gather(const void* latent_pages, const void* rope_pages,
                               const int32_t* page_table, const int32_t* row_offsets,
                               const int32_t* starts, const pda_latent_rows_params* params,
                               void* latent, void* rope, pda_stream_t stream) {
  return pda::rows_call(params, false, latent, rope, row_offsets, page_table, starts,
                        const_cast<void*>(latent_pages), const_cast<void*>(rope_pages), stream);
}

}  // extern "C"
