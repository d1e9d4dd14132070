// Tensor maps for TMA tile loads (host).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

namespace pda {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry point, so the
// library does not link libcuda.
inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// A matrix of `rows` rows of `width` elements (elt bytes: 1 or 2 = bf16),
// `stride` elements apart, read in boxes of 128 bytes x box_rows rows with
// the 128-byte swizzle. A box that reaches past a row's end or the last row
// gets zeros there.
inline bool make_rows_map(CUtensorMap* map, const void* base, long long width, long long rows,
                          long long stride, int elt, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(stride * elt)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / elt), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of `heads` vectors of `width` bf16 each, contiguous, read in boxes of 64
// elements of one head x box_rows rows with the 128-byte swizzle; zeros past
// the ends.
inline bool make_heads_map(CUtensorMap* map, const void* base, long long width, long long heads,
                           long long rows, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)(width * 2), (cuuint64_t)(width * heads * 2)};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of `width` elements (elt bytes: 1 or 2 = bf16), contiguous, as [groups of
// 8 rows][128-byte columns][8 rows][128 bytes]: boxes of box_rows rows (a
// multiple of 8, as is `rows`) x box_cols columns arrive in that order, each 8 x
// 128 bytes swizzled.
inline bool make_tokens_map(CUtensorMap* map, const void* base, long long width, long long rows, int elt,
                            int box_rows, int box_cols) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t row = (cuuint64_t)(width * elt);
  const cuuint64_t dims[4] = {(cuuint64_t)(128 / elt), 8, row / 128, (cuuint64_t)(rows / 8)};
  const cuuint64_t strides[3] = {row, 128, 8 * row};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / elt), 8, (cuuint32_t)box_cols, (cuuint32_t)(box_rows / 8)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pda
