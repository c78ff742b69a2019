// Helpers shared by the operators around the token mixers (embedding, block
// norms, vocabulary loss).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "common.cuh"

namespace tpk {

// Most SMs of any part this library runs on (workspace sizes that must not
// depend on the current device count on it).
constexpr int kMaxSms = 256;

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// body() -> status, for the C entry points: nothing thrown on the host (out of
// memory, a mutex) leaves the library.
template <typename Body>
int guarded(Body body) {
  try {
    return body();
  } catch (...) {
    return TPK_E_HOST;
  }
}

// Tensor map over a row-major bf16 matrix [rows, cols] with row stride ld
// (elements), 128-byte swizzle, box of 64 columns (128 bytes) x box_rows rows.
// Elements outside the matrix read as zero and are not written.
inline int make_map_2d(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return TPK_E_CUDA;
  if (!aligned16(base) || ld % 8) return TPK_E_ARG;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estride[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estride,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TPK_OK : TPK_E_CUDA;
}

// Two fp32 values as a bf16 pair (round to nearest even), and back.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

}  // namespace tpk
