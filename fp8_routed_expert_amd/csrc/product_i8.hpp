// What the 8-bit integer products share: the multiplication and the arguments.
#pragma once

#include "gemm_tiles.hpp"

namespace moe {

__device__ __forceinline__ v4i mfma_i8(const v4i& a, const v4i& b, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, (h2){(_Float16)lo, (_Float16)hi});
}

// The arguments of a product.  offsets == nullptr: dense (one weight matrix,
// every row of it).  row_src != nullptr: buffer row r is row row_src[r] of a
// [src_rows, K], its scale a_scale[row_src[r]].
struct I8Args {
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* w;
  const float* w_scale;
  const int32_t* offsets;
  const int32_t* counts;
  const int32_t* row_src;
  int E, rows_total, N, K, src_rows;
  void* c;
  int c_type;
  int32_t* status;
};

}  // namespace moe
