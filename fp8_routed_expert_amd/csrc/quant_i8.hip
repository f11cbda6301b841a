// Rows in 8-bit integers with one scale each, from activations or weights
// (moe_quantize_int8), or from the gated activation between the two expert
// products (moe_act_requant_int8):
//
//   s = fp32(max_j |v_j| / 127), 1 for a row of zeros, at least 2^-126
//   q_j = the integer nearest v_j / s, ties to even
//
// One workgroup per row.  The first kKeep slices of eight values that a
// thread takes stay in its registers between the row's maximum and the
// codes; a longer row's others are read (and the activation computed) again,
// from the cache.  Reads 2 (or 4) bytes and writes one per value: bound by
// HBM bandwidth.
//
// The codes are decided exactly: rint(v * (1 / s)) is the right integer or
// off by one where v / s is near a border, and the residual d = v - q s is
// exact in one fma (q has 8 bits and |d| is at most about s, a multiple of
// the smaller of the two's last places), so comparing 2d with s moves q to
// the nearest integer and finds the ties.
//
// A row with an infinity or a NaN gets the scale NaN and zero codes, so
// that whatever is computed from it is NaN.
#include "device_common.hpp"

namespace moe {

constexpr int kQThreads = 256;
constexpr int kKeep = 4;

__device__ __forceinline__ void load8_as(int dtype, const void* x, size_t at, float (&v)[8]) {
  if (dtype == MOE_TYPE_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    return;
  }
  const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
  if (dtype == MOE_TYPE_F16) {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    const h8 h = __builtin_bit_cast(h8, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  } else {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(w[i] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// A row's scale from the bits of its largest magnitude (a NaN's are above an
// infinity's).
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (amax_bits == 0) return 1.f;
  return fmaxf(__uint_as_float(amax_bits) / 127.f, 0x1p-126f);
}

__device__ __forceinline__ uint32_t int8_code(float v, float s, float inv) {
  float q = rintf(v * inv);
  const float d = fmaf(-q, s, v);
  const float d2 = d + d, up = q + 1.f, down = q - 1.f;
  const bool odd = ((int)q & 1) != 0;
  q = (d2 > s || (d2 == s && odd)) ? up : (d2 < -s || (d2 == -s && odd)) ? down : q;
  return (uint32_t)(int)q & 0xffu;
}

__device__ __forceinline__ uint2 int8_codes(const float (&v)[8], float s, float inv) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= int8_code(v[i], s, inv) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// kAct: v = silu(h[j]) * h[cols + j] of a row [2 cols]; else the row itself.
template <int kType, bool kAct>
__device__ __forceinline__ void row_slice(const void* x, size_t row, int cols, int j,
                                          float (&v)[8]) {
  if constexpr (kAct) {
    float g[8], u[8];
    load8_as(kType, x, row * (size_t)(2 * (long long)cols) + j, g);
    load8_as(kType, x, row * (size_t)(2 * (long long)cols) + cols + j, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu_mul(g[i], u[i]);
  } else {
    load8_as(kType, x, row * (size_t)cols + j, v);
  }
}

template <int kType, bool kAct>
__global__ __launch_bounds__(kQThreads) void quant_int8_kernel(
    const void* __restrict__ x, int rows, int cols, uint8_t* __restrict__ q,
    float* __restrict__ scale, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ counts, int E, int32_t* __restrict__ status) {
  __shared__ uint32_t red[kQThreads / 64];
  if (kAct && blockIdx.x == 0 && threadIdx.x < 64 && status &&
      segments_bad(offsets, counts, E, threadIdx.x) && threadIdx.x == 0)
    atomicOr(status, MOE_ERR_BAD_INDEX);
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    if (kAct && !row_valid(offsets, counts, E, rows, row)) continue;   // uniform
    float v[kKeep][8];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int j = (u * kQThreads + (int)threadIdx.x) * 8;
      if (j < cols) {
        row_slice<kType, kAct>(x, row, cols, j, v[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[u][i]) & 0x7fffffffu);
      }
    }
    for (int j = (kKeep * kQThreads + (int)threadIdx.x) * 8; j < cols; j += kQThreads * 8) {
      float t[8];
      row_slice<kType, kAct>(x, row, cols, j, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(t[i]) & 0x7fffffffu);
    }
    for (int o = 32; o >= 1; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQThreads / 64; ++i) top = max(top, red[i]);
    __syncthreads();
    const float s = int8_scale(top);
    const bool fine = top < 0x7f800000u;
    const float inv = 1.f / s;
    if (threadIdx.x == 0) scale[row] = s;
    uint8_t* out = q + (size_t)row * cols;
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int j = (u * kQThreads + (int)threadIdx.x) * 8;
      if (j < cols)
        *reinterpret_cast<uint2*>(out + j) = fine ? int8_codes(v[u], s, inv) : make_uint2(0, 0);
    }
    for (int j = (kKeep * kQThreads + (int)threadIdx.x) * 8; j < cols; j += kQThreads * 8) {
      float t[8];
      row_slice<kType, kAct>(x, row, cols, j, t);
      *reinterpret_cast<uint2*>(out + j) = fine ? int8_codes(t, s, inv) : make_uint2(0, 0);
    }
  }
}

template <bool kAct>
static moe_status_t quantize_int8(const void* x, int dtype, int rows, int cols, int8_t* q,
                                  float* scale, const int32_t* offsets, const int32_t* counts,
                                  int E, int32_t* status, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(rows < (1 << 22) ? rows : (1 << 22))), block(kQThreads);
  uint8_t* qb = reinterpret_cast<uint8_t*>(q);
  if (dtype == MOE_TYPE_F32)
    hipLaunchKernelGGL((quant_int8_kernel<MOE_TYPE_F32, kAct>), grid, block, 0, st, x, rows, cols,
                       qb, scale, offsets, counts, E, status);
  else if (dtype == MOE_TYPE_BF16)
    hipLaunchKernelGGL((quant_int8_kernel<MOE_TYPE_BF16, kAct>), grid, block, 0, st, x, rows,
                       cols, qb, scale, offsets, counts, E, status);
  else
    hipLaunchKernelGGL((quant_int8_kernel<MOE_TYPE_F16, kAct>), grid, block, 0, st, x, rows, cols,
                       qb, scale, offsets, counts, E, status);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

static bool float_type(int dtype) {
  return dtype == MOE_TYPE_F32 || dtype == MOE_TYPE_BF16 || dtype == MOE_TYPE_F16;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_quantize_int8(const void* x, int dtype, int rows, int cols, int8_t* q,
                                          float* scale, void* stream) {
  if (!float_type(dtype) || rows < 0 || cols <= 0) return MOE_INVALID_ARG;
  if (cols % 16 != 0) return MOE_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_INVALID_ARG;
  if (((uintptr_t)x | (uintptr_t)q) & 15) return MOE_UNSUPPORTED_SHAPE;
  return quantize_int8<false>(x, dtype, rows, cols, q, scale, nullptr, nullptr, 0, nullptr,
                              stream);
}

extern "C" moe_status_t moe_act_requant_int8(const void* h, int dtype, const int32_t* offsets,
                                             const int32_t* counts, int E, int rows_total, int I,
                                             int8_t* q, float* q_scale, int32_t* status_dev,
                                             void* stream) {
  if (!float_type(dtype) || E <= 0 || E > MOE_MAX_EXPERTS || rows_total < 0 || I <= 0)
    return MOE_INVALID_ARG;
  if (I % 16 != 0 || I > (1 << 30)) return MOE_UNSUPPORTED_SHAPE;
  if (!offsets || !counts) return MOE_INVALID_ARG;
  if (rows_total == 0) return MOE_OK;
  if (!h || !q || !q_scale) return MOE_INVALID_ARG;
  if (((uintptr_t)h | (uintptr_t)q) & 15) return MOE_UNSUPPORTED_SHAPE;
  return quantize_int8<true>(h, dtype, rows_total, I, q, q_scale, offsets, counts, E, status_dev,
                             stream);
}

// ---- a whole linear: quantise the rows, then the product.  The workspace
// holds the codes [M, K] and, from the next multiple of 16 bytes, the scales.
extern "C" size_t moe_linear_int8_workspace_bytes(int M, int K) {
  if (M < 0 || K <= 0) return 0;
  const size_t codes = ((size_t)M * (size_t)K + 15) / 16 * 16;
  return codes + (size_t)M * sizeof(float);
}

extern "C" moe_status_t moe_linear_int8(const void* x, int dtype, const int8_t* w,
                                        const float* w_scale, int M, int N, int K, void* c,
                                        int c_type, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  if (!float_type(dtype) || !float_type(c_type) || M < 0 || N <= 0 || K <= 0)
    return MOE_INVALID_ARG;
  if (N % 16 != 0 || K % 16 != 0 || K > 131056) return MOE_UNSUPPORTED_SHAPE;
  if (!w || !w_scale) return MOE_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !c || !workspace || workspace_bytes < moe_linear_int8_workspace_bytes(M, K))
    return MOE_INVALID_ARG;
  if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)c | (uintptr_t)workspace) & 15)
    return MOE_UNSUPPORTED_SHAPE;
  int8_t* q = static_cast<int8_t*>(workspace);
  float* s = reinterpret_cast<float*>(q + ((size_t)M * (size_t)K + 15) / 16 * 16);
  const moe_status_t ok = quantize_int8<false>(x, dtype, M, K, q, s, nullptr, nullptr, 0, nullptr,
                                               stream);
  if (ok != MOE_OK) return ok;
  return moe_gemm_int8(q, s, w, w_scale, M, N, K, c, c_type, stream);
}
