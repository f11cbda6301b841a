// Rows in 8-bit integers with one scale each, from activations or weights
// (moe_quantize_int8), or from the gated activation between the two expert
// products (moe_act_requant_int8):
//
//   s = fp32(max_j |v_j| / 127), 1 for a row of zeros, at least 2^-126
//   q_j = the integer nearest v_j / s, ties to even
//
// A wave per row (no barrier) or the four waves of a workgroup.  The first
// kKeep slices of eight values that a lane takes stay in its registers between
// the row's maximum and the codes; the others of a longer row are read (and
// the activation computed) again, from the cache.  Reads 2 (or 4) bytes and
// writes one per value.  Large inputs are bound by HBM bandwidth (65536 rows of
// 7168 bf16 250 us, 5.6 TB/s; 16384 of 4096 5.9; the activation of 131072 rows of
// 2 x 2048 220 us, 6.1 TB/s); a few thousand rows by the chain of a row's slices,
// one load after the other (8191 rows of 2048 11.5 us, 4.4 TB/s; the activation of
// 5529 rows of 2 x 2048 15 us, of which the bytes are 9), and the activation of a
// masked or padded buffer takes as long as that of a full one.
#include <type_traits>

#include "rows_i8.hpp"

namespace moe {

constexpr int kQThreads = 256;
constexpr int kKeep = 4;

// kAct: v = silu(h[j]) * h[cols + j] of a row [2 cols]; else the row itself.
template <int kType, bool kAct, bool kStream>
__device__ __forceinline__ void row_slice(const void* x, size_t row, int cols, int j,
                                          float (&v)[8]) {
  if constexpr (kAct) {
    float g[8], u[8];
    load8_as<kStream>(kType, x, row * (size_t)(2 * (long long)cols) + j, g);
    load8_as<kStream>(kType, x, row * (size_t)(2 * (long long)cols) + cols + j, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu_mul(g[i], u[i]);
  } else {
    load8_as<kStream>(kType, x, row * (size_t)cols + j, v);
  }
}

// kWaves: waves per row (1 or 4); kStream: the rows are read past the caches.
template <int kType, bool kAct, int kWaves, bool kStream>
__global__ __launch_bounds__(kQThreads) void quant_int8_kernel(
    const void* __restrict__ x, int rows, int cols, uint8_t* __restrict__ q,
    float* __restrict__ scale, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ counts, int E, int32_t* __restrict__ status) {
  constexpr int kRows = kQThreads / 64 / kWaves;   // rows of a workgroup
  constexpr int kStep = kWaves * 64 * 8;           // values a row's lanes take at once
  __shared__ uint32_t red[kQThreads / 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (kAct && blockIdx.x == 0 && threadIdx.x < 64 && status &&
      segments_bad(offsets, counts, E, threadIdx.x) && threadIdx.x == 0)
    atomicOr(status, MOE_ERR_BAD_INDEX);
  const int j0 = kWaves == 1 ? (threadIdx.x & 63) * 8 : threadIdx.x * 8;
  for (long long at = (long long)blockIdx.x * kRows + (kWaves == 1 ? wave : 0); at < rows;
       at += (long long)gridDim.x * kRows) {
    const int row = (int)at;
    // Slice by slice (lanes past the row read its first one again): each test of
    // a slice is a branch, so the compiler waits for its load and converts it
    // (or evaluates the activation) before the next slice's load goes out.  The
    // row's segment is looked up last, so rows outside the segments are read and
    // computed like the others, and then dropped.
    float v[kKeep][8];
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int j = u * kStep + j0;
      if (u * kStep < cols) row_slice<kType, kAct, kStream>(x, row, cols, j < cols ? j : 0, v[u]);
    }
    if (kAct && !row_valid(offsets, counts, E, rows, row)) continue;   // the same for the row
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kKeep; ++u)
      if (u * kStep < cols) top = max_bits(v[u], top);
    for (int j = kKeep * kStep + j0; j < cols; j += kStep) {
      float t[8];
      row_slice<kType, kAct, kStream>(x, row, cols, j, t);
      top = max_bits(t, top);
    }
    top = wave_max(top);
    if (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) red[wave] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWaves; ++i) top = max(top, red[i]);
      __syncthreads();
    }
    const float s = int8_scale(top);
    const bool fine = top < 0x7f800000u;
    const float inv = 1.f / s;
    if (j0 == 0) scale[row] = s;
    uint8_t* out = q + (size_t)row * cols;
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int j = u * kStep + j0;
      if (j < cols)
        *reinterpret_cast<uint2*>(out + j) = fine ? int8_codes(v[u], s, inv) : make_uint2(0, 0);
    }
    for (int j = kKeep * kStep + j0; j < cols; j += kStep) {
      float t[8];
      row_slice<kType, kAct, kStream>(x, row, cols, j, t);
      *reinterpret_cast<uint2*>(out + j) = fine ? int8_codes(t, s, inv) : make_uint2(0, 0);
    }
  }
}

template <int kType, bool kAct>
static void launch_quant(const void* x, int rows, int cols, uint8_t* q, float* scale,
                         const int32_t* offsets, const int32_t* counts, int E, int32_t* status,
                         hipStream_t st) {
  // a wave per row where the lanes of four would idle, or where there are
  // enough rows to fill the CUs, with a row's slices loaded one after the other
  // as they are (bf16, 8191 rows of 2048: 11.5 us against 12.8
  // with four waves, 2048 rows 4.5 against 5.0; 96 rows 3.7 against 2.9, all
  // latency; 8191 rows of 1024 6.1 against 10.5, 96 rows 3.0 against 2.9)
  const bool one = cols <= 1024 || (cols <= kKeep * 64 * 8 && rows > 1536);
  const long long blocks = one ? ((long long)rows + 3) / 4 : rows;
  const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : (1 << 22))), block(kQThreads);
  // Past the caches where h is more than the memory-side cache (256 MB) holds:
  // 131072 rows of 2 x 2048 220 us against 254, but 16384 34 against 31.  (The
  // plain rows gain nothing: 65536 of 7168 bf16 254 against 248.  Codes stored
  // past the caches cost the product that reads them next more than they give.)
  const bool past = kAct && 2LL * rows * cols * (kType == MOE_TYPE_F32 ? 4 : 2) > (512LL << 20);
  auto run = [&](auto waves, auto stream) {
    hipLaunchKernelGGL((quant_int8_kernel<kType, kAct, waves.value, stream.value>), grid, block, 0,
                       st, x, rows, cols, q, scale, offsets, counts, E, status);
  };
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  if (past && one)
    run(One(), std::integral_constant<bool, kAct>());
  else if (past)
    run(Four(), std::integral_constant<bool, kAct>());
  else if (one)
    run(One(), std::false_type());
  else
    run(Four(), std::false_type());
}

template <bool kAct>
static moe_status_t quantize_int8(const void* x, int dtype, int rows, int cols, int8_t* q,
                                  float* scale, const int32_t* offsets, const int32_t* counts,
                                  int E, int32_t* status, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  uint8_t* qb = reinterpret_cast<uint8_t*>(q);
  if (dtype == MOE_TYPE_F32)
    launch_quant<MOE_TYPE_F32, kAct>(x, rows, cols, qb, scale, offsets, counts, E, status, st);
  else if (dtype == MOE_TYPE_BF16)
    launch_quant<MOE_TYPE_BF16, kAct>(x, rows, cols, qb, scale, offsets, counts, E, status, st);
  else
    launch_quant<MOE_TYPE_F16, kAct>(x, rows, cols, qb, scale, offsets, counts, E, status, st);
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
  // (the kernel's index into a row goes a step past its end)
  if (cols % 16 != 0 || cols > 0x7ffff000) return MOE_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_INVALID_ARG;
  if ((((uintptr_t)x | (uintptr_t)q) & 15) || ((uintptr_t)scale & 3)) return MOE_UNSUPPORTED_SHAPE;
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
  if ((((uintptr_t)h | (uintptr_t)q) & 15) || ((uintptr_t)q_scale & 3))
    return MOE_UNSUPPORTED_SHAPE;
  return quantize_int8<true>(h, dtype, rows_total, I, q, q_scale, offsets, counts, E, status_dev,
                             stream);
}
