// The experts' products in fp32, bf16 and fp16, and their gradients, over the
// expert segments:
//
//   product            c[m, n] = sum_k a[m, k] w[e, n, k]
//   rows' gradient     da[m, k] = sum_n dc[m, n] w[e, n, k]
//   weights' gradient  dw[e, n, k] = sum of dc[m, n] a[m, k] over segment e
//
// All three are out(i, j) = sum_l P(i, l) Q(j, l) with the output contiguous
// along j; in the first both operands are contiguous along l, in the second Q
// is contiguous along j, in the third P is along i as well.  Sums are fp32, on
// the matrix cores, rounded once when stored.
#include <type_traits>

#include "gemm_tiles.hpp"

namespace moe {

enum { kProduct = 0, kRowsGrad = 1, kWeightsGrad = 2 };

struct FloatArgs {
  const uint8_t* p;   // a; dc in both gradients
  const uint8_t* q;   // w; w; a
  const int32_t* offsets;
  const int32_t* counts;
  int E, rows, N, K;
  uint8_t* out;
  int out_type;
  int32_t* status;
};

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// sums += 16 x 16 x 32 products of eight elements per lane: lane (g, r) holds
// elements l = 8 g .. 8 g + 7 of row r of each operand (in fp32 an instruction
// takes one element of every lane: l = 8 g + i, the same for both operands).
template <int kType, typename Frag>
__device__ __forceinline__ v4f multiply8(const Frag& a, const Frag& b, v4f c) {
  if constexpr (kType == MOE_TYPE_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  } else if constexpr (kType == MOE_TYPE_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
}

template <int kType>
using Elem = std::conditional_t<kType == MOE_TYPE_F32, float, uint16_t>;
template <int kType>
using Frag8 = std::conditional_t<kType == MOE_TYPE_F32, float __attribute__((ext_vector_type(8))),
                                 uint16_t __attribute__((ext_vector_type(8)))>;

// A 64 x 64 tile by four waves of 32 x 32, l advancing 32 a step through LDS.
template <int kType, int kMode>
__global__ __launch_bounds__(256) void float_tile_kernel(FloatArgs p) {
  typedef Elem<kType> El;
  typedef Frag8<kType> Frag;
  constexpr int BM = 64, BN = 64, BL = 32, kPitch = BL + 8;
  __shared__ __attribute__((aligned(16))) El sp[BM][kPitch], sq[BN][kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0 && threadIdx.x < 64 && p.status &&
      segments_bad(p.offsets, p.counts, p.E, lane) && lane == 0)
    atomicOr(p.status, MOE_ERR_BAD_INDEX);
  // operands of the tile: rows [i0, i_end) of P, [j0, j_end) of Q, L products
  const int width = kMode == kProduct ? p.N : p.K;
  const int n_tiles = (width + BN - 1) / BN;
  const int tile_i = blockIdx.x / n_tiles;
  const int j0 = (blockIdx.x - tile_i * n_tiles) * BN, j_end = width;
  int e = 0, i0 = 0, i_end = 0, L;
  const El* P = reinterpret_cast<const El*>(p.p);
  const El* Q = reinterpret_cast<const El*>(p.q);
  size_t pp, qp;   // elements from one row of memory to the next
  if (kMode == kWeightsGrad) {
    int s, en;
    const int i_tiles = (p.N + BM - 1) / BM;
    e = tile_i / i_tiles;
    expert_rows(p.offsets, p.counts, e, p.rows, s, en);
    i0 = (tile_i - e * i_tiles) * BM;
    i_end = p.N;
    L = en - s;
    pp = p.N;
    qp = p.K;
    P += (size_t)s * pp;
    Q += (size_t)s * qp;
  } else {
    find_mtile<BM>(p.offsets, p.counts, p.E, p.rows, tile_i, lane, e, i0, i_end);
    if (e < 0) return;
    L = kMode == kProduct ? p.K : p.N;
    pp = L;
    qp = p.K;
    Q += (size_t)e * p.N * p.K;
  }
  const El zero = (El)0;
  // eight elements of memory a thread and step: along l, or along the row
  auto stage = [&](El (*tile)[kPitch], const El* base, size_t pitch, bool along_l, int r0,
                   int r_end, int l0) {
    const int fast = along_l ? (threadIdx.x & 3) * 8 : (threadIdx.x & 7) * 8;
    const int slow = along_l ? threadIdx.x >> 2 : threadIdx.x >> 3;
    const int r = r0 + (along_l ? slow : fast), l = l0 + (along_l ? fast : slow);
    El v[8];
    const bool in = r < r_end && l < L;   // (both are in steps of eight along memory)
    const El* src = base + (along_l ? (size_t)r * pitch + l : (size_t)l * pitch + r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = in ? src[i] : zero;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (along_l)
        tile[slow][fast + i] = v[i];
      else
        tile[fast + i][slow] = v[i];
  };
  v4f acc[2][2] = {};
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int g = lane >> 4, r16 = lane & 15;
  for (int l0 = 0; l0 < L; l0 += BL) {
    __syncthreads();
    stage(sp, P, pp, kMode != kWeightsGrad, i0, i_end, l0);
    stage(sq, Q, qp, kMode == kProduct, j0, j_end, l0);
    __syncthreads();
    Frag fp[2], fq[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      __builtin_memcpy(&fp[u], &sp[wm + 16 * u + r16][8 * g], sizeof(Frag));
      __builtin_memcpy(&fq[u], &sq[wn + 16 * u + r16][8 * g], sizeof(Frag));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 2; ++v) acc[u][v] = multiply8<kType>(fq[v], fp[u], acc[u][v]);
  }
  // sums (u, v) of a lane: row r16 of P, four neighbours 4 g .. 4 g + 3 of Q
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int i = i0 + wm + 16 * u + r16, j = j0 + wn + 16 * v + 4 * g;
      if (i >= i_end || j >= j_end) continue;
      const size_t at = ((kMode == kWeightsGrad ? (size_t)e * p.N : 0) + i) * width + j;
      const v4f s = acc[u][v];
      if (p.out_type == MOE_TYPE_F32) {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) =
            make_float4(s[0], s[1], s[2], s[3]);
      } else {
        uint2 o;
        if (kType == MOE_TYPE_F16) {
          typedef _Float16 h2 __attribute__((ext_vector_type(2)));
          o.x = __builtin_bit_cast(uint32_t, (h2){(_Float16)s[0], (_Float16)s[1]});
          o.y = __builtin_bit_cast(uint32_t, (h2){(_Float16)s[2], (_Float16)s[3]});
        } else {
          o = make_uint2(pack2_bf16(s[0], s[1]), pack2_bf16(s[2], s[3]));
        }
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at) = o;
      }
    }
}

// Rows that no expert has, set to zero: a wave to a row.
__global__ __launch_bounds__(256) void zero_rest_kernel(const int32_t* offsets,
                                                        const int32_t* counts, int E, int rows,
                                                        long long row_bytes, uint8_t* out) {
  const int lane = threadIdx.x & 63;
  for (long long m = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); m < rows;
       m += (long long)gridDim.x * 4) {
    if (row_valid(offsets, counts, E, rows, (int)m)) continue;
    for (long long c = lane; c < row_bytes / 16; c += 64)
      reinterpret_cast<uint4*>(out + m * row_bytes)[c] = make_uint4(0, 0, 0, 0);
  }
}

static bool float_type(int dtype) {
  return dtype == MOE_TYPE_F32 || dtype == MOE_TYPE_BF16 || dtype == MOE_TYPE_F16;
}

template <int kMode>
static moe_status_t launch_float(const FloatArgs& p, int dtype, hipStream_t st) {
  const int width = kMode == kProduct ? p.N : p.K;
  const dim3 block(256);
  const long long tiles_i =
      kMode == kWeightsGrad ? (long long)p.E * ((p.N + 63) / 64) : (long long)p.rows / 64 + p.E;
  const long long tiles = tiles_i * ((width + 63) / 64);
  if (tiles * 256 > 0xffffffffLL) return MOE_UNSUPPORTED_SHAPE;   // threads of a launch
  const dim3 grid((unsigned)tiles);
  if (dtype == MOE_TYPE_F32)
    hipLaunchKernelGGL((float_tile_kernel<MOE_TYPE_F32, kMode>), grid, block, 0, st, p);
  else if (dtype == MOE_TYPE_BF16)
    hipLaunchKernelGGL((float_tile_kernel<MOE_TYPE_BF16, kMode>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((float_tile_kernel<MOE_TYPE_F16, kMode>), grid, block, 0, st, p);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

constexpr int kMaxFloatDim = 1 << 20;     // N and K

static moe_status_t float_args(const FloatArgs& p, int dtype) {
  if (!float_type(dtype) || p.E <= 0 || p.E > MOE_MAX_EXPERTS || p.rows < 0 || p.N <= 0 ||
      p.K <= 0)
    return MOE_INVALID_ARG;
  if (p.N % 8 != 0 || p.K % 8 != 0 || p.N > kMaxFloatDim || p.K > kMaxFloatDim)
    return MOE_UNSUPPORTED_SHAPE;
  if (!p.offsets || !p.counts) return MOE_INVALID_ARG;
  if (((uintptr_t)p.p | (uintptr_t)p.q | (uintptr_t)p.out) & 15) return MOE_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

template <int kMode>
static moe_status_t float_rows(const FloatArgs& p, int dtype, int zero_rest, void* stream) {
  const moe_status_t ok = float_args(p, dtype);
  if (ok != MOE_OK) return ok;
  if (!p.q) return MOE_INVALID_ARG;
  if (p.rows == 0) return MOE_OK;
  if (!p.p || !p.out) return MOE_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (zero_rest) {
    const long long blocks = ((long long)p.rows + 3) / 4;
    const long long bytes =
        (long long)(kMode == kProduct ? p.N : p.K) * (dtype == MOE_TYPE_F32 ? 4 : 2);
    hipLaunchKernelGGL(zero_rest_kernel, dim3((unsigned)(blocks < (1 << 22) ? blocks : (1 << 22))),
                       dim3(256), 0, st, p.offsets, p.counts, p.E, p.rows, bytes, p.out);
  }
  return launch_float<kMode>(p, dtype, st);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_grouped_gemm_float(const void* a, const void* w, int dtype,
                                               const int32_t* offsets, const int32_t* counts,
                                               int E, int rows_total, int N, int K, void* c,
                                               int zero_rest, int32_t* status_dev, void* stream) {
  const FloatArgs p{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(w), offsets,
                    counts, E, rows_total, N, K, static_cast<uint8_t*>(c), dtype, status_dev};
  return float_rows<kProduct>(p, dtype, zero_rest, stream);
}

extern "C" moe_status_t moe_grouped_gemm_float_grad_rows(const void* dc, const void* w, int dtype,
                                                         const int32_t* offsets,
                                                         const int32_t* counts, int E,
                                                         int rows_total, int N, int K, void* da,
                                                         int zero_rest, int32_t* status_dev,
                                                         void* stream) {
  const FloatArgs p{static_cast<const uint8_t*>(dc), static_cast<const uint8_t*>(w), offsets,
                    counts, E, rows_total, N, K, static_cast<uint8_t*>(da), dtype, status_dev};
  return float_rows<kRowsGrad>(p, dtype, zero_rest, stream);
}

extern "C" size_t moe_grouped_gemm_float_workspace_bytes(int E, int rows_total, int N, int K) {
  (void)E; (void)rows_total; (void)N; (void)K;
  return 0;
}

extern "C" moe_status_t moe_grouped_gemm_float_grad_weights(
    const void* dc, const void* a, int dtype, const int32_t* offsets, const int32_t* counts, int E,
    int rows_total, int N, int K, void* dw, int dw_type, void* workspace, size_t workspace_bytes,
    int32_t* status_dev, void* stream) {
  const FloatArgs p{static_cast<const uint8_t*>(dc), static_cast<const uint8_t*>(a), offsets,
                    counts, E, rows_total, N, K, static_cast<uint8_t*>(dw), dw_type, status_dev};
  const moe_status_t ok = float_args(p, dtype);
  if (ok != MOE_OK) return ok;
  if (dw_type != dtype && dw_type != MOE_TYPE_F32) return MOE_INVALID_ARG;
  if (!dw || (rows_total > 0 && (!dc || !a))) return MOE_INVALID_ARG;
  const size_t need = moe_grouped_gemm_float_workspace_bytes(E, rows_total, N, K);
  if (need && (!workspace || workspace_bytes < need)) return MOE_INVALID_ARG;
  if ((uintptr_t)workspace & 15) return MOE_UNSUPPORTED_SHAPE;
  return launch_float<kWeightsGrad>(p, dtype, reinterpret_cast<hipStream_t>(stream));
}
