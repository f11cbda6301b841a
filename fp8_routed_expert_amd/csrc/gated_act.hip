// The gated activation between the experts' two products, and its gradient,
// in fp32, bf16 and fp16, for the valid rows of the expert segments.
//
//   q = silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g))
//   dg = dq u s (1 + g (1 - s)),  du = dq g s
//
// h [rows, 2I] holds g in its first I columns and u in the others.  Every value
// is read and written once: bound by HBM bandwidth.
#include "row_chunks.hpp"

namespace moe {

struct ActArgs {
  const uint8_t* h;
  const uint8_t* dq;
  const int32_t* offsets;
  const int32_t* counts;
  int E, rows, I;
  uint8_t* out;      // q, or dh
  int zero_rest;
  int32_t* status;
};

// sigmoid(g) and 1 - sigmoid(g), both without cancellation, from
// e = exp(-|g|): 1 / (1 + e) and e / (1 + e), the larger one sigmoid of |g|.
// |g| log2(e) is kept in two parts (the exponential would scale its rounding
// up by |g|) and the base-2 exponential taken of its half and squared, so that
// e may be subnormal, which the hardware's instruction flushes.  The hardware's
// exponential and reciprocal are good to about 1 ulp each.
__device__ __forceinline__ void sigmoid(float g, float& s, float& rest) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.9259629911266175e-8f;
  const float a = fminf(fabsf(g), 256.f);
  const float t = a * kLog2e;
  const float low = fmaf(a, kLog2e, -t) + a * kLog2eLow;
  const float h = __builtin_amdgcn_exp2f(-0.5f * t);
  const float e = h * (h * fmaf(low, -0.693147182464599609375f, 1.f));
  const float big = __builtin_amdgcn_rcpf(1.f + e);
  const float small = e * big;
  s = g < 0.f ? small : big;
  rest = g < 0.f ? big : small;
}

// A lane takes a chunk (16 bytes of each operand), a wave 64 neighbouring ones
// of a row and the next.  Up to 64 experts (kFew), the wave's lanes hold their
// segments, so that the rows are looked up without a search through memory:
// a search for every row took 9.3 us at a decode share of 1193 rows on 32
// experts, and takes 6.8 (floor 2.4: the vector units are active in 77% of the
// cycles, mostly for waves that find their rows not valid).  More experts are
// searched for: 131040 rows of 2048 bf16 on 65 351 us, the gradient
// 452, on 256 386 and 474; on 9 260 and 446.
template <typename El, bool kGrad, bool kStream, bool kFew>
__global__ __launch_bounds__(256) void gated_act_kernel(ActArgs p) {
  constexpr int N = El::kN;
  const int lane = threadIdx.x & 63;
  const unsigned per_row = (unsigned)(p.I / N);
  int first = 0, end = 0;
  if (kFew && lane < p.E) expert_rows(p.offsets, p.counts, lane, p.rows, first, end);
  if (blockIdx.x == 0 && threadIdx.x < 64 && p.status &&
      segments_bad(p.offsets, p.counts, p.E, lane) && lane == 0)
    atomicOr(p.status, MOE_ERR_BAD_INDEX);
  const size_t row = (size_t)p.I * El::kSize;
  const long long waves = ((long long)p.rows * per_row + 63) / 64;
  for (long long u = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       u < waves; u += (long long)gridDim.x * 4) {
    const int m0 = (int)(u * 64 / per_row);
    const unsigned in = (unsigned)(u * 64 - (long long)m0 * per_row) + lane;
    const unsigned past = in / per_row;
    const int m = m0 + (int)past;
    const unsigned c = in - past * per_row;
    bool valid = false;
    if (kFew) {
      const int last = __builtin_amdgcn_readlane(m, 63);
      for (int q = m0; q <= last; ++q) {
        const bool v = __ballot(q >= first && q < end) != 0;
        if (q == m) valid = v;
      }
    } else if (m < p.rows) {
      valid = row_valid(p.offsets, p.counts, p.E, p.rows, m);
    }
    if (m >= p.rows || (!valid && !p.zero_rest)) continue;
    uint8_t* out = p.out + chunk_at(m, kGrad ? 2 * row : row, c);
    if (!valid) {
      store_chunk<true>(out, 16, make_uint4(0, 0, 0, 0));
      if (kGrad) store_chunk<true>(out + row, 16, make_uint4(0, 0, 0, 0));
      continue;
    }
    const uint8_t* h = p.h + chunk_at(m, 2 * row, c);
    float g[N], v[N], d[N];
    El::unpack(load_chunk<true, kStream>(h, 16), g);
    El::unpack(load_chunk<true, kStream>(h + row, 16), v);
    if (kGrad) {
      const uint8_t* dq = p.dq + chunk_at(m, row, c);
      El::unpack(load_chunk<true, kStream>(dq, 16), d);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float s, rest;
        sigmoid(g[i], s, rest);
        const float gate = d[i] * v[i] * s * fmaf(g[i], rest, 1.f);
        v[i] = d[i] * g[i] * s;
        g[i] = gate;
      }
      store_chunk<true>(out, 16, pack_row<El>(g));
      store_chunk<true>(out + row, 16, pack_row<El>(v));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float s, rest;
        sigmoid(g[i], s, rest);
        g[i] = g[i] * s * v[i];
      }
      store_chunk<true>(out, 16, pack_row<El>(g));
    }
  }
}

template <bool kGrad>
static moe_status_t gated_act(const ActArgs& p, int dtype, hipStream_t st) {
  if ((dtype != MOE_TYPE_F32 && dtype != MOE_TYPE_BF16 && dtype != MOE_TYPE_F16) || p.E <= 0 ||
      p.E > MOE_MAX_EXPERTS || p.rows < 0 || p.I <= 0)
    return MOE_INVALID_ARG;
  // (a wave's last row may lie 64 behind the last one)
  if (p.I % 8 != 0 || p.I > (1 << 28) || p.rows > 0x7fff0000) return MOE_UNSUPPORTED_SHAPE;
  if (!p.offsets || !p.counts) return MOE_INVALID_ARG;
  if (p.rows == 0) return MOE_OK;
  if (!p.h || !p.out || (kGrad && !p.dq)) return MOE_INVALID_ARG;
  if (((uintptr_t)p.h | (uintptr_t)p.dq | (uintptr_t)p.out) & 15) return MOE_UNSUPPORTED_SHAPE;
  const int n = dtype == MOE_TYPE_F32 ? 4 : 8;
  const long long units = ((long long)p.rows * (p.I / n) + 255) / 256;
  // Workgroups that end after a few chunks: with as few as the CUs hold at once,
  // whose waves wait for one chunk after the other, the gradient of a prefill
  // share took 511 us, with 16384 466, with 65536 442, without a limit 461 (and
  // the activation 323, 299, 293, 307).
  constexpr long long kMost = 65536;
  const dim3 grid((unsigned)(units < kMost ? units : kMost)), block(256);
  // past the caches where the rows are more than the memory-side cache holds
  const bool past = (long long)p.rows * p.I * (kGrad ? 3 : 2) * (16 / n) > (400LL << 20);
  auto run = [&](auto el) {
    using El = decltype(el);
    if (p.E > 64)
      hipLaunchKernelGGL((gated_act_kernel<El, kGrad, false, false>), grid, block, 0, st, p);
    else if (past)
      hipLaunchKernelGGL((gated_act_kernel<El, kGrad, true, true>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((gated_act_kernel<El, kGrad, false, true>), grid, block, 0, st, p);
  };
  if (dtype == MOE_TYPE_F32)
    run(F32());
  else if (dtype == MOE_TYPE_BF16)
    run(BF16());
  else
    run(F16());
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_gated_act(const void* h, int dtype, const int32_t* offsets,
                                      const int32_t* counts, int E, int rows_total, int I, void* q,
                                      int zero_rest, int32_t* status_dev, void* stream) {
  const ActArgs p{static_cast<const uint8_t*>(h), nullptr, offsets, counts, E, rows_total, I,
                  static_cast<uint8_t*>(q), zero_rest, status_dev};
  return gated_act<false>(p, dtype, reinterpret_cast<hipStream_t>(stream));
}

extern "C" moe_status_t moe_gated_act_grad(const void* dq, const void* h, int dtype,
                                           const int32_t* offsets, const int32_t* counts, int E,
                                           int rows_total, int I, void* dh, int zero_rest,
                                           int32_t* status_dev, void* stream) {
  const ActArgs p{static_cast<const uint8_t*>(h), static_cast<const uint8_t*>(dq), offsets, counts,
                  E, rows_total, I, static_cast<uint8_t*>(dh), zero_rest, status_dev};
  return gated_act<true>(p, dtype, reinterpret_cast<hipStream_t>(stream));
}
