// Rows in 8-bit integers: a row's scale and its values' codes, as the
// quantiser, the gated activation and the one-launch linear compute them.
//
//   s = fp32(max_j |v_j| / 127), 1 for a row of zeros, at least 2^-126
//   q_j = the integer nearest v_j / s, ties to even
//
// The codes are decided exactly: rint(v * (1 / s)) is the right integer or
// off by one where v / s is near a border, and the residual d = v - q s is
// exact in one fma (q has 8 bits and |d| is at most about s, a multiple of
// the smaller of the two's last places), so comparing 2d with s moves q to
// the nearest integer and finds the ties.
//
// A row with an infinity or a NaN gets the scale NaN and zero codes, so
// that whatever is computed from it is NaN.
#pragma once

#include "device_common.hpp"

namespace moe {

// Eight consecutive values of type `dtype` from element `at`; kStream: past the
// caches.
template <bool kStream = false>
__device__ __forceinline__ void load8_as(int dtype, const void* x, size_t at, float (&v)[8]) {
  if (dtype == MOE_TYPE_F32) {
    typedef float f4 __attribute__((ext_vector_type(4)));
    const f4* p = reinterpret_cast<const f4*>(static_cast<const float*>(x) + at);
    const f4 a = kStream ? __builtin_nontemporal_load(p) : p[0];
    const f4 b = kStream ? __builtin_nontemporal_load(p + 1) : p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
    return;
  }
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const u4* p = reinterpret_cast<const u4*>(static_cast<const uint16_t*>(x) + at);
  const u4 a = kStream ? __builtin_nontemporal_load(p) : *p;
  if (dtype == MOE_TYPE_F16) {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    const h8 h = __builtin_bit_cast(h8, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(a[i] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
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

// Eight codes.  v * inv + 1.5 * 2^23 rounds to an integer whose two's
// complement is in the low bits.  Where a residual reaches half a step (a tie,
// or a quotient so near one that inv's rounding shows) the integer moves
// towards the residual if twice its magnitude is past s, or is s and the
// integer odd: as bit patterns of positive floats, |2d| + odd > s.  (bf16
// rows have ties often: with branches for each kind of move 16384 rows of 1024
// took 14.8 us against 11.3.)
__device__ __forceinline__ uint2 int8_codes(const float (&v)[8], float s, float inv) {
  constexpr float kShift = 12582912.f;
  float t[8], d[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(v[i], inv, kShift);
    d[i] = fmaf(kShift - t[i], s, v[i]);
    far = fmaxf(far, fabsf(d[i]));
  }
  if (far + far >= s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t d2 = __float_as_uint(fabsf(d[i] + d[i])) + (__float_as_uint(t[i]) & 1u);
      t[i] += d2 > __float_as_uint(s) ? copysignf(1.f, d[i]) : 0.f;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {   // the low bytes of four
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 1]),
                                              __float_as_uint(t[4 * h]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 3]),
                                              __float_as_uint(t[4 * h + 2]), 0x04000c0cu);
    w[h] = lo | hi;
  }
  return make_uint2(w[0], w[1]);
}

// The largest magnitude among eight values and `top`, as bits.
__device__ __forceinline__ uint32_t max_bits(const float (&v)[8], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return top;
}

// The largest of a wave's values, in every lane: within rows of 16 lanes by
// moves that need no LDS, then across the four rows.
__device__ __forceinline__ uint32_t wave_max(uint32_t top) {
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xb1, 0xf, 0xf, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4e, 0xf, 0xf, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x141, 0xf, 0xf, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x140, 0xf, 0xf, true));
  const uint32_t a = __builtin_amdgcn_readlane((int)top, 0);
  const uint32_t b = __builtin_amdgcn_readlane((int)top, 16);
  const uint32_t c = __builtin_amdgcn_readlane((int)top, 32);
  const uint32_t e = __builtin_amdgcn_readlane((int)top, 48);
  return max(max(a, b), max(c, e));
}

}  // namespace moe
