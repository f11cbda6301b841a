// Rows of any length in 32-, 16- and 8-bit types, read and written in 16-byte
// chunks.
//
// A row is a run of H elements cut into 16-byte chunks.  Rows whose length in
// bytes is no multiple of 16 (or whose buffers are not 16-byte aligned) are
// read through unaligned 16-byte accesses, and their last chunk starts 16
// bytes before the row's end: it overlaps the one before it, so that every
// access is wide and none leaves the row.  The overlap writes the same values
// twice and is left out of sums.  Rows shorter than 16 bytes are one chunk of
// single bytes.
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace moe {

typedef unsigned int row_chunk __attribute__((ext_vector_type(4)));

struct F32 {
  static constexpr int kSize = 4, kN = 4;
  __device__ __forceinline__ static void unpack(const uint4& v, float (&f)[kN]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[kN]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

// 16-bit types: eight elements, rounded to nearest even once, when stored.
struct BF16 {
  static constexpr int kSize = 2, kN = 8;
  __device__ __forceinline__ static void unpack(const uint4& v, float (&f)[kN]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_to_f32(w[i] & 0xffffu);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[kN]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = f32_to_bf16(f[2 * i]) | ((uint32_t)f32_to_bf16(f[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct F16 {
  static constexpr int kSize = 2, kN = 8;
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  __device__ __forceinline__ static void unpack(const uint4& v, float (&f)[kN]) {
    const h8 h = __builtin_bit_cast(h8, v);
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = (float)h[i];
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[kN]) {
    h8 h;
#pragma unroll
    for (int i = 0; i < kN; ++i) h[i] = (_Float16)f[i];
    return __builtin_bit_cast(uint4, h);
  }
};

// A chunk of rounded values; bf16 in the hardware's conversion (to nearest
// even, as BF16::pack, a NaN stays one).
template <typename El>
__device__ __forceinline__ uint4 pack_row(const float (&f)[El::kN]) {
  if constexpr (std::is_same<El, BF16>::value) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_bit_cast(
          uint32_t, __builtin_convertvector((f32x2){f[2 * i], f[2 * i + 1]}, bf16x2));
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return El::pack(f);
  }
}

// A row's chunks: chunk c starts at byte start(c).
struct RowShape {
  int bytes;    // of a row
  int chunks;   // ceil(bytes / 16)
  __device__ __forceinline__ int start(int c) const {
    return bytes >= 16 ? min(16 * c, bytes - 16) : 0;
  }
};

// The byte at which chunk c of row m starts in a matrix of whole chunks, in 64
// bits: rows times bytes leave 31, and so does twice a row number.
__host__ __device__ __forceinline__ size_t chunk_at(int m, size_t row_bytes, unsigned c) {
  return (size_t)m * row_bytes + (size_t)c * 16;
}

// Sixteen bytes at p (all of the row where it is shorter).  kAligned: p is
// 16-byte aligned and the row a multiple of 16 bytes.  kStream: past the
// caches (see streamed()).
template <bool kAligned, bool kStream = false>
__device__ __forceinline__ uint4 load_chunk(const uint8_t* p, int row_bytes) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (kAligned) {
    const row_chunk* c = reinterpret_cast<const row_chunk*>(p);
    v = __builtin_bit_cast(uint4, kStream ? __builtin_nontemporal_load(c) : *c);
  } else if (row_bytes >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < row_bytes; ++i) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

// Outputs are written past the caches: nothing here reads them again, and a
// prefill share's permute took 536 us so against 547.
template <bool kAligned>
__device__ __forceinline__ void store_chunk(uint8_t* p, int row_bytes, const uint4& v) {
  if (kAligned) {
    __builtin_nontemporal_store(__builtin_bit_cast(row_chunk, v), reinterpret_cast<row_chunk*>(p));
  } else if (row_bytes >= 16) {
    __builtin_memcpy(p, &v, 16);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < row_bytes; ++i) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

}  // namespace moe
