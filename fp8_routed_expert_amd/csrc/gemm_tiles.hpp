// What the matrix-product kernels share: tile loads into LDS, the tiles'
// chunk permutation and fragment reads, and the search for a tile's expert.
#pragma once

#include "device_common.hpp"

namespace moe {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBK = 128;
constexpr int kXcds = 8;
constexpr int kLdsBytes = 160 * 1024;   // LDS per workgroup (gfx950)

// Workgroup barrier for the tile pipeline.  __syncthreads() (and even an
// LDS-scoped fence, since loads into LDS count as vector-memory operations)
// makes every wave wait for all its outstanding vector loads -- including
// the tile loads meant to stay in flight across the barrier.  Here the wave
// waits for its own LDS reads (lgkmcnt) and meets the others; completion of
// the tile loads is waited for explicitly with wait_loads<n>() before it.
// Both are compiler memory barriers (asm with a memory clobber), so no
// memory access is moved across them.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

typedef int v4i __attribute__((ext_vector_type(4)));
// Raw buffer descriptor: base, stride 0, num_records bytes (offsets at or
// past it read as zero), 32-bit data format.
__device__ __forceinline__ v4i make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  v4i r;
  r[0] = (int)(uint32_t)b;
  r[1] = (int)((b >> 32) & 0xffffu);
  r[2] = (int)bytes;
  r[3] = 0x00020000;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(r[i]);
  return r;
}
// 16 bytes per lane from a buffer into LDS at lds + 16 * lane (one wave
// instruction fills 1 KB).  M0 holds the LDS address; nothing else in these
// kernels reads M0 (gfx9 LDS instructions do not use it), so the clobber is
// safe.  The buffer offset is split into a per-lane part, XOR-ed with a
// wave-uniform 0 or 16 (the chunk permutation of the odd 8-row half of a
// 16-row group), and a wave-uniform part, combined inside the asm: the
// compiler cannot then hoist one offset register per chunk (or per parity)
// out of the K loop (the address is read when the load issues, so the
// temporary is free right after).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // (the m0 clobber is meant)
__device__ __forceinline__ void dma16_split(v4i rsrc, uint8_t* lds, uint32_t vlane,
                                            uint32_t sxor, uint32_t suni) {
  const uint32_t m = (uint32_t)(uintptr_t)(lds_void*)lds;
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(rsrc[i]);
  uint32_t t;
  asm volatile("v_xor_b32_e32 %0, %1, %2\n\tv_add_u32_e32 %0, %3, %0\n\ts_mov_b32 m0, %4\n\t"
               "buffer_load_dwordx4 %0, %5, 0 offen lds"
               : "=&v"(t) : "s"(sxor), "v"(vlane), "s"(suni), "s"(m), "s"(r) : "memory", "m0");
}
// The same with the per-lane part used as it is, and with the whole offset
// per lane.
__device__ __forceinline__ void dma16_add(v4i rsrc, uint8_t* lds, uint32_t vlane, uint32_t suni) {
  const uint32_t m = (uint32_t)(uintptr_t)(lds_void*)lds;
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(rsrc[i]);
  uint32_t t;
  asm volatile("v_add_u32_e32 %0, %2, %1\n\ts_mov_b32 m0, %3\n\t"
               "buffer_load_dwordx4 %0, %4, 0 offen lds"
               : "=&v"(t) : "v"(vlane), "s"(suni), "s"(m), "s"(r) : "memory", "m0");
}
__device__ __forceinline__ void dma16(v4i rsrc, uint8_t* lds, uint32_t voff) {
  const uint32_t m = (uint32_t)(uintptr_t)(lds_void*)lds;
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(rsrc[i]);
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(m), "v"(voff), "s"(r) : "memory", "m0");
}
#pragma clang diagnostic pop

// Wait until at most N vector-memory operations of this wave are outstanding
// (they complete in issue order).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Wait until at most N vector-memory operations of this wave are
// outstanding (they complete in issue order), and publish the registers of
// the asynchronous register loads issued before them (see load_scales).
template <int N, int M>
__device__ __forceinline__ void wait_loads(float (&r)[M]) {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
#pragma unroll
  for (int i = 0; i < M; ++i) asm volatile("" : "+v"(r[i]));
}

// The lane's index in its wave, read afresh from the hardware (the asm keeps
// the compiler from reusing, and so keeping live, an earlier copy), so that
// an epilogue need not hold its lane position in a register through the
// whole K loop.
__device__ __forceinline__ int lane_id_fresh() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// Two fp32 values to packed bf16, round to nearest even (one
// v_cvt_pk_bf16_f32; a NaN stays a NaN, its payload is not canonicalised).
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}

// Physical position of logical 16-byte chunk c of tile row r: chunks are
// XOR-permuted by (r & 7) ^ ((r >> 3) & 1).  A fragment read has lane
// (q, g) read chunk 2g (then 2g + 1) of row 16 b + q; with this permutation
// the LDS serves it without bank conflicts (4 cycles per 1 KB wave read on
// gfx950, against 8 for the (r >> 1) & 7 and r & 7 permutations).
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// A lane's byte offsets, within a stage, of the two 16-byte chunks (logical
// 2g and 2g + 1) it reads from row row0 + r16 of a swizzled tile.  For any
// row0 that is a multiple of 16 the permutation of row row0 + 16 i + r16
// is that of r16, so the fragment of subtile row i lies a fixed 16 i * 128
// bytes further: one pair of offsets serves every subtile of a wave.
struct FragLane {
  uint32_t lo, hi;
};
__device__ __forceinline__ FragLane frag_lane(int row0, int r16, int g) {
  const uint32_t r = (uint32_t)(row0 + r16) * kBK;
  const int sw = swz(r16);
  return {r + (uint32_t)(((2 * g) ^ sw) << 4), r + (uint32_t)(((2 * g + 1) ^ sw) << 4)};
}

// 32 bytes of a fragment: the lane's two chunks, `off` bytes (a multiple of
// 16 rows) past its offsets in stage `tile`.
__device__ __forceinline__ v8i load_frag_at(const uint8_t* tile, int off, FragLane fl) {
  const uint8_t* base = tile + off;
  uint4 lo = *reinterpret_cast<const uint4*>(base + fl.lo);
  uint4 hi = *reinterpret_cast<const uint4*>(base + fl.hi);
  v8i r;
  r[0] = (int)lo.x; r[1] = (int)lo.y; r[2] = (int)lo.z; r[3] = (int)lo.w;
  r[4] = (int)hi.x; r[5] = (int)hi.y; r[6] = (int)hi.z; r[7] = (int)hi.w;
  return r;
}

// The experts' m-tiles: expert e has ceil(valid rows / BM) of them,
// numbered expert by expert.  Each wave evaluates it on its own, 64 experts
// per pass with lane l holding expert base + l (one round of vector loads,
// then shuffles), so a tile is located in about one memory latency rather
// than a chain of dependent scalar loads per expert.  All results are
// wave-uniform.
struct SegLane {
  int s, en, nt;   // this lane's expert: valid rows [s, en), m-tiles
};

template <int BM>
__device__ __forceinline__ SegLane seg_lane(const int32_t* offsets, const int32_t* counts,
                                            int E, int rows_total, int e) {
  SegLane r{0, 0, 0};
  if (e < E) {
    expert_rows(offsets, counts, e, rows_total, r.s, r.en);
    r.nt = (r.en - r.s + BM - 1) / BM;
  }
  return r;
}

__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

__device__ __forceinline__ int wave_inclusive_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(x, d);
    if (lane >= d) x += t;
  }
  return x;
}

// Total number of m-tiles.
template <int BM>
__device__ __forceinline__ int total_mtiles(const int32_t* offsets, const int32_t* counts,
                                            int E, int rows_total, int lane) {
  int total = 0;
  for (int base = 0; base < E; base += 64)
    total += wave_sum(seg_lane<BM>(offsets, counts, E, rows_total, base + lane).nt);
  return __builtin_amdgcn_readfirstlane(total);
}

// The third A stage, an LDS object only where the kernel has one (a tile
// whose two A and two B stages already fill the LDS declares none).
template <int kBytes>
struct ThirdStage {
  __device__ __forceinline__ static uint8_t* get() {
    __shared__ __attribute__((aligned(1024))) uint8_t s[kBytes];
    return s;
  }
};
template <>
struct ThirdStage<0> {
  __device__ __forceinline__ static uint8_t* get() { return nullptr; }
};

// Expert, first row and segment end of m-tile mt (e_sel = -1 if none).
template <int BM>
__device__ __forceinline__ void find_mtile(const int32_t* offsets, const int32_t* counts,
                                           int E, int rows_total, int mt, int lane,
                                           int& e_sel, int& row0, int& row_end) {
  e_sel = -1;
  int before = 0;   // m-tiles of the experts of earlier passes
  for (int base = 0; base < E; base += 64) {
    const SegLane g = seg_lane<BM>(offsets, counts, E, rows_total, base + lane);
    const int incl = before + wave_inclusive_scan(g.nt, lane);
    // the first lane whose running count passes mt holds the expert (its
    // count is non-zero: the running count steps there)
    const uint64_t hit = __ballot(incl > mt);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      e_sel = base + l;
      row0 = __builtin_amdgcn_readlane(g.s, l) +
             (mt - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(g.nt, l))) * BM;
      row_end = __builtin_amdgcn_readlane(g.en, l);
      return;
    }
    before = __builtin_amdgcn_readlane(incl, 63);
  }
}

}  // namespace moe
