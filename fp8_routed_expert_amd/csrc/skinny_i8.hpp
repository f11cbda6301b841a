// Products in 8-bit integers of few rows with many channels: bound by the
// weights' one pass through HBM, not by the matrix cores.
#pragma once

#include "gemm_tiles.hpp"
#include "product_i8.hpp"
#include "rows_i8.hpp"

namespace moe {

// A workgroup computes 16 NT channels of at most 16 MT rows.  Its eight
// waves share out K, so that every CU has many waves' weight loads in flight
// (a wave's fragments go from global memory straight to its registers: each
// weight is used by one wave, and staging it would only add a step), and add
// their integer sums in LDS, where the order does not matter.
constexpr int kSkinnyWaves = 8;
constexpr int kSlab = 64;   // k of one multiplication: 16 bytes of 4 lanes

// The shares of K: wave w takes slabs [first, last), pairs of slabs (one
// 128-byte line) kept together.
__device__ __forceinline__ void slab_range(int K, int wave, int& first, int& last) {
  const int lines = (K + 2 * kSlab - 1) / (2 * kSlab);
  first = 2 * (int)((long long)lines * wave / kSkinnyWaves);
  last = min(2 * (int)((long long)lines * (wave + 1) / kSkinnyWaves), (K + kSlab - 1) / kSlab);
}

__device__ __forceinline__ v4i load_frag16(const uint8_t* p, bool in) {
  const v4i z = {0, 0, 0, 0};
  return in ? *reinterpret_cast<const v4i*>(p) : z;
}

// Sixteen bytes at a buffer's offset, zero past its end (no branch).
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ v4i load16(Rsrc r, uint32_t off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
constexpr uint32_t kNowhere = 0x80000000u;   // past the end of every buffer

// Adds a wave's sums to the workgroup's: register (i, j, q) of lane l at
// ((i NT + j) 4 + q) 64 + l, so that the lanes of an addition meet no bank
// twice.  (Laid out as rows of channels they met eightfold: 32 rows of 512
// channels took 3.9 us instead of 3.2.)
template <int MT, int NT>
__device__ __forceinline__ void add_sums(int32_t* sums, const v4i (&acc)[MT][NT], int lane) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        atomicAdd(&sums[((i * NT + j) * 4 + q) * 64 + lane], acc[i][j][q]);
}

// Four channels of a row.
__device__ __forceinline__ void store4(void* c, int c_type, size_t at, const float (&v)[4]) {
  if (c_type == MOE_TYPE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(c) + at) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
  uint2 o;
  if (c_type == MOE_TYPE_F16)
    o = make_uint2(pack2_f16(v[0], v[1]), pack2_f16(v[2], v[3]));
  else
    o = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c) + at) = o;
}

// Four channels of a row: sums (i, j, 0..3) of lane l are channels
// 16 j + 4 (l / 16) + 0..3 of row 16 i + l % 16.
__device__ __forceinline__ void scaled4(const int32_t* sums, int ij, int l, float sa,
                                        const float* sw, float (&v)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = (float)sums[(ij * 4 + q) * 64 + l] * (sa * sw[q]);
}

template <int MT, int NT, bool kGather>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_i8_kernel(I8Args p) {
  constexpr int kAhead = MT == 1 ? 8 : 4;   // slabs loaded at once
  __shared__ int32_t sums[MT * 16 * NT * 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = p.N, K = p.K;
  const int n_tiles = (N + 16 * NT - 1) / (16 * NT);
  const bool dense = p.offsets == nullptr;
  const int tile_m = blockIdx.x / n_tiles, tile_n = blockIdx.x - tile_m * n_tiles;
  if (!dense && blockIdx.x == 0 && threadIdx.x < 64 && p.status &&
      segments_bad(p.offsets, p.counts, p.E, lane) && lane == 0)
    atomicOr(p.status, MOE_ERR_BAD_INDEX);
  int e_sel = 0, row0 = tile_m * 16 * MT, row_end = p.rows_total;
  if (!dense) {
    find_mtile<16 * MT>(p.offsets, p.counts, p.E, p.rows_total, tile_m, lane, e_sel, row0,
                        row_end);
    if (e_sel < 0) return;
  }
  const int n0 = tile_n * 16 * NT;
  const int g = lane >> 4, r16 = lane & 15;
  for (int i = threadIdx.x; i < MT * 16 * NT * 16; i += 64 * kSkinnyWaves) sums[i] = 0;
  __syncthreads();

  // (plain loads under a condition: through buffer descriptors, which would
  // need none, these kernels measured 3-10% slower)
  const uint8_t* wp[NT];
  bool w_in[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = n0 + j * 16 + r16;
    w_in[j] = n < N;
    wp[j] = p.w + ((size_t)e_sel * N + (w_in[j] ? n : 0)) * K + 16 * g;
  }
  const uint8_t* ap[MT];
  bool a_in[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int r = row0 + i * 16 + r16;
    a_in[i] = r < row_end;
    if (kGather && a_in[i]) {
      r = p.row_src[r];
      a_in[i] = r >= 0 && r < p.src_rows;
    }
    ap[i] = p.a + (size_t)(a_in[i] ? r : 0) * K + 16 * g;
  }
  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
  int first, last;
  slab_range(K, wave, first, last);
  for (int s0 = first; s0 < last; s0 += kAhead) {
    // both halves of a line are asked for one after the other
    v4i wf[kAhead][NT], af[kAhead][MT];
#pragma unroll
    for (int u0 = 0; u0 < kAhead; u0 += 2) {
      bool in[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) in[u] = s0 + u0 + u < last && (s0 + u0 + u) * kSlab + 16 * g < K;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          wf[u0 + u][j] = load_frag16(wp[j] + (s0 + u0 + u) * kSlab, in[u] && w_in[j]);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          af[u0 + u][i] = load_frag16(ap[i] + (s0 + u0 + u) * kSlab, in[u] && a_in[i]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma_i8(wf[u][j], af[u][i], acc[i][j]);
  }
  add_sums<MT, NT>(sums, acc, lane);
  __syncthreads();
  for (int u = threadIdx.x; u < MT * NT * 64; u += 64 * kSkinnyWaves) {
    const int l = u & 63, ij = u >> 6;
    const int r = row0 + ij / NT * 16 + (l & 15), n = n0 + ij % NT * 16 + 4 * (l >> 4);
    if (r >= row_end || n >= N) continue;
    int at = r;
    if (kGather) {
      at = p.row_src[r];
      if (at >= p.src_rows) at = -1;
    }
    float v[4];
    scaled4(sums, ij, l, at >= 0 ? p.a_scale[at] : 0.f, p.w_scale + (size_t)e_sel * N + n, v);
    store4(p.c, p.c_type, (size_t)r * N + n, v);
  }
}

constexpr int kLinearRows = 4;

// The whole linear of at most kLinearRows rows in one launch: each workgroup asks for
// its weights, then quantises the rows into LDS while they are on their way.
// (Every workgroup does that again: for so few rows it costs less than a
// launch of its own.)  kType: x's type.
constexpr int kLinearAhead = 16;   // slabs a wave asks for before it quantises
constexpr int kLinearKeep = 4;     // slices of eight values a lane keeps for their codes

template <int kType>
__global__ __launch_bounds__(64 * kSkinnyWaves) void linear_i8_kernel(
    const void* __restrict__ x, const uint8_t* __restrict__ w, const float* __restrict__ w_scale,
    int M, int N, int K, void* __restrict__ c, int c_type) {
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];   // [M][K + 16]
  __shared__ int32_t sums[16 * 16];
  __shared__ uint32_t top[kLinearRows];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  const int n0 = blockIdx.x * 16;
  // every row to 8, 4 or 2 of the eight waves
  const int per_row = M == 1 ? 8 : M == 2 ? 4 : 2;
  const int m = wave / per_row, m_at = m < M ? m : M - 1;
  const int j0 = ((wave % per_row) * 64 + lane) * 8, jstep = per_row * 64 * 8;
  // the row's values are asked for before the weights: loads return in
  // order, and the quantisation must not wait for the weights
  float v[kLinearKeep][8];
#pragma unroll
  for (int u = 0; u < kLinearKeep; ++u) {
    const int j = j0 + u * jstep;
    load8_as(kType, x, (size_t)m_at * K + (j < K ? j : 0), v[u]);
  }
  int first, last;
  slab_range(K, wave, first, last);
  const Rsrc rw = buffer(w + (size_t)n0 * K, (uint32_t)min(16, N - n0) * K);
  const uint32_t wo = (uint32_t)r16 * (uint32_t)K + 16 * g;
  auto weights = [&](int s) {
    return load16(rw, s < last && s * kSlab + 16 * g < K ? wo + (uint32_t)s * kSlab : kNowhere);
  };
  __builtin_amdgcn_sched_barrier(0);
  v4i wf[kLinearAhead];
#pragma unroll
  for (int u = 0; u < kLinearAhead; ++u) wf[u] = weights(first + u);
  __builtin_amdgcn_sched_barrier(0);
  for (int i = threadIdx.x; i < 256; i += 64 * kSkinnyWaves) sums[i] = 0;
  if (threadIdx.x < kLinearRows) top[threadIdx.x] = 0;
  uint32_t t = 0;
#pragma unroll
  for (int u = 0; u < kLinearKeep; ++u)
    if (j0 + u * jstep < K) t = max_bits(v[u], t);
  for (int j = j0 + kLinearKeep * jstep; j < K; j += jstep) {
    float r[8];
    load8_as(kType, x, (size_t)m_at * K + j, r);
    t = max_bits(r, t);
  }
  t = wave_max(t);
  __syncthreads();
  if (lane == 0) atomicMax(&top[m_at], t);
  __syncthreads();
  const int pitch = K + 16;
  const float s = int8_scale(top[m_at]);
  const float inv = 1.f / s;
  const bool fine = top[m_at] < 0x7f800000u;
  if (m < M) {
#pragma unroll
    for (int u = 0; u < kLinearKeep; ++u) {
      const int j = j0 + u * jstep;
      if (j < K)
        *reinterpret_cast<uint2*>(codes + m * pitch + j) =
            fine ? int8_codes(v[u], s, inv) : make_uint2(0, 0);
    }
    for (int j = j0 + kLinearKeep * jstep; j < K; j += jstep) {
      float r[8];
      load8_as(kType, x, (size_t)m * K + j, r);
      *reinterpret_cast<uint2*>(codes + m * pitch + j) =
          fine ? int8_codes(r, s, inv) : make_uint2(0, 0);
    }
  }
  __syncthreads();
  v4i acc[1][1] = {{{0, 0, 0, 0}}};
  const uint8_t* ap = codes + (r16 < M ? r16 : 0) * pitch;
  // (lanes past M or K multiply some other codes: by no row that is stored,
  // or by weights that were read as zero)
  auto row = [&](int s) {
    const int k = s * kSlab + 16 * g;
    return *reinterpret_cast<const v4i*>(ap + (k < K ? k : 0));
  };
#pragma unroll
  for (int u = 0; u < kLinearAhead; ++u)
    if (first + u < last) acc[0][0] = mfma_i8(wf[u], row(first + u), acc[0][0]);
  // (past K = 8192: one load at a time, each waited for before the next; times
  // at one_launch)
  for (int sl = first + kLinearAhead; sl < last; ++sl)
    acc[0][0] = mfma_i8(weights(sl), row(sl), acc[0][0]);
  add_sums<1, 1>(sums, acc, lane);
  __syncthreads();
  if (threadIdx.x < 64) {
    const int n = n0 + 4 * g;
    if (r16 < M && n < N) {
      float o[4];
      scaled4(sums, 0, lane, int8_scale(top[r16]), w_scale + n, o);
      store4(c, c_type, (size_t)r16 * N + n, o);
    }
  }
}

}  // namespace moe
