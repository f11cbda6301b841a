// Matrix products in 8-bit integers with one scale per token and one per
// output channel, dense and over the expert segments:
//
//   c[m, n] = round( a_scale[m] * w_scale[e, n] * sum_k a[m, k] * w[e, n, k] )
//
// The sums are exact 32-bit integers (|a|, |w| <= 128: K may reach 131,056),
// so the order of K does not matter, and neither does any split of it; the
// scales are applied once, in fp32, when a tile is stored.
//
// Tiles, as the FP8 products have them (gfx950): a workgroup multiplies a
// BM x BN tile with waves of WM x WN, K advancing 128 bytes a step.  The
// tile's rows of a and w come from global memory straight into LDS
// (buffer_load ... lds), a's a step further ahead than w's; a wave reads
// fragments of 16 rows x 32 bytes and v_mfma_i32_16x16x64_i8 consumes 16 of
// the 32 at a time (which 64 of the 128 k an instruction takes is free, as
// long as both operands agree).  The weights are the first operand, so a
// lane's four sums are four channels of one token.
//
// K need only be a multiple of 16: where it is none of 128 (kRagged) every
// load compares its place in the row with K, and lanes past the end take an
// offset out of the descriptor's range, which reads zero.  Channels past N
// lie past the weight descriptor's range in the same way.
#include <type_traits>

#include "product_i8.hpp"
#include "skinny_i8.hpp"

namespace moe {

constexpr uint32_t kOutOfRange = 0x80000000u;

template <int i>
using Int = std::integral_constant<int, i>;

// f(Int<a>), ..., f(Int<b - 1>)
template <int a, int b, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (a < b) {
    f(Int<a>());
    each<a + 1, b>(f);
  }
}

// Stage i of an operand: an LDS object of its own, so that accesses to one
// are known not to touch another.
template <int kBytes, int kOperand, int i>
struct Stage {
  __device__ __forceinline__ static uint8_t* get() {
    __shared__ __attribute__((aligned(1024))) uint8_t s[kBytes];
    return s;
  }
};

// kDeep: 0, or the number of stages of both operands for launches of few
// tiles: with one workgroup to a CU at most, nothing else hides the latency of
// a step's loads, so they are issued kDeep - 1 steps ahead.
// kPersist: a workgroup walks the tiles blockIdx + i gridDim.  Between two
// tiles it issues the next one's first two steps' loads before it stores the
// last one's outputs, so that the stores drain under the next tile's
// multiplications instead of before the next workgroup's start (a wave ends
// only when its stores have).
template <int BM, int BN, int WM, int WN, int GM, int kDeep, bool kPersist, bool kGather,
          bool kRagged>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void grouped_gemm_i8_kernel(I8Args p) {
  constexpr int NWM = BM / WM;
  constexpr int NWN = BN / WN;
  constexpr int NW = NWM * NWN;
  constexpr int MI = WM / 16;
  constexpr int NJ = WN / 16;
  constexpr int CA = BM / 8 / NW;   // 1 KB chunks (8 rows) of a stage per wave
  constexpr int CB = BN / 8 / NW;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "chunks must split evenly");
  static_assert(MI >= 2, "the late loads need a subtile row before the barrier");
  constexpr int SA_B = BM * kBK, SB_B = BN * kBK;
  constexpr int NSA = kDeep ? kDeep : 3 * SA_B + 2 * SB_B <= kLdsBytes ? 3 : 2;
  constexpr int NSB = kDeep ? kDeep : 2;
  static_assert(NSA * SA_B + NSB * SB_B <= kLdsBytes, "tile stages exceed the LDS");
  static_assert(6 % NSA == 0 && 6 % NSB == 0, "the K loop is unrolled by 6");
  auto stA = [&](auto i) { return Stage<SA_B, 0, decltype(i)::value % NSA>::get(); };
  auto stB = [&](auto i) { return Stage<SB_B, 1, decltype(i)::value % NSB>::get(); };

  // ---- which tile (the tile list's order is that of the FP8 products)
  const int N = p.N, K = p.K, rows_total = p.rows_total;
  const int lane = threadIdx.x & 63;
  const int n_tiles = (N + BN - 1) / BN;
  const bool dense = p.offsets == nullptr;
  const int total_m = dense ? (rows_total + BM - 1) / BM
                            : total_mtiles<BM>(p.offsets, p.counts, p.E, rows_total, lane);
  if (!dense && blockIdx.x == 0 && threadIdx.x < 64 && p.status &&
      segments_bad(p.offsets, p.counts, p.E, lane) && lane == 0)
    atomicOr(p.status, MOE_ERR_BAD_INDEX);
  const long long total = (long long)total_m * n_tiles;
  // kPersist: at most 64 experts, each lane holding one, so that a tile is
  // found without reading memory
  SegLane seg{0, 0, 0};
  int seg_incl = 0;
  if (kPersist && !dense) {
    seg = seg_lane<BM>(p.offsets, p.counts, p.E, rows_total, lane);
    seg_incl = wave_inclusive_scan(seg.nt, lane);
  }
  struct Tile {
    int e, row0, row_end, n0;
  };
  auto locate = [&](long long logical, Tile& t) -> bool {
    if (logical >= total) return false;
    const int group = (int)logical / (GM * n_tiles);
    const int in_group = (int)logical - group * (GM * n_tiles);
    const int gm_cnt = min(GM, total_m - group * GM);
    const int tile_n = in_group / gm_cnt;
    const int tile_m = group * GM + (in_group - tile_n * gm_cnt);
    t = {0, tile_m * BM, rows_total, tile_n * BN};
    if (dense) return true;
    if constexpr (kPersist) {
      const uint64_t hit = __ballot(seg_incl > tile_m);
      if (!hit) return false;
      const int l = __builtin_ctzll(hit);
      t.e = l;
      const int start = __builtin_amdgcn_readlane(seg.s, l);
      t.row_end = __builtin_amdgcn_readlane(seg.en, l);
      const int before = __builtin_amdgcn_readlane(seg_incl, l) - (t.row_end - start + BM - 1) / BM;
      t.row0 = start + (tile_m - before) * BM;
    } else {
      find_mtile<BM>(p.offsets, p.counts, p.E, rows_total, tile_m, lane, t.e, t.row0, t.row_end);
      if (t.e < 0) return false;
    }
    return true;
  };
  Tile tile;
  if (!locate(blockIdx.x, tile)) return;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / NWN;
  const int wn = wave - wm * NWN;
  const int Kb = (K + kBK - 1) / kBK;
  const int g = lane >> 4, r16 = lane & 15;

  // ---- tile rows of w: row 16 j + 4 g + q of a wave's 64 holds channel
  //   channel(j, g, q) = 32 (j / 2) + 8 g + 4 (j % 2) + q,
  // so that a lane's sums of two neighbouring subtiles are eight neighbouring
  // channels and can be stored as they are (staging them through LDS, to
  // write whole rows, took the memory that the next tile's loads want).
  //
  // ---- tile loads.  A chunk is 8 rows; the lane's row is lane / 8, its
  // 16-byte piece the one that belongs at place lane % 8 of that row in an
  // even (odd) 8-row half.
  const int piece0 = (lane & 7) ^ (lane >> 3);
  uint32_t vl[2], vb[2];
  int lim[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    vl[o] = (uint32_t)(lane >> 3) * (uint32_t)K + (uint32_t)((piece0 ^ o) << 4);
    vb[o] = (uint32_t)(8 * (lane >> 5) + ((lane >> 3) & 3)) * (uint32_t)K +
            (uint32_t)((piece0 ^ o) << 4);
    lim[o] = K - ((piece0 ^ o) << 4);
  }
  v4i rsrc_a, rsrc_b;
  uint32_t a_off[kGather ? CA : 1];
  int a_row[MI];   // the rows of a whose scales the lane needs, -1: none
  auto prepare = [&](const Tile& t) __attribute__((always_inline)) {
    const long long a_bytes =
        kGather ? (long long)p.src_rows * K : (long long)(rows_total - t.row0) * K;
    rsrc_a = make_rsrc(kGather ? p.a : p.a + (size_t)t.row0 * K,
                       (uint32_t)(a_bytes > 0x7ffff000LL ? 0x7ffff000LL : a_bytes));
    rsrc_b = make_rsrc(p.w + ((size_t)t.e * N + t.n0) * K,
                       (uint32_t)((long long)min(BN, N - t.n0) * K));
    auto source = [&](int r) {
      if (r >= t.row_end) return -1;
      if (!kGather) return r;
      const int src = p.row_src[r];
      return src < p.src_rows ? src : -1;
    };
#pragma unroll
    for (int i = 0; i < MI; ++i) a_row[i] = source(t.row0 + wm * WM + i * 16 + r16);
    if constexpr (kGather) {
#pragma unroll
      for (int u = 0; u < CA; ++u) {
        const int c = wave * CA + u;
        const int src = source(t.row0 + c * 8 + (lane >> 3));
        a_off[u] = src >= 0 ? (uint32_t)src * (uint32_t)K + (uint32_t)((piece0 ^ (c & 1)) << 4)
                            : kOutOfRange;
      }
      // the offsets (and so the compiler's wait for row_src) are ready before
      // the first tile load is issued
#pragma unroll
      for (int u = 0; u < CA; ++u) asm volatile("" : "+v"(a_off[u]));
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) asm volatile("" : "+v"(a_row[i]));
  };
  // 16 bytes per lane: v + uni, or zero where the step does not exist or the
  // lane's piece (parity o) lies past K.  A sum that wraps (out of range plus
  // out of range) reads inside the buffer into a stage that is not read.
  auto stage16 = [&](const v4i& rsrc, uint8_t* lds, uint32_t v, uint32_t uni, int kofs, int o,
                    bool live) {
    if constexpr (kRagged) {
      const bool in = live && kofs < lim[o];
      dma16(rsrc, lds, in ? v + uni : kOutOfRange);
    } else {
      dma16_add(rsrc, lds, v, __builtin_amdgcn_readfirstlane(live ? uni : kOutOfRange));
    }
  };
  auto issue_a = [&](int kb, uint8_t* tA, bool live) {
#pragma unroll
    for (int u = 0; u < CA; ++u) {
      const int c = wave * CA + u;
      const int o = CA % 2 == 0 ? (u & 1) : (c & 1);
      if constexpr (kGather)
        stage16(rsrc_a, tA + c * 1024, a_off[u], (uint32_t)kb * kBK, kb * kBK, o, live);
      else
        stage16(rsrc_a, tA + c * 1024, o ? vl[1] : vl[0],
               (uint32_t)(c * 8) * (uint32_t)K + (uint32_t)kb * kBK, kb * kBK, o, live);
    }
  };
  auto issue_b = [&](int kb, uint8_t* tB, bool live) {
#pragma unroll
    for (int u = 0; u < CB; ++u) {
      const int c = wave * CB + u;
      const int o = CB % 2 == 0 ? (u & 1) : (c & 1);
      // the chunk's channels (see channel()): the lane's part is in vb
      const int first = c / 8 * 64 + ((c >> 2) & 1) * 32 + (c & 1) * 16 + ((c >> 1) & 1) * 4;
      stage16(rsrc_b, tB + c * 1024, o ? vb[1] : vb[0],
             (uint32_t)first * (uint32_t)K + (uint32_t)kb * kBK, kb * kBK, o, live);
    }
  };

  FragLane fa = frag_lane(wm * WM, r16, g);
  FragLane fb = frag_lane(wn * WN, r16, g);
  v4i acc[MI][NJ];
  v8i bf[NJ];
  v8i af_next;
  auto lo = [](const v8i& v) { return (v4i){v[0], v[1], v[2], v[3]}; };
  auto hi = [](const v8i& v) { return (v4i){v[4], v[5], v[6], v[7]}; };
  // One subtile (both halves of its 128 k), and a row of them.  Successive
  // multiplications share as much as they can -- the sums, else a half of the
  // token's fragment, and across rows the channels' fragment -- because large
  // products are bound by power: the same instructions with the halves in the
  // outer loop run 2% faster on zeros (600 us against 612 for 16384 x 8192 x
  // 8192) and 2.5% slower on random codes (774 against 755), and 32 x 32 x 32
  // ones 3% faster and 9% slower.
  auto subtile = [&](int i, int j, bool hi_first, const v8i& af) __attribute__((always_inline)) {
    if (hi_first) {
      acc[i][j] = mfma_i8(hi(bf[j]), hi(af), acc[i][j]);
      acc[i][j] = mfma_i8(lo(bf[j]), lo(af), acc[i][j]);
    } else {
      acc[i][j] = mfma_i8(lo(bf[j]), lo(af), acc[i][j]);
      acc[i][j] = mfma_i8(hi(bf[j]), hi(af), acc[i][j]);
    }
  };
  auto multiply = [&](int i, const v8i& af) __attribute__((always_inline)) {
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      subtile(i, (i & 1) ? NJ - 1 - jj : jj, jj & 1, af);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // One K step, as the packed-scale FP8 product's: the next step's loads go
  // out first (w) and after a subtile row (a); the step's barrier comes once
  // the wave's last LDS read of it has landed, and the next step's fragments
  // are read under the last subtile row's multiplications.
  constexpr int kLateRow = MI >= 3 ? 1 : 0;
  // loads that the step's barrier leaves in flight: all issued after the next
  // step's
  constexpr int kInFlight = kDeep ? (kDeep - 2) * (CA + CB) : NSA == 3 ? CA : 0;
  // kPersist: behind a tile's first two steps' loads come the last tile's
  // stores (`carried`; two per subtile row, none of them conditional) and the
  // scales' loads, so the first two waits count those too.
  constexpr bool kLateSw = kPersist && (kGather || kRagged);   // see load_scales
  constexpr int kStores = 2 * MI, kScales = kLateSw ? MI : MI + NJ;
  static_assert(!kPersist || (NSA == 3 && NSB == 2), "stages of the persistent form");
  bool carried = false;
  auto step = [&](int kb, auto unrolled) __attribute__((always_inline)) {
    constexpr int U = decltype(unrolled)::value;
    // formed anew each step, so that no address per stage and subtile is kept
    asm volatile("" : "+v"(fa.lo), "+v"(fa.hi), "+v"(fb.lo), "+v"(fb.hi));
    if (kRagged) asm volatile("" : "+v"(vl[0]), "+v"(vl[1]), "+v"(vb[0]), "+v"(vb[1]));
    const uint8_t* tA = stA(Int<U>());
    const uint8_t* tAn = stA(Int<U + 1>());
    const uint8_t* tBn = stB(Int<U + 1>());
    if (!(kPersist && U == 0 && kb == 0))   // (its second step's are under way)
      issue_b(kb + NSB - 1, stB(Int<U + NSB - 1>()), kb + NSB - 1 < Kb);
#pragma unroll
    for (int i = 0; i < MI - 1; ++i) {
      if (i == kLateRow) issue_a(kb + NSA - 1, stA(Int<U + NSA - 1>()), kb + NSA - 1 < Kb);
      const v8i af = af_next;
      af_next = load_frag_at(tA, (i + 1) * 16 * kBK, fa);
      multiply(i, af);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < MI - 1; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(acc[i][j]));
    if (kPersist && U == 0 && kb == 0) {
      if (carried)
        wait_vm<kStores + kScales + CA>();
      else
        wait_vm<kScales + CA>();
    } else {
      wait_vm<kInFlight>();
    }
    lds_barrier();
    const v8i af = af_next;
    // (the step's w fragments are replaced one by one, after their last use)
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const int j = (MI & 1) ? jj : NJ - 1 - jj;
      subtile(MI - 1, j, jj & 1, af);
      bf[j] = load_frag_at(tBn, j * 16 * kBK, fb);
    }
    af_next = load_frag_at(tAn, 0, fa);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(acc[MI - 1][j]));
  };

  auto issue_first = [&]() __attribute__((always_inline)) {
    issue_b(0, stB(Int<0>()), true);
    issue_a(0, stA(Int<0>()), true);
    if constexpr (kDeep != 0) {
      each<1, kDeep - 1>([&](auto i) {
        constexpr int k = decltype(i)::value;
        issue_b(k, stB(i), k < Kb);
        issue_a(k, stA(i), k < Kb);
      });
    } else if constexpr (NSA == 3) {
      if (kPersist) issue_b(1, stB(Int<1>()), Kb > 1);
      issue_a(1, stA(Int<1>()), Kb > 1);
    }
  };
  // a tile's sums, its first loads issued
  auto multiply_tile = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = (v4i){0, 0, 0, 0};
    if constexpr (kPersist) {
      if (carried)
        wait_vm<kStores + kScales + CA + CB>();
      else
        wait_vm<kScales + CA + CB>();
    } else {
      wait_vm<kInFlight>();
    }
    lds_barrier();
#pragma unroll
    for (int j = 0; j < NJ; ++j) bf[j] = load_frag_at(stB(Int<0>()), j * 16 * kBK, fb);
    af_next = load_frag_at(stA(Int<0>()), 0, fa);
    // unrolled by 6, a multiple of every number of stages, so that every step
    // names its stages statically
    for (int kb = 0; kb < Kb; kb += 6)
      each<0, 6>([&](auto u) __attribute__((always_inline)) {
        constexpr int U = decltype(u)::value;
        if (U == 0 || kb + U < Kb) step(kb + U, u);
      });
    // The last step's loads past K (zeros, into this wave's own chunks of the
    // stages) are waited for.  No wave needs a stage any more: every read of
    // the last step's came before its barrier.
    wait_vm<0>();
  };

  // ---- epilogue: scales, conversion, and stores straight from the lanes
  // that hold the sums: sums (i, j, 0..3) and (i, j + 1, 0..3) with j even are
  // eight neighbouring channels of row r16, 16 bytes in 16 bits, and the four
  // lanes of a row write 64 bytes together.
  static_assert(NJ == 4, "a wave's channels are two pieces of 32");
  float sw[NJ][4], sa[MI];
  // Loads of the scales: one per row and one per four channels, whatever the
  // lane (a row or channel that is none reads zero past the buffer's end).
  // kPersist: they are loaded before a tile's K loop; where registers are
  // short (kLateSw) the channels' only after it, under the next tile's search.
  auto load_sa = [&](const Tile&) __attribute__((always_inline)) {
    const long long rows = kGather ? p.src_rows : rows_total;
    const Rsrc ra = buffer(p.a_scale, (uint32_t)(rows * 4));   // (the host bounds the rows)
#pragma unroll
    for (int i = 0; i < MI; ++i)
      sa[i] = __int_as_float((int)__builtin_amdgcn_raw_buffer_load_b32(
          ra, a_row[i] >= 0 ? a_row[i] * 4 : (int)kNowhere, 0, 0));
  };
  auto load_sw = [&](const Tile& t) __attribute__((always_inline)) {
    const Rsrc rw = buffer(p.w_scale + (size_t)t.e * N + t.n0, (uint32_t)min(BN, N - t.n0) * 4u);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const v4i v = load16(rw, (uint32_t)(wn * WN + 8 * g + 32 * (j >> 1) + 4 * (j & 1)) * 4u);
#pragma unroll
      for (int q = 0; q < 4; ++q) sw[j][q] = __int_as_float(v[q]);
    }
  };
  auto load_scales = [&](const Tile& t) __attribute__((always_inline)) {
    load_sa(t);
    if (!kLateSw) load_sw(t);
  };
  auto store_as = [&](const Tile& t, auto type) __attribute__((always_inline)) {
    constexpr int kType = decltype(type)::value;
    const int wcol = t.n0 + wn * WN + 8 * g;
    // (the tile's rows of c from its first channel on)
    const Rsrc rc = buffer(static_cast<uint16_t*>(p.c) + (size_t)t.row0 * N + t.n0,
                           (uint32_t)((long long)min(BM, t.row_end - t.row0) * N - t.n0) * 2u);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      float v[2][8];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          v[s][q] = (float)acc[i][2 * s + (q >> 2)][q & 3] *
                    (sa[i] * sw[2 * s + (q >> 2)][q & 3]);
      const int top = t.row0 + wm * WM + i * 16;
      if constexpr (kType == MOE_TYPE_F32) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int row = top + r16, n = wcol + 32 * s;
          if (row < t.row_end && n < N) {
            float4* c4 = reinterpret_cast<float4*>(static_cast<float*>(p.c) + (size_t)row * N + n);
            c4[0] = make_float4(v[s][0], v[s][1], v[s][2], v[s][3]);
            c4[1] = make_float4(v[s][4], v[s][5], v[s][6], v[s][7]);
          }
        }
        continue;
      }
      constexpr bool half = kType == MOE_TYPE_F16;
      // lanes of rows 0..7 exchange their second piece for the first piece of
      // the row 8 further: a store then writes eight rows' whole 128 bytes
      // (sixteen rows' 64 bytes took 3-7% longer where the stores weigh)
      const bool low = r16 < 8;
      u32x4 first, second;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w0 = half ? pack2_f16(v[0][2 * q], v[0][2 * q + 1])
                                 : pack2_bf16(v[0][2 * q], v[0][2 * q + 1]);
        const uint32_t w1 = half ? pack2_f16(v[1][2 * q], v[1][2 * q + 1])
                                 : pack2_bf16(v[1][2 * q], v[1][2 * q + 1]);
        const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(
            0, (int)(low ? w1 : w0), 0x128, 0xf, 0xf, false);   // row_ror:8
        first[q] = low ? w0 : got;
        second[q] = low ? got : w1;
      }
      const int n = wcol + (low ? 0 : 32);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int row = top + (r16 & 7) + 8 * s;
        if constexpr (kPersist) {
          const uint32_t in =
              ((uint32_t)(row - t.row0) * (uint32_t)N + (uint32_t)(n - t.n0)) * 2u;
          const uint32_t at = row < t.row_end && n < N ? in : kNowhere;
          __builtin_amdgcn_raw_buffer_store_b128(s ? second : first, rc, (int)at, 0, 2);   // nt
        } else if (row < t.row_end && n < N) {
          u32x4* c4 = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.c) + (size_t)row * N + n);
          __builtin_nontemporal_store(s ? second : first, c4);
        }
      }
    }
  };

  auto store_tile = [&](const Tile& t) __attribute__((always_inline)) {
    if (p.c_type == MOE_TYPE_F16)
      store_as(t, Int<MOE_TYPE_F16>());
    else if (kPersist || p.c_type == MOE_TYPE_BF16)
      store_as(t, Int<MOE_TYPE_BF16>());
    else
      store_as(t, Int<MOE_TYPE_F32>());
  };

  prepare(tile);
  issue_first();
  if constexpr (!kPersist) {
    multiply_tile();
    load_sa(tile);
    load_sw(tile);
    store_tile(tile);
  } else {
    load_scales(tile);
    for (long long logical = blockIdx.x;;) {
      multiply_tile();
      // the compiler's own waits for the scales go before the next tile's loads
#pragma unroll
      for (int i = 0; i < MI; ++i) asm volatile("" : "+v"(sa[i]));
      if (kLateSw) load_sw(tile);
      Tile next;
      logical += gridDim.x;
      const bool more = locate(logical, next);
      if (more) prepare(next);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(sw[j][q]));
      if (more) issue_first();
      store_tile(tile);
      if (!more) return;
      load_scales(next);
      tile = next;
      carried = true;
    }
  }
}

constexpr long long kRoundTilesI8 = 256;   // one workgroup to a CU of an MI355X

template <int BM, int BN, int WM, int WN, int GM, int kDeep = 0, bool kPersist = false>
static moe_status_t launch_i8(const I8Args& p, hipStream_t st) {
  const long long m_tiles = p.offsets ? (long long)p.rows_total / BM + p.E
                                      : ((long long)p.rows_total + BM - 1) / BM;
  constexpr int threads = 64 * (BM / WM) * (BN / WN);
  long long blocks = m_tiles * ((p.N + BN - 1) / BN);
  blocks = (blocks + kXcds - 1) / kXcds * kXcds;
  if (blocks > 0x7fffffffLL) return MOE_UNSUPPORTED_SHAPE;
  if (kPersist && blocks > kRoundTilesI8) blocks = kRoundTilesI8;
  if (blocks * threads > 0xffffffffLL) return MOE_UNSUPPORTED_SHAPE;
  const dim3 grid((unsigned)blocks), block(threads);
  const bool ragged = p.K % kBK != 0;
  if (p.row_src && ragged) {
    if constexpr (kPersist)
      return MOE_INVALID_ARG;   // not asked for: its offsets do not fit the registers
    else
      hipLaunchKernelGGL((grouped_gemm_i8_kernel<BM, BN, WM, WN, GM, kDeep, kPersist, true, true>),
                         grid, block, 0, st, p);
  } else if (p.row_src) {
    hipLaunchKernelGGL((grouped_gemm_i8_kernel<BM, BN, WM, WN, GM, kDeep, kPersist, true, false>),
                       grid, block, 0, st, p);
  } else if (ragged) {
    hipLaunchKernelGGL((grouped_gemm_i8_kernel<BM, BN, WM, WN, GM, kDeep, kPersist, false, true>),
                       grid, block, 0, st, p);
  } else {
    hipLaunchKernelGGL((grouped_gemm_i8_kernel<BM, BN, WM, WN, GM, kDeep, kPersist, false, false>),
                       grid, block, 0, st, p);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

template <int MT, int NT>
static moe_status_t launch_skinny(const I8Args& p, hipStream_t st) {
  const long long m_tiles = p.offsets ? (long long)p.rows_total / (16 * MT) + p.E
                                      : ((long long)p.rows_total + 16 * MT - 1) / (16 * MT);
  const long long blocks = m_tiles * ((p.N + 16 * NT - 1) / (16 * NT));
  if (blocks * 64 * kSkinnyWaves > 0xffffffffLL) return MOE_UNSUPPORTED_SHAPE;
  const dim3 grid((unsigned)blocks), block(64 * kSkinnyWaves);
  if (p.row_src)
    hipLaunchKernelGGL((skinny_i8_kernel<MT, NT, true>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((skinny_i8_kernel<MT, NT, false>), grid, block, 0, st, p);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

// Launches the product in tiles chosen from the sizes alone (the same inside
// graph capture).  `rows` is a dense product's, or a segment's on average: of
// the buffer, whose rows the host knows, not of the tokens.  The capacity of
// masked segments and the padding between contiguous ones (up to 127 rows of
// an expert) count as rows, so few tokens in a contiguous buffer run in the
// tiles of a hundred or more.  Dense products of 9 to 64 rows go from 64 x 64
// to 128 x 128 tiles past 16384 channels (one round of the former is full), which
// leaves CUs without a tile up to some 32768 channels.
// Times are of products whose weights come from HBM, N x K (experts x N x K),
// in us.
//
//   * Few rows: the kernel that takes the weights straight to registers, up to
//     16 rows (1 row of 4096 x 7168 and 7168 x 2048: 8.0 and 6.1; as 64 x 128
//     tiles 46 and 17), and up to 32 (with more than 8 rows) where the tiles
//     below would be few (32 rows: 15.2 and 7.9; 8192 x 8192 21.2 both ways, 16384 x
//     7168 33.0 against 23.2).  Its workgroups take 16 channels, or 32 where
//     there are enough of them and each has more to do than to stream (search
//     its segment, read rows, start on a short K): 32 x 4096 x 7168 of 16 rows
//     177 against 219, one expert's 16 rows of 32768 x 4096 31.5 against 36.0 (a
//     dense product of that many channels has tiles from 9 rows on); but 1 row
//     28.0 against 26.4, and 4096 x 7168, too few, 11.5 against 8.0.
//     Where even those are short-lived and many, 64 x 128 tiles: 32 x 7168 x
//     2048 of 16 rows 97 against 124, 64 x 7168 x 3584 296 against 388, one
//     row of 65536 x 1024 15.9 against 17.7; but 32 x 4096 x 4096 132 against
//     124, one row of 152064 x 2048 65 against 52.  With one row of each of few
//     experts and K <= 2048 the rule loses: 6 x 7168 x 2048 18.7 against 14.1, 8 x
//     7168 x 2048 (half of them empty) 13.4 against 12.1.
//   * One round of small tiles, loaded five steps ahead: 64 x 64 (128 rows:
//     20.4 and 9.6; two and three stages of 64 x 128 tiles 45 and 17), then
//     128 x 64 (512 and 256 rows: 27 and 11.5; 64 x 64 tiles 41 and 17), then
//     128 x 128 two steps ahead (1024 rows of 4096 x 7168: 32; without the
//     third stage of weights 40).  A CU takes in some 20 bytes a cycle
//     whatever it runs, so as many of them as possible have to share the bytes.
//   * 256 x 256 once that gives more than half the CUs a tile and segments
//     have 256 rows: twice the work per byte of two 128 x 128 tiles (prefill
//     gate/up 3.27 ms against 4.32); and from 128 rows where those would take
//     more than a round (32 x 4096 x 7168 of 256 rows 329 against 383, 8 x 7168
//     x 2048 of 200 33.6 against 44.3; masked segments of capacity 192 win a
//     third when 80% full, 31 against 43, and lose it when 30% full, 30
//     against 23).  192 x 256 where both fit one round and
//     K is long (the EP72 share's gate/up: 67 against 78; but 1536 rows of
//     7168 x 2048 35.9 against 27.8).
//   * else 64 x 128 up to 64 rows (32 x 4096 x 7168: 170 against 195, 64 x
//     7168 x 3584 302 against 337), and 128 x 128, two workgroups to a CU (segments
//     of 48 to 96 rows, 32 x 7168 x 2048: 111 against 143, as 64 rows do not
//     hold them; half empty ones 107 against 97).
static moe_status_t product_i8(const I8Args& p, hipStream_t st) {
  const long long rows = ((long long)p.rows_total + p.E - 1) / p.E;
  const bool grouped = p.offsets != nullptr;
  auto tiles = [&](int bm, int bn) {
    return p.E * ((rows + bm - 1) / bm) * ((p.N + bn - 1) / bn);
  };
  const long long slices = (long long)p.E * ((p.N + 15) / 16);   // of 16 channels
  const long long wide = (long long)p.E * ((p.N + 127) / 128);
  if (rows <= 16 && wide > 256 &&
      (p.K <= 1024 || (grouped && (p.K <= 2048 || wide > 1024))))
    return launch_i8<64, 128, 32, 64, 4>(p, st);
  // (a launch holds 2^32 threads: past 2^21 slices tiles follow)
  if (rows <= 16 && slices < (1 << 21) && (rows <= 8 || grouped || tiles(64, 64) <= 128))
    return slices >= 448 && (grouped || rows > 4 || p.K <= 1024) ? launch_skinny<1, 2>(p, st)
                                                                 : launch_skinny<1, 1>(p, st);
  if (rows <= 32 && tiles(64, 64) <= 128)
    return (long long)p.E * p.N >= 192 * 32 ? launch_skinny<2, 2>(p, st)
                                            : launch_skinny<2, 1>(p, st);
  // (segments differ and end anywhere in a tile: half a tile more each, on
  // average, once they are nearly as long as one; those of a buffer that is as
  // many whole tiles per expert are taken to be its parts)
  auto ragged = [&](int bm, int bn) {
    return !grouped || 4 * rows <= 3 * bm || p.rows_total % ((long long)p.E * bm) == 0
               ? tiles(bm, bn)
               : (p.E * (2 * rows + bm) + 2 * bm - 1) / (2 * bm) * ((p.N + bn - 1) / bn);
  };
  if (ragged(64, 64) <= 256) return launch_i8<64, 64, 32, 64, 4, 6>(p, st);
  if (ragged(128, 64) <= 256) return launch_i8<128, 64, 32, 64, 4, 6>(p, st);
  if (ragged(128, 128) <= 256) return launch_i8<128, 128, 64, 64, 4, 3>(p, st);
  if ((rows >= 256 && tiles(256, 256) > 128) ||
      (grouped && rows > 128 && ragged(128, 128) > 512)) {
    if (p.K > 4096 && ragged(192, 256) <= 256) return launch_i8<192, 256, 96, 64, 2>(p, st);
    // walked by one workgroup per CU where the kernel's counted loads and
    // stores allow (down products 2.7% faster: 1826 us against 1877, 113
    // against 115; long K 1%)
    if (p.E <= 64 && p.c_type != MOE_TYPE_F32 && p.N <= (1 << 20) &&
        !(p.row_src && p.K % kBK != 0))
      return launch_i8<256, 256, 128, 64, 2, 0, true>(p, st);
    return launch_i8<256, 256, 128, 64, 2>(p, st);
  }
  if (rows <= 64) return launch_i8<64, 128, 32, 64, 4>(p, st);
  return launch_i8<128, 128, 64, 64, 4>(p, st);
}

constexpr int kMaxChannels = 0x7fffff00;
constexpr int kMaxRows = 0x1ffffc00;   // the row scales are addressed with 32-bit byte offsets

// The checks that every product shares: sizes, then pointers.
static moe_status_t product_args(const I8Args& p, bool grouped) {
  if (p.E <= 0 || p.E > MOE_MAX_EXPERTS || p.rows_total < 0 || p.N <= 0 || p.K <= 0)
    return MOE_INVALID_ARG;
  if (p.c_type != MOE_TYPE_F32 && p.c_type != MOE_TYPE_BF16 && p.c_type != MOE_TYPE_F16)
    return MOE_INVALID_ARG;
  // 128 * 128 * K stays below 2^31, and so does N with a tile's channels added
  if (p.N % 16 != 0 || p.K % 16 != 0 || p.K > 131056 || p.N > kMaxChannels)
    return MOE_UNSUPPORTED_SHAPE;
  if (p.rows_total > kMaxRows || p.src_rows > kMaxRows) return MOE_UNSUPPORTED_SHAPE;
  if (grouped && (!p.offsets || !p.counts)) return MOE_INVALID_ARG;
  if (!p.w || !p.w_scale) return MOE_INVALID_ARG;
  if (p.row_src) {
    if (p.src_rows < 0 || (p.src_rows > 0 && !p.a)) return MOE_INVALID_ARG;
    if ((long long)p.src_rows * p.K > 0x7ffff000LL) return MOE_UNSUPPORTED_SHAPE;
  } else if (p.rows_total > 0 && !p.a) {
    return MOE_INVALID_ARG;
  }
  if (p.rows_total > 0 && ((!p.a_scale && !(p.row_src && p.src_rows == 0)) || !p.c))
    return MOE_INVALID_ARG;
  if (((uintptr_t)p.a | (uintptr_t)p.w | (uintptr_t)p.c) & 15) return MOE_UNSUPPORTED_SHAPE;
  if (((uintptr_t)p.a_scale | (uintptr_t)p.w_scale) & 3) return MOE_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_gemm_int8(const int8_t* a, const float* a_scale, const int8_t* w,
                                      const float* w_scale, int M, int N, int K, void* c,
                                      int c_type, void* stream) {
  const I8Args p{reinterpret_cast<const uint8_t*>(a), a_scale, reinterpret_cast<const uint8_t*>(w),
                 w_scale, nullptr, nullptr, nullptr, 1, M, N, K, 0, c, c_type, nullptr};
  const moe_status_t ok = product_args(p, false);
  if (ok != MOE_OK || M == 0) return ok;
  return product_i8(p, reinterpret_cast<hipStream_t>(stream));
}

extern "C" moe_status_t moe_grouped_gemm_int8(const int8_t* a, const float* a_scale,
                                              const int8_t* w, const float* w_scale,
                                              const int32_t* offsets, const int32_t* counts,
                                              int E, int rows_total, int N, int K, void* c,
                                              int c_type, int32_t* status_dev, void* stream) {
  const I8Args p{reinterpret_cast<const uint8_t*>(a), a_scale, reinterpret_cast<const uint8_t*>(w),
                 w_scale, offsets, counts, nullptr, E, rows_total, N, K, 0, c, c_type,
                 status_dev};
  const moe_status_t ok = product_args(p, true);
  if (ok != MOE_OK || rows_total == 0) return ok;
  return product_i8(p, reinterpret_cast<hipStream_t>(stream));
}

extern "C" moe_status_t moe_grouped_gemm_int8_gather(
    const int8_t* x, const float* x_scale, int T, const int32_t* row_src, const int8_t* w,
    const float* w_scale, const int32_t* offsets, const int32_t* counts, int E, int rows_total,
    int N, int K, void* c, int c_type, int32_t* status_dev, void* stream) {
  if (!row_src && rows_total != 0) return MOE_INVALID_ARG;
  const I8Args p{reinterpret_cast<const uint8_t*>(x), x_scale, reinterpret_cast<const uint8_t*>(w),
                 w_scale, offsets, counts, row_src, E, rows_total, N, K, T, c, c_type,
                 status_dev};
  const moe_status_t ok = product_args(p, true);
  if (ok != MOE_OK || rows_total == 0) return ok;
  return product_i8(p, reinterpret_cast<hipStream_t>(stream));
}

// ---- a whole linear: quantise the rows, then the product.  The workspace
// holds the codes [M, K] and, from the next multiple of 16 bytes, the scales.
extern "C" size_t moe_linear_int8_workspace_bytes(int M, int K) {
  if (M < 0 || K <= 0) return 0;
  const size_t codes = ((size_t)M * (size_t)K + 15) / 16 * 16;
  return codes + (size_t)M * sizeof(float);
}

// One launch for few rows, and no more channels than three workgroups to a CU
// have: later workgroups would quantise the rows again with no weights under way
// (us, weights from HBM, one launch against two; 1 row of 4096 x 7168 (N x K)
// 8.5 : 11.7, 4 rows 10.6 : 12.7; 12288 x 4096 15.0 : 15.3, 16384 x 4096
// 19.5 : 18.5, 32768 x 1024 19.4 : 13.8, 152064 x 2048 97 : 54).  Past K = 8192,
// where a wave asks for its weights one load at a time, the two come out even:
// 8192 x 14336 1 row 26.5 : 31.0, 4 rows 34.1 : 33.1; 8192 x 28672 53.1 : 57.7,
// 2 rows 60.6 : 60.8; but 4096 x 28672 35.9 : 35.4, 2 rows 39.4 : 35.8.
static bool one_launch(int M, int N, int K) {
  return M <= kLinearRows && N <= 3 * 256 * 16 &&
         (long long)M * (K + 16) <= 61440;   // of 64 KB
}

static moe_status_t linear_in_one(const void* x, int dtype, const int8_t* w, const float* w_scale,
                                  int M, int N, int K, void* c, int c_type, hipStream_t st) {
  const dim3 grid((unsigned)((N + 15) / 16)), block(64 * kSkinnyWaves);
  const size_t lds = (size_t)M * (K + 16);
  const uint8_t* wb = reinterpret_cast<const uint8_t*>(w);
  if (dtype == MOE_TYPE_F32)
    hipLaunchKernelGGL((linear_i8_kernel<MOE_TYPE_F32>), grid, block, lds, st, x, wb, w_scale, M,
                       N, K, c, c_type);
  else if (dtype == MOE_TYPE_BF16)
    hipLaunchKernelGGL((linear_i8_kernel<MOE_TYPE_BF16>), grid, block, lds, st, x, wb, w_scale, M,
                       N, K, c, c_type);
  else
    hipLaunchKernelGGL((linear_i8_kernel<MOE_TYPE_F16>), grid, block, lds, st, x, wb, w_scale, M,
                       N, K, c, c_type);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

static bool float_type(int dtype) {
  return dtype == MOE_TYPE_F32 || dtype == MOE_TYPE_BF16 || dtype == MOE_TYPE_F16;
}

extern "C" moe_status_t moe_linear_int8(const void* x, int dtype, const int8_t* w,
                                        const float* w_scale, int M, int N, int K, void* c,
                                        int c_type, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  if (!float_type(dtype) || !float_type(c_type) || M < 0 || N <= 0 || K <= 0)
    return MOE_INVALID_ARG;
  if (N % 16 != 0 || K % 16 != 0 || K > 131056 || N > kMaxChannels || M > kMaxRows)
    return MOE_UNSUPPORTED_SHAPE;
  if (!w || !w_scale) return MOE_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !c || !workspace || workspace_bytes < moe_linear_int8_workspace_bytes(M, K))
    return MOE_INVALID_ARG;
  if ((((uintptr_t)x | (uintptr_t)w | (uintptr_t)c | (uintptr_t)workspace) & 15) ||
      ((uintptr_t)w_scale & 3))
    return MOE_UNSUPPORTED_SHAPE;
  if (one_launch(M, N, K))
    return linear_in_one(x, dtype, w, w_scale, M, N, K, c, c_type,
                         reinterpret_cast<hipStream_t>(stream));
  int8_t* q = static_cast<int8_t*>(workspace);
  float* s = reinterpret_cast<float*>(q + ((size_t)M * (size_t)K + 15) / 16 * 16);
  const moe_status_t ok = moe_quantize_int8(x, dtype, M, K, q, s, stream);
  if (ok != MOE_OK) return ok;
  return moe_gemm_int8(q, s, w, w_scale, M, N, K, c, c_type, stream);
}
