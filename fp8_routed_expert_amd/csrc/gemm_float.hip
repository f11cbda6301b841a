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
// the matrix cores, rounded once when stored.  Large ones are bound by power
// (131040 x 4096 x 7168 bf16 1358 TF/s, the gradients 1270), few rows by the
// weights' one pass through HBM (256 x 32 x 4096 x 7168 bf16 6.0 TB/s).
#include <type_traits>

#include "float_tile.hpp"
#include "gemm_tiles.hpp"

namespace moe {

struct FloatArgs {
  const uint8_t* p;   // a; dc in both gradients
  const uint8_t* q;   // w; w; a
  const int32_t* offsets;
  const int32_t* counts;
  int E, rows, N, K;
  uint8_t* out;
  int out_type;
  int32_t* status;
  int splits;   // of a segment, for the weights' gradient: 1, or as many fp32 outputs
};

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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

constexpr uint32_t kOutOfRange = 0x80000000u;

// An operand of a tile: B rows of a step's l's (64, in fp32 32) in 128 B bytes of
// LDS.
//
// Contiguous along l (kSlow false): as the 8-bit products have it, a row of
// the tile is 128 bytes of LDS, its 16-byte pieces permuted (swz), and a lane's
// fragment is pieces 2 g and 2 g + 1: l = 16 g .. 16 g + 15 (fp32: 8 g .. 8 g + 7).
//
// Contiguous along the rows (kSlow true), fp32: the step's l's are lines of
// 4 B bytes, of which a lane reads its row's element of eight.  (The four g's
// meet in a bank; the matrix cores take eight times as long in fp32 and hide it.)
//
// The same in 16 bits: the step's 64 values of l are lines of 2 B bytes.  Line
// 16 u + 4 t + g of the stage holds l = 16 g + 4 u + t, so that the four lines t
// of a group of 16 lanes, which ds_read_b64_tr_b16 turns into four l of 16 rows,
// belong to the same g as the other operand's fragment.
// Those 16 lanes read 32 bytes of each of the lines t = 0 .. 3, and the group
// next to them (g + 1) of four others: the 32-byte columns of a line are
// permuted by 2 t + g % 2 (64-byte-row lines: by t; neighbours then lie in
// other banks by themselves), so the eight lines lie in different banks.
template <int B, bool kSlow, int kSize>
struct Operand {
  static constexpr int kStepL = kBK / kSize;      // l's of a step
  static constexpr int kLine = kSize * B;         // bytes of a line (slow)
  static constexpr int kPieces = kLine / 16;      // of a line
  static constexpr int kReads = !kSlow ? 2 : kSize == 2 ? 4 : 8;   // LDS reads of a fragment
  uint32_t vl[2];     // a lane's offset in a chunk's memory, by the chunk's parity
  int lim[2];         // (along l) l's left behind the lane's piece, in bytes
  FragLane frag;      // (slow: lo only)
  // slow: the rest of the matrix, from this step's first line on
  uint64_t base;
  long long bytes;
  long long step;
  v4i rsrc;

  // pitch: bytes from a row of memory to the next; w0: the wave's first row
  __device__ __forceinline__ void lanes(int lane, uint32_t pitch, int L, int w0) {
    const int g = lane >> 4, r16 = lane & 15;
    if constexpr (!kSlow) {
      const int piece = (lane & 7) ^ (lane >> 3);
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        vl[o] = (uint32_t)(lane >> 3) * pitch + (uint32_t)((piece ^ o) << 4);
        lim[o] = kSize * L - ((piece ^ o) << 4);
      }
      frag = frag_lane(w0, r16, g);
    } else if constexpr (kSize == 4) {
      vl[0] = vl[1] = (uint32_t)(lane / kPieces) * pitch + (uint32_t)((lane % kPieces) << 4);
      frag.lo = (uint32_t)(8 * g * kLine + (w0 + r16) * 4);
      frag.hi = 0;
    } else {
      const int at = lane % kPieces, line = lane / kPieces;
      if constexpr (B == 256) {        // lines g % 2
        vl[0] = vl[1] = (uint32_t)line * 16u * pitch + (uint32_t)((at ^ (2 * line)) << 4);
      } else if constexpr (B == 128) { // lines g
        vl[0] = vl[1] = (uint32_t)line * 16u * pitch + (uint32_t)((at ^ (2 * (line & 1))) << 4);
      } else {                         // lines 4 (t % 2) + g
        const int tl = line >> 2;
#pragma unroll
        for (int o = 0; o < 2; ++o)
          vl[o] = (uint32_t)(line & 3) * 16u * pitch + (uint32_t)tl * pitch +
                  (uint32_t)((at ^ (2 * (2 * o + tl))) << 4);
      }
      const int t = r16 >> 2, q = r16 & 3;
      const int sl = B >= 128 ? (g & 1) | (t << 1) : t;
      const uint32_t in = (uint32_t)((4 * t + g) * kLine + sl * 32 + (q >> 1) * 16 + (q & 1) * 8);
      const int w = w0 / 16;
      frag.lo = (in ^ (uint32_t)((w & 7) * 32)) + (uint32_t)((w >> 3) * 256);
      frag.hi = 0;
    }
  }
  // the tile's memory: first element, and the bytes from there to the end of
  // what may be read
  __device__ __forceinline__ void tile(const void* p, long long n, uint32_t pitch) {
    if constexpr (!kSlow) {
      rsrc = make_rsrc(p, (uint32_t)(n > 0x7ffff000LL ? 0x7ffff000LL : n));
    } else {
      base = (uint64_t)(uintptr_t)p;
      bytes = n;
      step = (long long)kStepL * pitch;
    }
  }
  // chunks [wave * kC, wave * kC + kC) of step kb into its stage; steps are
  // issued in order
  template <int kC, bool kRagged>
  __device__ __forceinline__ void issue(int kb, uint8_t* stage, int wave, uint32_t pitch,
                                        bool live) {
    if constexpr (!kSlow) {
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const int c = wave * kC + u;
        const int o = kC % 2 == 0 ? (u & 1) : (c & 1);
        const uint32_t uni = (uint32_t)(c * 8) * pitch + (uint32_t)kb * kBK;
        if constexpr (kRagged) {
          const bool in = live && kb * kBK < lim[o];
          dma16(rsrc, stage + c * 1024, in ? (o ? vl[1] : vl[0]) + uni : kOutOfRange);
        } else {
          dma16_add(rsrc, stage + c * 1024, o ? vl[1] : vl[0],
                    __builtin_amdgcn_readfirstlane(live ? uni : kOutOfRange));
        }
      }
    } else {
      // (past the last step nothing is left: the loads read zeros)
      const long long left = bytes < 0 ? 0 : bytes > 0x7ffff000LL ? 0x7ffff000LL : bytes;
      const v4i r = make_rsrc(reinterpret_cast<const void*>((uintptr_t)base), (uint32_t)left);
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const int c = wave * kC + u;
        if constexpr (kSize == 4) {
          dma16_add(r, stage + c * 1024, vl[0],
                    __builtin_amdgcn_readfirstlane((uint32_t)(c * (64 / kPieces)) * pitch));
        } else if constexpr (B == 256) {
          const uint32_t t = (uint32_t)((c >> 1) & 3);
          dma16_split(r, stage + c * 1024, vl[0], __builtin_amdgcn_readfirstlane(t * 64u),
                      __builtin_amdgcn_readfirstlane(
                          (uint32_t)(32 * (c & 1) + 4 * (c >> 3)) * pitch + t * pitch));
        } else if constexpr (B == 128) {
          const uint32_t t = (uint32_t)(c & 3);
          dma16_split(r, stage + c * 1024, vl[0], __builtin_amdgcn_readfirstlane(t * 64u),
                      __builtin_amdgcn_readfirstlane((uint32_t)(4 * (c >> 2)) * pitch + t * pitch));
        } else {
          dma16_add(r, stage + c * 1024, (kC % 2 == 0 ? u & 1 : c & 1) ? vl[1] : vl[0],
                    __builtin_amdgcn_readfirstlane((uint32_t)(4 * (c >> 1) + 2 * (c & 1)) * pitch));
        }
      }
      base += (uint64_t)step;
      bytes -= step;
    }
  }
  // the fragment of the wave's 16-row subtile i
  __device__ __forceinline__ v8i load(const uint8_t* stage, int i) const {
    if constexpr (!kSlow) {
      return load_frag_at(stage, i * 16 * kBK, frag);
    } else if constexpr (kSize == 4) {
      v8i r;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        r[u] = *reinterpret_cast<const int*>(stage + frag.lo + u * kLine + i * 64);
      return r;
    } else {
      typedef short s4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s4 lds_s4;
      const uint8_t* at = stage + (frag.lo ^ (uint32_t)(i * 32));
      v8i r;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s4*)(lds_void*)(at + u * 16 * kLine));
        const uint2 w = __builtin_bit_cast(uint2, v);
        r[2 * u] = (int)w.x;
        r[2 * u + 1] = (int)w.y;
      }
      return r;
    }
  }
  __device__ __forceinline__ void fresh() {
    asm volatile("" : "+v"(frag.lo));
    if constexpr (!kSlow) asm volatile("" : "+v"(frag.hi));
  }
};

// c += the products of half h of two fragments (16 bits: eight l's of a lane in
// one instruction; fp32: four, one of every lane to an instruction).
template <int kType, int h>
__device__ __forceinline__ v4f multiply_half(const v8i& a, const v8i& b, v4f c) {
  if constexpr (kType == MOE_TYPE_F32) {
#pragma unroll
    for (int i = 4 * h; i < 4 * h + 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[i]), __int_as_float(b[i]), c, 0, 0,
                                               0);
    return c;
  } else {
    const v4i x = {a[4 * h], a[4 * h + 1], a[4 * h + 2], a[4 * h + 3]};
    const v4i y = {b[4 * h], b[4 * h + 1], b[4 * h + 2], b[4 * h + 3]};
    if constexpr (kType == MOE_TYPE_BF16)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                     __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                    __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
  }
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, (h2){(_Float16)lo, (_Float16)hi});
}

// A BM x BN tile by waves of WM x WN, l advancing 128 bytes a step.  The
// operands go from global memory straight into LDS, P's a step further ahead
// than Q's; the pipeline is that of the 8-bit products (waits and barriers are
// explained there): the next step's loads go out first, the step's barrier comes
// once a wave's last LDS read of it has landed, and the next step's fragments
// are read under the last subtile row's multiplications.
// kDeep: 0, or the stages of both operands for launches of few tiles.
template <int kType, int kMode, int BM, int BN, int WM, int WN, int GM, int kDeep, bool kRagged>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void float_tile_kernel(FloatArgs p) {
  constexpr int kSize = kType == MOE_TYPE_F32 ? 4 : 2;
  constexpr int kStepL = kBK / kSize;
  constexpr int NWN = BN / WN;
  constexpr int NW = BM / WM * NWN;
  constexpr int MI = WM / 16, NJ = WN / 16;
  constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;   // 1 KB chunks of a stage per wave
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "chunks must split evenly");
  static_assert(MI >= 2 && NJ == 4, "late loads; a wave's stores are whole pieces");
  constexpr int SA_B = BM * kBK, SB_B = BN * kBK;
  constexpr int NSA = kDeep ? kDeep : 3 * SA_B + 2 * SB_B <= kLdsBytes ? 3 : 2;
  constexpr int NSB = kDeep ? kDeep : 2;
  static_assert(NSA * SA_B + NSB * SB_B <= kLdsBytes, "tile stages exceed the LDS");
  static_assert(6 % NSA == 0 && 6 % NSB == 0, "the loop over l is unrolled by 6");
  auto stA = [&](auto i) { return Stage<SA_B, 0, decltype(i)::value % NSA>::get(); };
  auto stB = [&](auto i) { return Stage<SB_B, 1, decltype(i)::value % NSB>::get(); };

  // ---- which tile: columns within groups of GM row tiles
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int width = kMode == kProduct ? p.N : p.K;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 64 && p.status &&
      segments_bad(p.offsets, p.counts, p.E, lane) && lane == 0)
    atomicOr(p.status, MOE_ERR_BAD_INDEX);
  const int n_tiles = (width + BN - 1) / BN;
  const int i_tiles = (p.N + BM - 1) / BM;   // of an expert's weights
  const int total_m = kMode == kWeightsGrad
                          ? p.E * i_tiles
                          : total_mtiles<BM>(p.offsets, p.counts, p.E, p.rows, lane);
  if ((long long)blockIdx.x >= (long long)total_m * n_tiles) return;
  const int group = (int)blockIdx.x / (GM * n_tiles);
  const int in_group = (int)blockIdx.x - group * (GM * n_tiles);
  const int gm_cnt = min(GM, total_m - group * GM);
  const int tile_n = in_group / gm_cnt;
  const int tile_m = group * GM + (in_group - tile_n * gm_cnt);
  const int n0 = tile_n * BN;
  int e, row0, row_end, L, s0 = 0;   // rows of P and of the output; s0: the segment's first row
  if (kMode == kWeightsGrad) {
    int en;
    e = tile_m / i_tiles;
    expert_rows(p.offsets, p.counts, e, p.rows, s0, en);
    s0 = __builtin_amdgcn_readfirstlane(s0);
    L = __builtin_amdgcn_readfirstlane(en) - s0;
    if (p.splits > 1) {
      // this workgroup's steps of the segment
      const int steps = (L + kStepL - 1) / kStepL;
      const int per = (steps + p.splits - 1) / p.splits * kStepL;
      const int skip = min(L, per * (int)blockIdx.y);
      s0 += skip;
      L = min(L - skip, per);
    }
    row0 = (tile_m - e * i_tiles) * BM;
    row_end = p.N;
  } else {
    find_mtile<BM>(p.offsets, p.counts, p.E, p.rows, tile_m, lane, e, row0, row_end);
    if (e < 0) return;
    L = kMode == kProduct ? p.K : p.N;
  }

  // ---- operands
  constexpr bool kSlowA = kMode == kWeightsGrad, kSlowB = kMode != kProduct;
  Operand<BM, kSlowA, kSize> A;
  Operand<BN, kSlowB, kSize> B;
  const uint32_t pitch_a = (uint32_t)kSize * (uint32_t)(kMode == kProduct ? p.K : p.N);
  const uint32_t pitch_b = (uint32_t)kSize * (uint32_t)p.K;
  const int wm = wave / NWN, wn = wave - wm * NWN;
  A.lanes(lane, pitch_a, L, wm * WM);
  B.lanes(lane, pitch_b, L, wn * WN);
  if constexpr (kMode == kWeightsGrad)
    A.tile(p.p + (size_t)s0 * pitch_a + kSize * row0, (long long)L * pitch_a - kSize * row0,
           pitch_a);
  else
    A.tile(p.p + (size_t)row0 * pitch_a, (long long)(p.rows - row0) * pitch_a, pitch_a);
  const uint8_t* we = p.q + (size_t)e * p.N * pitch_b;
  if constexpr (kMode == kProduct)
    B.tile(we + (size_t)n0 * pitch_b, (long long)min(BN, p.N - n0) * pitch_b, pitch_b);
  else if constexpr (kMode == kRowsGrad)
    B.tile(we + kSize * n0, (long long)L * pitch_b - kSize * n0, pitch_b);
  else
    B.tile(p.q + (size_t)s0 * pitch_b + kSize * n0, (long long)L * pitch_b - kSize * n0, pitch_b);
  const int Lb = (L + kStepL - 1) / kStepL;
  auto issue_a = [&](int kb, uint8_t* st) {
    A.template issue<CA, kRagged>(kb, st, wave, pitch_a, kb < Lb);
  };
  auto issue_b = [&](int kb, uint8_t* st) {
    B.template issue<CB, kRagged>(kb, st, wave, pitch_b, kb < Lb);
  };

  v4f acc[MI][NJ] = {};
  v8i bf[NJ];
  v8i af_next;
  auto subtile = [&](int i, int j, bool hi_first, const v8i& af) __attribute__((always_inline)) {
    if (hi_first) {
      acc[i][j] = multiply_half<kType, 1>(bf[j], af, acc[i][j]);
      acc[i][j] = multiply_half<kType, 0>(bf[j], af, acc[i][j]);
    } else {
      acc[i][j] = multiply_half<kType, 0>(bf[j], af, acc[i][j]);
      acc[i][j] = multiply_half<kType, 1>(bf[j], af, acc[i][j]);
    }
  };
  constexpr int kLateRow = MI >= 3 ? 1 : 0;
  constexpr int kInFlight = kDeep ? (kDeep - 2) * (CA + CB) : NSA == 3 ? CA : 0;
  auto step = [&](int kb, auto unrolled) __attribute__((always_inline)) {
    constexpr int U = decltype(unrolled)::value;
    A.fresh();
    B.fresh();
    const uint8_t* tA = stA(Int<U>());
    const uint8_t* tAn = stA(Int<U + 1>());
    const uint8_t* tBn = stB(Int<U + 1>());
    issue_b(kb + NSB - 1, stB(Int<U + NSB - 1>()));
#pragma unroll
    for (int i = 0; i < MI - 1; ++i) {
      if (i == kLateRow) issue_a(kb + NSA - 1, stA(Int<U + NSA - 1>()));
      const v8i af = af_next;
      af_next = A.load(tA, i + 1);
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) {
        subtile(i, (i & 1) ? NJ - 1 - jj : jj, jj & 1, af);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int i = 0; i < MI - 1; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(acc[i][j]));
    wait_vm<kInFlight>();
    lds_barrier();
    const v8i af = af_next;
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const int j = (MI & 1) ? jj : NJ - 1 - jj;
      subtile(MI - 1, j, jj & 1, af);
      bf[j] = B.load(tBn, j);
    }
    af_next = A.load(tAn, 0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x008, kSize == 2 ? 2 : 8, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, decltype(B)::kReads, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, decltype(A)::kReads, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(acc[MI - 1][j]));
  };

  issue_b(0, stB(Int<0>()));
  issue_a(0, stA(Int<0>()));
  if constexpr (kDeep != 0) {
    each<1, kDeep - 1>([&](auto i) {
      issue_b(decltype(i)::value, stB(i));
      issue_a(decltype(i)::value, stA(i));
    });
  } else if constexpr (NSA == 3) {
    issue_a(1, stA(Int<1>()));
  }
  wait_vm<kInFlight>();
  lds_barrier();
#pragma unroll
  for (int j = 0; j < NJ; ++j) bf[j] = B.load(stB(Int<0>()), j);
  af_next = A.load(stA(Int<0>()), 0);
  // fp32: an instruction adds four products to a sum, so a long sum is a chain of
  // l / 4 roundings; one of 48 is added to a total every six steps instead (over
  // 7168 l's the error falls from 1.3e-6 to 3e-7 of the result).
  v4f total[kSize == 4 ? MI : 1][kSize == 4 ? NJ : 1] = {};
  for (int kb = 0; kb < Lb; kb += 6) {
    each<0, 6>([&](auto u) __attribute__((always_inline)) {
      constexpr int U = decltype(u)::value;
      if (U == 0 || kb + U < Lb) step(kb + U, u);
    });
    if constexpr (kSize == 4)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          total[i][j] += acc[i][j];
          acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
  }
  wait_vm<0>();   // (the loads past the last step)
  if constexpr (kSize == 4)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = total[i][j];

  // ---- epilogue: sums (i, j) of a lane are four columns 4 g .. 4 g + 3 of row
  // r16.  In 16 bits two subtiles' halves are exchanged between neighbouring
  // rows of 16 lanes, so that a lane holds eight columns, then lanes of rows
  // 0..7 exchange their second piece for the first piece of the row 8 further:
  // a store writes eight rows' whole 128 bytes, past the caches.  In fp32 a row's
  // 128 bytes take two stores, which the cache has to put together (past it, 32
  // x 4096 x 7168 of few rows 1063 us against 719).
  const int g = lane >> 4, r16 = lane & 15;
  const size_t out0 =
      kMode == kWeightsGrad ? ((size_t)blockIdx.y * p.E + (size_t)e) * (size_t)p.N : 0;
  const int top = row0 + wm * WM, left = n0 + wn * WN;
  if (kType == MOE_TYPE_F32 || p.out_type == MOE_TYPE_F32) {
    float* out = reinterpret_cast<float*>(p.out);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int row = top + 16 * i + r16, col = left + 16 * j + 4 * g;
        if (row < row_end && col < width)
          *reinterpret_cast<v4f*>(out + (out0 + row) * width + col) = acc[i][j];
      }
    return;
  }
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out);
  const bool low = r16 < 8;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    u32x4 piece[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t a[2], b[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const v4f& x = acc[i][2 * s];
        const v4f& y = acc[i][2 * s + 1];
        a[q] = kType == MOE_TYPE_F16 ? pack2_f16(x[2 * q], x[2 * q + 1])
                                     : pack2_bf16(x[2 * q], x[2 * q + 1]);
        b[q] = kType == MOE_TYPE_F16 ? pack2_f16(y[2 * q], y[2 * q + 1])
                                     : pack2_bf16(y[2 * q], y[2 * q + 1]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const auto r = __builtin_amdgcn_permlane16_swap(a[q], b[q], false, false);
        piece[s][q] = r[0];
        piece[s][2 + q] = r[1];
      }
    }
    u32x4 first, second;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(
          0, (int)(low ? piece[1][q] : piece[0][q]), 0x128, 0xf, 0xf, false);   // row_ror:8
      first[q] = low ? piece[0][q] : got;
      second[q] = low ? got : piece[1][q];
    }
    const int col = left + (low ? 0 : 32) + 16 * (g & 1) + 8 * (g >> 1);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int row = top + 16 * i + (r16 & 7) + 8 * s;
      if (row < row_end && col < width)
        __builtin_nontemporal_store(
            s ? second : first, reinterpret_cast<u32x4*>(out + (out0 + row) * width + col));
    }
  }
}

// Products of a few rows of every expert in 16 bits, 16 of them to a workgroup,
// where tiles would be too few to keep the memory busy: bound by the weights'
// way from HBM, once for 16 rows.  A workgroup computes 16 NT channels; its
// eight waves share out K, so that every CU has many waves' weight loads in
// flight (a wave's fragments go from global memory straight to its registers:
// each weight is used by one wave), and their sums are added in LDS in the
// order of the waves.
constexpr int kSkinnyWaves = 8;
constexpr int kSlab = 64;   // bytes of a row that one multiplication takes: 16 of four lanes

template <int kType, int NT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_float_kernel(FloatArgs p) {
  constexpr int kAhead = 8;   // slabs loaded at once
  __shared__ float sums[kSkinnyWaves][NT * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = p.N, bytes = 2 * p.K;   // of a row
  const int n_tiles = (N + 16 * NT - 1) / (16 * NT);
  const int tile_m = blockIdx.x / n_tiles, n0 = (blockIdx.x - tile_m * n_tiles) * 16 * NT;
  if (blockIdx.x == 0 && threadIdx.x < 64 && p.status &&
      segments_bad(p.offsets, p.counts, p.E, lane) && lane == 0)
    atomicOr(p.status, MOE_ERR_BAD_INDEX);
  int e, row0, row_end;
  find_mtile<16>(p.offsets, p.counts, p.E, p.rows, tile_m, lane, e, row0, row_end);
  if (e < 0) return;
  const int g = lane >> 4, r16 = lane & 15;
  const uint8_t* wp[NT];
  bool w_in[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = n0 + j * 16 + r16;
    w_in[j] = n < N;
    wp[j] = p.q + ((size_t)e * N + (w_in[j] ? n : 0)) * bytes + 16 * g;
  }
  const bool a_in = row0 + r16 < row_end;
  const uint8_t* ap = p.p + (size_t)(a_in ? row0 + r16 : row0) * bytes + 16 * g;
  auto load = [](const uint8_t* at, bool in) {
    const v4i z = {0, 0, 0, 0};
    return in ? *reinterpret_cast<const v4i*>(at) : z;
  };
  v4f acc[NT] = {};
  // wave w takes slabs [first, last), pairs of them (one 128-byte line) together
  const int lines = (bytes + 2 * kSlab - 1) / (2 * kSlab);
  const int first = 2 * (int)((long long)lines * wave / kSkinnyWaves);
  const int last = min(2 * (int)((long long)lines * (wave + 1) / kSkinnyWaves),
                       (bytes + kSlab - 1) / kSlab);
  for (int s0 = first; s0 < last; s0 += kAhead) {
    v4i wf[kAhead][NT], af[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool in = s0 + u < last && (s0 + u) * kSlab + 16 * g < bytes;
#pragma unroll
      for (int j = 0; j < NT; ++j) wf[u][j] = load(wp[j] + (s0 + u) * kSlab, in && w_in[j]);
      af[u] = load(ap + (s0 + u) * kSlab, in && a_in);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (kType == MOE_TYPE_BF16)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wf[u][j]),
                                                           __builtin_bit_cast(bf16x8, af[u]),
                                                           acc[j], 0, 0, 0);
        else
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, wf[u][j]),
                                                          __builtin_bit_cast(f16x8, af[u]),
                                                          acc[j], 0, 0, 0);
      }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) sums[wave][4 * j + q][lane] = acc[j][q];
  __syncthreads();
  // channels 16 j + 4 (l / 16) + 0 .. 3 of row l % 16
  for (int u = threadIdx.x; u < NT * 64; u += 64 * kSkinnyWaves) {
    const int j = u >> 6, l = u & 63;
    const int row = row0 + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (row >= row_end || n >= N) continue;
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = sums[0][4 * j + q][l];
#pragma unroll
      for (int w = 1; w < kSkinnyWaves; ++w) v[q] += sums[w][4 * j + q][l];
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + (size_t)row * N + n) =
        kType == MOE_TYPE_F16 ? make_uint2(pack2_f16(v[0], v[1]), pack2_f16(v[2], v[3]))
                              : make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
  }
}

// The weights' gradient from `n` fp32 parts of it, added in order.
__global__ __launch_bounds__(256) void join_parts_kernel(const float* __restrict__ parts, int n,
                                                         long long values, uint8_t* out,
                                                         int out_type) {
  for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4; i < values;
       i += (long long)gridDim.x * 1024) {
    v4f s = *reinterpret_cast<const v4f*>(parts + i);
#pragma unroll 4
    for (int k = 1; k < n; ++k) s += *reinterpret_cast<const v4f*>(parts + k * values + i);
    if (out_type == MOE_TYPE_F32)
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(out) + i) = s;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + i) =
          out_type == MOE_TYPE_F16 ? make_uint2(pack2_f16(s[0], s[1]), pack2_f16(s[2], s[3]))
                                   : make_uint2(pack2_bf16(s[0], s[1]), pack2_bf16(s[2], s[3]));
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

template <int kType, int kMode, int BM, int BN, int WM, int WN, int GM, int kDeep>
static moe_status_t launch_tiles(const FloatArgs& p, hipStream_t st) {
  constexpr int threads = 64 * (BM / WM) * (BN / WN);
  const long long blocks = tiles_of(kMode, p.E, p.rows, p.N, p.K, BM, BN);
  if (blocks * threads > 0xffffffffLL || blocks > 0x7fffffffLL) return MOE_UNSUPPORTED_SHAPE;
  const dim3 grid((unsigned)blocks, (unsigned)p.splits), block(threads);
  // (a weights' gradient ends where its operands' descriptors end)
  const int l = kMode == kProduct ? p.K : p.N;
  const bool ragged = kMode != kWeightsGrad && l % (kType == MOE_TYPE_F32 ? 32 : 64) != 0;
  if constexpr (kMode != kWeightsGrad) {
    if (ragged) {
      hipLaunchKernelGGL((float_tile_kernel<kType, kMode, BM, BN, WM, WN, GM, kDeep, true>), grid,
                         block, 0, st, p);
      return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
    }
  }
  hipLaunchKernelGGL((float_tile_kernel<kType, kMode, BM, BN, WM, WN, GM, kDeep, false>), grid,
                     block, 0, st, p);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

template <int kType, int NT>
static moe_status_t launch_skinny(const FloatArgs& p, hipStream_t st) {
  const long long blocks =
      ((long long)p.rows / 16 + p.E) * ((p.N + 16 * NT - 1) / (16 * NT));
  if (blocks * 64 * kSkinnyWaves > 0xffffffffLL) return MOE_UNSUPPORTED_SHAPE;
  hipLaunchKernelGGL((skinny_float_kernel<kType, NT>), dim3((unsigned)blocks),
                     dim3(64 * kSkinnyWaves), 0, st, p);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

template <int kType, int kMode>
static moe_status_t launch_float(const FloatArgs& p, hipStream_t st) {
  const FloatTile t = float_tile(kMode, kType == MOE_TYPE_F32, p.E, p.rows, p.N, p.K, p.splits);
  if constexpr (kType == MOE_TYPE_F32) {
    if (t.cols == 64) return launch_tiles<kType, kMode, 64, 64, 32, 64, 4, 6>(p, st);
    return launch_tiles<kType, kMode, 64, 128, 32, 64, 4, 0>(p, st);
  } else {
    if constexpr (kMode == kProduct)
      if (t.rows == 16)
        return t.cols == 32 ? launch_skinny<kType, 2>(p, st) : launch_skinny<kType, 1>(p, st);
    if constexpr (kMode != kWeightsGrad)
      if (t.rows == 64)
        return t.cols == 64 ? launch_tiles<kType, kMode, 64, 64, 32, 64, 4, 6>(p, st)
                            : launch_tiles<kType, kMode, 64, 128, 32, 64, 4, 0>(p, st);
    if (t.rows == 256) return launch_tiles<kType, kMode, 256, 256, 128, 64, 2, 0>(p, st);
    if constexpr (kMode != kRowsGrad)
      if (t.ahead == 0) return launch_tiles<kType, kMode, 128, 128, 64, 64, 4, 0>(p, st);
    return launch_tiles<kType, kMode, 128, 128, 64, 64, 4, 3>(p, st);
  }
}

template <int kMode>
static moe_status_t launch_float(const FloatArgs& p, int dtype, hipStream_t st) {
  if (dtype == MOE_TYPE_BF16) return launch_float<MOE_TYPE_BF16, kMode>(p, st);
  if (dtype == MOE_TYPE_F16) return launch_float<MOE_TYPE_F16, kMode>(p, st);
  return launch_float<MOE_TYPE_F32, kMode>(p, st);
}

constexpr int kMaxFloatDim = 1 << 20;     // N and K
constexpr int kMaxFloatRows = 0x7fff0000; // rounded up to tiles, 32 bits still hold them

static moe_status_t float_args(const FloatArgs& p, int dtype) {
  if (!float_type(dtype) || p.E <= 0 || p.E > MOE_MAX_EXPERTS || p.rows < 0 || p.N <= 0 ||
      p.K <= 0)
    return MOE_INVALID_ARG;
  if (p.N % 8 != 0 || p.K % 8 != 0 || p.N > kMaxFloatDim || p.K > kMaxFloatDim ||
      p.rows > kMaxFloatRows)
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
                    counts, E, rows_total, N, K, static_cast<uint8_t*>(c), dtype, status_dev, 1};
  return float_rows<kProduct>(p, dtype, zero_rest, stream);
}

extern "C" moe_status_t moe_grouped_gemm_float_grad_rows(const void* dc, const void* w, int dtype,
                                                         const int32_t* offsets,
                                                         const int32_t* counts, int E,
                                                         int rows_total, int N, int K, void* da,
                                                         int zero_rest, int32_t* status_dev,
                                                         void* stream) {
  const FloatArgs p{static_cast<const uint8_t*>(dc), static_cast<const uint8_t*>(w), offsets,
                    counts, E, rows_total, N, K, static_cast<uint8_t*>(da), dtype, status_dev, 1};
  return float_rows<kRowsGrad>(p, dtype, zero_rest, stream);
}

extern "C" size_t moe_grouped_gemm_float_workspace_bytes(int E, int rows_total, int N, int K) {
  if (E <= 0 || rows_total < 0 || N <= 0 || K <= 0) return 0;
  const int n = weight_splits(E, rows_total, N, K);
  return n > 1 ? (size_t)n * E * N * K * sizeof(float) : 0;
}

extern "C" moe_status_t moe_grouped_gemm_float_grad_weights(
    const void* dc, const void* a, int dtype, const int32_t* offsets, const int32_t* counts, int E,
    int rows_total, int N, int K, void* dw, int dw_type, void* workspace, size_t workspace_bytes,
    int32_t* status_dev, void* stream) {
  FloatArgs p{static_cast<const uint8_t*>(dc), static_cast<const uint8_t*>(a), offsets, counts, E,
              rows_total, N, K, static_cast<uint8_t*>(dw), dw_type, status_dev, 1};
  moe_status_t ok = float_args(p, dtype);
  if (ok != MOE_OK) return ok;
  if (dw_type != dtype && dw_type != MOE_TYPE_F32) return MOE_INVALID_ARG;
  if (!dw || (rows_total > 0 && (!dc || !a))) return MOE_INVALID_ARG;
  const size_t need = moe_grouped_gemm_float_workspace_bytes(E, rows_total, N, K);
  if (need && (!workspace || workspace_bytes < need)) return MOE_INVALID_ARG;
  if ((uintptr_t)workspace & 15) return MOE_UNSUPPORTED_SHAPE;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  p.splits = weight_splits(E, rows_total, N, K);
  if (p.splits == 1) return launch_float<kWeightsGrad>(p, dtype, st);
  p.out = static_cast<uint8_t*>(workspace);
  p.out_type = MOE_TYPE_F32;
  ok = launch_float<kWeightsGrad>(p, dtype, st);
  if (ok != MOE_OK) return ok;
  const long long values = (long long)E * N * K;
  const long long blocks = (values + 1023) / 1024;
  hipLaunchKernelGGL(join_parts_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256),
                     0, st, static_cast<const float*>(workspace), p.splits, values,
                     static_cast<uint8_t*>(dw), dw_type);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}
