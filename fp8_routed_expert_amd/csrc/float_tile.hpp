// Which tiles the products in fp32, bf16 and fp16 and their gradients take
// (gemm_float.hip), from the sizes alone: plain host code.
#pragma once

namespace moe {

enum { kProduct = 0, kRowsGrad = 1, kWeightsGrad = 2 };

// Tiles of a launch: those of every expert's rows, rounded up.
inline long long tiles_of(int mode, int E, int rows, int N, int K, int bm, int bn) {
  const int width = mode == kProduct ? N : K;
  const long long m = mode == kWeightsGrad ? (long long)E * ((N + bm - 1) / bm)
                                            : (long long)rows / bm + E;
  return m * ((width + bn - 1) / bn);
}

// Parts that the weights' gradient splits its segments into: where the experts'
// 128 x 128 tiles are fewer than a round of the CUs (two workgroups to each),
// and segments (of the buffer, on average) long enough for at least 512 rows
// in a part.  (65536 rows of one expert, 512 x 512 bf16: 306 us whole, 73 in 32
// parts, their join included.)
inline int weight_splits(int E, int rows, int N, int K) {
  const long long tiles = (long long)E * ((N + 127) / 128) * ((K + 127) / 128);
  long long n = tiles < 256 ? 512 / tiles : 1;
  const long long parts = rows / E / 512;
  if (n > parts) n = parts;
  return n < 1 ? 1 : n > 32 ? 32 : (int)n;
}

// Tiles are chosen from the sizes alone (the same inside graph capture).  `rows`
// is a segment's on average: the buffer's, less the 127 that a contiguous one
// has for the padding between segments (a capacity of 128 rows or more counts
// as less than it may hold).  Times in us, weights from HBM, rows x experts x N
// x K, bf16; p: product, r: rows' gradient, w: weights' gradient.
//
//   * Few rows: 64 x 128 tiles, several workgroups to a CU, once there are more
//     of them than CUs (p 256 x 32 x 4096 x 7168 318, 64 x 64 tiles loaded five
//     steps ahead 366, 128 x 128 354; r 357, 450, 375) or l is short; else 64 x
//     64 (r 8 x 8 x 7168 x 2048 36, 64 x 128 68, 128 x 128 55); and where
//     there are so few channels that those leave CUs idle, the product
//     without tiles (p 1 x 1 x 4096 x 7168 14, 64 x 64 31; 1 x 1 x 7168 x 2048
//     9.6 and 12; 8 x 8 x 4096 x 7168 66 and 80; but 4 x 4 36 and 32).  That
//     one reads the weights once for every 16 rows.  A buffer of 128 to 143
//     rows to an expert may be a contiguous one of few rows or hold full
//     segments (x 4096 x 7168, experts x rows of each, without tiles and 64 x
//     64: 4 x 1 50 and 47, 4 x 128 316 and 80; 8 x 1 95 and 94, 8 x 128 629 and
//     162; but 1 x 1 14 and 36, 1 x 128 104 and 36; 2 x 1 26 and 39, 2 x 128 161
//     and 41): it takes 64 x 64 tiles where these are as many as the CUs, and
//     with fewer channels stays without, for the few rows.
//   * else 256 x 256 or 128 x 128, whichever takes less time by their rounds of
//     the CUs: a step of 256 tiles of 256 x 256 takes 1.59 us at the rate of
//     large products, one of 256 tiles of 128 x 128 0.605 (p 1024 x 8 x 4096 x
//     7168 185 and 152, r 117 and 140; p 4096 x 32 571 and 483; 6144 x 6 x
//     7168 x 2048 p 163 and 210, r 185 and 229; prefill shares 131040 x 9 x 4096
//     x 7168 p 5700 and 9090).  128 x 128 with two workgroups to a CU, or, for
//     the rows' gradient and where there are no two, loaded two steps ahead
//     (r 4096 x 32 x 7168 x 2048 243 and 301; p 8192 x 32 402 and 372).
//   * fp32: 64 x 128, or 64 x 64 where those are few (16384 x 8 x 1024 x 1024 p
//     294, 64 x 64 591, 128 x 128 329, 256 x 256 485: its steps have half the
//     l's and eight times the multiplications, so the loads hide in any tile and
//     what counts is that the last round is full).
struct FloatTile {
  int rows, cols;   // rows 16: without tiles
  int ahead;        // stages of both operands, or 0
};

inline FloatTile float_tile(int mode, bool f32, int E, int rows_total, int N, int K, int splits) {
  const int width = mode == kProduct ? N : K;
  if (f32) {
    if (tiles_of(mode, E, rows_total, N, K, 64, 64) <= 512 && splits == 1) return {64, 64, 6};
    return {64, 128, 0};
  }
  const long long most = ((long long)rows_total + E - 1) / E;
  const long long rows = most >= 128 ? most - 127 : most;
  if (mode != kWeightsGrad && rows <= 48) {
    const long long wide = (long long)E * ((width + 127) / 128);
    const int L = mode == kProduct ? K : N;
    if (wide > 256 || (wide > 128 && L <= 1024)) return {64, 128, 0};
    if (mode == kProduct && rows <= 16 && (most <= 16 || (long long)E * N < 256 * 64))
      return {16, (long long)E * N >= 448 * 16 ? 32 : 16, 0};
    return {64, 64, 6};
  }
  // (segments differ, and end anywhere in a tile: six tenths of one more each,
  // but a tile at least.  One expert's 100 rows x 4096 x 7168 counted as none
  // took 256 x 256 tiles, p 152 us, and take 62.)
  auto tiles = [&](int b) {
    const long long few = E * (10 * rows + 6 * b) / (10 * b);
    const long long m = mode == kWeightsGrad ? (long long)E * ((N + b - 1) / b) : few ? few : 1;
    return m * ((width + b - 1) / b);
  };
  auto rounds = [](long long n) { return (n + 255) / 256; };
  if (splits == 1 && rounds(tiles(256)) * 159 <= rounds(tiles(128)) * 60) return {256, 256, 0};
  return {128, 128, mode != kRowsGrad && tiles(128) > 256 ? 0 : 3};
}

}  // namespace moe
