// Layer norm of rows, and its gradient, in fp32, bf16 and fp16.
//
//   mu = sum_h x_h / H,  v = sum_h (x_h - mu)^2 / H,  r = 1 / sqrt(v + eps)
//   y_h = (x_h - mu) r w_h + b_h
//
//   with g_h = dy_h w_h and z_h = (x_h - mu) r:
//   dx_h = r (g_h - sum_j g_j / H - z_h sum_j g_j z_j / H)
//   dw_h = sum_t dy_th z_th,   db_h = sum_t dy_th
//
// A row is read once and kept in registers, so that the variance is the sum of
// the squared distances from the mean that was found before (the difference of
// two sums loses everything where the mean is large).  Sums are fp32: a lane's
// own values in order, then the lanes of a wave, then (rows shared by several
// waves) the waves in order, of 16 waves the pairs first (row_total).  Nothing
// is added with atomics: the gradients of w and b are kept by column in each
// workgroup's registers over all the rows that it walks, written once as partial
// sums, and joined by a second kernel in the order of the workgroups.  Bound by HBM bandwidth: 65536 rows of 7168
// bf16 336 us (5.6 TB/s), the gradient of 32768 242 (5.8 TB/s).
#include "row_chunks.hpp"

namespace moe {

constexpr int kNormParts = 512;     // workgroups that keep partial sums, at most
constexpr int kNormRows = 4;        // rows that make another such workgroup worth its sums
constexpr int kNormLong = 32768;    // bytes of a row that the registers of a workgroup hold

struct NormArgs {
  const uint8_t* x;
  const uint8_t* dy;
  const uint8_t* w;
  const uint8_t* b;
  int T, H;
  RowShape row;
  float eps;
  uint8_t* y;        // dx in the gradient
  float* mean;
  float* rstd;
  float* parts;      // [workgroups][2][H]
  float* stats;      // [T][2], long rows
};

// The wave's sum, in every lane: rows of 16 lanes by lane permutations, then
// their four sums.
__device__ __forceinline__ float wave_add(float v) {
  v += dpp_row<0xb1>(v);
  v += dpp_row<0x4e>(v);
  v += dpp_row<0x141>(v);
  v += dpp_row<0x140>(v);
  const int i = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(i, 0)) +
          __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(i, 32)) +
          __int_as_float(__builtin_amdgcn_readlane(i, 48)));
}

// The sums of the kWaves waves that share a row, in every lane of them.  Two
// sums that follow one another take two buffers, so that a sum costs one
// barrier: whoever writes a buffer again has passed the barrier behind which
// its last values were read.
template <int kWaves, int kN>
__device__ __forceinline__ void row_add(float (&v)[kN], float (*red)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = wave_add(v[i]);
  if constexpr (kWaves > 1) {
    const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) % kWaves;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < kN; ++i) red[wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float s = red[0][i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += red[w][i];
      v[i] = s;
    }
  }
}

// The row's sum, in every lane of its waves.  Rows of 513 to 1024 chunks are
// taken by 16 waves of one chunk to a lane or, where there are many, by eight of
// two (launch_norm): wave w of the sixteen and wave w + 8 hold what wave w of the
// eight has in its first and second chunks.  Both add these two waves' sums
// first (kSums: the eight have a sum for each chunk; kPairs: the sixteen), so
// that a row's bits do not depend on its batch.  (second: the wave has second
// chunks; the sum of none is 0.)
template <int kWaves, int kSums, bool kPairs>
__device__ __forceinline__ float row_total(const float (&v)[kSums], bool second, float* red) {
  float s = wave_add(v[0]);
  if constexpr (kSums == 2)
    if (second) s += wave_add(v[1]);
  if constexpr (kWaves > 1) {
    const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) % kWaves;
    if (lane == 0) red[wave] = s;
    __syncthreads();
    constexpr int kHalf = kPairs ? kWaves / 2 : kWaves;
    s = kPairs ? red[0] + red[kHalf] : red[0];
#pragma unroll
    for (int w = 1; w < kHalf; ++w) s += kPairs ? red[w] + red[w + kHalf] : red[w];
  }
  return s;
}

// Values [at, at + n) of a weight or bias, n <= kN of them.
template <typename W, int kN>
__device__ __forceinline__ void load_param(const uint8_t* p, int at, int n, float (&v)[kN]) {
  const uint8_t* src = p + (size_t)at * W::kSize;
  if (n >= kN) {
    constexpr int kBytes = kN * W::kSize;
#pragma unroll
    for (int u = 0; u < (kBytes + 15) / 16; ++u) {
      uint4 c = make_uint4(0, 0, 0, 0);
      __builtin_memcpy(&c, src + 16 * u, kBytes < 16 ? kBytes : 16);
      float f[W::kN];
      W::unpack(c, f);
#pragma unroll
      for (int i = 0; i < W::kN && u * W::kN + i < kN; ++i) v[u * W::kN + i] = f[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    uint4 c = make_uint4(0, 0, 0, 0);
    if (i < n) __builtin_memcpy(&c, src + i * W::kSize, W::kSize);
    float f[W::kN];
    W::unpack(c, f);
    v[i] = f[0];
  }
}

// Rows: shorter than a chunk; of any longer length, read and written through
// unaligned 16-byte accesses; of whole aligned chunks.  (65536 rows of 2050 bf16
// 124 us, the gradient 194; with a mask for every element and narrow accesses
// 149 and 256; rows of 2048 88 and 139.)
enum { kShortRows = 0, kLooseRows = 1, kWholeRows = 2 };

template <int kKind, bool kStream = false>
__device__ __forceinline__ uint4 load_row(const uint8_t* p, int row_bytes) {
  if constexpr (kKind == kLooseRows) {
    uint4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
  } else {
    return load_chunk<kKind == kWholeRows, kStream>(p, row_bytes);
  }
}

template <int kKind>
__device__ __forceinline__ void store_row(uint8_t* p, int row_bytes, const uint4& v) {
  if constexpr (kKind == kLooseRows)
    __builtin_memcpy(p, &v, 16);
  else
    store_chunk<kKind == kWholeRows>(p, row_bytes, v);
}

// The elements of chunk c that count: [lo, hi) of its El::kN (a last chunk
// overlaps the one before it, a row shorter than a chunk ends inside it).
template <typename El>
__device__ __forceinline__ void chunk_range(const RowShape& row, int c, int& lo, int& hi) {
  lo = (16 * c - row.start(c)) / El::kSize;
  hi = row.bytes >= 16 ? El::kN : row.bytes / El::kSize;
}

// The weight (or bias, missing: `none`) of a lane's chunk c.
template <typename El, typename W, int kKind>
__device__ __forceinline__ void chunk_param(const uint8_t* p, const NormArgs& a, int c, float none,
                                            float (&v)[El::kN]) {
#pragma unroll
  for (int i = 0; i < El::kN; ++i) v[i] = none;
  if (!p || c >= a.row.chunks) return;
  const int at = a.row.start(c) / El::kSize;
  load_param<W, El::kN>(p, at, kKind != kShortRows ? El::kN : min(El::kN, a.H - at), v);
}

// kWaves waves to a row, which its lanes hold in kCh chunks each.  A workgroup
// walks rows, so that a lane keeps the weight and bias of its columns, and the
// next row is on its way while this one is summed.
// Waves of a SIMD that the registers are shared out to, and the workgroups that
// a CU then holds: a launch has no more, since a second round of workgroups
// that walk would leave most CUs idle.
constexpr int norm_waves(int waves, int ch) { return ch == 1 ? 8 : waves == 8 ? 6 : 4; }
constexpr int norm_threads(int waves) { return waves == 1 ? 256 : 64 * waves; }
constexpr int norm_groups(int waves, int ch) {
  return 256 * 4 * norm_waves(waves, ch) * 64 / norm_threads(waves);
}

template <typename El, typename W, int kWaves, int kCh, int kKind, bool kStream>
__global__ __launch_bounds__(norm_threads(kWaves), norm_waves(kWaves, kCh)) void
norm_kernel(NormArgs p) {
  constexpr int N = El::kN, kStep = 64 * kWaves;
  constexpr int kPer = kWaves == 1 ? 4 : 1;   // rows of a workgroup
  constexpr int kSums = kWaves == 8 && kCh == 2 ? 2 : 1;   // (see row_total)
  constexpr bool kPairs = kWaves == 16 && kCh == 1;
  __shared__ float red[2][kWaves];
  const int at = threadIdx.x % kStep;
  const bool second = __builtin_amdgcn_readfirstlane(threadIdx.x & -64) + kStep < p.row.chunks;
  const float over = 1.f / (float)p.H;
  const long long step = (long long)gridDim.x * kPer;
  long long t = (long long)blockIdx.x * kPer + (kPer > 1 ? threadIdx.x / kStep : 0);
  if (t >= p.T) return;   // (all waves of a row)
  uint4 raw[kCh];
  auto load = [&](long long row) __attribute__((always_inline)) {
    const uint8_t* src = p.x + row * p.row.bytes;
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = at + u * kStep;
      raw[u] = load_row<kKind, kStream>(src + p.row.start(c < p.row.chunks ? c : 0), p.row.bytes);
    }
  };
  load(t);
  float w[kCh][N], b[kCh][N];
  int lo[kCh], hi[kCh];   // the elements of a chunk that count
#pragma unroll
  for (int u = 0; u < kCh; ++u) {
    const int c = at + u * kStep;
    chunk_param<El, W, kKind>(p.w, p, c, 1.f, w[u]);
    chunk_param<El, W, kKind>(p.b, p, c, 0.f, b[u]);
    lo[u] = 0;
    hi[u] = N;
    if (kKind != kWholeRows) chunk_range<El>(p.row, c, lo[u], hi[u]);
    if (c >= p.row.chunks) hi[u] = 0;
  }
  // The row's end is among the lanes' last chunks, so that the others need no
  // mask: loose rows go without (8192 x 4099 bf16 29 us, with it 33, of spills).
  // Whole rows keep it: at the memory's rate they are slower without (65536 x
  // 7168 bf16 347 us, with it 333).
  auto whole = [&](int u) __attribute__((always_inline)) {
    return (kKind == kLooseRows && u < kCh - 1) || hi[u] - lo[u] == N;
  };
  for (; t < p.T; t += step) {
    float v[kCh][N];
#pragma unroll
    for (int u = 0; u < kCh; ++u) El::unpack(raw[u], v[u]);
    load(t + step < p.T ? t + step : t);
    // (all of a chunk, but for the lane with the row's end)
    float s[kSums] = {};
#pragma unroll
    for (int u = 0; u < kCh; ++u)
      if (whole(u)) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[u % kSums] += v[u][i];
      } else if (kKind != kWholeRows && hi[u]) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i >= lo[u] && i < hi[u]) s[u % kSums] += v[u][i];
      }
    // (divided: the mean of equal values is that value, and no product with a
    // rounded 1 / H that the subtraction below could be contracted with)
    const float mu = row_total<kWaves, kSums, kPairs>(s, second, red[0]) / (float)p.H;
#pragma unroll
    for (int u = 0; u < kSums; ++u) s[u] = 0.f;
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[u][i] -= mu;
      if (whole(u)) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[u % kSums] = fmaf(v[u][i], v[u][i], s[u % kSums]);
      } else if (kKind != kWholeRows && hi[u]) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i >= lo[u] && i < hi[u]) s[u % kSums] = fmaf(v[u][i], v[u][i], s[u % kSums]);
      }
    }
    const float r =
        1.f / sqrtf(fmaf(row_total<kWaves, kSums, kPairs>(s, second, red[1]), over, p.eps));
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = at + u * kStep;
#pragma unroll
      for (int i = 0; i < N; ++i) v[u][i] = fmaf(v[u][i] * r, w[u][i], b[u][i]);
      if (c < p.row.chunks)
        store_row<kKind>(p.y + t * p.row.bytes + p.row.start(c), p.row.bytes,
                         pack_row<El>(v[u]));
    }
    if (at == 0) {
      if (p.mean) p.mean[t] = mu;
      if (p.rstd) p.rstd[t] = r;
    }
  }
}

// Rows of any length, read again for each of their sums.  (8192 rows of 32768
// bf16 313 us, 3.4 TB/s; of 16384, in registers, 82, 6.6 TB/s.)
template <typename El, typename W>
__global__ __launch_bounds__(256) void norm_long_kernel(NormArgs p) {
  constexpr int N = El::kN;
  __shared__ float red[2][4][1];
  const float over = 1.f / (float)p.H;
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
    const uint8_t* src = p.x + t * p.row.bytes;
    auto sum = [&](float (*buffer)[1], auto f) __attribute__((always_inline)) {
      float s[1] = {0.f};
      for (int c = threadIdx.x; c < p.row.chunks; c += 256) {
        float e[N];
        El::unpack(load_chunk<false>(src + p.row.start(c), p.row.bytes), e);
        int lo, hi;
        chunk_range<El>(p.row, c, lo, hi);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i >= lo && i < hi) s[0] += f(e[i]);
      }
      row_add<4>(s, buffer);
      return s[0];
    };
    const float mu = sum(red[0], [](float e) { return e; }) / (float)p.H;
    const float var = sum(red[1], [&](float e) { return (e - mu) * (e - mu); }) * over;
    const float r = 1.f / sqrtf(var + p.eps);
    for (int c = threadIdx.x; c < p.row.chunks; c += 256) {
      float e[N], w[N], b[N];
      El::unpack(load_chunk<false>(src + p.row.start(c), p.row.bytes), e);
      chunk_param<El, W, kShortRows>(p.w, p, c, 1.f, w);
      chunk_param<El, W, kShortRows>(p.b, p, c, 0.f, b);
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = fmaf((e[i] - mu) * r, w[i], b[i]);
      store_chunk<false>(p.y + t * p.row.bytes + p.row.start(c), p.row.bytes, pack_row<El>(e));
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[t] = mu;
      if (p.rstd) p.rstd[t] = r;
    }
  }
}

// The gradient: a workgroup walks rows, kRows at a time, kWaves waves to a row,
// their lanes holding the same kCh chunks of every row, and so the sums over the
// rows of their columns.  The next row is on its way while this one is summed.
// (Rows of 64 chunks: 512 workgroups of one wave, one row at a time, left most
// of the memory idle: 65536 rows of 512 bf16 66 us.  Two chunks to a lane, rows
// of 16 to 32 KB, do not fit the registers of 16 waves in 16 bits: 8192 rows of
// 12288 bf16 201 us, 3.0 TB/s, of 16384 208, 3.9; of 8192 70, 5.7.)
template <typename El, typename W, int kRows, int kWaves, int kCh, int kKind, bool kStream>
__global__ __launch_bounds__(64 * kWaves * kRows) void norm_grad_kernel(NormArgs p) {
  constexpr int N = El::kN, kStep = 64 * kWaves;
  __shared__ float red[2][kRows * kWaves][2];
  __shared__ float joined[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? 2 * kCh * N : 1]
                         [kRows > 1 ? kStep : 1];
  const int at = threadIdx.x % kStep, part = threadIdx.x / kStep;
  const float over = 1.f / (float)p.H;
  uint4 raw_x[kCh], raw_g[kCh];
  float mu, r;
  auto load = [&](long long t) __attribute__((always_inline)) {
    if (t >= p.T) t = p.T - 1;
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = at + u * kStep;
      const long long off = t * p.row.bytes + p.row.start(c < p.row.chunks ? c : 0);
      raw_x[u] = load_row<kKind, kStream>(p.x + off, p.row.bytes);
      raw_g[u] = load_row<kKind, kStream>(p.dy + off, p.row.bytes);
    }
    mu = p.mean[t];
    r = p.rstd[t];
  };
  const long long step = (long long)gridDim.x * kRows;
  long long t = (long long)blockIdx.x * kRows + part;
  load(t);
  float w[kCh][N], dw[kCh][N], db[kCh][N];
  int lo[kCh], hi[kCh];   // the elements of a chunk that count
#pragma unroll
  for (int u = 0; u < kCh; ++u) {
    const int c = at + u * kStep;
    chunk_param<El, W, kKind>(p.w, p, c, 1.f, w[u]);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[u][i] = db[u][i] = 0.f;
    lo[u] = 0;
    hi[u] = N;
    if (kKind != kWholeRows) chunk_range<El>(p.row, c, lo[u], hi[u]);
    if (c >= p.row.chunks) hi[u] = 0;
  }
  int parity = 0;
  for (; t - part < p.T; t += step) {   // (the same for all of a workgroup's rows)
    const bool live = t < p.T;
    float z[kCh][N], g[kCh][N];
    const float rt = r, mut = mu;
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      El::unpack(raw_x[u], z[u]);
      El::unpack(raw_g[u], g[u]);
    }
    load(t + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[u][i] = (z[u][i] - mut) * rt;
      // (what does not count, in few waves: zeros)
      if (!live || hi[u] - lo[u] != N)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (!live || i < lo[u] || i >= hi[u]) g[u][i] = z[u][i] = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dw[u][i] = fmaf(g[u][i], z[u][i], dw[u][i]);
        db[u][i] += g[u][i];
        g[u][i] *= w[u][i];
        s[0] += g[u][i];
        s[1] = fmaf(g[u][i], z[u][i], s[1]);
      }
    }
    if (!p.y) continue;
    row_add<kWaves>(s, red[parity] + part * kWaves);
    parity ^= 1;
    const float c1 = s[0] * over, c2 = s[1] * over;
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = at + u * kStep;
      float d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = rt * (g[u][i] - c1 - z[u][i] * c2);
      if (c >= p.row.chunks || !live) continue;
      uint8_t* out = p.y + t * p.row.bytes + p.row.start(c);
      if (kKind == kWholeRows || lo[u] == 0) {
        store_row<kKind>(out, p.row.bytes, pack_row<El>(d));
      } else {
        // (the elements that the chunk before holds too were left out here)
        const uint4 v = pack_row<El>(d);
        alignas(16) uint8_t byte[16];
        __builtin_memcpy(byte, &v, 16);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i >= lo[u] * El::kSize) out[i] = byte[i];
      }
    }
  }
  if (!p.parts) return;
  if constexpr (kRows > 1) {
    if (part > 0)
#pragma unroll
      for (int u = 0; u < kCh; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          joined[part - 1][2 * (u * N + i)][at] = dw[u][i];
          joined[part - 1][2 * (u * N + i) + 1][at] = db[u][i];
        }
    __syncthreads();
    if (part > 0) return;
    for (int q = 0; q < kRows - 1; ++q)
#pragma unroll
      for (int u = 0; u < kCh; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dw[u][i] += joined[q][2 * (u * N + i)][at];
          db[u][i] += joined[q][2 * (u * N + i) + 1][at];
        }
  }
  float* out = p.parts + (size_t)blockIdx.x * 2 * p.H;
#pragma unroll
  for (int u = 0; u < kCh; ++u) {
    const int c = at + u * kStep;
    if (c >= p.row.chunks) continue;
    const int first = p.row.start(c) / El::kSize;
    if (kKind == kWholeRows) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        *reinterpret_cast<float4*>(out + first + i) =
            make_float4(dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]);
        *reinterpret_cast<float4*>(out + p.H + first + i) =
            make_float4(db[u][i], db[u][i + 1], db[u][i + 2], db[u][i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= lo[u] && i < hi[u]) {
          out[first + i] = dw[u][i];
          out[p.H + first + i] = db[u][i];
        }
    }
  }
}

// Rows too long for registers: their two sums first, then column by column.
// (8192 rows of 32768 bf16 574 us, 2.8 TB/s.)
template <typename El, typename W>
__global__ __launch_bounds__(256) void norm_grad_sums_kernel(NormArgs p) {
  constexpr int N = El::kN;
  __shared__ float red[2][4][2];
  int parity = 0;
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
    const float mu = p.mean[t], r = p.rstd[t];
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < p.row.chunks; c += 256) {
      const long long off = t * p.row.bytes + p.row.start(c);
      float x[N], g[N], w[N];
      El::unpack(load_chunk<false>(p.x + off, p.row.bytes), x);
      El::unpack(load_chunk<false>(p.dy + off, p.row.bytes), g);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = 1.f;
      if (p.w) load_param<W, N>(p.w, p.row.start(c) / El::kSize, N, w);
      int lo, hi;
      chunk_range<El>(p.row, c, lo, hi);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= lo && i < hi) {
          s[0] = fmaf(g[i], w[i], s[0]);
          s[1] = fmaf(g[i] * w[i], (x[i] - mu) * r, s[1]);
        }
    }
    row_add<4>(s, red[parity]);
    parity ^= 1;
    if (threadIdx.x == 0) {
      p.stats[2 * t] = s[0];
      p.stats[2 * t + 1] = s[1];
    }
  }
}

// grid (strips of 256 chunks, parts)
template <typename El, typename W>
__global__ __launch_bounds__(256) void norm_grad_strip_kernel(NormArgs p) {
  constexpr int N = El::kN;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.row.chunks) return;
  const float over = 1.f / (float)p.H;
  const int first = p.row.start(c) / El::kSize;
  int lo, hi;
  chunk_range<El>(p.row, c, lo, hi);
  float w[N], dw[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = 1.f, dw[i] = db[i] = 0.f;
  if (p.w) load_param<W, N>(p.w, first, N, w);
  for (long long t = blockIdx.y; t < p.T; t += gridDim.y) {
    const float mu = p.mean[t], r = p.rstd[t];
    const float c1 = p.stats ? p.stats[2 * t] * over : 0.f;
    const float c2 = p.stats ? p.stats[2 * t + 1] * over : 0.f;
    const long long off = t * p.row.bytes + p.row.start(c);
    float x[N], g[N];
    El::unpack(load_chunk<false>(p.x + off, p.row.bytes), x);
    El::unpack(load_chunk<false>(p.dy + off, p.row.bytes), g);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = (x[i] - mu) * r;
      dw[i] = fmaf(g[i], z, dw[i]);
      db[i] += g[i];
      g[i] = r * (g[i] * w[i] - c1 - z * c2);
    }
    if (p.y) store_chunk<false>(p.y + off, p.row.bytes, pack_row<El>(g));
  }
  if (!p.parts) return;
  float* out = p.parts + (size_t)blockIdx.y * 2 * p.H;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i >= lo && i < hi) {
      out[first + i] = dw[i];
      out[p.H + first + i] = db[i];
    }
}

// dw and db from the partial sums: 32 columns to a workgroup, four to a lane;
// its 32 groups of eight lanes each add every 32nd part, in order, and their
// sums are added in order too.
template <typename W, bool kWide>
__global__ __launch_bounds__(256) void norm_join_kernel(const float* __restrict__ parts, int n,
                                                        int H, uint8_t* __restrict__ dw,
                                                        uint8_t* __restrict__ db) {
  __shared__ float red[32][33];
  const int col = (threadIdx.x & 7) * 4, group = threadIdx.x >> 3;
  const long long all = 2LL * H;
  const long long j = (long long)blockIdx.x * 32 + col;   // dw's columns, then db's
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (j < all) {
#pragma unroll 8
    for (int i = group; i < n; i += 32) {
      const float* p = parts + i * all + j;
      if (kWide) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] += j + u < all ? p[u] : 0.f;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) red[group][col + u] = s[u];
  __syncthreads();
  if (threadIdx.x >= 32) return;
  float sum = red[0][threadIdx.x];
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += red[i][threadIdx.x];
  const long long at = (long long)blockIdx.x * 32 + threadIdx.x;
  if (at >= all) return;
  uint8_t* out = at < H ? dw : db;
  if (!out) return;
  float v[W::kN] = {sum};
  const uint4 c = W::pack(v);
  __builtin_memcpy(out + (at < H ? at : at - H) * W::kSize, &c, W::kSize);
}

static int norm_type_size(int dtype) {
  return dtype == MOE_TYPE_F32 ? 4 : dtype == MOE_TYPE_BF16 || dtype == MOE_TYPE_F16 ? 2 : 0;
}

static moe_status_t norm_args(int dtype, int w_dtype, int T, int H, RowShape* row) {
  const int es = norm_type_size(dtype);
  if (es == 0 || norm_type_size(w_dtype) == 0) return MOE_INVALID_ARG;
  if (w_dtype != dtype && w_dtype != MOE_TYPE_F32) return MOE_INVALID_ARG;
  if (T < 0 || H <= 0) return MOE_INVALID_ARG;
  if ((long long)H * es > 0x7fffffffLL - 64) return MOE_UNSUPPORTED_SHAPE;
  row->bytes = H * es;
  row->chunks = (row->bytes + 15) / 16;
  return MOE_OK;
}

// f(El(), W()) for the rows' type and the weights'.
template <typename F>
static void by_type(int dtype, int w_dtype, F f) {
  if (dtype == MOE_TYPE_F32)
    f(F32(), F32());
  else if (dtype == MOE_TYPE_BF16 && w_dtype == MOE_TYPE_F32)
    f(BF16(), F32());
  else if (dtype == MOE_TYPE_BF16)
    f(BF16(), BF16());
  else if (w_dtype == MOE_TYPE_F32)
    f(F16(), F32());
  else
    f(F16(), F16());
}

static bool whole_rows(const NormArgs& p) {
  return p.row.bytes % 16 == 0 &&
         (((uintptr_t)p.x | (uintptr_t)p.dy | (uintptr_t)p.y) & 15) == 0;
}

static unsigned walk(long long n) {
  return (unsigned)(n < 1 ? 1 : n > (1 << 22) ? (1 << 22) : n);
}

// Reads past the caches where they are more than the memory-side cache (256
// MB) keeps: 65536 rows of 7168 bf16 343 us against 352, the gradient of 32768
// 270 against 279; but 65536 rows of 2048 96 against 88.
static bool norm_streams(const NormArgs& p) {
  return (long long)p.T * p.row.bytes * (p.dy ? 2 : 1) > (400LL << 20);
}

template <typename El, typename W, int kWaves, int kCh, int kKind>
static void launch_norm_as(const NormArgs& p, hipStream_t st) {
  constexpr long long most = norm_groups(kWaves, kCh);
  constexpr int kPer = kWaves == 1 ? 4 : 1;
  const long long blocks = ((long long)p.T + kPer - 1) / kPer;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(norm_threads(kWaves));
  if (norm_streams(p))
    hipLaunchKernelGGL((norm_kernel<El, W, kWaves, kCh, kKind, true>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((norm_kernel<El, W, kWaves, kCh, kKind, false>), grid, block, 0, st, p);
}

template <typename El, typename W, int kKind>
static void launch_norm(const NormArgs& p, hipStream_t st) {
  const int c = p.row.chunks;
  if (p.row.bytes > kNormLong)
    hipLaunchKernelGGL((norm_long_kernel<El, W>), dim3(walk(p.T)), dim3(256), 0, st, p);
  else if (kKind == kShortRows || c <= 64)   // (a short row is one chunk)
    launch_norm_as<El, W, 1, 1, kKind>(p, st);
  else if constexpr (kKind == kShortRows)
    return;
  else if (c <= 128)
    launch_norm_as<El, W, 2, 1, kKind>(p, st);
  else if (c <= 256)
    launch_norm_as<El, W, 4, 1, kKind>(p, st);
  else if (c <= 512)
    launch_norm_as<El, W, 8, 1, kKind>(p, st);
  // (few rows: one as fast as it goes; us for rows of 7168 bf16, 16 waves to a
  // row and 8: 1 row 3.0 and 3.6, 512 5.1 and 5.5, 2048 11.1 and 10.6, 8192 40.6
  // and 38.2)
  else if (c <= 1024 && p.T <= 512)
    launch_norm_as<El, W, 16, 1, kKind>(p, st);
  else if (c <= 1024)
    launch_norm_as<El, W, 8, 2, kKind>(p, st);
  else
    launch_norm_as<El, W, 16, 2, kKind>(p, st);
}

template <typename El, typename W, int kRows, int kWaves, int kCh, int kKind>
static void launch_norm_grad_as(const NormArgs& p, int parts, hipStream_t st) {
  const dim3 grid((unsigned)parts), block(64 * kWaves * kRows);
  if (norm_streams(p))
    hipLaunchKernelGGL((norm_grad_kernel<El, W, kRows, kWaves, kCh, kKind, true>), grid, block, 0,
                       st, p);
  else
    hipLaunchKernelGGL((norm_grad_kernel<El, W, kRows, kWaves, kCh, kKind, false>), grid, block,
                       0, st, p);
}

// Workgroups with partial sums: as many as the CUs hold at once, each with
// enough rows to be worth its sums.
static int norm_parts(const NormArgs& p) {
  const long long least = (long long)p.T / kNormRows + (p.T % kNormRows != 0);
  const int most = p.row.chunks > 512 ? kNormParts / 2 : kNormParts;
  return (int)(least < most ? least : most);
}

template <typename El, typename W, int kKind>
static void launch_norm_grad(const NormArgs& p, int parts, hipStream_t st) {
  const int c = p.row.chunks;
  if (kKind == kShortRows || c <= 64)
    launch_norm_grad_as<El, W, 8, 1, 1, kKind>(p, parts, st);
  else if constexpr (kKind == kShortRows)
    return;
  else if (c <= 128)
    launch_norm_grad_as<El, W, 4, 2, 1, kKind>(p, parts, st);
  else if (c <= 256)
    launch_norm_grad_as<El, W, 2, 4, 1, kKind>(p, parts, st);
  else if (c <= 512)
    launch_norm_grad_as<El, W, 1, 8, 1, kKind>(p, parts, st);
  else if (c <= 1024)
    launch_norm_grad_as<El, W, 1, 16, 1, kKind>(p, parts, st);
  else
    launch_norm_grad_as<El, W, 1, 16, 2, kKind>(p, parts, st);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_layer_norm(const void* x, int dtype, int T, int H, const void* weight,
                                       const void* bias, int w_dtype, float eps, void* y,
                                       float* mean, float* rstd, void* stream) {
  NormArgs p{};
  const moe_status_t ok = norm_args(dtype, w_dtype, T, H, &p.row);
  if (ok != MOE_OK) return ok;
  if (!(eps >= 0.f)) return MOE_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !y) return MOE_INVALID_ARG;
  if ((((uintptr_t)x | (uintptr_t)y) & (norm_type_size(dtype) - 1)) ||
      (((uintptr_t)weight | (uintptr_t)bias) & (norm_type_size(w_dtype) - 1)) ||
      (((uintptr_t)mean | (uintptr_t)rstd) & 3))
    return MOE_UNSUPPORTED_SHAPE;
  p.x = static_cast<const uint8_t*>(x);
  p.w = static_cast<const uint8_t*>(weight);
  p.b = static_cast<const uint8_t*>(bias);
  p.T = T;
  p.H = H;
  p.eps = eps;
  p.y = static_cast<uint8_t*>(y);
  p.mean = mean;
  p.rstd = rstd;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  by_type(dtype, w_dtype, [&](auto el, auto w) {
    if (p.row.bytes < 16)
      launch_norm<decltype(el), decltype(w), kShortRows>(p, st);
    else if (whole_rows(p))
      launch_norm<decltype(el), decltype(w), kWholeRows>(p, st);
    else
      launch_norm<decltype(el), decltype(w), kLooseRows>(p, st);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

// Partial sums of the gradients of w and b, then (rows that are too long for
// registers in some type) two sums per row.
extern "C" size_t moe_layer_norm_workspace_bytes(int T, int H) {
  if (T < 0 || H <= 0) return 0;
  const size_t parts = T < kNormParts ? T : kNormParts;
  return parts * 2 * (size_t)H * sizeof(float) +
         (H > kNormLong / 4 ? (size_t)T * 2 * sizeof(float) : 0);
}

extern "C" moe_status_t moe_layer_norm_grad(const void* dy, const void* x, int dtype, int T, int H,
                                            const void* weight, int w_dtype, const float* mean,
                                            const float* rstd, void* dx, void* dweight,
                                            void* dbias, void* workspace, size_t workspace_bytes,
                                            void* stream) {
  NormArgs p{};
  const moe_status_t ok = norm_args(dtype, w_dtype, T, H, &p.row);
  if (ok != MOE_OK) return ok;
  const bool params = dweight || dbias;
  if (!dx && !params) return T == 0 ? MOE_OK : MOE_INVALID_ARG;
  // (the joining launch has 256 threads to 32 columns of both gradients)
  if (params && (2LL * H + 31) / 32 * 256 > 0xffffffffLL) return MOE_UNSUPPORTED_SHAPE;
  if (T > 0 && (!dy || !x || !mean || !rstd)) return MOE_INVALID_ARG;
  const bool is_long = p.row.bytes > kNormLong;
  if (T > 0 && (params || is_long) &&
      (!workspace || workspace_bytes < moe_layer_norm_workspace_bytes(T, H)))
    return MOE_INVALID_ARG;
  if ((((uintptr_t)dy | (uintptr_t)x | (uintptr_t)dx) & (norm_type_size(dtype) - 1)) ||
      (((uintptr_t)weight | (uintptr_t)dweight | (uintptr_t)dbias) &
       (norm_type_size(w_dtype) - 1)) ||
      (((uintptr_t)mean | (uintptr_t)rstd) & 3) || ((uintptr_t)workspace & 15))
    return MOE_UNSUPPORTED_SHAPE;
  if (T == 0 && !params) return MOE_OK;
  p.x = static_cast<const uint8_t*>(x);
  p.dy = static_cast<const uint8_t*>(dy);
  p.w = static_cast<const uint8_t*>(weight);
  p.T = T;
  p.H = H;
  const int parts = norm_parts(p);
  p.y = static_cast<uint8_t*>(dx);
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  float* ws = static_cast<float*>(workspace);
  p.parts = params ? ws : nullptr;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (T > 0 && is_long) {
    p.stats = dx ? ws + (size_t)parts * 2 * H : nullptr;
    by_type(dtype, w_dtype, [&](auto el, auto w) {
      using El = decltype(el);
      using W = decltype(w);
      if (dx)
        hipLaunchKernelGGL((norm_grad_sums_kernel<El, W>), dim3(walk(T)), dim3(256), 0, st, p);
      hipLaunchKernelGGL((norm_grad_strip_kernel<El, W>),
                         dim3((unsigned)((p.row.chunks + 255) / 256), (unsigned)parts), dim3(256),
                         0, st, p);
    });
  } else if (T > 0) {
    by_type(dtype, w_dtype, [&](auto el, auto w) {
      if (p.row.bytes < 16)
        launch_norm_grad<decltype(el), decltype(w), kShortRows>(p, parts, st);
      else if (whole_rows(p))
        launch_norm_grad<decltype(el), decltype(w), kWholeRows>(p, parts, st);
      else
        launch_norm_grad<decltype(el), decltype(w), kLooseRows>(p, parts, st);
    });
  }
  if (params) {
    const dim3 grid((unsigned)((2LL * H + 31) / 32));
    uint8_t* dw = static_cast<uint8_t*>(dweight);
    uint8_t* db = static_cast<uint8_t*>(dbias);
    by_type(w_dtype, w_dtype, [&](auto el, auto) {
      if (H % 2 == 0)
        hipLaunchKernelGGL((norm_join_kernel<decltype(el), true>), grid, dim3(256), 0, st, ws,
                           parts, H, dw, db);
      else
        hipLaunchKernelGGL((norm_join_kernel<decltype(el), false>), grid, dim3(256), 0, st, ws,
                           parts, H, dw, db);
    });
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}
