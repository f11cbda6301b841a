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
// waves) the waves in order.  Nothing is added with atomics: the gradients of
// w and b are kept by column in each workgroup's registers over all the rows
// that it walks, written once as partial sums, and joined by a second kernel
// in the order of the workgroups.  Bound by HBM bandwidth.
#include "row_chunks.hpp"

namespace moe {

constexpr int kNormParts = 512;     // workgroups that keep partial sums, at most
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

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The sums of the kWaves waves that share a row, in every lane of them.
template <int kWaves, int kN>
__device__ __forceinline__ void row_add(float (&v)[kN], float (*red)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = wave_add(v[i]);
  if constexpr (kWaves > 1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();   // the last sum has been read
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

// The elements of chunk c that count: [lo, hi) of its El::kN (a last chunk
// overlaps the one before it, a row shorter than a chunk ends inside it).
template <typename El>
__device__ __forceinline__ void chunk_range(const RowShape& row, int c, int& lo, int& hi) {
  lo = (16 * c - row.start(c)) / El::kSize;
  hi = row.bytes >= 16 ? El::kN : row.bytes / El::kSize;
}

// y of a chunk.
template <typename El, typename W, bool kWhole>
__device__ __forceinline__ void norm_store(const NormArgs& p, long long t, int c, float mu, float r,
                                           float (&v)[El::kN]) {
  constexpr int N = El::kN;
  const int at = p.row.start(c) / El::kSize;
  const int n = kWhole ? N : min(N, p.H - at);
  float w[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = 1.f, b[i] = 0.f;
  if (p.w) load_param<W, N>(p.w, at, n, w);
  if (p.b) load_param<W, N>(p.b, at, n, b);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = fmaf((v[i] - mu) * r, w[i], b[i]);
  store_chunk<kWhole>(p.y + t * p.row.bytes + p.row.start(c), p.row.bytes, El::pack(v));
}

// kWaves waves to a row, which its lanes hold in kCh chunks each; kCh 0: a row
// of any length, read again for each of its sums.
template <typename El, typename W, int kWaves, int kCh, bool kWhole>
__global__ __launch_bounds__(kWaves > 4 ? 64 * kWaves : 256) void norm_kernel(NormArgs p) {
  constexpr int N = El::kN, kStep = 64 * kWaves;
  constexpr int kPer = kWaves >= 4 ? 1 : 4 / kWaves;   // rows of a workgroup
  __shared__ float red[kWaves][1];
  const int at = threadIdx.x % kStep;
  const float over = 1.f / (float)p.H;
  for (long long t0 = (long long)blockIdx.x * kPer; t0 < p.T; t0 += (long long)gridDim.x * kPer) {
    const long long t = t0 + (kPer > 1 ? threadIdx.x / kStep : 0);
    if (kPer > 1 && t >= p.T) continue;   // (a wave of its own)
    const uint8_t* src = p.x + t * p.row.bytes;
    float v[kCh ? kCh : 1][N];
    auto load = [&](int c, float (&f)[N]) {
      El::unpack(load_chunk<kWhole>(src + p.row.start(c < p.row.chunks ? c : 0), p.row.bytes), f);
    };
    auto each = [&](auto f) __attribute__((always_inline)) {
      if constexpr (kCh != 0) {
#pragma unroll
        for (int u = 0; u < kCh; ++u) f(at + u * kStep, v[u]);
      } else {
        for (int c = at; c < p.row.chunks; c += kStep) {
          load(c, v[0]);
          f(c, v[0]);
        }
      }
    };
    // the sum of f over the row's elements, each once
    auto sum = [&](auto f) __attribute__((always_inline)) {
      float s[1] = {0.f};
      each([&](int c, float (&e)[N]) {
        int lo = 0, hi = N;
        if (!kWhole) chunk_range<El>(p.row, c, lo, hi);
        if (c < p.row.chunks)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (kWhole || (i >= lo && i < hi)) s[0] += f(e[i]);
      });
      row_add<kWaves>(s, red);
      return s[0];
    };
    if constexpr (kCh != 0)
#pragma unroll
      for (int u = 0; u < kCh; ++u) load(at + u * kStep, v[u]);
    const float mu = sum([](float e) { return e; }) * over;
    const float var = sum([&](float e) { return (e - mu) * (e - mu); }) * over;
    const float r = 1.f / sqrtf(var + p.eps);
    each([&](int c, float (&e)[N]) {
      if (c < p.row.chunks) norm_store<El, W, kWhole>(p, t, c, mu, r, e);
    });
    if (at == 0) {
      if (p.mean) p.mean[t] = mu;
      if (p.rstd) p.rstd[t] = r;
    }
  }
}

// The gradient: a workgroup of kWaves waves walks rows, its lanes holding the
// same kCh chunks of every row, and so the sums over the rows of their
// columns.
template <typename El, typename W, int kWaves, int kCh, bool kWhole>
__global__ __launch_bounds__(64 * kWaves) void norm_grad_kernel(NormArgs p) {
  constexpr int N = El::kN, kStep = 64 * kWaves;
  __shared__ float red[kWaves][2];
  const int at = threadIdx.x;
  const float over = 1.f / (float)p.H;
  float dw[kCh][N], db[kCh][N];
#pragma unroll
  for (int u = 0; u < kCh; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[u][i] = db[u][i] = 0.f;
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
    const float mu = p.mean[t], r = p.rstd[t];
    float z[kCh][N], g[kCh][N];
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = at + u * kStep;
      const long long off = t * p.row.bytes + p.row.start(c < p.row.chunks ? c : 0);
      El::unpack(load_chunk<kWhole>(p.x + off, p.row.bytes), z[u]);
      El::unpack(load_chunk<kWhole>(p.dy + off, p.row.bytes), g[u]);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = at + u * kStep;
      int lo = 0, hi = N;
      if (!kWhole) chunk_range<El>(p.row, c, lo, hi);
      if (c >= p.row.chunks) hi = 0;
      const int first = p.row.start(c < p.row.chunks ? c : 0) / El::kSize;
      float w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = 1.f;
      if (p.w) load_param<W, N>(p.w, first, kWhole ? N : min(N, p.H - first), w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool in = kWhole ? hi != 0 : i >= lo && i < hi;
        z[u][i] = (z[u][i] - mu) * r;
        if (in) {
          dw[u][i] = fmaf(g[u][i], z[u][i], dw[u][i]);
          db[u][i] += g[u][i];
        }
        g[u][i] *= w[i];
        if (in) {
          s[0] += g[u][i];
          s[1] = fmaf(g[u][i], z[u][i], s[1]);
        }
      }
    }
    if (p.y) {
      row_add<kWaves>(s, red);
      const float c1 = s[0] * over, c2 = s[1] * over;
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        const int c = at + u * kStep;
        float d[N];
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = r * (g[u][i] - c1 - z[u][i] * c2);
        if (c < p.row.chunks)
          store_chunk<kWhole>(p.y + t * p.row.bytes + p.row.start(c), p.row.bytes, El::pack(d));
      }
    }
  }
  if (!p.parts) return;
  float* out = p.parts + (size_t)blockIdx.x * 2 * p.H;
#pragma unroll
  for (int u = 0; u < kCh; ++u) {
    const int c = at + u * kStep;
    if (c >= p.row.chunks) continue;
    int lo = 0, hi = N;
    if (!kWhole) chunk_range<El>(p.row, c, lo, hi);
    const int first = p.row.start(c) / El::kSize;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (kWhole || (i >= lo && i < hi)) {
        out[first + i] = dw[u][i];
        out[p.H + first + i] = db[u][i];
      }
  }
}

// Rows too long for registers: their two sums first, then column by column.
template <typename El, typename W>
__global__ __launch_bounds__(256) void norm_grad_sums_kernel(NormArgs p) {
  constexpr int N = El::kN;
  __shared__ float red[4][2];
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
    row_add<4>(s, red);
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
    if (p.y) store_chunk<false>(p.y + off, p.row.bytes, El::pack(g));
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

// dw and db from the partial sums: 32 columns to a workgroup, whose eight
// groups of 32 lanes each add every eighth part, in order.
template <typename W>
__global__ __launch_bounds__(256) void norm_join_kernel(const float* __restrict__ parts, int n,
                                                        int H, uint8_t* __restrict__ dw,
                                                        uint8_t* __restrict__ db) {
  __shared__ float red[8][32];
  const int col = threadIdx.x & 31, group = threadIdx.x >> 5;
  const long long all = 2LL * H;
  const long long j = (long long)blockIdx.x * 32 + col;   // dw's columns, then db's
  float s = 0.f;
  if (j < all)
    for (int i = group; i < n; i += 8) s += parts[i * all + j];
  red[group][col] = s;
  __syncthreads();
  if (group != 0 || j >= all) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += red[i][col];
  uint8_t* out = j < H ? dw : db;
  if (!out) return;
  float v[W::kN] = {s};
  const uint4 c = W::pack(v);
  __builtin_memcpy(out + (j < H ? j : j - H) * W::kSize, &c, W::kSize);
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

template <typename El, typename W, bool kWhole>
static void launch_norm(const NormArgs& p, hipStream_t st) {
  const int c = p.row.chunks;
  if (c <= 64)
    hipLaunchKernelGGL((norm_kernel<El, W, 1, 1, kWhole>), dim3(walk((p.T + 3LL) / 4)), dim3(256),
                       0, st, p);
  else if (c <= 256)
    hipLaunchKernelGGL((norm_kernel<El, W, 4, 1, kWhole>), dim3(walk(p.T)), dim3(256), 0, st, p);
  else if (c <= 1024)
    hipLaunchKernelGGL((norm_kernel<El, W, 4, 4, kWhole>), dim3(walk(p.T)), dim3(256), 0, st, p);
  else if (p.row.bytes <= kNormLong)
    hipLaunchKernelGGL((norm_kernel<El, W, 16, 2, kWhole>), dim3(walk(p.T)), dim3(1024), 0, st, p);
  else
    hipLaunchKernelGGL((norm_kernel<El, W, 4, 0, kWhole>), dim3(walk(p.T)), dim3(256), 0, st, p);
}

template <typename El, typename W, bool kWhole>
static void launch_norm_grad(const NormArgs& p, int parts, hipStream_t st) {
  const int c = p.row.chunks;
  const dim3 grid((unsigned)parts);
  if (c <= 64)
    hipLaunchKernelGGL((norm_grad_kernel<El, W, 1, 1, kWhole>), grid, dim3(64), 0, st, p);
  else if (c <= 256)
    hipLaunchKernelGGL((norm_grad_kernel<El, W, 4, 1, kWhole>), grid, dim3(256), 0, st, p);
  else if (c <= 512)
    hipLaunchKernelGGL((norm_grad_kernel<El, W, 8, 1, kWhole>), grid, dim3(512), 0, st, p);
  else if (c <= 1024)
    hipLaunchKernelGGL((norm_grad_kernel<El, W, 8, 2, kWhole>), grid, dim3(512), 0, st, p);
  else
    hipLaunchKernelGGL((norm_grad_kernel<El, W, 16, 2, kWhole>), grid, dim3(1024), 0, st, p);
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
    if (whole_rows(p))
      launch_norm<decltype(el), decltype(w), true>(p, st);
    else
      launch_norm<decltype(el), decltype(w), false>(p, st);
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
  const int parts = T < kNormParts ? T : kNormParts;
  p.x = static_cast<const uint8_t*>(x);
  p.dy = static_cast<const uint8_t*>(dy);
  p.w = static_cast<const uint8_t*>(weight);
  p.T = T;
  p.H = H;
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
      if (whole_rows(p))
        launch_norm_grad<decltype(el), decltype(w), true>(p, parts, st);
      else
        launch_norm_grad<decltype(el), decltype(w), false>(p, parts, st);
    });
  }
  if (params) {
    const dim3 grid((unsigned)((2LL * H + 31) / 32));
    uint8_t* dw = static_cast<uint8_t*>(dweight);
    uint8_t* db = static_cast<uint8_t*>(dbias);
    by_type(w_dtype, w_dtype, [&](auto el, auto) {
      hipLaunchKernelGGL((norm_join_kernel<decltype(el)>), grid, dim3(256), 0, st, ws, parts, H,
                         dw, db);
    });
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}
