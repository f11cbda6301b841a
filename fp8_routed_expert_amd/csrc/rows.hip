// Rows sorted by expert and back, with their gradients, in 32-, 16- and 8-bit
// types: the row movement of the dispatch and the weighted sum of the combine
// for layers that are trained or that keep their activations in other types
// than FP8 (whose own calls are moe_dispatch_layout and moe_combine).
//
//   permute          a[slot(t, k)] = x[t]
//   permute, grad    dx[t] = sum_k da[slot(t, k)]
//   combine          out[t] = sum_k w[t, k] y[slot(t, k)]
//   combine, grad    dy[slot(t, k)] = w[t, k] dout[t]
//                    dw[t, k] = <dout[t], y[slot(t, k)]>
//
// All four walk the source tokens: a token's row is read or written once, and
// each of its slots' rows once, so a call moves every byte it has to and no
// other; sums are gathers in ascending k, held in fp32, with no atomics, so a
// call's result does not depend on its schedule.  Bound by HBM bandwidth.
#include <type_traits>

#include "row_chunks.hpp"

namespace moe {

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;

// How a row is shared out: a wave (kLanes 64) takes a piece of at most 64
// kCh chunks, or each of its four groups of 16 lanes a whole short row.
//
// The token's picks: lane k of the wave or group holds pick k's slot.  valid
// is a bit mask of those that are rows; every lane of the group has the same.
template <int kLanes>
struct Picks {
  int s;
  unsigned long long valid;
  bool bad;   // a slot past the buffer
  int base;   // the group's first lane
  __device__ __forceinline__ Picks(const int32_t* slot_of, long long t, int K, int rows_total,
                                   bool live) {
    const int lane = threadIdx.x & 63, at = lane % kLanes;
    base = lane - at;
    s = live && at < K ? slot_of[t * K + at] : -1;
    unsigned long long b = __ballot(s >= rows_total);
    valid = __ballot(s >= 0 && s < rows_total);
    if (kLanes < 64) {
      constexpr unsigned long long kMask = (1ull << (kLanes & 63)) - 1;
      valid = (valid >> base) & kMask;
      b = (b >> base) & kMask;
    }
    bad = b != 0;
  }
  // the value that pick k's lane holds
  __device__ __forceinline__ int of(int v, int k) const {
    return kLanes == 64 ? __builtin_amdgcn_readlane(v, k) : __shfl(v, base + k);
  }
  __device__ __forceinline__ float of(float v, int k) const {
    return __int_as_float(of(__float_as_int(v), k));
  }
};

// Rows of the buffer that no token goes to are set to zero: one wave per 64
// rows reads their sources and clears those without one, row after row (12-17 us
// where nearly all 64 are empty: 777 x 3 picks of 509 fp32, the gradient with
// the clearing 22.0 us, without 5.4).
__device__ __forceinline__ void zero_rows(long long w, const int32_t* __restrict__ row_src,
                                          int rows_total, long long row_bytes, uint8_t* a) {
  const int lane = threadIdx.x & 63;
  const long long r0 = w * 64;
  const long long r = r0 + lane;
  unsigned long long m = __ballot(r < rows_total && row_src[r < rows_total ? r : 0] < 0);
  while (m) {
    const int i = __ffsll((long long)m) - 1;
    m &= m - 1;
    uint8_t* p = a + (r0 + i) * row_bytes;
    // the row's 16-byte aligned part by 16, its ends byte by byte
    const long long head = min((long long)((16 - ((uintptr_t)p & 15)) & 15), row_bytes);
    const long long mid = (row_bytes - head) / 16;
    for (long long c = lane; c < mid; c += 64)
      reinterpret_cast<uint4*>(p + head)[c] = make_uint4(0, 0, 0, 0);
    if (lane < head) p[lane] = 0;
    const long long tail = head + mid * 16 + lane;
    if (lane < 16 && tail < row_bytes) p[tail] = 0;
  }
}

template <int kLanes, int kCh, bool kAligned>
__global__ __launch_bounds__(kRowThreads) void permute_rows_kernel(
    const uint8_t* __restrict__ x, const int32_t* __restrict__ slot_of, int T, int K,
    RowShape row, int pieces, int plen, int rows_total, uint8_t* __restrict__ a,
    const int32_t* __restrict__ row_src, long long zero_waves, int32_t* __restrict__ status) {
  constexpr int kGroups = 64 / kLanes;   // rows of a wave
  const int at = threadIdx.x & (kLanes - 1);
  const long long units = zero_waves + ((long long)T * pieces + kGroups - 1) / kGroups;
  for (long long w = (long long)blockIdx.x * kRowWaves + (threadIdx.x >> 6); w < units;
       w += (long long)gridDim.x * kRowWaves) {
    if (w < zero_waves) {
      zero_rows(w, row_src, rows_total, row.bytes, a);
      continue;
    }
    const long long u0 = (w - zero_waves) * kGroups + (threadIdx.x & 63) / kLanes;
    const bool live = kLanes == 64 || u0 < T;
    const long long t = live ? u0 / pieces : 0;
    const int c0 = kLanes == 64 ? (int)(u0 - t * pieces) * plen : 0;
    const int cend = min(c0 + plen, row.chunks);
    const Picks<kLanes> picks(slot_of, t, K, rows_total, live);
    if (picks.bad && at == 0 && c0 == 0) atomicOr(status, MOE_ERR_BAD_INDEX);
    const uint8_t* src = x + t * (long long)row.bytes;
    uint4 v[kCh];
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = c0 + at + u * kLanes;
      v[u] = load_chunk<kAligned>(src + row.start(c < cend ? c : c0), row.bytes);
    }
    for (unsigned long long m = picks.valid; m; m &= m - 1) {
      const int k = __ffsll((long long)m) - 1;
      uint8_t* dst = a + (long long)picks.of(picks.s, k) * row.bytes;
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        const int c = c0 + at + u * kLanes;
        if (c < cend) store_chunk<kAligned>(dst + row.start(c), row.bytes, v[u]);
      }
    }
  }
}

// out[t] = sum over the valid picks, in ascending k, of (w[t, k] *) y[slot]:
// the combine, and (kWeighted false) the gradient of the permute.  Rows are
// taken in pairs, but only the combine in fp16 and fp32 (aligned rows, a wave
// each) has both rows' loads in flight: in bf16, and in the permute's gradient
// in every type, the compiler moves the first row's conversion (fp32: its
// addition) ahead of the second load, and so waits for one row at a time.
template <typename El, int kLanes, int kCh, bool kAligned, bool kStream, bool kWeighted>
__global__ __launch_bounds__(kRowThreads) void gather_sum_kernel(
    const uint8_t* __restrict__ y, int rows_total, const int32_t* __restrict__ slot_of,
    const float* __restrict__ topk_w, int T, int K, RowShape row, int pieces, int plen,
    uint8_t* __restrict__ out, int32_t* __restrict__ status) {
  constexpr int N = El::kN;
  constexpr int kGroups = 64 / kLanes;
  const int at = threadIdx.x & (kLanes - 1);
  const long long units = ((long long)T * pieces + kGroups - 1) / kGroups;
  for (long long w = (long long)blockIdx.x * kRowWaves + (threadIdx.x >> 6); w < units;
       w += (long long)gridDim.x * kRowWaves) {
    const long long u0 = w * kGroups + (threadIdx.x & 63) / kLanes;
    const bool live = kLanes == 64 || u0 < T;
    const long long t = live ? u0 / pieces : 0;
    const int c0 = kLanes == 64 ? (int)(u0 - t * pieces) * plen : 0;
    const int cend = min(c0 + plen, row.chunks);
    const Picks<kLanes> picks(slot_of, t, K, rows_total, live);
    const float wt = kWeighted && live && at < K ? topk_w[t * K + at] : 1.f;
    if (picks.bad && at == 0 && c0 == 0) atomicOr(status, MOE_ERR_BAD_INDEX);
    float acc[kCh][N];
#pragma unroll
    for (int u = 0; u < kCh; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[u][i] = 0.f;
    auto load = [&](int k, uint4 (&v)[kCh]) {
      const uint8_t* src = y + (long long)picks.of(picks.s, k) * row.bytes;
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        const int c = c0 + at + u * kLanes;
        v[u] = load_chunk<kAligned, kStream>(src + row.start(c < cend ? c : c0), row.bytes);
      }
    };
    auto add = [&](int k, const uint4 (&v)[kCh]) {
      const float wk = picks.of(wt, k);
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        float f[N];
        El::unpack(v[u], f);
#pragma unroll
        for (int i = 0; i < N; ++i)
          acc[u][i] = kWeighted ? fmaf(wk, f[i], acc[u][i]) : acc[u][i] + f[i];
      }
    };
    unsigned long long m = picks.valid;
    while (m) {
      const int k0 = __ffsll((long long)m) - 1;
      m &= m - 1;
      uint4 v0[kCh], v1[kCh];
      load(k0, v0);
      if (m) {
        const int k1 = __ffsll((long long)m) - 1;
        m &= m - 1;
        load(k1, v1);
        add(k0, v0);
        add(k1, v1);
      } else {
        add(k0, v0);
      }
    }
    uint8_t* dst = out + t * (long long)row.bytes;
#pragma unroll
    for (int u = 0; u < kCh; ++u) {
      const int c = c0 + at + u * kLanes;
      if (c < cend && live) store_chunk<kAligned>(dst + row.start(c), row.bytes, El::pack(acc[u]));
    }
  }
}

// Sum over the kLanes lanes of a group, in every one of them.
template <int kLanes>
__device__ __forceinline__ float group_sum(float d) {
#pragma unroll
  for (int o = kLanes / 2; o >= 1; o >>= 1) d += __shfl_xor(d, o);
  return d;
}

// Gradient of the combine: a token's dout row is read once and its chunks kept
// in registers; each of its y rows is read and its dy row written in the same
// pass.  A lane's products of a row are summed first, then its group's lanes,
// then (kBlock: the workgroup's waves share a token) the waves in order: no
// atomics.  Rows longer than the registers hold are walked in parts.
//
// Few chunks per lane leave room for many waves, which is what keeps the
// memory busy (a prefill share, 5.0 GB: 925 us with 512 threads of one chunk,
// 955 with 256 of two, 1014 with 256 of four; two rows' loads in flight
// 945-965).  Unaligned rows took 280 us with 256 threads of two chunks against
// 356.
constexpr int grad_threads(bool block, bool aligned) { return block && aligned ? 512 : 256; }

template <typename El, int kLanes, bool kBlock, bool kAligned, bool kStream>
__global__ __launch_bounds__(grad_threads(kBlock, kAligned)) void combine_grad_kernel(
    const uint8_t* __restrict__ dout, const uint8_t* __restrict__ y, int rows_total,
    const int32_t* __restrict__ slot_of, const float* __restrict__ topk_w, int T, int K,
    RowShape row, uint8_t* __restrict__ dy, float* __restrict__ dw,
    const int32_t* __restrict__ row_src, long long zero_units, int32_t* __restrict__ status) {
  constexpr int N = El::kN;
  constexpr int kThreads = grad_threads(kBlock, kAligned), kWaves = kThreads / 64;
  constexpr int kCh = kThreads == 512 ? 1 : 2;
  constexpr int kStep = kBlock ? kThreads : kLanes;   // lanes on a row
  constexpr int kPer = kBlock ? 1 : kRowThreads / kLanes;   // tokens of a workgroup
  __shared__ float part[kBlock ? kWaves : 1][MOE_MAX_TOPK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = kBlock ? (int)threadIdx.x : (int)threadIdx.x & (kLanes - 1);
  const long long units = zero_units + ((long long)T + kPer - 1) / kPer;
  for (long long b = blockIdx.x; b < units; b += gridDim.x) {
    if (b < zero_units) {
      zero_rows(b * kWaves + wave, row_src, rows_total, row.bytes, dy);
      continue;
    }
    const long long t0 = (b - zero_units) * kPer + (kBlock ? 0 : (int)threadIdx.x / kLanes);
    const bool live = t0 < T;
    const long long t = live ? t0 : 0;
    const Picks<kLanes> picks(slot_of, t, K, rows_total, live);
    const int pick = lane & (kLanes - 1);
    const float wt = topk_w && live && pick < K ? topk_w[t * K + pick] : 0.f;
    if (picks.bad && at == 0) atomicOr(status, MOE_ERR_BAD_INDEX);
    float dots = 0.f;   // of pick `pick`
    for (int c0 = 0; c0 < row.chunks; c0 += kStep * kCh) {
      int off[kCh];
      uint4 g[kCh];
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        const int c = c0 + at + u * kStep;
        off[u] = row.start(c < row.chunks ? c : 0);
        if (c0 + u * kStep < row.chunks)
          g[u] = load_chunk<kAligned, kStream>(dout + t * (long long)row.bytes + off[u], row.bytes);
      }
      auto load = [&](int k, uint4 (&v)[kCh]) {
        const uint8_t* src = y + (long long)picks.of(picks.s, k) * row.bytes;
#pragma unroll
        for (int u = 0; u < kCh; ++u)
          if (c0 + u * kStep < row.chunks)
            v[u] = load_chunk<kAligned, kStream>(src + off[u], row.bytes);
      };
      auto finish = [&](int k, const uint4 (&v)[kCh]) {
        uint8_t* dst = dy + (long long)picks.of(picks.s, k) * row.bytes;
        const float wk = picks.of(wt, k);
        float d = 0.f;
#pragma unroll
        for (int u = 0; u < kCh; ++u) {
          const int c = c0 + at + u * kStep;
          if (c >= row.chunks) continue;
          float f[N], e[N];
          El::unpack(g[u], f);
          if (dw) {
            El::unpack(v[u], e);
            // elements of this chunk that the chunk before it has too
            const int skip = kAligned ? 0 : (16 * c - off[u]) / El::kSize;
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (kAligned || i >= skip) d = fmaf(f[i], e[i], d);
          }
          if (dy) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] *= wk;
            store_chunk<kAligned>(dst + off[u], row.bytes, El::pack(f));
          }
        }
        if (dw) {
          d = group_sum<kLanes>(d);
          if (pick == k) dots += d;
        }
      };
      for (unsigned long long m = picks.valid; m; m &= m - 1) {
        const int k = __ffsll((long long)m) - 1;
        uint4 v[kCh];
        if (dw) load(k, v);
        finish(k, v);
      }
    }
    if (!dw) continue;
    if constexpr (kBlock) {
      part[wave][lane] = dots;
      __syncthreads();
      if (threadIdx.x < K) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) d += part[i][threadIdx.x];
        dw[t * K + threadIdx.x] = d;
      }
      __syncthreads();
    } else if (live && pick < K) {
      dw[t * K + pick] = dots;
    }
  }
}

static int type_size(int dtype) {
  switch (dtype) {
    case MOE_TYPE_F32: return 4;
    case MOE_TYPE_BF16:
    case MOE_TYPE_F16: return 2;
    case MOE_TYPE_U8: return 1;
    default: return 0;
  }
}

// Workgroups of a launch over `units` units, `per` of them to a workgroup:
// a grid past 2^22 workgroups walks (HIP bounds a launch's threads by 2^32).
static unsigned grid_for(long long units, int per) {
  const long long b = (units + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b > (1 << 22) ? (1 << 22) : b);
}

// Pieces of a row for one wave each, and their length in chunks.
static void cut(const RowShape& row, int& pieces, int& plen) {
  pieces = (row.chunks + 63) / 64;
  plen = (row.chunks + pieces - 1) / pieces;
}

// Groups of 16 lanes for rows of up to 512 bytes, where a wave would be half
// idle (60,000 tokens of 130 bf16: combine 32 us with a wave each).
static bool short_rows(const RowShape& row, int K) { return row.chunks <= 32 && K <= 16; }

// Reading past the caches pays where the rows are more than the memory-side
// cache holds (256 MB): combine of 2.8 GB 506 us against 534, but of 32 MB
// 7.1 against 5.9 and of 147 MB 26 against 25, as there the caches may hold
// what the caller has just written.
static bool streamed(long long rows_total, const RowShape& row) {
  return rows_total * row.bytes > (512LL << 20);
}

// The checks that the four calls share.  Sizes first, then (by the caller)
// the pointers that the sizes make necessary.
static moe_status_t row_args(int dtype, int T, int K, int H, int rows_total, bool bytes_too,
                             RowShape* row) {
  const int es = type_size(dtype);
  if (es == 0 || (es == 1 && !bytes_too)) return MOE_INVALID_ARG;
  if (T < 0 || K <= 0 || K > MOE_MAX_TOPK || H <= 0 || rows_total < 0) return MOE_INVALID_ARG;
  if ((long long)H * es > 0x7fffffffLL - 64) return MOE_UNSUPPORTED_SHAPE;
  if ((long long)T * K > 0x7fffffffLL) return MOE_UNSUPPORTED_SHAPE;
  row->bytes = H * es;
  row->chunks = (row->bytes + 15) / 16;
  return MOE_OK;
}

static bool wide(const RowShape& row, uintptr_t pointers) {
  return row.bytes % 16 == 0 && (pointers & 15) == 0;
}

static moe_status_t launched() {
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

template <typename El, bool kWeighted>
static moe_status_t gather_sum(const void* y, int rows_total, const int32_t* slot_of,
                               const float* topk_w, int T, int K, const RowShape& row, void* out,
                               int32_t* status, hipStream_t st) {
  const dim3 block(kRowThreads);
  const uint8_t* yb = static_cast<const uint8_t*>(y);
  uint8_t* ob = static_cast<uint8_t*>(out);
  const bool al = wide(row, (uintptr_t)y | (uintptr_t)out);
  if (short_rows(row, K)) {
    const dim3 grid(grid_for(T, 4 * kRowWaves));
    if (al)
      hipLaunchKernelGGL((gather_sum_kernel<El, 16, 2, true, false, kWeighted>), grid, block, 0,
                         st, yb, rows_total, slot_of, topk_w, T, K, row, 1, 32, ob, status);
    else
      hipLaunchKernelGGL((gather_sum_kernel<El, 16, 2, false, false, kWeighted>), grid, block, 0,
                         st, yb, rows_total, slot_of, topk_w, T, K, row, 1, 32, ob, status);
    return launched();
  }
  int pieces, plen;
  cut(row, pieces, plen);
  const dim3 grid(grid_for((long long)T * pieces, kRowWaves));
  if (al && streamed(rows_total, row))
    hipLaunchKernelGGL((gather_sum_kernel<El, 64, 1, true, true, kWeighted>), grid, block, 0, st,
                       yb, rows_total, slot_of, topk_w, T, K, row, pieces, plen, ob, status);
  else if (al)
    hipLaunchKernelGGL((gather_sum_kernel<El, 64, 1, true, false, kWeighted>), grid, block, 0, st,
                       yb, rows_total, slot_of, topk_w, T, K, row, pieces, plen, ob, status);
  else
    hipLaunchKernelGGL((gather_sum_kernel<El, 64, 1, false, false, kWeighted>), grid, block, 0, st,
                       yb, rows_total, slot_of, topk_w, T, K, row, pieces, plen, ob, status);
  return launched();
}

template <bool kWeighted>
static moe_status_t gather_sum_any(int dtype, const void* y, int rows_total,
                                   const int32_t* slot_of, const float* topk_w, int T, int K,
                                   const RowShape& row, void* out, int32_t* status,
                                   void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == MOE_TYPE_F32)
    return gather_sum<F32, kWeighted>(y, rows_total, slot_of, topk_w, T, K, row, out, status, st);
  if (dtype == MOE_TYPE_BF16)
    return gather_sum<BF16, kWeighted>(y, rows_total, slot_of, topk_w, T, K, row, out, status,
                                       st);
  return gather_sum<F16, kWeighted>(y, rows_total, slot_of, topk_w, T, K, row, out, status, st);
}

template <typename El, int kLanes, bool kBlock>
static void launch_combine_grad(bool al, bool stream, const uint8_t* dout, const uint8_t* y,
                                int rows_total, const int32_t* slot_of, const float* topk_w,
                                int T, int K, const RowShape& row, uint8_t* dy, float* dw,
                                const int32_t* row_src, int32_t* status, hipStream_t st) {
  const int per = kBlock ? 1 : kRowThreads / kLanes;
  const long long tokens = ((long long)T + per - 1) / per;
  auto run = [&](auto aligned, auto past) {
    constexpr int kThreads = grad_threads(kBlock, aligned.value);
    const long long zero = row_src && dy ? ((long long)rows_total + kThreads - 1) / kThreads : 0;
    hipLaunchKernelGGL((combine_grad_kernel<El, kLanes, kBlock, aligned.value, past.value>),
                       dim3(grid_for(zero + tokens, 1)), dim3(kThreads), 0, st, dout, y,
                       rows_total, slot_of, topk_w, T, K, row, dy, dw, row_src, zero, status);
  };
  if (al && stream)
    run(std::true_type(), std::true_type());
  else if (al)
    run(std::true_type(), std::false_type());
  else
    run(std::false_type(), std::false_type());
}

// A workgroup per token for rows past 256 chunks (4 KB), else a wave, or 16
// lanes for short rows.
template <typename El>
static moe_status_t combine_grad(const void* dout, const void* y, int rows_total,
                                 const int32_t* slot_of, const float* topk_w, int T, int K,
                                 const RowShape& row, void* dy, float* dw,
                                 const int32_t* row_src, int32_t* status, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const uint8_t* db = static_cast<const uint8_t*>(dout);
  const uint8_t* yb = static_cast<const uint8_t*>(y);
  uint8_t* gb = static_cast<uint8_t*>(dy);
  const bool al = wide(row, (uintptr_t)dout | (uintptr_t)y | (uintptr_t)dy);
  const bool past = streamed(rows_total, row);
  if (short_rows(row, K))
    launch_combine_grad<El, 16, false>(al, false, db, yb, rows_total, slot_of, topk_w, T, K, row,
                                       gb, dw, row_src, status, st);
  else if (row.chunks <= 256)
    launch_combine_grad<El, 64, false>(al, past, db, yb, rows_total, slot_of, topk_w, T, K, row,
                                       gb, dw, row_src, status, st);
  else
    launch_combine_grad<El, 64, true>(al, past, db, yb, rows_total, slot_of, topk_w, T, K, row,
                                      gb, dw, row_src, status, st);
  return launched();
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_permute_rows(const void* x, int dtype, int T, int K, int H,
                                         const int32_t* slot_of, int rows_total, void* a,
                                         const int32_t* row_src, int32_t* status_dev,
                                         void* stream) {
  RowShape row;
  const moe_status_t ok = row_args(dtype, T, K, H, rows_total, true, &row);
  if (ok != MOE_OK) return ok;
  if (rows_total == 0 && T == 0) return MOE_OK;
  if (!status_dev || (T > 0 && (!x || !slot_of)) || (rows_total > 0 && !a))
    return MOE_INVALID_ARG;
  if (((uintptr_t)x | (uintptr_t)a) & (type_size(dtype) - 1)) return MOE_UNSUPPORTED_SHAPE;
  const bool few = short_rows(row, K);
  int pieces = 1, plen = 32;
  if (!few) cut(row, pieces, plen);
  const long long zero = row_src ? ((long long)rows_total + 63) / 64 : 0;
  const long long units = zero + (few ? ((long long)T + 3) / 4 : (long long)T * pieces);
  if (units == 0) return MOE_OK;
  const dim3 grid(grid_for(units, kRowWaves)), block(kRowThreads);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const uint8_t* xb = static_cast<const uint8_t*>(x);
  uint8_t* ab = static_cast<uint8_t*>(a);
  const bool al = wide(row, (uintptr_t)x | (uintptr_t)a);
  if (few && al)
    hipLaunchKernelGGL((permute_rows_kernel<16, 2, true>), grid, block, 0, st, xb, slot_of, T, K,
                       row, pieces, plen, rows_total, ab, row_src, zero, status_dev);
  else if (few)
    hipLaunchKernelGGL((permute_rows_kernel<16, 2, false>), grid, block, 0, st, xb, slot_of, T, K,
                       row, pieces, plen, rows_total, ab, row_src, zero, status_dev);
  else if (al)
    hipLaunchKernelGGL((permute_rows_kernel<64, 1, true>), grid, block, 0, st, xb, slot_of, T, K,
                       row, pieces, plen, rows_total, ab, row_src, zero, status_dev);
  else
    hipLaunchKernelGGL((permute_rows_kernel<64, 1, false>), grid, block, 0, st, xb, slot_of, T, K,
                       row, pieces, plen, rows_total, ab, row_src, zero, status_dev);
  return launched();
}

extern "C" moe_status_t moe_permute_rows_grad(const void* da, int dtype, int rows_total,
                                              const int32_t* slot_of, int T, int K, int H,
                                              void* dx, int32_t* status_dev, void* stream) {
  RowShape row;
  const moe_status_t ok = row_args(dtype, T, K, H, rows_total, false, &row);
  if (ok != MOE_OK) return ok;
  if (T == 0) return MOE_OK;
  if (!slot_of || !dx || !status_dev || (rows_total > 0 && !da)) return MOE_INVALID_ARG;
  if (((uintptr_t)da | (uintptr_t)dx) & (type_size(dtype) - 1)) return MOE_UNSUPPORTED_SHAPE;
  return gather_sum_any<false>(dtype, da, rows_total, slot_of, nullptr, T, K, row, dx,
                               status_dev, stream);
}

extern "C" moe_status_t moe_combine_rows(const void* y, int dtype, int rows_total,
                                         const int32_t* slot_of, const float* topk_w, int T,
                                         int K, int H, void* out, int32_t* status_dev,
                                         void* stream) {
  RowShape row;
  const moe_status_t ok = row_args(dtype, T, K, H, rows_total, false, &row);
  if (ok != MOE_OK) return ok;
  if (T == 0) return MOE_OK;
  if (!slot_of || !topk_w || !out || !status_dev || (rows_total > 0 && !y))
    return MOE_INVALID_ARG;
  if (((uintptr_t)y | (uintptr_t)out) & (type_size(dtype) - 1)) return MOE_UNSUPPORTED_SHAPE;
  return gather_sum_any<true>(dtype, y, rows_total, slot_of, topk_w, T, K, row, out, status_dev,
                              stream);
}

extern "C" moe_status_t moe_combine_rows_grad(const void* dout, const void* y, int dtype,
                                              int rows_total, const int32_t* slot_of,
                                              const float* topk_w, int T, int K, int H, void* dy,
                                              float* dtopk_w, const int32_t* row_src,
                                              int32_t* status_dev, void* stream) {
  RowShape row;
  const moe_status_t ok = row_args(dtype, T, K, H, rows_total, false, &row);
  if (ok != MOE_OK) return ok;
  // (an output without elements may be NULL as well)
  if (!dy && !dtopk_w) return T == 0 || rows_total == 0 ? MOE_OK : MOE_INVALID_ARG;
  if (!status_dev || (T > 0 && (!dout || !slot_of))) return MOE_INVALID_ARG;
  if (dy && T > 0 && !topk_w) return MOE_INVALID_ARG;
  if (dtopk_w && rows_total > 0 && !y) return MOE_INVALID_ARG;
  if (((uintptr_t)dout | (uintptr_t)(dtopk_w ? y : nullptr) | (uintptr_t)dy) &
      (type_size(dtype) - 1))
    return MOE_UNSUPPORTED_SHAPE;
  if (T == 0 && !(row_src && dy && rows_total > 0)) return MOE_OK;
  if (!dtopk_w) y = nullptr;   // not read
  if (dtype == MOE_TYPE_F32)
    return combine_grad<F32>(dout, y, rows_total, slot_of, topk_w, T, K, row, dy, dtopk_w,
                             row_src, status_dev, stream);
  if (dtype == MOE_TYPE_BF16)
    return combine_grad<BF16>(dout, y, rows_total, slot_of, topk_w, T, K, row, dy, dtopk_w,
                              row_src, status_dev, stream);
  return combine_grad<F16>(dout, y, rows_total, slot_of, topk_w, T, K, row, dy, dtopk_w,
                           row_src, status_dev, stream);
}
