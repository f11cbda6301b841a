// The router: tokens' scores over the experts, the K experts each token goes
// to with their weights, and the gradient with respect to the logits.
//
//   softmax  s_e = exp(l_e - max l) / sum_f exp(l_f - max l)
//   sigmoid  s_e = 1 / (1 + exp(-l_e))
//   key_e = s_e + b_e, the picks are the K highest keys (of the top groups)
//   w_k = scale s_k [/ max(sum_j s_j, 2^-64)]
//
//   with S = sum_j s_j and c = scale, g_e = ds_e + sum of d_k over the k whose
//   pick is e, where d_k = c dw_k; renormalised c / S (dw_k - sum_j dw_j s_j / S),
//   or c 2^64 dw_k where S <= 2^-64:
//   softmax  dl_e = s_e (g_e - sum_f s_f g_f)
//   sigmoid  dl_e = s_e (1 - s_e) g_e
//
// Keys are compared as 64-bit numbers: which expert a token goes to does not
// hang on the last bit of an exponential.  A wave takes a token, lane l holding
// experts l, l + 64, ...
#include "row_chunks.hpp"

namespace moe {

constexpr int kRouteWaves = 4;
constexpr float kLeastSum = 0x1p-64f;

struct RouteArgs {
  const uint8_t* logits;
  const float* bias;
  int T, E, K;
  int softmax, groups, top_groups, group_best, renorm;
  float scale;
  int first, local;
  int32_t* idx;
  int32_t* local_idx;
  float* w;
  float* scores;
  int32_t* status;
  const float* dw;
  const float* dscores;
  uint8_t* dlogits;
};

template <typename El>
__device__ __forceinline__ float load_one(const uint8_t* p, size_t at) {
  uint4 c = make_uint4(0, 0, 0, 0);
  __builtin_memcpy(&c, p + at * El::kSize, El::kSize);
  float f[El::kN];
  El::unpack(c, f);
  return f[0];
}

template <typename El>
__device__ __forceinline__ void store_one(uint8_t* p, size_t at, float v) {
  float f[El::kN] = {v};
  const uint4 c = El::pack(f);
  __builtin_memcpy(p + at * El::kSize, &c, El::kSize);
}

__device__ __forceinline__ double wave_add(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The highest (key, lowest index on a tie) of the wave's candidates, in every
// lane; index -1 where no lane has one.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const double k = __shfl_xor(key, d);
    const int i = __shfl_xor(idx, d);
    if (i >= 0 && (idx < 0 || k > key || (k == key && i < idx))) {
      key = k;
      idx = i;
    }
  }
}

template <typename El, int kPer>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs p) {
  extern __shared__ double shared[];   // [waves][E], only where there are groups
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int size = p.E / p.groups;     // experts of a group
  double* keys = shared + (size_t)wave * p.E;
  for (long long t = (long long)blockIdx.x * kRouteWaves + wave; t < p.T;
       t += (long long)gridDim.x * kRouteWaves) {
    float l[kPer];
    bool pick[kPer], nan = false;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < p.E ? load_one<El>(p.logits, (size_t)t * p.E + e) : -INFINITY;
      nan |= l[i] != l[i];
      if (l[i] != l[i]) l[i] = -INFINITY;
      l[i] = fminf(l[i], 3.402823466e38f);
      pick[i] = l[i] > -INFINITY;
      top = fmaxf(top, l[i]);
    }
    double s[kPer], key[kPer];
    if (p.softmax) {
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
      double sum = 0.;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        s[i] = pick[i] ? exp((double)l[i] - (double)top) : 0.;
        sum += s[i];
      }
      sum = wave_add(sum);
#pragma unroll
      for (int i = 0; i < kPer; ++i) s[i] = pick[i] ? s[i] / sum : 0.;
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) s[i] = pick[i] ? 1. / (1. + exp(-(double)l[i])) : 0.;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 64 * i;
      const float b = p.bias && e < p.E ? p.bias[e] : 0.f;
      nan |= b != b;
      pick[i] = pick[i] && b > -INFINITY;   // (nor a NaN)
      key[i] = pick[i] ? s[i] + (double)b : -INFINITY;
      if (p.scores && e < p.E) p.scores[(size_t)t * p.E + e] = (float)s[i];
    }
    if (__ballot(nan) && lane == 0) atomicOr(p.status, MOE_ERR_NAN);

    if (p.groups > 1) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 64 * i < p.E) keys[lane + 64 * i] = key[i];
      __threadfence_block();
      // lane g's group (and g + 64's, ...): up to 1024 groups of one
      uint32_t kept = 0;   // bit j: group lane + 64 j
      double total[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int g = lane + 64 * j;
        double first = -INFINITY, second = -INFINITY;
        if (g < p.groups)
          for (int m = 0; m < size; ++m) {
            const double k = keys[g * size + m];
            second = k > first ? first : k > second ? k : second;
            first = k > first ? k : first;
          }
        total[j] = p.group_best > 1 && size > 1 ? first + second : first;
      }
      for (int n = 0; n < p.top_groups; ++n) {
        double k = 0.;
        int g = -1;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int at = lane + 64 * j;
          if (at < p.groups && !(kept >> j & 1) && (g < 0 || total[j] > k)) {
            k = total[j];
            g = at;
          }
        }
        wave_best(k, g);
        if (g >= 0 && (g & 63) == lane) kept |= 1u << (g >> 6);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int g = min(lane + 64 * i, p.E - 1) / size;
        const uint32_t bits = (uint32_t)__shfl((int)kept, g & 63);
        pick[i] = pick[i] && (bits >> (g >> 6) & 1);
      }
      __threadfence_block();
    }

    int mine = -1;      // lane k: pick k and its score
    double mine_s = 0.;
    for (int k = 0; k < p.K; ++k) {
      double best = 0.;
      int e = -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (pick[i] && (e < 0 || key[i] > best)) {
          best = key[i];
          e = lane + 64 * i;
        }
      wave_best(best, e);
      if (e < 0) break;
      double got = 0.;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (e == lane + 64 * i) {
          got = s[i];
          pick[i] = false;
        }
      got = __shfl(got, e & 63);
      if (lane == k) {
        mine = e;
        mine_s = got;
      }
    }
    double w = mine_s;
    if (p.renorm) {
      double sum = 0.;
      for (int k = 0; k < p.K; ++k) sum += __shfl(mine_s, k);
      w /= sum > (double)kLeastSum ? sum : (double)kLeastSum;
    }
    if (lane < p.K) {
      const size_t at = (size_t)t * p.K + lane;
      p.idx[at] = mine;
      if (p.local_idx) {
        const int here = mine - p.first;
        p.local_idx[at] = mine >= 0 && here >= 0 && here < p.local ? here : -1;
      }
      p.w[at] = mine >= 0 ? (float)(w * (double)p.scale) : 0.f;
    }
  }
}

template <typename El, int kPer>
__global__ __launch_bounds__(64 * kRouteWaves) void route_grad_kernel(RouteArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (long long t = (long long)blockIdx.x * kRouteWaves + wave; t < p.T;
       t += (long long)gridDim.x * kRouteWaves) {
    float s[kPer], g[kPer];
    bool live[kPer];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 64 * i;
      float l = e < p.E ? load_one<El>(p.logits, (size_t)t * p.E + e) : -INFINITY;
      if (l != l) l = -INFINITY;
      s[i] = fminf(l, 3.402823466e38f);
      live[i] = l > -INFINITY;
      top = fmaxf(top, s[i]);
      g[i] = live[i] && p.dscores ? p.dscores[(size_t)t * p.E + e] : 0.f;
    }
    if (p.softmax) {
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        s[i] = live[i] ? expf(s[i] - top) : 0.f;
        sum += s[i];
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
#pragma unroll
      for (int i = 0; i < kPer; ++i) s[i] = live[i] ? s[i] / sum : 0.f;
    }
    float rest[kPer];   // 1 - s, without cancellation (sigmoid)
    if (!p.softmax) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float e = expf(-fabsf(s[i])), big = 1.f / (1.f + e);
        rest[i] = s[i] < 0.f ? big : e * big;
        s[i] = !live[i] ? 0.f : s[i] < 0.f ? e * big : big;
      }
    }
    // lane k: pick k, its weight's gradient and its score
    int idx = lane < p.K ? p.idx[(size_t)t * p.K + lane] : -1;
    const bool bad = idx < -1 || idx >= p.E;
    if (__ballot(bad) && lane == 0) atomicOr(p.status, MOE_ERR_BAD_EXPERT);
    if (bad) idx = -1;
    float d = idx >= 0 ? p.dw[(size_t)t * p.K + lane] * p.scale : 0.f;
    if (p.renorm) {
      float sk = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float got = __shfl(s[i], idx & 63);
        if (idx >= 0 && idx >> 6 == i) sk = got;
      }
      float sum = sk, dot = d * sk;
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) {
        sum += __shfl_xor(sum, o);
        dot += __shfl_xor(dot, o);
      }
      d = sum > kLeastSum ? (d - dot / sum) / sum : d / kLeastSum;
      if (idx < 0) d = 0.f;
    }
    for (int k = 0; k < p.K; ++k) {
      const int e = __builtin_amdgcn_readlane(idx, k);
      const float dk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), k));
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (e == lane + 64 * i && live[i]) g[i] += dk;
    }
    float dot = 0.f;
    if (p.softmax) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) dot = fmaf(s[i], g[i], dot);
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) dot += __shfl_xor(dot, o);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 64 * i;
      const float dl = p.softmax ? s[i] * (g[i] - dot) : s[i] * rest[i] * g[i];
      if (e < p.E) store_one<El>(p.dlogits, (size_t)t * p.E + e, live[i] ? dl : 0.f);
    }
  }
}

static int route_type_size(int dtype) {
  return dtype == MOE_TYPE_F32 ? 4 : dtype == MOE_TYPE_BF16 || dtype == MOE_TYPE_F16 ? 2 : 0;
}

static moe_status_t route_args(const RouteArgs& p, int dtype, int score) {
  const int es = route_type_size(dtype);
  if (es == 0 || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID))
    return MOE_INVALID_ARG;
  if (p.T < 0 || p.E <= 0 || p.E > MOE_MAX_EXPERTS || p.K <= 0 || p.K > MOE_MAX_TOPK || p.K > p.E)
    return MOE_INVALID_ARG;
  if (((uintptr_t)p.logits | (uintptr_t)p.dlogits) & (es - 1)) return MOE_UNSUPPORTED_SHAPE;
  if (((uintptr_t)p.bias | (uintptr_t)p.idx | (uintptr_t)p.local_idx | (uintptr_t)p.w |
       (uintptr_t)p.scores | (uintptr_t)p.dw | (uintptr_t)p.dscores) & 3)
    return MOE_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

template <typename El, int kPer>
static void launch_route(const RouteArgs& p, bool grad, hipStream_t st) {
  const long long blocks = ((long long)p.T + kRouteWaves - 1) / kRouteWaves;
  const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : (1 << 22))), block(64 * kRouteWaves);
  const size_t lds = p.groups > 1 ? kRouteWaves * (size_t)p.E * sizeof(double) : 0;
  if (grad)
    hipLaunchKernelGGL((route_grad_kernel<El, kPer>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((route_kernel<El, kPer>), grid, block, lds, st, p);
}

template <typename El>
static moe_status_t launch_route(const RouteArgs& p, bool grad, hipStream_t st) {
  if (p.E <= 64)
    launch_route<El, 1>(p, grad, st);
  else if (p.E <= 128)
    launch_route<El, 2>(p, grad, st);
  else if (p.E <= 256)
    launch_route<El, 4>(p, grad, st);
  else if (p.E <= 512)
    launch_route<El, 8>(p, grad, st);
  else
    launch_route<El, 16>(p, grad, st);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_HIP_ERROR;
}

static moe_status_t launch_route(const RouteArgs& p, int dtype, bool grad, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == MOE_TYPE_F32) return launch_route<F32>(p, grad, st);
  if (dtype == MOE_TYPE_BF16) return launch_route<BF16>(p, grad, st);
  return launch_route<F16>(p, grad, st);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_route_tokens(const void* logits, int dtype, int T, int E,
                                         const float* bias, int score, int groups, int top_groups,
                                         int group_best, int K, int renorm, float scale,
                                         int first_expert, int local_experts, int32_t* topk_idx,
                                         int32_t* local_idx, float* topk_w, float* scores,
                                         int32_t* status_dev, void* stream) {
  RouteArgs p{};
  p.logits = static_cast<const uint8_t*>(logits);
  p.bias = bias;
  p.T = T;
  p.E = E;
  p.K = K;
  p.softmax = score == MOE_SCORE_SOFTMAX;
  p.groups = groups;
  p.top_groups = top_groups;
  p.group_best = group_best;
  p.renorm = renorm;
  p.scale = scale;
  p.first = first_expert;
  p.local = local_experts;
  p.idx = topk_idx;
  p.local_idx = local_idx;
  p.w = topk_w;
  p.scores = scores;
  p.status = status_dev;
  const moe_status_t ok = route_args(p, dtype, score);
  if (ok != MOE_OK) return ok;
  if (groups <= 0 || E % groups != 0 || top_groups <= 0 || top_groups > groups ||
      (group_best != 1 && group_best != 2))
    return MOE_INVALID_ARG;
  if (local_idx && (first_expert < 0 || local_experts <= 0 || local_experts > E - first_expert))
    return MOE_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w || !status_dev) return MOE_INVALID_ARG;
  return launch_route(p, dtype, false, stream);
}

extern "C" moe_status_t moe_route_tokens_grad(const void* logits, int dtype, int T, int E,
                                              const int32_t* topk_idx, int K, int score,
                                              int renorm, float scale, const float* dtopk_w,
                                              const float* dscores, void* dlogits,
                                              int32_t* status_dev, void* stream) {
  RouteArgs p{};
  p.logits = static_cast<const uint8_t*>(logits);
  p.T = T;
  p.E = E;
  p.K = K;
  p.softmax = score == MOE_SCORE_SOFTMAX;
  p.groups = 1;
  p.renorm = renorm;
  p.scale = scale;
  p.idx = const_cast<int32_t*>(topk_idx);
  p.dw = dtopk_w;
  p.dscores = dscores;
  p.dlogits = static_cast<uint8_t*>(dlogits);
  p.status = status_dev;
  const moe_status_t ok = route_args(p, dtype, score);
  if (ok != MOE_OK) return ok;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !dtopk_w || !dlogits || !status_dev) return MOE_INVALID_ARG;
  return launch_route(p, dtype, true, stream);
}
