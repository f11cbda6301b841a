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
#include <type_traits>

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

// Maximum over the wave, in every lane: rows of 16 lanes as in group16_max, then
// their results.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
  const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32);
  const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
  return max(max(a, b), max(c, d));
}

// The index of the highest key (the lowest index on a tie) of the wave's
// candidates, -1 where no lane has one (idx -1): the keys' upper halves first,
// the lower ones and the indices among the lanes that are left.
__device__ __forceinline__ int wave_best(double key, int idx) {
  uint64_t bits = __builtin_bit_cast(uint64_t, key + 0.0);   // (no -0)
  bits ^= (uint64_t)((int64_t)bits >> 63) | 0x8000000000000000ull;
  bool in = idx >= 0;
  uint64_t left = __ballot(in);
  if (!left) return -1;
  uint32_t m = wave_max(in ? (uint32_t)(bits >> 32) : 0u);
  in = in && (uint32_t)(bits >> 32) == m;
  left = __ballot(in);
  if (left & (left - 1)) {
    m = wave_max(in ? (uint32_t)bits : 0u);
    in = in && (uint32_t)bits == m;
    left = __ballot(in);
    if (left & (left - 1)) return (int)~wave_max(in ? ~(uint32_t)idx : 0u);
  }
  return __builtin_amdgcn_readlane(idx, __builtin_ctzll(left));
}

// A logit as the router counts it: NaN as -infinity, +infinity as the largest
// fp32 number.
__device__ __forceinline__ float clean(float l, bool& nan) {
  nan |= l != l;
  return l == l ? fminf(l, 3.402823466e38f) : -INFINITY;
}

// Pick k of token t: expert e (-1: none) with weight w.
__device__ __forceinline__ void put_pick(const RouteArgs& p, long long t, int k, int e, float w) {
  const size_t at = (size_t)t * p.K + k;
  p.idx[at] = e;
  if (p.local_idx) {
    const int here = e - p.first;
    p.local_idx[at] = e >= 0 && here >= 0 && here < p.local ? here : -1;
  }
  p.w[at] = w;
}

// ---- the exact form: a token to a wave, lane l on experts l, l + 64, ..., keys
// in 64 bits throughout, in E doubles of LDS.  It takes the tokens that the
// fast form below cannot decide, so its loops are short code, not fast: 65536
// tokens of 256 equal logits, all of which take it, 273 us (random ones 26), and
// 4096 44.
template <typename El>
__device__ __forceinline__ void route_exact(const RouteArgs& p, long long t, double* keys) {
  const int lane = threadIdx.x & 63;
  const size_t row = (size_t)t * p.E;
  bool nan = false;
  float top = -INFINITY;
  double all = 0.;
  if (p.softmax) {
#pragma unroll 1
    for (int e = lane; e < p.E; e += 64)
      top = fmaxf(top, clean(load_one<El>(p.logits, row + e), nan));
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    top = fmaxf(top, -3.402823466e38f);   // (a row of -infinity)
#pragma unroll 1
    for (int e = lane; e < p.E; e += 64)
      all += exp((double)clean(load_one<El>(p.logits, row + e), nan) - (double)top);
    all = wave_add(all);
    if (!(all > 0.)) all = 1.;
  }
  auto score = [&](int e, bool& pick) {
    const float l = clean(load_one<El>(p.logits, row + e), nan);
    pick = l > -INFINITY;
    const double x = exp(p.softmax ? (double)l - (double)top : -(double)l);
    return !pick ? 0. : p.softmax ? x / all : 1. / (1. + x);
  };
#pragma unroll 1
  for (int e = lane; e < p.E; e += 64) {
    bool pick;
    const double s = score(e, pick);
    const float b = p.bias ? p.bias[e] : 0.f;
    nan |= b != b;
    keys[e] = pick && b > -INFINITY ? s + (double)b : -INFINITY;   // (nor a NaN)
    if (p.scores) p.scores[row + e] = (float)s;
  }
  if (__ballot(nan) && lane == 0) atomicOr(p.status, MOE_ERR_NAN);
  __threadfence_block();

  if (p.groups > 1) {
    const int size = p.E / p.groups;
    // lane g has groups g, g + 64, ...; bit j of kept: group lane + 64 j
    auto total = [&](int g) {
      double first = -INFINITY, second = -INFINITY;
#pragma unroll 4
      for (int m = 0; m < size; ++m) {
        const double k = keys[g * size + m];
        second = k > first ? first : k > second ? k : second;
        first = k > first ? k : first;
      }
      return p.group_best > 1 && size > 1 ? first + second : first;
    };
    uint32_t kept = 0;
    const double own = lane < p.groups ? total(lane) : 0.;
#pragma unroll 1
    for (int n = 0; n < p.top_groups; ++n) {
      double k = own;
      int g = lane < p.groups && !(kept & 1) ? lane : -1;
#pragma unroll 1
      for (int at = lane + 64; at < p.groups; at += 64)
        if (!(kept >> (at >> 6) & 1)) {
          const double o = total(at);
          if (g < 0 || o > k) {
            k = o;
            g = at;
          }
        }
      g = wave_best(k, g);
      if (g >= 0 && (g & 63) == lane) kept |= 1u << (g >> 6);
    }
    __threadfence_block();
#pragma unroll 1
    for (int g = lane; g < p.groups; g += 64)
      if (!(kept >> (g >> 6) & 1))
        for (int m = 0; m < size; ++m) keys[g * size + m] = -INFINITY;
    __threadfence_block();
  }

  int mine = -1;      // lane k: pick k and its score
  double mine_s = 0.;
#pragma unroll 1
  for (int k = 0; k < p.K; ++k) {
    double best = -INFINITY;
    int e = -1;
#pragma unroll 4
    for (int at = lane; at < p.E; at += 64)
      if (keys[at] > best) {
        best = keys[at];
        e = at;
      }
    e = wave_best(best, e);
    if (e < 0) break;
    if (lane == k) mine = e;
    if (lane == 0) keys[e] = -INFINITY;
    __threadfence_block();
  }
  bool pick;
  if (mine >= 0) mine_s = score(mine, pick);
  const double sum = wave_add(mine_s);
  if (p.renorm) mine_s /= sum > (double)kLeastSum ? sum : (double)kLeastSum;
  if (lane < p.K) put_pick(p, t, lane, mine, (float)(mine_s * (double)p.scale));
  __threadfence_block();
}

template <typename El>
__global__ __launch_bounds__(64 * kRouteWaves) void route_exact_kernel(RouteArgs p) {
  extern __shared__ double shared[];   // [waves][E]
  const int wave = threadIdx.x >> 6;
  for (long long t = (long long)blockIdx.x * kRouteWaves + wave; t < p.T;
       t += (long long)gridDim.x * kRouteWaves)
    route_exact<El>(p, t, shared + (size_t)wave * p.E);
}

// ---- the fast form: kLanes lanes to a token, each holding up to kN
// neighbouring experts of one group.
//
// Keys are fp32 here.  The K highest of every lane's two best keys bound the
// K-th highest key from below, and the experts above that bound (less the keys'
// error) are candidates, hardly more than K of them.  A candidate goes to a
// lane, which ranks it by counting the higher ones.  Where two candidates are
// closer than their error, or tie, their keys are formed again in 64 bits; what
// is still open goes to route_exact: groups whose scores are closer than their
// error, more candidates than fit, and, for a softmax with a bias, whose sum
// is fp32, candidates that are close.
//
// Bound by instruction issue: the vector units are active in 82% of the cycles
// that the CUs are busy (65536 tokens of 256 experts in 8 groups fp32, 33 us), with
// 866 vector instructions for four tokens; the three waves of a unit hide each
// other's waits, 45% of their cycles.  Scores are stored one by one: asked for,
// they add 55 us.
constexpr float kU = 0x1p-24f;

// The larger of two numbers that are no NaN: a median with infinity, where fmaxf
// first quiets what might be a signalling NaN, one instruction more per operand.
// (Where the compiler turns it back into a maximum, it quiets one as well.)
__device__ __forceinline__ float larger(float a, float b) {
  return __builtin_amdgcn_fmed3f(a, b, INFINITY);
}

// Maximum over the aligned group of kLanes lanes, in all of them (no NaN).
// Rows of 16 lanes exchange as in group16_max, the exchange a part of the
// instruction that compares; a lane's new value can be exchanged two wait
// states later.
template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
  asm("s_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_mirror row_mask:0xf bank_mask:0xf"
      : "+v"(v));
  if constexpr (kLanes == 64) {
    v = larger(v, __shfl_xor(v, 16));
    v = larger(v, __shfl_xor(v, 32));
  }
  return v;
}

template <int kLanes>
__device__ __forceinline__ float lanes_add(float v) {
  v += dpp_row<0xb1>(v);
  v += dpp_row<0x4e>(v);
  v += dpp_row<0x141>(v);
  v += dpp_row<0x140>(v);
  if constexpr (kLanes == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}

constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.9259629911266175e-8f;
constexpr float kLn2 = 0.693147182464599609375f;

// exp(x) for x in [-1000, 88], within 3 roundings down to 2^-126, 0 below: x
// log2(e) in two parts, since the exponential would scale the rounding of one
// up by |x|.
__device__ __forceinline__ float exp32(float x) {
  const float t = x * kLog2e;
  const float low = fmaf(x, kLog2e, -t) + x * kLog2eLow;
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, low * kLn2, e);
}

// 1 / x for x in [1, 2^12].
__device__ __forceinline__ float inverse(float x) {
  const float y = __builtin_amdgcn_rcpf(x);
  return fmaf(fmaf(-x, y, 1.f), y, y);
}

// A score within 8 roundings (softmax: of the exponential; l - top adds |l - top|).
__device__ __forceinline__ float score32(float l, bool softmax, float top, float inv) {
  if (softmax) return exp32(fmaxf(l - top, -1000.f)) * inv;
  const float e = exp32(fmaxf(-fabsf(l), -1000.f));
  const float r = inverse(1.f + e);
  return l < 0.f ? e * r : r;
}

// An fp32 number as an unsigned one of the same order.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// A candidate: of two, the one of the higher key, or of the same and the lower
// index, has the higher `order`.  key64 takes its place once it has been formed.
struct __attribute__((aligned(16))) Candidate {
  uint64_t order;
  float key;
  union {
    float error;
    int e;
  };
};

// Waves of a SIMD that the registers are shared out to.  (16 experts to each of
// 16 lanes: three 41 us for 65536 tokens of 256 experts in groups, four, with
// spills, 45.  Later steps brought the first to 33.)
constexpr int route_waves(int lanes, int n) { return lanes == 16 && n == 16 ? 3 : 4; }

template <typename El, int kLanes, int kN, bool kWide>
__global__ __launch_bounds__(64 * kRouteWaves, route_waves(kLanes, kN)) void
route_kernel(RouteArgs p, int lanes_per_group, int per_lane) {
  constexpr int kTokens = 64 / kLanes;          // of a wave
  constexpr int kCap = kLanes == 16 ? 32 : 64;  // candidates of a token
  constexpr int kMine = kCap / kLanes;          // of them to a lane
  __shared__ Candidate cand[kRouteWaves][kTokens][kCap];
  __shared__ __attribute__((aligned(16))) float totals[kRouteWaves][64];
  extern __shared__ double shared[];   // [waves][E], of route_exact
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = lane % kLanes, seg = lane / kLanes, base = lane - at;
  const int size = p.E / p.groups;
  const int group = at / lanes_per_group, sub = at - group * lanes_per_group;
  const int first = group * size + sub * per_lane;   // the lane's experts
  const int mine = group < p.groups ? max(0, min(per_lane, size - sub * per_lane)) : 0;
  Candidate* list = cand[wave][seg];
  const bool softmax = p.softmax;

  float bias[kN], reach = 0.f;   // reach: the largest finite bias in magnitude
  bool bias_nan = false;
#pragma unroll
  for (int i = 0; i < kN; ++i) bias[i] = 0.f;
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      bias[i] = p.bias[kWide ? (mine ? first : 0) + i : i < mine ? first + i : 0];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      bias_nan |= i < mine && bias[i] != bias[i];
      bias[i] = bias[i] == bias[i] ? bias[i] : -INFINITY;
      if (i < mine && fabsf(bias[i]) < INFINITY) reach = larger(reach, fabsf(bias[i]));
    }
  }
  reach = lanes_max<kLanes>(reach);
  // an fp32 key's error where v = |key| + 2 reach bounds both the key and its
  // score.  Sigmoid: 9 roundings (exponential 3, sum, reciprocal 2, bias), and
  // of the exponent's low part, left out here, 0.22 per unit of the argument,
  // which is -ln(score) at most where it counts.  Softmax: the exponential's and
  // the sum's, and one per unit of the argument.  Scores below e^-88 are 0,
  // within 1e-37.  (Two keys with |sum| + 4 reach <= v together: the same.)  v is
  // 0 where all scores that it bounds are and there is no bias: its logarithm
  // is taken of the least normal number then, since 0 times -log 0 is NaN.
  auto error = [&](float v) {
    const float units = larger(0.f, -0.7f * __builtin_amdgcn_logf(larger(v, 0x1p-126f)));
    const float roundings = softmax ? 25.f + kN + units : fmaf(0.22f, units, 9.f);
    return fmaf(v, roundings * kU, 1e-37f);
  };
  uint32_t absent = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) absent |= (i < mine ? 0u : 1u) << i;

  for (long long t0 = ((long long)blockIdx.x * kRouteWaves + wave) * kTokens; t0 < p.T;
       t0 += (long long)gridDim.x * kRouteWaves * kTokens) {
    const long long t = t0 + seg;
    const bool live = t < p.T;
    const size_t row = (size_t)(live ? t : t0) * p.E;
    // ---- logits; `odd`: there are infinities or NaN among them
    float key[kN];
    bool nan = bias_nan;
    float odd = 0.f;
    if constexpr (kWide) {
#pragma unroll
      for (int c = 0; c < kN * El::kSize / 16; ++c) {
        float f[El::kN];
        const uint8_t* src = p.logits + (row + first) * El::kSize + 16 * c;
        El::unpack(*reinterpret_cast<const uint4*>(mine > 0 ? src : p.logits), f);
#pragma unroll
        for (int i = 0; i < El::kN; ++i) key[c * El::kN + i] = f[i];
      }
      if (mine == 0) key[0] = INFINITY;   // (a lane without experts)
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        key[i] = i < mine ? load_one<El>(p.logits, row + first + i) : INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) odd = fmaf(key[i], key[i], odd);
    uint32_t masked = absent;   // bit i: expert i is none, or not to be picked
    const bool special = __ballot(!(odd < INFINITY)) != 0;
    if (special) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        nan |= key[i] != key[i] && !(absent >> i & 1);
        masked |= (key[i] > -INFINITY ? 0u : 1u) << i;
        key[i] = __builtin_amdgcn_fmed3f(key[i], -3.402823466e38f, 3.402823466e38f);
        if (softmax) key[i] = masked >> i & 1 ? -INFINITY : key[i];
      }
    }
    // ---- scores and keys
    float top = 0.f, inv = 1.f;
    if (softmax) {
      top = -3.402823466e38f;   // (of a row of -infinity)
#pragma unroll
      for (int i = 0; i < kN; ++i) top = larger(top, key[i]);
      top = lanes_max<kLanes>(top);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        key[i] = exp32(larger(key[i] - top, -1000.f));
        sum += key[i];
      }
      sum = lanes_add<kLanes>(sum);
      inv = 1.f / fmaxf(sum, 1.f);
      if (p.scores && live)
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (i < mine) p.scores[row + first + i] = key[i] * inv;
#pragma unroll
      for (int i = 0; i < kN; ++i) key[i] = fmaf(key[i], inv, bias[i]);
    } else {
      if (p.scores && live)
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (i < mine)
            p.scores[row + first + i] = masked >> i & 1 ? 0.f : score32(key[i], false, 0.f, 1.f);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float x = -__builtin_amdgcn_fmed3f(key[i], -88.f, 88.f);
        const float u = x * kLog2e;
        const float e = __builtin_amdgcn_exp2f(u);
        const float e1 = fmaf(e, fmaf(x, kLog2e, -u) * kLn2, e);
        key[i] = __builtin_amdgcn_rcpf(1.f + e1) + bias[i];
      }
    }
    if (special) {
#pragma unroll
      for (int i = 0; i < kN; ++i) key[i] = masked >> i & 1 ? -INFINITY : key[i];
    }

    // ---- the lane's two best, and its group's
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      b = __builtin_amdgcn_fmed3f(a, b, key[i]);
      a = larger(a, key[i]);
    }
    bool slow = false;
    if (p.groups > 1) {
      float ga = a, gb = b;
      for (int d = 1; d < lanes_per_group; ++d) {
        const int s2 = sub + d < lanes_per_group ? sub + d : sub + d - lanes_per_group;
        const int from = base + group * lanes_per_group + s2;
        const float oa = __shfl(a, from), ob = __shfl(b, from);
        gb = larger(__builtin_amdgcn_fmed3f(ga, oa, gb), ob);
        ga = larger(ga, oa);
      }
      // (clamped, so that differences are no NaN.  Both keys' scores and
      // magnitudes together are at most |total| + 4 reach: a key below 0 is
      // one of -reach at least.)
      float total = p.group_best > 1 && size > 1 ? ga + gb : ga;
      total = __builtin_amdgcn_fmed3f(total, -3e38f, 3e38f);
      const float margin = 2.f * error(fabsf(total) + 4.f * reach);
      // (what is no group is lower than all)
      totals[wave][lane] = -INFINITY;
      if (sub == 0 && group < p.groups) totals[wave][base + group] = total;
      __threadfence_block();
      int higher = 0, near = -1;   // (itself)
      for (int g = 0; g < p.groups; g += 4) {
        const float4 o = *reinterpret_cast<const float4*>(&totals[wave][base + g]);
        const float d[4] = {o.x - total, o.y - total, o.z - total, o.w - total};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          higher += d[i] > margin;
          near += fabsf(d[i]) <= margin;
        }
      }
      // surely kept: fewer than top_groups higher ones even if all near ones are
      // higher; surely dropped: top_groups surely higher ones
      const bool kept = higher + near < p.top_groups;
      slow = group < p.groups && ga > -INFINITY && !kept && higher < p.top_groups;
      if (!kept) {
        a = b = -INFINITY;
#pragma unroll
        for (int i = 0; i < kN; ++i) key[i] = -INFINITY;
      }
    }
    // ---- a lower bound of the K-th highest key
    float bound = lanes_max<kLanes>(a);
    {
      float a1 = a, b1 = b;
      for (int k = 1; k < p.K; ++k) {
        const bool popped = a1 == bound;
        a1 = popped ? b1 : a1;
        b1 = popped ? -INFINITY : b1;
        bound = lanes_max<kLanes>(a1);
      }
    }
    bound -= 2.f * error(fabsf(bound) + 2.f * reach);
    // (never -infinity: masked keys are no candidates)
    bound = larger(bound == bound ? bound : -INFINITY, -3.402823466e38f);
    // ---- candidates, in the order of the lanes
    uint32_t in = 0;
#pragma unroll
    for (int i = kN - 1; i >= 0; --i) in = in + in + (key[i] >= bound ? 1u : 0u);
    const int n = __builtin_popcount(in);
    int pos = n;
    if constexpr (kLanes == 16) {
      // inclusive sum over rows of 16 lanes
      pos += __builtin_amdgcn_update_dpp(0, pos, 0x111, 0xf, 0xf, true);
      pos += __builtin_amdgcn_update_dpp(0, pos, 0x112, 0xf, 0xf, true);
      pos += __builtin_amdgcn_update_dpp(0, pos, 0x114, 0xf, 0xf, true);
      pos += __builtin_amdgcn_update_dpp(0, pos, 0x118, 0xf, 0xf, true);
    } else {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(pos, d);
        if (lane >= d) pos += o;
      }
    }
    const int total_n = __shfl(pos, base + kLanes - 1);
    pos -= n;
    while (in) {
      if (pos < kCap) list[pos].e = first + __builtin_ctz(in);
      in &= in - 1;
      ++pos;
    }
    slow |= total_n > kCap;
    const int cands = min(total_n, kCap);
    int most = cands;   // of the wave's tokens
#pragma unroll
    for (int d = kLanes; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
    most = __builtin_amdgcn_readfirstlane(most);
    __threadfence_block();
    // ---- candidate at (and kLanes further): its score again, a few roundings
    // off, and its rank.  Places behind a token's candidates rank below all.
    int ce[kMine], rank[kMine];
    float cl[kMine], cs[kMine], ck[kMine], err[kMine];
    uint64_t order[kMine];
    auto form = [&](auto at_u) __attribute__((always_inline)) {
      constexpr int u = decltype(at_u)::value;
      const int c = at + u * kLanes;
      ce[u] = -1;
      rank[u] = 0;
      cl[u] = cs[u] = 0.f;
      ck[u] = -INFINITY;
      order[u] = 0;
      if (c < cands) {
        ce[u] = list[c].e;
        bool none = false;
        cl[u] = clean(load_one<El>(p.logits, row + ce[u]), none);
        cs[u] = score32(cl[u], softmax, top, inv);
        ck[u] = cs[u] + (p.bias ? p.bias[ce[u]] : 0.f);
        order[u] = (uint64_t)ordered(ck[u]) << 32 | (uint32_t)~ce[u];
      }
      err[u] = 0.f;
      if (c < cands)
        err[u] = fmaf(cs[u], (softmax ? 18.f + kN + (top - cl[u]) : 12.f) * kU,
                      fmaf(fabsf(ck[u]), kU, 1e-37f));
      list[c].order = order[u];
      list[c].key = ck[u];
      list[c].error = err[u];
    };
    // how many of the candidates rank higher, and how many are close (itself
    // among them)
    int close = 0;
    auto count = [&](int upto, auto at_u) __attribute__((always_inline)) {
      constexpr int u = decltype(at_u)::value;
      int n_close = 0;
#pragma unroll 4
      for (int c = 0; c < upto; ++c) {
        const uint64_t o = list[c].order;
        const float ok = list[c].key;
        rank[u] += o > order[u];
        n_close += !(fabsf(ok - ck[u]) > list[c].error + err[u]);
      }
      if (ce[u] >= 0) close |= n_close - 1;
    };
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, kMine - 1>;
    const bool two = kMine > 1 && most > kLanes;
    form(First());
    if (kMine > 1) {
      ce[kMine - 1] = kMine > 1 ? -1 : ce[0];
      if (two) form(Second());
    }
    __threadfence_block();
    count(most, First());
    if (two) count(most, Second());
    if (__ballot(close != 0 && live)) {
      // keys in 64 bits.  (A softmax's sum, the same for all, does not change
      // the order of its scores.)
      if (softmax && p.bias) slow |= close != 0;
      double key64[kMine];
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        key64[u] = 0.;
        if (ce[u] < 0) continue;
        const double l = (double)cl[u];
        const double x = exp(softmax ? l - (double)top : -l);
        key64[u] = !softmax ? 1. / (1. + x) : p.bias ? x * (double)inv : x;
        if (p.bias) key64[u] += (double)p.bias[ce[u]];
        list[at + u * kLanes].order = __builtin_bit_cast(uint64_t, key64[u]);
        list[at + u * kLanes].e = ce[u];
        rank[u] = 0;
      }
      __threadfence_block();
#pragma unroll 1
      for (int c = 0; c < most; ++c) {
        const double ok = __builtin_bit_cast(double, list[c].order);
        const int oe = list[c].e;
#pragma unroll
        for (int u = 0; u < kMine; ++u)
          if (ce[u] >= 0)
            rank[u] += c < cands && (ok > key64[u] || (ok == key64[u] && oe < ce[u]));
      }
    }
    // ---- weights
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < kMine; ++u)
      if (ce[u] >= 0 && rank[u] < p.K) sum += cs[u];
    sum = lanes_add<kLanes>(sum);
    const unsigned long long slow_bits = __ballot(slow && live);
    constexpr unsigned long long kSeg = kLanes == 64 ? ~0ull : (1ull << (kLanes & 63)) - 1;
    const bool seg_slow = (slow_bits >> base & kSeg) != 0;
    if (live && !seg_slow) {
      const float by = p.renorm ? p.scale / fmaxf(sum, kLeastSum) : p.scale;
#pragma unroll
      for (int u = 0; u < kMine; ++u)
        if (ce[u] >= 0 && rank[u] < p.K) put_pick(p, t, rank[u], ce[u], cs[u] * by);
      // (fewer candidates than picks: none)
      for (int k = cands + at; k < p.K; k += kLanes) put_pick(p, t, k, -1, 0.f);
      if (nan) atomicOr(p.status, MOE_ERR_NAN);
    }
    if (slow_bits) {
#pragma unroll 1
      for (int q = 0; q < kTokens; ++q)
        if (slow_bits >> (q * kLanes) & kSeg)
          route_exact<El>(p, t0 + q, shared + (size_t)wave * p.E);
    }
    __threadfence_block();   // (the list is written again)
  }
}

// The gradient, bound by instruction issue (16384 x 72 bf16 6.7 us: 605 vector
// instructions for four tokens, the vector units active in 75% of the cycles):
// kLanes lanes to a token, each holding kN neighbouring experts
// (kWide: whole 16-byte pieces of a row) or experts at, at + kLanes, ...; lane k
// holds pick k.
template <typename El, int kLanes, int kN, bool kWide>
__global__ __launch_bounds__(64 * kRouteWaves) void route_grad_kernel(RouteArgs p) {
  constexpr int kTokens = 64 / kLanes;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = lane % kLanes, seg = lane / kLanes, base = lane - at;
  const int first = kWide ? at * kN : at;
  const int mine = kWide ? (first < p.E ? kN : 0) : max(0, (p.E - at + kLanes - 1) / kLanes);
  constexpr int kNext = kWide ? 1 : kLanes;   // from one of the lane's experts to the next
  const bool softmax = p.softmax;
  for (long long t0 = ((long long)blockIdx.x * kRouteWaves + wave) * kTokens; t0 < p.T;
       t0 += (long long)gridDim.x * kRouteWaves * kTokens) {
    const long long t = t0 + seg;
    const bool live = t < p.T;
    const size_t row = (size_t)(live ? t : t0) * p.E;
    float s[kN], g[kN], rest[kN];   // rest: 1 - s, without cancellation (sigmoid)
    bool none = false;
    if constexpr (kWide) {
#pragma unroll
      for (int c = 0; c < kN * El::kSize / 16; ++c) {
        float f[El::kN];
        const uint8_t* src = p.logits + (row + first) * El::kSize + 16 * c;
        El::unpack(*reinterpret_cast<const uint4*>(mine > 0 ? src : p.logits), f);
#pragma unroll
        for (int i = 0; i < El::kN; ++i) s[c * El::kN + i] = f[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        s[i] = load_one<El>(p.logits, row + (i < mine ? first + i * kNext : 0));
    }
    int idx = live && at < p.K ? p.idx[(size_t)t * p.K + at] : -1;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      g[i] = p.dscores ? p.dscores[row + (i < mine ? first + i * kNext : 0)] : 0.f;
    const bool bad = idx < -1 || idx >= p.E;
    if (__ballot(bad) && lane == 0) atomicOr(p.status, MOE_ERR_BAD_EXPERT);
    if (bad) idx = -1;
    float d = idx >= 0 ? p.dw[(size_t)t * p.K + at] * p.scale : 0.f;
    const float picked = load_one<El>(p.logits, row + (idx >= 0 ? idx : 0));
    // (a logit that counts as -infinity: score and gradient 0)
    bool dead[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      s[i] = i < mine ? clean(s[i], none) : -INFINITY;
      dead[i] = !(s[i] > -INFINITY);
      if (dead[i]) g[i] = 0.f;
    }
    float top = -3.402823466e38f, inv = 1.f;
    if (softmax) {
#pragma unroll
      for (int i = 0; i < kN; ++i) top = larger(top, s[i]);
      top = lanes_max<kLanes>(top);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        s[i] = exp32(larger(s[i] - top, -1000.f));
        sum += s[i];
      }
      sum = lanes_add<kLanes>(sum);
      inv = 1.f / fmaxf(sum, 1.f);
#pragma unroll
      for (int i = 0; i < kN; ++i) s[i] *= inv;
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float e = exp32(larger(-fabsf(s[i]), -1000.f));
        const float big = inverse(1.f + e), small = e * big;
        rest[i] = s[i] < 0.f ? big : small;
        s[i] = dead[i] ? 0.f : s[i] < 0.f ? small : big;
      }
    }
    if (p.renorm) {
      const float l = clean(picked, none);
      const float sk = idx >= 0 && l > -INFINITY ? score32(l, softmax, top, inv) : 0.f;
      const float sum = lanes_add<kLanes>(sk);
      const float dot = lanes_add<kLanes>(d * sk);
      d = sum > kLeastSum ? (d - dot / sum) / sum : d / kLeastSum;
      if (idx < 0) d = 0.f;
    }
    for (int k = 0; k < p.K; ++k) {
      const int e = __shfl(idx, base + k) - first;
      const float dk = __shfl(d, base + k);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (e == i * kNext && i < mine && !dead[i]) g[i] += dk;
    }
    float dot = 0.f;
    if (softmax) {
#pragma unroll
      for (int i = 0; i < kN; ++i) dot = fmaf(s[i], g[i], dot);
      dot = lanes_add<kLanes>(dot);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      g[i] = softmax ? s[i] * (g[i] - dot) : s[i] * rest[i] * g[i];
      if (dead[i]) g[i] = 0.f;
    }
    if (!live) continue;
    if constexpr (kWide) {
      if (mine > 0)
#pragma unroll
        for (int c = 0; c < kN * El::kSize / 16; ++c) {
          float f[El::kN];
#pragma unroll
          for (int i = 0; i < El::kN; ++i) f[i] = g[c * El::kN + i];
          *reinterpret_cast<uint4*>(p.dlogits + (row + first) * El::kSize + 16 * c) =
              pack_row<El>(f);
        }
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i < mine) store_one<El>(p.dlogits, row + first + i * kNext, g[i]);
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

static dim3 route_grid(long long units, long long most) {
  const long long blocks = (units + kRouteWaves - 1) / kRouteWaves;
  return dim3((unsigned)(blocks < most ? blocks : most));
}

template <typename El, int kLanes, int kN>
static void launch_fast(const RouteArgs& p, int lanes_per_group, int per_lane, hipStream_t st) {
  constexpr int kTokens = 64 / kLanes;
  // as many workgroups as the CUs hold, so that a wave loads its experts'
  // biases once for several tokens
  const dim3 grid = route_grid(((long long)p.T + kTokens - 1) / kTokens,
                               256LL * route_waves(kLanes, kN));
  const dim3 block(64 * kRouteWaves);
  const size_t lds = kRouteWaves * (size_t)p.E * sizeof(double);
  // every lane's experts are whole 16-byte pieces of a row
  const bool wide = per_lane == kN && p.E / p.groups % kN == 0 &&
                    (size_t)p.E * El::kSize % 16 == 0 && ((uintptr_t)p.logits & 15) == 0;
  if constexpr (kN * El::kSize % 16 == 0) {
    if (wide) {
      hipLaunchKernelGGL((route_kernel<El, kLanes, kN, true>), grid, block, lds, st, p,
                         lanes_per_group, per_lane);
      return;
    }
  }
  hipLaunchKernelGGL((route_kernel<El, kLanes, kN, false>), grid, block, lds, st, p,
                     lanes_per_group, per_lane);
}

template <typename El>
static void launch_exact(const RouteArgs& p, hipStream_t st) {
  const size_t lds = kRouteWaves * (size_t)p.E * sizeof(double);
  hipLaunchKernelGGL((route_exact_kernel<El>), route_grid(p.T, 1 << 22),
                     dim3(64 * kRouteWaves), lds, st, p);
}

// 16 lanes to a token where they hold its experts, 16 at most each, else 64,
// else the exact form.  Four tokens to a wave share its instructions, which
// bound many tokens (us, 16 and 64 lanes: 65536 x 256 in 8 groups 33 and 86,
// without groups 26 and 60, 65536 x 64 16 and 57; 4096 x 256 in groups 15 and
// 16).  For few tokens a lane's longer list shows (1 x 256 in groups 5.8 and
// 5.4, 1024 x 256 6.6 and 5.7; 1 x 64 4.0 and 4.6); the rule leaves T out, so
// that a token's scores and weights have the same bits in every batch.
template <typename El>
static void launch_route(const RouteArgs& p, hipStream_t st) {
  const int size = p.E / p.groups;
  const int g16 = p.groups <= 16 ? 16 / p.groups : 0, g64 = p.groups <= 64 ? 64 / p.groups : 0;
  const int n16 = g16 ? (size + g16 - 1) / g16 : 1 << 20;
  const int n64 = g64 ? (size + g64 - 1) / g64 : 1 << 20;
  if (n16 <= 16 && p.K <= 16) {
    if (n16 <= 2)
      launch_fast<El, 16, 2>(p, g16, n16, st);
    else if (n16 <= 4)
      launch_fast<El, 16, 4>(p, g16, n16, st);
    else if (n16 <= 8)
      launch_fast<El, 16, 8>(p, g16, n16, st);
    else
      launch_fast<El, 16, 16>(p, g16, n16, st);
  } else if (n64 <= 16) {
    if (n64 <= 4)
      launch_fast<El, 64, 4>(p, g64, n64, st);
    else if (n64 <= 8)
      launch_fast<El, 64, 8>(p, g64, n64, st);
    else
      launch_fast<El, 64, 16>(p, g64, n64, st);
  } else {
    launch_exact<El>(p, st);
  }
}

template <typename El, int kLanes, int kN>
static void launch_route_grad(const RouteArgs& p, hipStream_t st) {
  constexpr int kTokens = 64 / kLanes;
  const dim3 grid = route_grid(((long long)p.T + kTokens - 1) / kTokens, 1 << 22);
  const dim3 block(64 * kRouteWaves);
  const bool wide = (p.E + kLanes - 1) / kLanes == kN && p.E % kN == 0 &&
                    (size_t)p.E * El::kSize % 16 == 0 &&
                    (((uintptr_t)p.logits | (uintptr_t)p.dlogits) & 15) == 0;
  if constexpr (kN * El::kSize % 16 == 0) {
    if (wide) {
      hipLaunchKernelGGL((route_grad_kernel<El, kLanes, kN, true>), grid, block, 0, st, p);
      return;
    }
  }
  hipLaunchKernelGGL((route_grad_kernel<El, kLanes, kN, false>), grid, block, 0, st, p);
}

// (72 bf16 experts, 16384 tokens with six picks and the scores' gradients: 16
// lanes to a token 8.9 us, 64 lanes 11.1)
template <typename El>
static moe_status_t launch_route(const RouteArgs& p, bool grad, hipStream_t st) {
  if (!grad)
    launch_route<El>(p, st);
  else if (p.K <= 16 && p.E <= 32)
    launch_route_grad<El, 16, 2>(p, st);
  else if (p.K <= 16 && p.E <= 64)
    launch_route_grad<El, 16, 4>(p, st);
  else if (p.K <= 16 && p.E <= 128)
    launch_route_grad<El, 16, 8>(p, st);
  else if (p.K <= 16 && p.E <= 256)
    launch_route_grad<El, 16, 16>(p, st);
  else if (p.E <= 256)
    launch_route_grad<El, 64, 4>(p, st);
  else if (p.E <= 512)
    launch_route_grad<El, 64, 8>(p, st);
  else
    launch_route_grad<El, 64, 16>(p, st);
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
