// route_kernels.h -- the experts of each token, and the gradient of their
// weights.
//
//   forward   s = softmax(l) or sigmoid(l),  c = l or s + bias,
//             top_k of c within the best groups,  w = scale s_i (/ sum of s_i)
//   backward  with p_i = s_i / sum of the chosen s, g the gradients of w:
//     softmax, renormalized  dl_i = scale p_i (g_i - sum_j p_j g_j), chosen only
//     softmax                dl_i = scale s_i (g_i - sum_j s_j g_j), all experts
//     sigmoid, renormalized  dl_i = scale p_i (1 - s_i) (g_i - sum_j p_j g_j)
//     sigmoid                dl_i = scale s_i (1 - s_i) g_i
//
// Instructions bound the forward, so a token belongs to 16 lanes (64 past 256
// experts or 15 choices): 4 tokens share each one.  A lane holds up to 16
// consecutive experts as 32-bit keys in the order of c, the number within the lane
// in the lowest 4 bits, so that a maximum is one instruction and names its expert.
// The first top_k + 1 of them are put in order by their exact logits or sums in 64
// bits; where one more might belong to them, or the groups' sizes are too close
// for fp32 (about one token in 10^4), the wave does the token again in 64 bits.
//
// Renormalized weights are quotients of the chosen scores, formed from
// scores over a power of e that the chosen have in common (choice_top), since the
// scores themselves may lie below fp32: sigmoids of logits below -88, and with a
// bias softmax's of logits that far below the largest.
//
// 16384 tokens of 256 experts, sigmoid, bias, 4 of 8 groups, 8 chosen: 17.7 us
// forward (the vector unit is busy for 75% of it) and 11.6 backward (44%: a lane's
// stores are a line apart); forward by a wave a token 28.7, all in 64 bits 48.8.
#pragma once

#include "kv_common.h"

namespace fp4q {

constexpr int kRouteThreads = 256, kRouteWaves = kRouteThreads / 64;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t stride, tokens;
  int experts, top_k, groups, top_groups, group_top, renormalize, sigmoid;
  int per_lane, group_lanes;             // experts of a lane; lanes of a group
  float scale;
};

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
  const uint32_t o =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  return v > o ? v : o;
}
// The largest of a (fully active) wave, uniform.
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
  v = dpp_max_u32<0x111, 0xF>(v);        // row_shr 1, 2, 4, 8
  v = dpp_max_u32<0x112, 0xF>(v);
  v = dpp_max_u32<0x114, 0xF>(v);
  v = dpp_max_u32<0x118, 0xF>(v);
  v = dpp_max_u32<0x142, 0xA>(v);        // row_bcast 15, 31
  v = dpp_max_u32<0x143, 0xC>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ double wave_total(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Keys in the order of the numbers, 0 for no candidate.
__device__ __forceinline__ uint32_t key_of(float v) {      // 0 is below every number's key
  const uint32_t b = __float_as_uint(v + 0.0f);            // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float number_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  else return ((const float*)p)[i];
}

// A lane's V values from row + V lane on, `none` past n.  Rows begin anywhere.
template <int V, bool BF16>
__device__ __forceinline__ void load_lane(const void* p, int64_t row, int n, float none, float (&x)[V]) {
  const int e = ((int)threadIdx.x & 63) * V;
  if (e + V <= n) {
    if constexpr (BF16) {
      uint16_t h[V];
      __builtin_memcpy(h, (const uint16_t*)p + row + e, sizeof(h));
#pragma unroll
      for (int v = 0; v < V; v++) x[v] = __uint_as_float((uint32_t)h[v] << 16);
    } else {
      __builtin_memcpy(x, (const float*)p + row + e, sizeof(x));
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < V; v++) x[v] = e + v < n ? logit_at<BF16>(p, row + e + v) : none;
}

// Lowest lane of the wave's largest key, or -1 if all keys are 0.
__device__ __forceinline__ int best_lane(uint64_t key) {
  const uint32_t up = (uint32_t)(key >> 32), hi = wave_top(up);
  if (hi == 0) return -1;
  uint64_t m = __ballot(up == hi);
  if (m & (m - 1)) {
    const uint32_t lo = wave_top(up == hi ? (uint32_t)key : 0);
    m = __ballot(up == hi && (uint32_t)key == lo);
  }
  return __builtin_ctzll(m);
}

// A chosen score over e^m, with m the largest choice_top(l) of a token's chosen: of
// softmax e^(l - m), of sigmoid e^(min(l, 0) - m) / (1 + e^-|l|).  Sigmoids that
// are all below e^kLeastSigmoid, the range of 64 bits, count as 0.
constexpr float kLeastSigmoid = -708.0f;
template <typename T>
__device__ __forceinline__ T choice_top(T l, int sigmoid) {
  return sigmoid && l > (T)0 ? (T)0 : l;
}
__device__ __forceinline__ float choice_score(float l, float m, int sigmoid) {
  if (!sigmoid) return expf(l - m);
  if (m < kLeastSigmoid) return 0.0f;
  return expf(choice_top(l, 1) - m) / (1.0f + expf(-fabsf(l)));
}
__device__ __forceinline__ double choice_score(double l, double m, int sigmoid) {
  if (!sigmoid) return exp(l - m);
  if (m < (double)kLeastSigmoid) return 0.0;
  return exp(choice_top(l, 1) - m) / (1.0 + exp(-fabs(l)));
}

// A score as a term of its group's size: where softmax's are NaN, all of them
// are, and all groups are of one size.
template <typename T>
__device__ __forceinline__ T size_term(T s) {
  return s == s ? s : (T)0;
}

// A lane's value in every lane.
__device__ __forceinline__ float from_lane(float v, int l) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
}
__device__ __forceinline__ double from_lane(double v, int l) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), l);
  return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

// A token by the whole wave in 64 bits, whatever its groups: lane l holds its
// experts from V l on.  Lane j gets the j-th expert and its weight but for the scale
// (-1 and 0 if there is none).
template <int V, bool BF16>
__device__ __forceinline__ void choose64(const RouteArgs& a, int64_t tok, double& mine_s, int& mine_e) {
  const int lane = (int)threadIdx.x & 63;
  float x[V], bias[V];
  load_lane<V, BF16>(a.logits, tok * a.stride, a.experts, -INFINITY, x);
#pragma unroll
  for (int v = 0; v < V; v++) bias[v] = 0.0f;
  if (a.bias) load_lane<V, false>(a.bias, 0, a.experts, 0.0f, bias);
  double s[V], c[V];
  double t = 0.0;                        // softmax's sum
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; v++) s[v] = 1.0 / (1.0 + exp(-(double)x[v]));
  } else {
    float m = x[0];                      // a NaN reaches the sum by itself
#pragma unroll
    for (int v = 1; v < V; v++) m = fmaxf(m, x[v]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    const double top = m == -INFINITY ? 0.0 : (double)m;
#pragma unroll
    for (int v = 0; v < V; v++) {
      s[v] = exp((double)x[v] - top);
      t += s[v];
    }
    t = wave_total(t);
    const double r = t == 0.0 ? 0.0 : 1.0 / t;       // all masked: scores 0
#pragma unroll
    for (int v = 0; v < V; v++) s[v] *= r;
  }
  uint64_t key[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    c[v] = a.bias ? s[v] + (double)bias[v] : (double)x[v];
    const bool open = x[v] > -INFINITY && c[v] > -INFINITY;      // neither -inf nor NaN
    key[v] = open ? key_of(c[v]) : 0;
  }
  if (a.groups > 1) {
    const int per = a.experts / a.groups, lanes = per / V;
    if (per % V == 0 && (lanes & (lanes - 1)) == 0) {
      // a group is a run of a power of two of lanes: all groups' two largest at once
      double t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; v++) {
        const double w = key[v] == 0 ? -INFINITY : (a.bias || a.group_top == 1 ? c[v] : size_term(s[v]));
        t2 = fmax(t2, fmin(t1, w));
        t1 = fmax(t1, w);
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const double o1 = __shfl_xor(t1, d, 64), o2 = __shfl_xor(t2, d, 64);
        t2 = fmax(fmax(t2, o2), fmin(t1, o1));
        t1 = fmax(t1, o1);
      }
      const double size = a.group_top == 2 && t2 > -INFINITY ? t1 + t2 : t1;
      int ahead = 0;
      for (int g = 0; g < a.groups; g++) {
        const double o = from_lane(size, g * lanes);
        ahead += o > size || (o == size && g < lane / lanes);
      }
      if (!(t1 > -INFINITY && ahead < a.top_groups))
#pragma unroll
        for (int v = 0; v < V; v++) key[v] = 0;
    } else {
    // one after another; lane g keeps group g's size
    uint64_t size = 0;
    for (int g = 0; g < a.groups; g++) {
      uint64_t best = 0, second = 0;
      double b1 = 0.0, b2 = 0.0;
#pragma unroll
      for (int v = 0; v < V; v++) {
        const int e = lane * V + v;
        if (e < g * per || e >= (g + 1) * per) continue;
        const double w = a.bias ? c[v] : size_term(s[v]);
        if (key[v] > best) {
          second = best;
          b2 = b1;
          best = key[v];
          b1 = w;
        } else if (key[v] > second) {
          second = key[v];
          b2 = w;
        }
      }
      const int l = best_lane(best);
      if (l < 0) continue;
      uint64_t total = __shfl(best, l, 64);
      if (a.group_top == 2) {
        double t = from_lane(b1, l);
        if (lane == l) {
          best = second;
          b1 = b2;
        }
        const int l2 = best_lane(best);
        if (l2 >= 0) t += from_lane(b1, l2);
        total = key_of(t);
      }
      if (lane == g) size = total;
    }
    uint64_t kept = 0;
    for (int i = 0; i < a.top_groups; i++) {
      const int l = best_lane(size);
      if (l < 0) break;
      kept |= 1ull << l;
      if (lane == l) size = 0;
    }
#pragma unroll
    for (int v = 0; v < V; v++)
      if (!((kept >> ((lane * V + v) / per & 63)) & 1)) key[v] = 0;
    }
  }
  mine_s = 0.0;
  mine_e = -1;
  for (int j = 0; j < a.top_k; j++) {
    uint64_t best = key[0];
    int at = 0;
    double bs = s[0];
#pragma unroll
    for (int v = 1; v < V; v++)
      if (key[v] > best) {
        best = key[v];
        at = v;
        bs = s[v];
      }
    const int l = best_lane(best);
    if (l < 0) break;
    const double won = from_lane(bs, l);
    const int e = l * V + __builtin_amdgcn_readlane(at, l);
    if (lane == j) {
      mine_s = won;
      mine_e = e;
    }
#pragma unroll
    for (int v = 0; v < V; v++) key[v] = lane == l && at == v ? 0 : key[v];
  }
  if (!a.renormalize) return;
  const double l = mine_e < 0 ? -INFINITY : (double)logit_at<BF16>(a.logits, tok * a.stride + mine_e);
  double m = choice_top(l, a.sigmoid);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmax(m, __shfl_xor(m, d, 64));
  mine_s = mine_e < 0 ? 0.0 : choice_score(l, m, a.sigmoid);
  if (mine_e >= 0 && t != t) mine_s = t;             // the whole token's NaN
  const double sum = wave_total(mine_s);
  mine_s = sum == 0.0 ? 0.0 : mine_s / sum;
}

// Reductions over the LPT lanes of a token; every lane gets the result.
template <int LPT>
__device__ __forceinline__ float token_max(float v) {
  v = fmaxf(v, dpp_f<kDppXor1>(v));
  v = fmaxf(v, dpp_f<kDppXor2>(v));
  v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
  v = fmaxf(v, dpp_f<kDppMirror>(v));
  if constexpr (LPT == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float token_sum(float v) {
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  v += dpp_f<kDppHalfMirror>(v);
  v += dpp_f<kDppMirror>(v);
  if constexpr (LPT == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t token_top(uint32_t v) {
  if constexpr (LPT == 64) return wave_top(v);
  v = max(v, dpp_row_u<kDppXor1>(v));
  v = max(v, dpp_row_u<kDppXor2>(v));
  v = max(v, dpp_row_u<kDppHalfMirror>(v));
  return max(v, dpp_row_u<kDppMirror>(v));
}

// How far from the truth fp32 leaves what a choice compares: scores are off by
// 2^-22 (sigmoid: exponential, sum, reciprocal) or 2^-19 (softmax: also a sum of up
// to 22 terms in a run) at most, a sum with a bias by 2^-24 of itself more, and
// a key drops up to 15 steps of 2^-24.  Two values further apart than `base`
// (1 + |value|) are in their true order.  A group's size of two of them is off by
// twice as much and 2^-24 of what it sums: by `base_sum` (1 + |terms|) at most.
__device__ __forceinline__ bool apart(float high, float low, float base) {
  return high - low > base * (1.0f + fabsf(high));
}

template <int LPT, int V, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void expert_route_kernel(RouteArgs a, float* weights,
                                                                     int32_t* experts) {
  constexpr int TOKENS = 64 / LPT;
  const int lane = (int)threadIdx.x & 63, sub = lane & (LPT - 1), row = lane / LPT;
  const int64_t first = ((int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6)) * TOKENS;
  if (first >= a.tokens) return;         // the whole wave
  const int64_t tok = first + row < a.tokens ? first + row : a.tokens - 1;
  const int n = a.per_lane, e0 = sub * n, mine = min(max(a.experts - e0, 0), n);
  float x[V], bias[V];
  const int64_t at = tok * a.stride + e0;
  if (n == V && mine == V) {             // whole vectors, beginning anywhere
    if constexpr (BF16) {
      uint16_t h[V];
      __builtin_memcpy(h, (const uint16_t*)a.logits + at, sizeof(h));
#pragma unroll
      for (int v = 0; v < V; v++) x[v] = __uint_as_float((uint32_t)h[v] << 16);
    } else {
      __builtin_memcpy(x, (const float*)a.logits + at, sizeof(x));
    }
    if (a.bias) __builtin_memcpy(bias, a.bias + e0, sizeof(bias));
  } else {
#pragma unroll
    for (int v = 0; v < V; v++) x[v] = v < mine ? logit_at<BF16>(a.logits, at + v) : -INFINITY;
    if (a.bias)
#pragma unroll
      for (int v = 0; v < V; v++) bias[v] = v < mine ? a.bias[e0 + v] : 0.0f;
  }
  // the largest logit and the sum of softmax, where scores of all are needed
  const bool all = a.bias || (a.groups > 1 && a.group_top == 2) || (!a.sigmoid && !a.renormalize);
  float top = 0.0f, total = 1.0f;
  float c[V];
#pragma unroll
  for (int v = 0; v < V; v++) c[v] = x[v];
  if (!a.sigmoid) {
    top = x[0];
#pragma unroll
    for (int v = 1; v < V; v++) top = fmaxf(top, x[v]);
    top = token_max<LPT>(top);
    top = top == -INFINITY ? 0.0f : top;
    if (all) {
      total = 0.0f;
#pragma unroll
      for (int v = 0; v < V; v++) {
        c[v] = __expf(x[v] - top);
        total += c[v];
      }
      total = token_sum<LPT>(total);
      const float r = total == 0.0f ? 0.0f : 1.0f / total;       // all masked: scores 0
#pragma unroll
      for (int v = 0; v < V; v++) c[v] *= r;
    }
  } else if (all) {
#pragma unroll
    for (int v = 0; v < V; v++) c[v] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[v]));
  }
  bool clear = true;
  const float base_sum = a.sigmoid ? 0x1p-21f : 0x1p-18f, base = base_sum + 0x1p-18f;
  constexpr bool TAGGED = BF16;          // a bf16 logit's key leaves room for the whole index
  const bool whole = TAGGED && !a.bias;
  uint32_t key[V];
  float t1 = -INFINITY, t2 = -INFINITY;  // the lane's largest, for the groups
  const bool by_score = a.bias || a.group_top == 2;
#pragma unroll
  for (int v = 0; v < V; v++) {
    if (a.bias) c[v] += bias[v];
    const float order = a.bias ? c[v] : x[v];
    const bool open = x[v] > -INFINITY && order > -INFINITY;     // neither -inf nor NaN
    key[v] = !open ? 0 : (whole ? (key_of(order) & ~0xFFFFu) | (0xFFFF - e0 - v)
                                : (key_of(order) & ~15u) | (15 - v));
    const float w = open ? (by_score ? size_term(c[v]) : x[v]) : -INFINITY;
    t2 = fmaxf(t2, fminf(t1, w));
    t1 = fmaxf(t1, w);
  }
  if (a.groups > 1) {
    // a group is a run of a power of two of lanes: all groups at once
    const int lanes = a.group_lanes;
    for (int d = 1; d < lanes; d <<= 1) {
      const float o1 = __shfl_xor(t1, d, 64), o2 = __shfl_xor(t2, d, 64);
      t2 = fmaxf(fmaxf(t2, o2), fminf(t1, o1));
      t1 = fmaxf(t1, o1);
    }
    const float size = a.group_top == 2 && t2 > -INFINITY ? t1 + t2 : t1;
    const int own = sub / lanes;
    int ahead = 0;
    for (int g = 0; g < a.groups; g++) {
      const float o = __shfl(size, row * LPT + g * lanes, 64);
      ahead += o > size || (o == size && g < own);
    }
    const bool stays = t1 > -INFINITY && ahead < a.top_groups;
    if (by_score) {
      // the smallest that stays and the largest that goes, each by as much as its terms,
      // which may cancel, can be off; infinite sizes are exact
      const float terms = fabsf(t1) + (a.group_top == 2 && t2 > -INFINITY ? fabsf(t2) : 0.0f);
      const float off = fabsf(size) < INFINITY ? base_sum * (1.0f + terms) : 0.0f;
      const float low = -token_max<LPT>(stays ? off - size : -INFINITY);
      const float high = token_max<LPT>(stays ? -INFINITY : size + off);
      if (low < INFINITY && high > -INFINITY && !(low > high)) clear = false;
    }
    if (!stays)
#pragma unroll
      for (int v = 0; v < V; v++) key[v] = 0;
  }
  // top_k + 1 candidates, lane j the j-th by key, and one more to see that none is missing
  int chosen = -1;
  float kth = INFINITY;                  // the value of the last place
  for (int j = 0; j < a.top_k + 2; j++) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; v++) best = max(best, key[v]);
    const uint32_t won = token_top<LPT>(best);
    const uint64_t m = __ballot(best == won);
    const int l = LPT == 64 ? __builtin_ctzll(m) : __builtin_ctz((uint32_t)(m >> (16 * row)) & 0xFFFFu);
    if (j == a.top_k - 1) kth = number_of(won & ~15u);
    if (j == a.top_k + 1) {
      const float next = number_of(won & ~15u);
      if (won && !whole && (a.bias ? !apart(kth, next, base) : next == kth)) clear = false;
      break;
    }
    if (sub == j && won) chosen = whole ? 0xFFFF - (int)(won & 0xFFFF) : l * n + 15 - (int)(won & 15);
    const uint32_t gone = sub == l && won ? won : 0xFFFFFFFFu;
#pragma unroll
    for (int v = 0; v < V; v++) key[v] = key[v] == gone ? 0 : key[v];
  }
  // the candidates' true order: of the logits, or of the sums in 64 bits
  const float l = chosen >= 0 ? logit_at<BF16>(a.logits, tok * a.stride + chosen) : -INFINITY;
  double c64 = (double)l;
  if (a.bias) {
    const double b = chosen >= 0 ? (double)a.bias[chosen] : -INFINITY;
    if (a.sigmoid) {
      c64 = 1.0 / (1.0 + exp(-(double)l)) + b;
    } else {                             // softmax's sum is fp32: what is close goes the long way
      c64 = chosen >= 0 ? (double)(expf(l - top) / total) + b : -INFINITY;
    }
  }
  int place = 0;
  for (int j = 0; j <= a.top_k; j++) {
    const double o = __shfl(c64, row * LPT + j, 64);
    const int oe = __shfl(chosen, row * LPT + j, 64);
    place += oe >= 0 && (o > c64 || (o == c64 && oe < chosen));
    if (a.bias && !a.sigmoid && oe >= 0 && chosen >= 0 && oe != chosen &&
        !apart((float)fmax(o, c64), (float)fmin(o, c64), base_sum))
      clear = false;
  }
  const bool in = chosen >= 0 && place < a.top_k;
  float s = 0.0f;
  if (a.renormalize) {
    // softmax's largest logit is chosen itself but for a bias or groups
    const float m = a.sigmoid || a.bias || a.groups > 1
                        ? token_max<LPT>(in ? choice_top(l, a.sigmoid) : -INFINITY) : top;
    if (in) s = choice_score(l, m, a.sigmoid);
  } else if (in) {
    s = a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / total;
  }
  if (!a.sigmoid && a.renormalize) {
    // the whole token's NaN and infinities, which its sum would carry
    bool bad = false;
#pragma unroll
    for (int v = 0; v < V; v++) bad |= !(x[v] < INFINITY);
    const uint64_t m = __ballot(bad);
    const uint64_t own = LPT == 64 ? ~0ull : 0xFFFFull << (16 * row);
    if ((m & own) && in) s = NAN;
  }
  const float sum = token_sum<LPT>(s);
  const int found = (int)token_sum<LPT>(in ? 1.0f : 0.0f);       // places past them have no expert
  const uint64_t again = __ballot(!clear);
  if (first + row < a.tokens) {
    if (in) {
      if (a.renormalize) s = sum == 0.0f ? 0.0f : s / sum;
      weights[tok * a.top_k + place] = a.scale * s;
      experts[tok * a.top_k + place] = chosen;
    }
    if (sub >= found && sub < a.top_k) {
      weights[tok * a.top_k + sub] = 0.0f;
      experts[tok * a.top_k + sub] = -1;
    }
  }
  if (!again) return;
  for (int i = 0; i < TOKENS; i++) {
    const uint64_t own = LPT == 64 ? ~0ull : 0xFFFFull << (16 * i);
    if (!(again & own) || first + i >= a.tokens) continue;
    double s64;
    int e;
    choose64<(LPT * V + 63) / 64, BF16>(a, first + i, s64, e);
    if (lane < a.top_k) {
      weights[(first + i) * a.top_k + lane] = e < 0 ? 0.0f : (float)((double)a.scale * s64);
      experts[(first + i) * a.top_k + lane] = e;
    }
  }
}

// Groups that no run of lanes holds: every token in 64 bits.
template <int V, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void expert_route64_kernel(RouteArgs a, float* weights,
                                                                       int32_t* experts) {
  const int lane = (int)threadIdx.x & 63;
  const int64_t tok = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  if (tok >= a.tokens) return;
  double s;
  int e;
  choose64<V, BF16>(a, tok, s, e);
  if (lane < a.top_k) {
    weights[tok * a.top_k + lane] = e < 0 ? 0.0f : (float)((double)a.scale * s);
    experts[tok * a.top_k + lane] = e;
  }
}

template <int LPT, int V, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void expert_route_backward_kernel(
    RouteArgs a, const float* dweights, const int32_t* experts, void* dlogits, int64_t ds) {
  constexpr int TOKENS = 64 / LPT;
  __shared__ float2 pick[kRouteWaves][64];           // a token's chosen experts and what they get
  const int lane = (int)threadIdx.x & 63, sub = lane & (LPT - 1), row = lane / LPT;
  const int64_t first = ((int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6)) * TOKENS;
  if (first >= a.tokens) return;
  const bool real = first + row < a.tokens;
  const int64_t tok = real ? first + row : a.tokens - 1;
  const int e = sub < a.top_k ? experts[tok * a.top_k + sub] : -1;
  const bool there = e >= 0 && e < a.experts;
  const float g = there ? dweights[tok * a.top_k + sub] : 0.0f;
  const float l = there ? logit_at<BF16>(a.logits, tok * a.stride + e) : -INFINITY;
  const int e0 = sub * V, mine = min(max(a.experts - e0, 0), V);
  float out[V];
#pragma unroll
  for (int v = 0; v < V; v++) out[v] = 0.0f;
  float d;                               // what lands on the lane's chosen expert
  if (a.renormalize) {
    const float m = token_max<LPT>(choice_top(l, a.sigmoid));
    float p = there ? choice_score(l, m == -INFINITY && !a.sigmoid ? 0.0f : m, a.sigmoid) : 0.0f;
    const float sum = token_sum<LPT>(p);
    p = sum == 0.0f ? 0.0f : p / sum;
    d = p * (g - token_sum<LPT>(p * g));
    if (a.sigmoid) d *= 1.0f / (1.0f + expf(l));
  } else if (a.sigmoid) {
    d = there ? 1.0f / (1.0f + expf(-l)) * (1.0f / (1.0f + expf(l))) * g : 0.0f;
  } else {
    float x[V];
    const int64_t at = tok * a.stride + e0;
    if (mine == V) {
      if constexpr (BF16) {
        uint16_t h[V];
        __builtin_memcpy(h, (const uint16_t*)a.logits + at, sizeof(h));
#pragma unroll
        for (int v = 0; v < V; v++) x[v] = __uint_as_float((uint32_t)h[v] << 16);
      } else {
        __builtin_memcpy(x, (const float*)a.logits + at, sizeof(x));
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; v++) x[v] = v < mine ? logit_at<BF16>(a.logits, at + v) : -INFINITY;
    }
    float m = x[0], sum = 0.0f;
#pragma unroll
    for (int v = 1; v < V; v++) m = fmaxf(m, x[v]);
    m = token_max<LPT>(m);
    m = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int v = 0; v < V; v++) {
      x[v] = expf(x[v] - m);
      sum += x[v];
    }
    sum = token_sum<LPT>(sum);
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
    d = there ? expf(l - m) * r * g : 0.0f;
    const float dot = token_sum<LPT>(d);
#pragma unroll
    for (int v = 0; v < V; v++) out[v] = -(x[v] * r * dot);
  }
  float2* const mine_picks = pick[threadIdx.x >> 6] + row * LPT;
  mine_picks[sub] = make_float2(__int_as_float(there ? e : -1), there ? d : 0.0f);
  wave_lds_sync();
  for (int j = 0; j < a.top_k; j++) {
    const float2 p = mine_picks[j];
    const int at = __float_as_int(p.x) - e0;
#pragma unroll
    for (int v = 0; v < V; v++) out[v] += at == v ? p.y : 0.0f;
  }
  if (!real) return;
#pragma unroll
  for (int v = 0; v < V; v++) out[v] *= a.scale;
  const int64_t to = tok * ds + e0;
  if constexpr (BF16) {
    uint16_t h[V];
#pragma unroll
    for (int v = 0; v < V; v++) h[v] = (uint16_t)bf16x2_of(out[v], out[v]);
    uint16_t* p = (uint16_t*)dlogits + to;
    if (mine == V) __builtin_memcpy(p, h, sizeof(h));
    else
#pragma unroll
      for (int v = 0; v < V; v++)
        if (v < mine) p[v] = h[v];
  } else {
    float* p = (float*)dlogits + to;
    if (mine == V) __builtin_memcpy(p, out, sizeof(out));
    else
#pragma unroll
      for (int v = 0; v < V; v++)
        if (v < mine) p[v] = out[v];
  }
}

}  // namespace fp4q
