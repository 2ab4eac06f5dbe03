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
// A wave takes a token, lane l its experts l, l + 64, ...  Scores without a
// bias are in their logits' order, so the choice compares the logits; with a
// bias two candidates next to each other are told apart in 64 bits, at the
// full rate of the vector units here.  The choice takes top_k rounds: each
// lane holds its best candidate, the wave's largest key is found by DPP
// maxima of its upper word, and only on a tie the lower word and the index.
#pragma once

#include "kv_common.h"

namespace fp4q {

constexpr int kRouteThreads = 256, kRouteWaves = kRouteThreads / 64;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t stride, tokens;
  int experts, top_k, groups, top_groups, group_top, renormalize;
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
__device__ __forceinline__ float wave_total(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
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
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  else return ((const float*)p)[i];
}

// T: the type of scores and keys (float: the logits decide, or double).
template <typename T>
struct RouteKey;
template <>
struct RouteKey<float> { using type = uint32_t; };
template <>
struct RouteKey<double> { using type = uint64_t; };

__device__ __forceinline__ uint32_t upper(uint32_t k) { return k; }
__device__ __forceinline__ uint32_t upper(uint64_t k) { return (uint32_t)(k >> 32); }
__device__ __forceinline__ uint32_t lower(uint32_t) { return 0; }
__device__ __forceinline__ uint32_t lower(uint64_t k) { return (uint32_t)k; }

// Lane of the wave's largest (key, then lowest index), or -1 if all keys are 0.
template <typename K>
__device__ __forceinline__ int best_lane(K key, int index) {
  const uint32_t hi = wave_top(upper(key));
  if (hi == 0) return -1;
  uint64_t m = __ballot(upper(key) == hi);
  if (__popcll(m) > 1) {
    bool in = upper(key) == hi;
    if constexpr (sizeof(K) == 8) {
      const uint32_t lo = wave_top(in ? lower(key) : 0);
      in = in && lower(key) == lo;
      m = __ballot(in);
    }
    if (__popcll(m) > 1) {
      const uint32_t first = wave_top(in ? ~(uint32_t)index : 0);
      m = __ballot(in && ~(uint32_t)index == first);
    }
  }
  return __builtin_ctzll(m);
}

// exp in the type of the scores; the library's functions.
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// Scores s[] of a token's logits x[] (lane's experts; those past `experts` hold
// -inf): softmax needs the whole token.
template <typename T, int V>
__device__ __forceinline__ void scores_of(const float (&x)[V], bool sigmoid, T (&s)[V]) {
  if (sigmoid) {
#pragma unroll
    for (int v = 0; v < V; v++) s[v] = T(1) / (T(1) + exp_of(-(T)x[v]));
    return;
  }
  float m = x[0];                        // a NaN reaches the sum below by itself
#pragma unroll
  for (int v = 1; v < V; v++) m = fmaxf(m, x[v]);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  const T top = m == -INFINITY ? T(0) : (T)m;
  T sum = 0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    s[v] = exp_of((T)x[v] - top);
    sum += s[v];
  }
  sum = wave_total(sum);
  const T r = sum == T(0) ? T(0) : T(1) / sum;       // all masked: scores 0
#pragma unroll
  for (int v = 0; v < V; v++) s[v] *= r;
}

template <typename T, int V, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void expert_route_kernel(RouteArgs a, int sigmoid,
                                                                     float* weights,
                                                                     int32_t* experts) {
  using K = typename RouteKey<T>::type;
  const int lane = (int)threadIdx.x & 63;
  const int64_t tok = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  if (tok >= a.tokens) return;
  float x[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = v * 64 + lane;
    x[v] = e < a.experts ? logit_at<BF16>(a.logits, tok * a.stride + e) : -INFINITY;
  }
  T s[V];
  scores_of<T, V>(x, sigmoid, s);
  K key[V];
  T c[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = v * 64 + lane;
    c[v] = a.bias && e < a.experts ? s[v] + (T)a.bias[e] : (T)x[v];
    const bool open = x[v] > -INFINITY && c[v] > -INFINITY;      // neither -inf nor NaN
    key[v] = open ? key_of(c[v]) : 0;
    if (!a.bias) c[v] = s[v];            // what a group's sum is made of
  }
  if (a.groups > 1) {
    // group sizes: lane g holds group g's (up to 64 groups a round)
    const int per = a.experts / a.groups;
    auto group_of = [&](int v) { return (v * 64 + lane) / per; };
    int gr[V];
#pragma unroll
    for (int v = 0; v < V; v++) gr[v] = group_of(v);
    K size = 0;                          // key of the size of group `lane`
    for (int g = 0; g < a.groups; g++) {
      K best = 0;
      int at = 0;
#pragma unroll
      for (int v = 0; v < V; v++)
        if (gr[v] == g && key[v] > best) {
          best = key[v];
          at = v;
        }
      const int l = best_lane(best, at * 64 + lane);
      if (l < 0) continue;
      K total;
      if (a.group_top == 2) {
        T sum = 0;
        T mine = 0;
#pragma unroll
        for (int v = 0; v < V; v++) mine = at == v ? c[v] : mine;
        sum = __shfl(mine, l, 64);
        K second = 0;
        int at2 = 0;
#pragma unroll
        for (int v = 0; v < V; v++)
          if (gr[v] == g && key[v] > second && !(lane == l && v == at)) {
            second = key[v];
            at2 = v;
          }
        const int l2 = best_lane(second, at2 * 64 + lane);
        if (l2 >= 0) {
#pragma unroll
          for (int v = 0; v < V; v++) mine = at2 == v ? c[v] : mine;
          sum += __shfl(mine, l2, 64);
        }
        total = key_of(sum);
      } else {
        total = __shfl(best, l, 64);
      }
      if (lane == g) size = total;
    }
    uint64_t kept = 0;
    for (int i = 0; i < a.top_groups; i++) {
      const int l = best_lane(size, lane);
      if (l < 0) break;
      kept |= 1ull << l;
      if (lane == l) size = 0;
    }
#pragma unroll
    for (int v = 0; v < V; v++)
      if (!((kept >> (gr[v] & 63)) & 1)) key[v] = 0;
  }
  T mine_s = 0, sum = 0;
  int mine_e = -1;
  for (int j = 0; j < a.top_k; j++) {
    K best = 0;
    int at = 0;
    T bs = 0;
#pragma unroll
    for (int v = 0; v < V; v++)
      if (key[v] > best) {
        best = key[v];
        at = v;
        bs = s[v];
      }
    const int l = best_lane(best, at * 64 + lane);
    if (l < 0) break;
    const T won = __shfl(bs, l, 64);
    const int e = __shfl(at, l, 64) * 64 + l;
    sum += won;
    if (lane == j) {
      mine_s = won;
      mine_e = e;
    }
#pragma unroll
    for (int v = 0; v < V; v++)
      if (lane == l && at == v) key[v] = 0;
  }
  if (lane < a.top_k) {
    if (a.renormalize) mine_s = sum == T(0) ? T(0) : mine_s / sum;
    weights[tok * a.top_k + lane] = mine_e < 0 ? 0.0f : (float)((T)a.scale * mine_s);
    experts[tok * a.top_k + lane] = mine_e;
  }
}

template <int V, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void expert_route_backward_kernel(
    RouteArgs a, int sigmoid, const float* dweights, const int32_t* experts, void* dlogits,
    int64_t ds) {
  const int lane = (int)threadIdx.x & 63;
  const int64_t tok = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  if (tok >= a.tokens) return;
  const int e = lane < a.top_k ? experts[tok * a.top_k + lane] : -1;
  const bool there = e >= 0 && e < a.experts;
  const float g = there ? dweights[tok * a.top_k + lane] : 0.0f;
  const float l = there ? logit_at<BF16>(a.logits, tok * a.stride + e) : -INFINITY;
  float out[V];
#pragma unroll
  for (int v = 0; v < V; v++) out[v] = 0.0f;
  float d;                               // what lands on the lane's chosen expert
  if (sigmoid) {
    const float s = there ? 1.0f / (1.0f + expf(-l)) : 0.0f;
    const float not_s = 1.0f / (1.0f + expf(l));
    if (a.renormalize) {
      const float sum = wave_total(s), p = sum == 0.0f ? 0.0f : s / sum;
      d = p * not_s * (g - wave_total(p * g));
    } else {
      d = s * not_s * g;
    }
  } else if (a.renormalize) {
    float m = l;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    float p = there ? expf(l - (m == -INFINITY ? 0.0f : m)) : 0.0f;
    const float sum = wave_total(p);
    p = sum == 0.0f ? 0.0f : p / sum;
    d = p * (g - wave_total(p * g));
  } else {
    float x[V], s[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
      const int i = v * 64 + lane;
      x[v] = i < a.experts ? logit_at<BF16>(a.logits, tok * a.stride + i) : -INFINITY;
    }
    scores_of<float, V>(x, false, s);
    float mine = 0.0f;                   // the chosen expert's score
    const int from = there ? e : 0;
#pragma unroll
    for (int v = 0; v < V; v++) {
      const float o = __shfl(s[v], from & 63, 64);
      mine = from / 64 == v ? o : mine;
    }
    d = there ? mine * g : 0.0f;
    const float dot = wave_total(d);
#pragma unroll
    for (int v = 0; v < V; v++) out[v] = -(s[v] * dot);
  }
  if (!there) d = 0.0f;
  for (int j = 0; j < a.top_k; j++) {
    const int ej = __shfl(there ? e : -1, j, 64);
    const float dj = __shfl(d, j, 64);
#pragma unroll
    for (int v = 0; v < V; v++)
      if (ej == v * 64 + lane) out[v] += dj;
  }
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int i = v * 64 + lane;
    if (i >= a.experts) continue;
    const float y = a.scale * out[v];
    if constexpr (BF16) ((uint16_t*)dlogits)[tok * ds + i] = (uint16_t)bf16x2_of(y, y);
    else ((float*)dlogits)[tok * ds + i] = y;
  }
}

}  // namespace fp4q
