// rope_kernels.h -- RMS norm of each query and key head with the position
// rotation in the same pass, forward and backward.
//
//   forward   n = x / sqrt(mean(x^2) + eps),  y = R (n w)
//   backward  g = R^T dy,  dx = r (w g - n mean(w g n)),  dw = sum g n,
//             r = 1 / sqrt(mean(x^2) + eps)
// with R the rotation of value pairs by the angles of the token's position
// (pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved); values past rot
// pass through.  Without a weight the norm is left out (r = w = 1).
//
// Mapping: a lane holds 8 consecutive values of a head (one 16-byte load), so
// a head of D values is a group of D/8 lanes (rounded up to a power of two)
// and its mean is a butterfly inside the group; the pair partner of the
// half-split rotation sits rot/16 lanes away.  A group takes several heads
// of one token, so the token's cosines and sines are read once for them.
// Everything is fp32 until the one rounding to bf16 at the store.
//
// Memory bounds it: 8192 tokens of 40 heads of 128 (84 MB a tensor) forward
// in 34.3 to 35.1 us (4.8 TB/s), backward in 53.4 (4.7 TB/s) and 5.1 for the
// join of the weight gradients.  With one head per lane group the cosines are read
// for every head and the pair takes 170 us instead of 93.
#pragma once

#include "kv_common.h"

namespace fp4q {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxGroups = 1024;     // workgroups of the backward pass: rows of partial dw

struct RopeArgs {
  const uint16_t *q, *k;
  const uint16_t *qw, *kw;               // NULL: no norm
  const int64_t* pos;
  const float* table;                    // [table_rows][rot/2] (cos, sin)
  int64_t qs, ks;                        // elements between tokens
  int64_t tokens, table_rows;
  int hq, hk, dim, rot;
  int hpg, chunks;                       // heads per lane group; groups per token
  float eps;
};

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LPH / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// v <- n = v r of one head.  Returns r.  Where the squares leave the range of
// fp32 (values past 2^60; with an eps below 2^-90 also small ones) the head is
// scaled by a power of two first; r itself may then be a subnormal.
template <int LPH>
__device__ __forceinline__ float norm_head(float* v, const RopeArgs& a) {
  float ss = 0.0f, c = 1.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) ss = __builtin_fmaf(v[i], v[i], ss);
  ss = group_sum<LPH>(ss) / (float)a.dim + a.eps;
  if (!(ss >= 0x1p-90f && ss <= 3.402823466e38f)) {
    c = ss < 1.0f ? 0x1p100f : 0x1p-80f;
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      v[i] *= c;
      ss = __builtin_fmaf(v[i], v[i], ss);
    }
    ss = group_sum<LPH>(ss) / (float)a.dim + a.eps * c * c;
  }
  const float r = 1.0f / sqrtf(ss);
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] *= r;
  return r * c;
}

// One lane's cosines and sines: its 8 values' pairs (half-split), or its 4
// pairs (interleaved).
template <bool INTER>
struct Turn {
  static constexpr int N = INTER ? 4 : 8;
  float c[N], s[N];
  bool on;                               // the lane's values are rotated
  bool second;                           // half-split: the pair's second members
  int partner;                           // half-split: lane with the other members
  __device__ __forceinline__ void load(const RopeArgs& a, int64_t row, int sub) {
    const int first = sub * 8;
    on = first < a.rot;
    second = !INTER && first >= a.rot / 2;
    const int lane = (int)(threadIdx.x & 63), half = a.rot / 16;
    partner = !on || INTER ? lane : (second ? lane - half : lane + half);
    const int pair = INTER ? sub * 4 : (second ? first - a.rot / 2 : first);
    if (!on) {
#pragma unroll
      for (int i = 0; i < N; i++) {
        c[i] = 1.0f;
        s[i] = 0.0f;
      }
      return;
    }
    const float4* t = (const float4*)(a.table + (row * (a.rot / 2) + pair) * 2);
#pragma unroll
    for (int i = 0; i < N / 2; i++) {
      const float4 v = t[i];
      c[2 * i] = v.x;
      s[2 * i] = v.y;
      c[2 * i + 1] = v.z;
      s[2 * i + 1] = v.w;
    }
  }
  // v <- R v (BACK: R^T v)
  template <bool BACK>
  __device__ __forceinline__ void apply(float* v) const {
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float sn = BACK ? -s[i] : s[i];
        const float x = v[2 * i], y = v[2 * i + 1];
        v[2 * i] = __builtin_fmaf(x, c[i], -(y * sn));
        v[2 * i + 1] = __builtin_fmaf(y, c[i], x * sn);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float o = __shfl(v[i], partner, 64);
        // first member: x c - o s; second: x c + o s
        const float sn = second != BACK ? s[i] : -s[i];
        v[i] = on ? __builtin_fmaf(v[i], c[i], o * sn) : v[i];
      }
    }
  }
};

struct HeadPtr {
  const uint16_t* x;
  int64_t off;                           // element offset of the head in its tensor
};

// Heads are numbered through: queries first, then keys.
__device__ __forceinline__ int64_t head_off(const RopeArgs& a, int64_t tok, int h, int64_t qs,
                                            int64_t ks) {
  return h < a.hq ? tok * qs + (int64_t)h * a.dim : tok * ks + (int64_t)(h - a.hq) * a.dim;
}

__device__ __forceinline__ int64_t table_row(const RopeArgs& a, int64_t tok) {
  if (a.rot == 0) return 0;              // no table
  const int64_t p = a.pos[tok];
  return p < 0 ? 0 : (p < a.table_rows ? p : a.table_rows - 1);
}

template <int LPH, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope_kernel(RopeArgs a, uint16_t* qo,
                                                                    int64_t qos, uint16_t* ko,
                                                                    int64_t kos) {
  const int sub = (int)threadIdx.x & (LPH - 1);
  const bool live = sub * 8 < a.dim;
  const int64_t item =
      (int64_t)blockIdx.x * (kRopeThreads / LPH) + (int64_t)(threadIdx.x / LPH);
  if (item >= a.tokens * a.chunks) return;
  const int64_t tok = item / a.chunks;
  const int h0 = (int)(item - tok * a.chunks) * a.hpg;
  const int h1 = min(h0 + a.hpg, a.hq + a.hk);
  const int64_t trow = table_row(a, tok);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](int h) {
    const uint16_t* x = (h < a.hq ? a.q : a.k) + head_off(a, tok, h, a.qs, a.ks);
    return live ? *(const uint4*)(x + sub * 8) : zero;
  };
  auto weight = [&](const uint16_t* w) {
    return w && live ? *(const uint4*)(w + sub * 8) : zero;
  };
  const uint4 wq = weight(a.qw), wk = weight(a.kw);
  uint4 next = load(h0);
  Turn<INTER> turn;                      // its rows wait for the position: last
  turn.load(a, trow, sub);
  for (int h = h0; h < h1; h++) {
    const uint4 raw = next;
    if (h + 1 < h1) next = load(h + 1);
    float v[8], w[8];
    unpack8(raw, v);
    if (h < a.hq ? a.qw != nullptr : a.kw != nullptr) {
      unpack8(h < a.hq ? wq : wk, w);
      norm_head<LPH>(v, a);
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] *= w[i];
    }
    turn.template apply<false>(v);
    uint16_t* y = (h < a.hq ? qo : ko) + head_off(a, tok, h, qos, kos);
    if (live) *(uint4*)(y + sub * 8) = pack8(v);
  }
}

// Partial weight gradients of workgroup b go to partial[b][0 = q, 1 = k][dim],
// or without it (one workgroup) the gradients to dqw and dkw.  A lane sums its
// own heads in fp32, in one run, and the workgroup's lanes after that; the
// workgroups are joined in 64 bits.  A run is at most tokens x heads x lanes a
// head / 2^18 terms and one group of heads: 20 for 8192 tokens of 40 heads of
// 128, 2560 for a million, an error of as many 2^-24 of sum |g n| at worst.
template <int LPH, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope_bwd_kernel(
    RopeArgs a, const uint16_t* dqo, int64_t dqos, const uint16_t* dko, int64_t dkos, uint16_t* dq,
    int64_t dqs, uint16_t* dk, int64_t dks, float* partial, float* dqw, float* dkw) {
  __shared__ float red[kRopeThreads / LPH][2][LPH * 8];
  const int sub = (int)threadIdx.x & (LPH - 1), grp = (int)threadIdx.x / LPH;
  const bool live = sub * 8 < a.dim;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto weight = [&](const uint16_t* w) {
    return w && live ? *(const uint4*)(w + sub * 8) : zero;
  };
  const uint4 wq = weight(a.qw), wk = weight(a.kw);
  float gq[8] = {}, gk[8] = {};
  const int64_t items = a.tokens * a.chunks;
  for (int64_t item = (int64_t)blockIdx.x * (kRopeThreads / LPH) + grp; item < items;
       item += (int64_t)gridDim.x * (kRopeThreads / LPH)) {
    const int64_t tok = item / a.chunks;
    const int h0 = (int)(item - tok * a.chunks) * a.hpg;
    const int h1 = min(h0 + a.hpg, a.hq + a.hk);
    const int64_t trow = table_row(a, tok);
    auto load_x = [&](int h) {
      const uint16_t* x = (h < a.hq ? a.q : a.k) + head_off(a, tok, h, a.qs, a.ks);
      return live ? *(const uint4*)(x + sub * 8) : zero;
    };
    auto load_g = [&](int h) {
      const uint16_t* g = (h < a.hq ? dqo : dko) + head_off(a, tok, h, dqos, dkos);
      return live ? *(const uint4*)(g + sub * 8) : zero;
    };
    uint4 nx = load_x(h0), ng = load_g(h0);
    Turn<INTER> turn;
    turn.load(a, trow, sub);
    for (int h = h0; h < h1; h++) {
      const uint4 rx = nx, rg = ng;
      if (h + 1 < h1) {
        nx = load_x(h + 1);
        ng = load_g(h + 1);
      }
      float g[8], x[8], w[8];
      unpack8(rg, g);
      turn.template apply<true>(g);
      const bool isq = h < a.hq;
      if (isq ? a.qw != nullptr : a.kw != nullptr) {
        unpack8(rx, x);
        unpack8(isq ? wq : wk, w);
        const float r = norm_head<LPH>(x, a);         // x is n now
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float t = g[i] * x[i];
          gq[i] += isq ? t : 0.0f;
          gk[i] += isq ? 0.0f : t;
          g[i] *= w[i];
          dot = __builtin_fmaf(g[i], x[i], dot);
        }
        const float mean = group_sum<LPH>(dot) / (float)a.dim;
#pragma unroll
        for (int i = 0; i < 8; i++) g[i] = r * __builtin_fmaf(-x[i], mean, g[i]);
      }
      uint16_t* y = (isq ? dq : dk) + head_off(a, tok, h, dqs, dks);
      if (live) *(uint4*)(y + sub * 8) = pack8(g);
    }
  }
  if (!partial && !dqw && !dkw) return;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    red[grp][0][sub * 8 + i] = gq[i];
    red[grp][1][sub * 8 + i] = gk[i];
  }
  __syncthreads();
  for (int j = (int)threadIdx.x; j < 2 * a.dim; j += kRopeThreads) {
    const int which = j >= a.dim, c = which ? j - a.dim : j;
    if (partial) {
      float t = 0.0f;
      for (int g = 0; g < kRopeThreads / LPH; g++) t += red[g][which][c];
      partial[(int64_t)blockIdx.x * 2 * a.dim + j] = t;
    } else if (float* out = which ? dkw : dqw) {
      double t = 0.0;
      for (int g = 0; g < kRopeThreads / LPH; g++) t += (double)red[g][which][c];
      out[c] = (float)t;
    }
  }
}

// dw = sum of the workgroups' partials, in a fixed order and 64 bits (the
// sum runs over every token): 8 columns per workgroup, 128 rows at a time, so
// that a thread's few loads are all on their way at once.
constexpr int kDwThreads = 1024, kDwCols = 8, kDwRows = kDwThreads / kDwCols;
__global__ __launch_bounds__(kDwThreads) void qk_norm_rope_dw_kernel(const float* partial, int rows,
                                                                     int dim, float* dqw,
                                                                     float* dkw) {
  __shared__ double red[kDwRows][kDwCols];
  const int c = (int)threadIdx.x % kDwCols, r = (int)threadIdx.x / kDwCols;
  const int j = (int)blockIdx.x * kDwCols + c;
  double t = 0.0;
  if (j < 2 * dim) {
    float x[kRopeMaxGroups / kDwRows];
#pragma unroll
    for (int i = 0; i < kRopeMaxGroups / kDwRows; i++) {
      const int row = r + i * kDwRows;
      x[i] = row < rows ? partial[(int64_t)row * 2 * dim + j] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kRopeMaxGroups / kDwRows; i++) t += (double)x[i];
  }
  red[r][c] = t;
  for (int half = kDwRows / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (r < half) red[r][c] = t += red[r + half][c];
  }
  if (r == 0 && j < 2 * dim) {
    float* out = j < dim ? dqw : dkw;
    if (out) out[j < dim ? j : j - dim] = (float)t;
  }
}

}  // namespace fp4q
