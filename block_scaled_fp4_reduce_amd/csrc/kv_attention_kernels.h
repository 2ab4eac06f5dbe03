// kv_attention_kernels.h -- attention of new tokens over the paged FP4 cache.
//
// Token i of a sequence's n new ones stands at position pos = len - n + i
// and sees the cached tokens j <= pos (with a window W also j > pos - W):
//   s_j = scale q . K_j,  s_j <- cap tanh(s_j / cap) with a cap,
//   p = softmax(s),  out = sum p_j V_j,  lse = log sum exp(s_j)
// K and V are the decoded values of the cache.  A token that sees nothing
// gets out = 0 and lse = -inf.
#pragma once

#include "kv_common.h"

namespace fp4q {

struct AttnArgs {
  KvView c;
  const uint16_t* q;
  const int32_t *pt, *lens, *cu;
  uint16_t* out;
  float* lse;                            // [tokens][hq] or NULL
  int64_t qs, os;                        // elements between tokens
  int64_t tokens, seqs, width;
  int hq, group, window;
  float scale, cap;                      // cap 0: none
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// The sequence that token `tok` belongs to: the last b with cu[b] <= tok.
__device__ __forceinline__ int64_t seq_of(const AttnArgs& a, int64_t tok) {
  if (!a.cu) return tok;
  int64_t lo = 0, hi = a.seqs;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.cu[mid] <= tok) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One wave per query row, a key at a time, D / 64 values per lane.
// MODE: 0 NVFP4, 1 NVFP4 with 4/6, 2 MXFP4.
template <int MODE, int D>
__global__ __launch_bounds__(kThreads) void kv_attention_kernel(AttnArgs a) {
  constexpr int G = MODE == 2 ? 32 : 16, VPL = D / 64;
  const int lane = (int)threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= a.tokens * a.hq) return;
  const int64_t tok = row / a.hq;
  const int head = (int)(row - tok * a.hq), h = head / a.group;
  const int64_t b = seq_of(a, tok);
  const int64_t n = a.cu ? a.cu[b + 1] - a.cu[b] : 1, i = a.cu ? tok - a.cu[b] : 0;
  const int P = 1 << a.c.page_shift;
  int64_t len = a.lens[b];
  if (len > a.width * P) len = a.width * P;
  const bool in_seq = i >= 0 && i < n;
  const int64_t pos = len - n + i;
  const int64_t hi = in_seq ? pos + 1 : 0;
  const int64_t lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
  const float C = MODE == 1 ? 256.0f : 448.0f;
  const float ka = MODE == 2 ? 1.0f : a.c.kam[h] / (6.0f * C);
  const float va = MODE == 2 ? 1.0f : a.c.vam[h] / (6.0f * C);
  auto grid = [](uint32_t code) {
    const uint32_t m = code & 7u;
    const float v = m < 4 ? 0.5f * (float)m : (m == 4 ? 2.0f : (m == 5 ? 3.0f : (m == 6 ? 4.0f : 6.0f)));
    return code & 8u ? -v : v;
  };
  auto scale_of = [](uint32_t code) {
    return MODE == 2 ? __builtin_ldexpf(1.0f, (int)code - 127) : e4m3_value(code & 0x7Fu);
  };
  float q[VPL], o[VPL] = {};
#pragma unroll
  for (int e = 0; e < VPL; e++)
    q[e] = __uint_as_float((uint32_t)a.q[tok * a.qs + head * D + lane * VPL + e] << 16);
  float m = -__builtin_inff(), l = 0.0f;
  for (int64_t j = lo; j < hi; j++) {
    const int64_t page = a.pt[b * a.width + (j >> a.c.page_shift)];
    if (page < 0 || page >= a.c.pages) continue;
    const int at = (int)(j & (P - 1));
    const int64_t ph = page * a.c.heads + h;
    float s = 0.0f, vv[VPL];
#pragma unroll
    for (int e = 0; e < VPL; e++) {
      const int ch = lane * VPL + e;
      const uint32_t kb = a.c.kc[(ph * P + at) * (D / 2) + ch / 2];
      const uint32_t vb = a.c.vc[(ph * (D / 2) + ch / 2) * P + at];
      const float kscale = scale_of(a.c.ks[(ph * P + at) * (D / G) + ch / G]);
      const float vscale = scale_of(a.c.vs[(ph * (D / G) + ch / G) * P + at]);
      s += q[e] * (grid(ch & 1 ? kb >> 4 : kb & 15u) * (ka * kscale));
      vv[e] = grid(ch & 1 ? vb >> 4 : vb & 15u) * (va * vscale);
    }
    s = wave_sum(s) * a.scale;
    if (a.cap > 0.0f) s = a.cap * tanhf(s / a.cap);
    const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < VPL; e++) o[e] = o[e] * f + p * vv[e];
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < VPL; e++) {
    const uint32_t w = bf16x2_of(l > 0.0f ? o[e] / l : 0.0f, 0.0f);
    a.out[tok * a.os + head * D + lane * VPL + e] = (uint16_t)w;
  }
  if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? m + logf(l) : -__builtin_inff();
}

}  // namespace fp4q
