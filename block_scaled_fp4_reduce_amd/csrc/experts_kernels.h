// experts_kernels.h -- sorting a batch's assignments by expert, and joining the
// experts' outputs of a token.
//
// An assignment a = t * top_k + j sends token t to expert ids[a].
#pragma once

#include "weights_common.h"

namespace fp4q {

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;

// Stable counting sort in one launch: workgroup e counts the assignments of
// expert e and those of the experts before it (every workgroup reads all ids,
// from L2), so off[e] needs no other workgroup; then it writes its own, in
// order, to order[off[e]] ...  Numbers outside [0, experts) are left out.
// Latency bounds it, so a wave asks for kPlanAhead runs of ids at once (24576
// assignments of 64 experts: one run at a time 17.0 us, 8 9.3).
constexpr int kPlanAhead = 8;

__global__ __launch_bounds__(kPlanThreads) void expert_plan_kernel(const int32_t* __restrict__ ids,
                                                                   int n, int experts,
                                                                   int32_t* __restrict__ off,
                                                                   int32_t* __restrict__ order) {
  __shared__ int mine_of[kPlanWaves], less_of[kPlanWaves];
  const int e = (int)blockIdx.x, t = (int)threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t per = ((int64_t)n + kPlanThreads - 1) / kPlanThreads * 64;   // ids of a wave
  const int64_t i0 = wave * per, i1 = i0 + per < n ? i0 + per : n;
  auto runs = [&](int64_t i, int (&id)[kPlanAhead]) {
#pragma unroll
    for (int r = 0; r < kPlanAhead; r++) {
      const int64_t at = i + 64 * r + lane;
      id[r] = ids[at < n ? at : n - 1];
      if (at >= i1) id[r] = -1;
    }
  };
  int mine = 0, less = 0;                // of the wave
  for (int64_t i = i0; i < i1; i += 64 * kPlanAhead) {
    int id[kPlanAhead];
    runs(i, id);
#pragma unroll
    for (int r = 0; r < kPlanAhead; r++) {
      mine += __popcll(__ballot(id[r] == e));
      less += __popcll(__ballot(id[r] >= 0 && id[r] < e));
    }
  }
  if (lane == 0) {
    mine_of[wave] = mine;
    less_of[wave] = less;
  }
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < kPlanWaves; w++) {
    at += less_of[w] + (w < wave ? mine_of[w] : 0);
    total += less_of[w];
  }
  if (t == 0) off[e] = total;
  if (e == experts - 1 && t == 0) {
    for (int w = 0; w < kPlanWaves; w++) total += mine_of[w];
    off[experts] = total;
  }
  if (!mine) return;
  for (int64_t i = i0; i < i1; i += 64 * kPlanAhead) {
    int id[kPlanAhead];
    runs(i, id);
#pragma unroll
    for (int r = 0; r < kPlanAhead; r++) {
      const uint64_t m = __ballot(id[r] == e);
      if (id[r] == e) order[at + __popcll(m & ((1ull << lane) - 1))] = (int32_t)(i + 64 * r + lane);
      at += __popcll(m);
    }
  }
}

// out[t] = sum_j weights[t][j] y[t * top_k + j] over the assignments that have
// an expert; y fp32 [assignments][cols].  A thread takes 4 columns of a token.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void experts_join_kernel(
    const float* __restrict__ y, const float* __restrict__ weights, const int32_t* __restrict__ ids,
    int64_t tokens, int top_k, int experts, int cols, uint16_t* __restrict__ out, int64_t os) {
  const int64_t per = cols / 4, i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int64_t t = i / per;
  if (t >= tokens) return;
  const int64_t c = (i - t * per) * 4;
  f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < top_k; j++) {
    const int64_t at = t * top_k + j;
    const int id = ids[at];
    if (id < 0 || id >= experts) continue;
    const float w = weights[at];
    const f32x4_t v = *(const f32x4_t*)(y + at * cols + c);
#pragma unroll
    for (int q = 0; q < 4; q++) sum[q] = __builtin_fmaf(w, v[q], sum[q]);
  }
  *(u32x2_t*)(out + t * os + c) = u32x2_t{bf16x2_of(sum[0], sum[1]), bf16x2_of(sum[2], sum[3])};
}

}  // namespace fp4q
