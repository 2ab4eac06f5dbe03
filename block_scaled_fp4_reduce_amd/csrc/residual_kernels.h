// residual_kernels.h -- the norms before and after a block with its gate and
// the scale of the residual stream, forward and backward.
//
//   forward   n = b rb wb,  y = s x + g n,  z = y r w
//   backward  u = w dz,  dY = dy + r (u - yh mean(u yh)),  dx = s dY,
//             h = g wb dY,  db = rb (h - bh mean(h bh)),
//             dw = sum dz yh,  dwb = sum g dY bh,  dg = sum dY n
// with rb = 1 / sqrt(mean(b^2) + eps), bh = b rb, r and yh alike for y; without
// a block weight n = b, db = g dY.  sum: over the tokens, for a token's gate
// over its channels.
//
// A row belongs to 1, 4 or 16 waves, a thread holds 8 consecutive values
// (one 16-byte load) of each of its CH chunks, and everything stays in registers
// between the one read and the one write, but for the backward pass of more than
// 8192 channels: a thread of 16 waves has 128 registers, and 641 values go to
// scratch (4096 tokens of 16384 channels 4.85 ms; of 8192 channels 0.12).  The
// backward pass reads x again and makes y from it: the same bytes as reading y,
// which is rounded.  All fp32 but for the squares' sums that leave its range (Rms
// below) and the tokens' sums, which are joined in 64 bits.  Memory bounds the rest:
// 8192 tokens of 4096 channels 50 us forward (5.4 TB/s), 95 backward (4.2 TB/s) and
// 7 for the weights' sums; forward 4096 tokens of 16384 channels 114 (4.7 TB/s).
#pragma once

#include "kv_common.h"

namespace fp4q {

constexpr int kResidualMaxGroups = 512;  // rows of partial weight gradients

struct ResidualArgs {
  const uint16_t *x, *b;
  const uint16_t *bw, *w, *gate;         // bw: NULL without a norm of the block; gate: NULL
  int64_t xs, bs, tokens;
  int dim, token_gate;
  float scale, eps;
};

// WPR waves a row; rows of a workgroup; threads.
template <int WPR>
struct RowShape {
  static constexpr int kRows = WPR == 1 ? 4 : 1, kThreadsRow = WPR * 64;
  static constexpr int kAll = kRows * kThreadsRow;
};

// Sums of N values over the threads of a row; every thread gets them.
template <int WPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds /* [2][WPR * N] */, int& turn) {
#pragma unroll
  for (int i = 0; i < N; i++)
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v[i] += __shfl_xor(v[i], d, 64);
  if constexpr (WPR > 1) {               // buffers alternate: one barrier a sum
    float* at = lds + (turn & 1) * (WPR * 4);
    turn++;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; i++) at[i * WPR + (threadIdx.x >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < WPR; w++) t += at[i * WPR + w];
      v[i] = t;
    }
  }
}

// 1 / sqrt(mean(v^2) + eps) of a row as r * c, v scaled by c where the squares
// leave the range of fp32 (c a power of two, usually 1): v r is normalized.
struct Rms {
  float r, c;
};
template <int WPR, int N>
__device__ __forceinline__ Rms row_rms(float (&v)[N], int dim, float eps, float* lds, int& turn) {
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < N; i++) ss[0] = __builtin_fmaf(v[i], v[i], ss[0]);
  row_sums<WPR>(ss, lds, turn);
  float m = ss[0] / (float)dim + eps, c = 1.0f;
  if (!(m >= 0x1p-90f && m <= 3.402823466e38f)) {    // the same for the whole row
    c = m < 1.0f ? 0x1p100f : 0x1p-80f;
    ss[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
      v[i] *= c;
      ss[0] = __builtin_fmaf(v[i], v[i], ss[0]);
    }
    row_sums<WPR>(ss, lds, turn);
    m = ss[0] / (float)dim + eps * c * c;
  }
  return {1.0f / sqrtf(m), c};
}

// A thread's columns: chunk j holds (j * threads + thread) * 8 .. + 7.
template <int WPR, int CH>
struct RowLane {
  int sub;                               // thread of the row
  __device__ __forceinline__ int col(int j) const {
    return (j * RowShape<WPR>::kThreadsRow + sub) * 8;
  }
  __device__ __forceinline__ void load(const uint16_t* row, int dim, float (&v)[CH * 8]) const {
    uint4 raw[CH];
#pragma unroll
    for (int j = 0; j < CH; j++)
      raw[j] = col(j) < dim ? *(const uint4*)(row + col(j)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < CH; j++) unpack8(raw[j], v + 8 * j);
  }
  __device__ __forceinline__ void store(uint16_t* row, int dim, const float (&v)[CH * 8]) const {
#pragma unroll
    for (int j = 0; j < CH; j++)
      if (col(j) < dim) *(uint4*)(row + col(j)) = pack8(v + 8 * j);
  }
};

// The gate of a row: NULL 1, a token's one number, or the channels'.
template <int CH>
__device__ __forceinline__ float token_gate(const ResidualArgs& a, int64_t row) {
  return a.gate && a.token_gate ? __uint_as_float((uint32_t)a.gate[row] << 16) : 1.0f;
}

template <int WPR, int CH>
__global__ __launch_bounds__(RowShape<WPR>::kAll) void residual_norm_kernel(ResidualArgs a,
                                                                            uint16_t* y, int64_t ys,
                                                                            uint16_t* z,
                                                                            int64_t zs) {
  using S = RowShape<WPR>;
  __shared__ float lds[WPR * 8];
  const int64_t row = (int64_t)blockIdx.x * S::kRows + threadIdx.x / S::kThreadsRow;
  if (row >= a.tokens) return;           // whole waves, and only where rows share no barrier
  const RowLane<WPR, CH> me{(int)threadIdx.x % S::kThreadsRow};
  int turn = 0;
  float x[CH * 8], b[CH * 8], w[CH * 8];
  me.load(a.x + row * a.xs, a.dim, x);
  me.load(a.b + row * a.bs, a.dim, b);
  me.load(a.w, a.dim, w);
  const float tg = token_gate<CH>(a, row);
  if (a.bw) {
    float bw[CH * 8];
    me.load(a.bw, a.dim, bw);
    const Rms q = row_rms<WPR>(b, a.dim, a.eps, lds, turn);
#pragma unroll
    for (int i = 0; i < CH * 8; i++) b[i] = b[i] * q.r * bw[i];
  }
  if (a.gate && !a.token_gate) {
    float g[CH * 8];
    me.load(a.gate, a.dim, g);
#pragma unroll
    for (int i = 0; i < CH * 8; i++) b[i] *= g[i];
  }
#pragma unroll
  for (int i = 0; i < CH * 8; i++) x[i] = __builtin_fmaf(tg, b[i], a.scale * x[i]);
  me.store(y + row * ys, a.dim, x);
  const Rms q = row_rms<WPR>(x, a.dim, a.eps, lds, turn);
#pragma unroll
  for (int i = 0; i < CH * 8; i++) x[i] = x[i] * q.r * w[i];
  me.store(z + row * zs, a.dim, x);
}

// Partial sums of workgroup i over its rows: partial[i][0][dim] of g dY bh (or,
// with a channel's gate, dY bh), partial[i][1][dim] of dz yh.  NULL: not wanted.
// A thread's run is tokens / 512 terms in fp32.
template <int WPR, int CH>
__global__ __launch_bounds__(RowShape<WPR>::kAll) void residual_norm_bwd_kernel(
    ResidualArgs a, const uint16_t* dy, int64_t dys, const uint16_t* dz, int64_t dzs, uint16_t* dx,
    int64_t dxs, uint16_t* db, int64_t dbs, float* partial, float* dgate) {
  using S = RowShape<WPR>;
  __shared__ float lds[WPR * 8];
  __shared__ float join[S::kRows > 1 ? S::kRows * 64 * 8 : 1];
  const RowLane<WPR, CH> me{(int)threadIdx.x % S::kThreadsRow};
  const int sub_row = (int)threadIdx.x / S::kThreadsRow;
  int turn = 0;
  float sum_b[CH * 8] = {}, sum_w[CH * 8] = {};
  const float inv = 1.0f / (float)a.dim;
  for (int64_t row = (int64_t)blockIdx.x * S::kRows + sub_row; row < a.tokens;
       row += (int64_t)gridDim.x * S::kRows) {
    float x[CH * 8], b[CH * 8], gy[CH * 8], gz[CH * 8];
    me.load(a.x + row * a.xs, a.dim, x);
    me.load(a.b + row * a.bs, a.dim, b);
    me.load(dy + row * dys, a.dim, gy);
    me.load(dz + row * dzs, a.dim, gz);
    const float tg = token_gate<CH>(a, row);
    Rms qb = {1.0f, 1.0f};
    if (a.bw) {
      qb = row_rms<WPR>(b, a.dim, a.eps, lds, turn);
#pragma unroll
      for (int i = 0; i < CH * 8; i++) b[i] *= qb.r;           // bh
    }
    // x becomes y: s x + tg wb gate bh
    float m[CH * 8];                     // wb gate, the factor of bh
#pragma unroll
    for (int i = 0; i < CH * 8; i++) m[i] = 1.0f;
    if (a.bw) me.load(a.bw, a.dim, m);
    if (a.gate && !a.token_gate) {
      float g[CH * 8];
      me.load(a.gate, a.dim, g);
#pragma unroll
      for (int i = 0; i < CH * 8; i++) m[i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < CH * 8; i++) x[i] = __builtin_fmaf(tg, b[i] * m[i], a.scale * x[i]);
    const Rms q = row_rms<WPR>(x, a.dim, a.eps, lds, turn);
    float w[CH * 8];
    me.load(a.w, a.dim, w);
    float t[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < CH * 8; i++) {
      x[i] *= q.r;                       // yh
      sum_w[i] = __builtin_fmaf(gz[i], x[i], sum_w[i]);
      gz[i] *= w[i];                     // u
      t[0] = __builtin_fmaf(gz[i], x[i], t[0]);
    }
    row_sums<WPR>(t, lds, turn);
    const float mean = t[0] * inv, r = q.r * q.c;
    t[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < CH * 8; i++) {
      gy[i] = __builtin_fmaf(r, __builtin_fmaf(-x[i], mean, gz[i]), gy[i]);      // dY
      const float d = gy[i] * b[i];
      sum_b[i] += tg * d;
      t[0] = __builtin_fmaf(m[i], d, t[0]);          // dY n
      x[i] = a.scale * gy[i];
    }
    me.store(dx + row * dxs, a.dim, x);
    if (a.bw || dgate) row_sums<WPR>(t, lds, turn);  // the same for the whole workgroup
    if (dgate && a.token_gate && me.sub == 0) dgate[row] = t[0];
    const float mb = a.bw ? tg * t[0] * inv : 0.0f, rb = qb.r * qb.c;
#pragma unroll
    for (int i = 0; i < CH * 8; i++)
      x[i] = rb * __builtin_fmaf(-b[i], mb, tg * m[i] * gy[i]);
    me.store(db + row * dbs, a.dim, x);
  }
  if (!partial) return;
  float* out = partial + (int64_t)blockIdx.x * 2 * a.dim;
#pragma unroll
  for (int h = 0; h < 2; h++)
#pragma unroll
    for (int j = 0; j < CH; j++) {
      float* v = (h ? sum_w : sum_b) + 8 * j;
      if constexpr (S::kRows > 1) {      // the rows of a workgroup in order
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; i++) join[(sub_row * 64 + me.sub) * 8 + i] = v[i];
        __syncthreads();
        if (sub_row == 0)
#pragma unroll
          for (int i = 0; i < 8; i++)
            for (int s = 1; s < S::kRows; s++) v[i] += join[(s * 64 + me.sub) * 8 + i];
      }
      if (sub_row == 0 && me.col(j) < a.dim)
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          *(float4*)(out + h * a.dim + me.col(j) + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// The workgroups' partials in order and 64 bits: 32 columns a workgroup, 32
// rows at a time.
constexpr int kResidualDwCols = 32, kResidualDwRows = 32;
__global__ __launch_bounds__(kResidualDwCols* kResidualDwRows) void residual_norm_dw_kernel(
    const float* partial, int rows, ResidualArgs a, float* dbw, float* dw, float* dgate) {
  __shared__ double red[kResidualDwRows][kResidualDwCols];
  const int c = (int)threadIdx.x % kResidualDwCols, r = (int)threadIdx.x / kResidualDwCols;
  const int64_t j = (int64_t)blockIdx.x * kResidualDwCols + c;
  double t = 0.0;
  if (j < 2 * (int64_t)a.dim)
    for (int row = r; row < rows; row += kResidualDwRows)
      t += (double)partial[(int64_t)row * 2 * a.dim + j];
  red[r][c] = t;
  for (int half = kResidualDwRows / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (r < half) red[r][c] = t += red[r + half][c];
  }
  if (r != 0 || j >= 2 * (int64_t)a.dim) return;
  if (j >= a.dim) {
    if (dw) dw[j - a.dim] = (float)t;
    return;
  }
  const bool channel = a.gate && !a.token_gate;
  auto bf = [](uint16_t v) { return (double)__uint_as_float((uint32_t)v << 16); };
  if (dbw) dbw[j] = (float)(channel ? t * bf(a.gate[j]) : t);
  if (dgate && channel) dgate[j] = (float)(a.bw ? t * bf(a.bw[j]) : t);
}

}  // namespace fp4q
