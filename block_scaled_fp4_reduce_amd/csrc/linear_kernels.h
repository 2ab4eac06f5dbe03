// linear_kernels.h -- products of a few activations with FP4 weights: decoding
// batches through a matrix or through their experts.
//
//   y[t][n] = alpha_n sum_k x[t][k] w[n][k]
//
// on the matrix instructions with 16 rows of weights as one operand and 16
// tokens as the other, whatever the number of tokens: the codes of a row are
// read once and decoded straight into operand registers, so memory bounds it
// and not the products.  A lane serves row lane % 16 and the 32 consecutive
// values (16 code bytes) number lane / 16 of 128; the order of the values
// inside a product does not matter as long as the activations are read in the
// same one.
//
// A workgroup of 8 waves takes a number of rows and cuts K over its waves
// (`wk` of them a row; the others take other rows), which meet in LDS: no
// workspace and no second launch, and the sum's order depends on sizes alone.
#pragma once

#include "weights_common.h"

namespace fp4q {

constexpr int kColsThreads = 512, kColsWaves = kColsThreads / 64;
constexpr int kColsStep = 256;           // values of K in a wave's step
constexpr int kInlineMost = 512;         // assignments that a workgroup sorts by itself

struct ColsArgs {
  WeightView w;
  const uint16_t* x;
  void* out;
  int64_t xs, os;                        // elements between rows of x and out
  int64_t tokens;
  const int32_t *ids, *off, *order;      // experts: [tokens][top_k], [E + 1], [tokens * top_k]
  int top_k, experts;
  int inner;                             // gated: F
  int wk;                                // waves that share a row's K
  int row_blocks;                        // of a matrix (or of F)
  int col_groups;                        // SRC 0: groups of tokens
  int out_f32, out_vec;                  // fp32 outputs; 4 of them may be stored at once
  int x_per_token;                       // experts: rows of x are tokens (else assignments)
};

// Where a workgroup's columns (tokens) come from.
enum { kDense = 0, kPlanned = 1, kInline = 2 };

// The assignments of the slot-th expert that has any, in their order, to list[];
// returns their number and the expert (all threads alike).
__device__ __forceinline__ int inline_rows(const ColsArgs& a, int slot, int* list, int& expert) {
  __shared__ uint32_t bits[32];
  __shared__ int wave_count[kColsWaves];
  const int t = (int)threadIdx.x, n = (int)(a.tokens * a.top_k), lane = t & 63;
  if (t < 32) bits[t] = 0;
  __syncthreads();
  const int id = t < n ? a.ids[t] : -1;
  if (id >= 0 && id < a.experts) atomicOr(&bits[id >> 5], 1u << (id & 31));
  __syncthreads();
  // word and bit of the slot-th set bit
  const uint32_t word = lane < 32 ? bits[lane] : 0;
  int upto = __popc(word);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up(upto, d, 64);
    if (lane >= d) upto += o;
  }
  const uint64_t past = __ballot(lane < 32 && upto > slot);
  if (!past) {
    expert = -1;
    return 0;
  }
  const int wd = __builtin_ctzll(past);
  uint32_t wv = (uint32_t)__shfl((int)word, wd, 64);
  const int before = __shfl(upto, wd, 64) - __popc(wv);
  for (int i = before; i < slot; i++) wv &= wv - 1;
  expert = __builtin_amdgcn_readfirstlane(wd * 32 + __builtin_ctz(wv));
  const bool mine = id == expert;
  const uint64_t m = __ballot(mine);
  if (lane == 0) wave_count[t >> 6] = __popcll(m);
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < kColsWaves; w++) {
    base += w < (t >> 6) ? wave_count[w] : 0;
    total += wave_count[w];
  }
  if (mine) list[base + __popcll(m & ((1ull << lane) - 1))] = t;
  __syncthreads();
  return total;
}

// FMT of the weights, NT tiles of 16 tokens, R tiles of 16 rows (GATED: R pairs
// of a gate's and an up projection's tile).
template <int FMT, int NT, int R, bool GATED, int SRC>
__global__ __launch_bounds__(kColsThreads) void fp4_cols_kernel(ColsArgs a) {
  constexpr int TR = GATED ? 2 * R : R, TILES = TR * NT;
  constexpr int BATCH = TILES < 4 ? TILES : 4;       // tiles joined at once
  __shared__ f32x4_t red[kColsWaves][BATCH][64];
  __shared__ int list[SRC == kInline ? kInlineMost : 1];
  const int t = (int)threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const uint32_t slot = blockIdx.x / (uint32_t)a.row_blocks;
  const int rb = (int)(blockIdx.x - slot * (uint32_t)a.row_blocks);
  int64_t e = 0, first = 0, count;
  if constexpr (SRC == kDense) {
    first = (int64_t)slot * (16 * NT);
    count = a.tokens - first < 16 * NT ? a.tokens - first : 16 * NT;
  } else if constexpr (SRC == kPlanned) {
    e = slot;
    first = a.off[slot];
    count = a.off[slot + 1] - first;
  } else {
    int found;
    count = inline_rows(a, (int)slot, list, found);
    e = found;
  }
  if (count <= 0) return;
  const int rows = GATED ? a.inner : a.w.rows;
  const int kpart = wave % a.wk, wr = kColsWaves / a.wk;
  const int n0 = (rb * wr + wave / a.wk) * 16 * R;
  const int K = a.w.cols, steps = (K + kColsStep - 1) / kColsStep;
  const uint8_t *crow[TR], *srow[TR];
#pragma unroll
  for (int i = 0; i < TR; i++) {
    const int n = n0 + 16 * (GATED ? i / 2 : i) + r;
    const int row = (n < rows ? n : rows - 1) + (GATED && (i & 1) ? rows : 0);
    crow[i] = code_row<FMT>(a.w, e, row);
    srow[i] = scale_row<FMT>(a.w, e, row);
  }
  const u32x4_t zero = {0, 0, 0, 0};

  for (int64_t c0 = 0; c0 < count; c0 += 16 * NT) {
    const uint16_t* xrow[NT];
    bool there[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int64_t c = c0 + 16 * j + r;
      there[j] = c < count;
      int64_t row = there[j] ? c : 0;
      if constexpr (SRC == kDense) {
        row += first;
      } else {
        row = SRC == kPlanned ? a.order[first + row] : list[row];
        if (a.x_per_token) row = (int64_t)((uint32_t)row / (uint32_t)a.top_k);
      }
      xrow[j] = a.x + row * a.xs;
    }
    f32x4_t acc[TR][NT] = {};
    for (int s = kpart; s < steps; s += a.wk) {
#pragma unroll
      for (int c = 0; c < kColsStep / 128; c++) {
        const int k = s * kColsStep + 128 * c + 32 * g;
        const bool in = k < K;
        u32x4_t code[TR];
        uint32_t sc[TR];
#pragma unroll
        for (int i = 0; i < TR; i++) {
          code[i] = in ? *(const u32x4_t*)(crow[i] + k / 2) : zero;
          sc[i] = in ? load_scales<FMT>(srow[i], k) : 0;
        }
        u32x4_t x[NT][4];
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int q = 0; q < 4; q++)
            x[j][q] = in && there[j] ? *(const u32x4_t*)(xrow[j] + k + 8 * q) : zero;
#pragma unroll
        for (int i = 0; i < TR; i++) {
          float sv[2];
          scale_values<FMT>(sc[i], sv);
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const u32x4_t op = decode8<FMT>(code[i][q], sv[q / 2]);
#pragma unroll
            for (int j = 0; j < NT; j++) acc[i][j] = mfma16_bf16(op, x[j][q], acc[i][j]);
          }
        }
      }
    }
    // join the waves of a row block: tiles in batches, one value of a lane each
#pragma unroll
    for (int b = 0; b < TILES; b += BATCH) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < BATCH; i++)    // tile order: pairs of a gate and an up tile together
        red[wave][i][lane] = acc[GATED ? 2 * ((b + i) / 2 / NT) + (b + i) % 2 : (b + i) / NT]
                                [GATED ? (b + i) / 2 % NT : (b + i) % NT];
      __syncthreads();
      constexpr int OUT = GATED ? BATCH / 2 : BATCH;
      for (int item = t; item < wr * OUT * 64; item += kColsThreads) {
        const int l = item & 63, tile = item / 64 % OUT, blk = item / (64 * OUT);
        f32x4_t v[GATED ? 2 : 1];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); h++) {
          v[h] = red[blk * a.wk][GATED ? 2 * tile + h : tile][l];
          for (int w = 1; w < a.wk; w++)
            v[h] += red[blk * a.wk + w][GATED ? 2 * tile + h : tile][l];
        }
        const int at = (GATED ? b / 2 : b) + tile;   // row tile and token tile
        const int n = (rb * wr + blk) * 16 * R + 16 * (at / NT) + 4 * (l >> 4);
        const int64_t c = c0 + 16 * (at % NT) + (l & 15);
        if (c >= count || n >= rows) continue;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int row = n + i < rows ? n + i : rows - 1;
          y[i] = v[0][i] * alpha_of(a.w, e, row);
          if constexpr (GATED) y[i] = silu_times(y[i], v[1][i] * alpha_of(a.w, e, row + rows));
        }
        int64_t orow = c;
        if constexpr (SRC == kDense) orow += first;
        else orow = SRC == kPlanned ? a.order[first + c] : list[c];
        const int64_t o = orow * a.os + n;
        if (a.out_f32) {
          float* p = (float*)a.out + o;
          if (a.out_vec && n + 3 < rows) {
            *(f32x4_t*)p = f32x4_t{y[0], y[1], y[2], y[3]};
          } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (n + i < rows) p[i] = y[i];
          }
        } else {
          uint16_t* p = (uint16_t*)a.out + o;
          const u32x2_t v2 = {bf16x2_of(y[0], y[1]), bf16x2_of(y[2], y[3])};
          if (a.out_vec && n + 3 < rows) {
            *(u32x2_t*)p = v2;
          } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (n + i < rows) p[i] = (uint16_t)(v2[i / 2] >> (16 * (i & 1)));
          }
        }
      }
    }
  }
}

}  // namespace fp4q
