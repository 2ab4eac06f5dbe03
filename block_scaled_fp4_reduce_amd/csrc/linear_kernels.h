// linear_kernels.h -- products of a few activations with FP4 weights: decoding
// batches through a matrix or through their experts.
//
//   y[t][n] = alpha_n sum_k x[t][k] w[n][k]
//
// on the matrix instructions with 16 rows of weights as one operand and 16
// tokens as the other, whatever the number of tokens: the codes of a row are
// read once and decoded straight into operand registers, so memory bounds it
// and not the products.  A lane loads the 32 consecutive values (16 code bytes)
// number lane / 16 of 128 of row lane % 16; the four lanes of a row then trade
// dwords, so that a product takes 32 values in a run and the activations are
// read in whole 64-byte pieces too (read as the codes lie, 16 bytes of every
// 64, they would take most of the cache's lookups).  It is the form for small
// matrices and few tokens, where a launch's latency is most of the time (1 token
// through 4096x4096: 5.7 us, of which reading the codes at 4.9 TB/s is 1.9), and
// for sizes that the others do not take; the streams and tiles of
// linear_stream_kernels.h and linear_tiled_kernels.h read by neighbouring lanes.
//
// A workgroup of 8 waves (experts: 4) takes a number of rows and cuts K over its waves
// (`wk` of them a row; the others take other rows), which meet in LDS: no
// workspace and no second launch, and the sum's order depends on sizes alone.
#pragma once

#include "weights_common.h"

namespace fp4q {

constexpr int kColsStep = 256;           // values of K that a wave reads at once
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
  int kseg_shift, span, blocks;          // streams: log2 of a segment of K, columns at a time, row blocks
  int row_blocks;                        // of a matrix (or of F)
  int out_f32, out_vec;                  // fp32 outputs; 4 of them may be stored at once
  int x_per_token;                       // experts: rows of x are tokens (else assignments)
  int64_t x_bytes;                       // experts: of x
};

// Where a workgroup's columns (tokens) come from.
enum { kDense = 0, kPlanned = 1, kInline = 2 };

// The slot-th of the experts that have assignments, by number: workgroups ask for
// it by themselves, without a launch before, and their list has no holes
// (hardware deals workgroups out to the XCDs in turn, and holes unbalance
// them).  -1 if there are fewer.  One token: the slot-th assignment's expert,
// so that there are as many slots as assignments.
template <int W>
__device__ __forceinline__ int inline_expert(const ColsArgs& a, int slot) {
  if (a.tokens == 1) {
    const int e = a.ids[slot];
    return e >= 0 && e < a.experts ? e : -1;
  }
  __shared__ uint32_t bits[32];
  const int t = (int)threadIdx.x, n = (int)(a.tokens * a.top_k), lane = t & 63;
  if (t < 32) bits[t] = 0;
  __syncthreads();
  for (int i = t; i < n; i += W * 64) {
    const int id = a.ids[i];
    if (id >= 0 && id < a.experts) atomicOr(&bits[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  const uint32_t word = lane < 32 ? bits[lane] : 0;
  int upto = __popc(word);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up(upto, d, 64);
    if (lane >= d) upto += o;
  }
  const uint64_t past = __ballot(lane < 32 && upto > slot);
  if (!past) return -1;
  const int at = __builtin_ctzll(past);
  uint32_t v = (uint32_t)__builtin_amdgcn_readlane((int)word, at);
  int skip = slot - (__builtin_amdgcn_readlane(upto, at) - __popc(v));
  for (; skip > 0; skip--) v &= v - 1;
  return __builtin_amdgcn_readfirstlane(at * 32 + __builtin_ctz(v));
}

// An expert's assignments in their order to list[] (every wave for itself);
// returns their number.  One token: 0 but for the first slot of its expert.
__device__ __forceinline__ int inline_rows(const ColsArgs& a, int slot, int expert, int* list) {
  const int n = (int)(a.tokens * a.top_k), lane = (int)threadIdx.x & 63;
  int total = 0;
  for (int i = 0; i < n; i += 64) {
    const bool mine = i + lane < n && a.ids[i + lane] == expert;
    const uint64_t m = __ballot(mine);
    if (a.tokens == 1 && m && i + __builtin_ctzll(m) < slot) return 0;
    if (mine) list[total + __popcll(m & ((1ull << lane) - 1))] = i + lane;
    total += __popcll(m);
  }
  wave_lds_sync();
  return total;
}

// Scale bytes of a row's 256 values, the same in the four lanes of a row.
template <int FMT>
struct StepScales {
  static constexpr int N = FMT == 0 ? 4 : 2;
  uint32_t v[N];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int off) {
    if constexpr (FMT == 0) {
      const u32x4_t x = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] = x[i];
    } else {
      const u32x2_t x = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
      v[0] = x[0];
      v[1] = x[1];
    }
  }
  // the last step of a row: `left` of its 256 values, byte by byte (lane g fetches
  // those of 64 values), so that nothing behind the row is touched
  __device__ __forceinline__ void load_tail(__amdgpu_buffer_rsrc_t r, int off, int left) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      v[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; b++)
        if ((4 * i + b) * WeightFmt<FMT>::G < left)            // uniform
          v[i] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, off + 4 * i + b, 0, 0) << (8 * b);
    }
  }
  // of the values 128 half + 32 q + 8 g ..
  __device__ __forceinline__ float at(int half, int q, int g) const {
    if constexpr (FMT == 0) {            // an E4M3 scale's sign bit is ignored
      const int w = (int)((v[2 * half + q / 2] & 0x7F7F7F7Fu) >> (8 * (g >> 1)));
      return q & 1 ? __builtin_amdgcn_cvt_f32_fp8(w, 2) : __builtin_amdgcn_cvt_f32_fp8(w, 0);
    } else {
      return __uint_as_float((v[half] >> (8 * q) & 0xFFu) << 23);
    }
  }
};

// Dword d of lane group g (lanes 16 g .. 16 g + 15) to dword g of group d.
__device__ __forceinline__ u32x4_t turn_groups(u32x4_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4_t{c[0], c[1], d[0], d[1]};
}

// The sums of rows n .. n + 3 (GATED: and of the same rows of the up projection)
// to row `orow` of the output.
template <bool GATED>
__device__ __forceinline__ void put_rows(const ColsArgs& a, int64_t e, int rows, int n, int64_t orow,
                                         float all, const f32x4_t (&v)[GATED ? 2 : 1]) {
  float y[4];
  auto sum = [&](int h, int i) {         // of projection h
    return v[h][i] * alpha_row(a.w, e, (n + i < rows ? n + i : rows - 1) + h * rows, all);
  };
  if constexpr (GATED) {
    silu_times(y, [&](int i) { return sum(0, i); }, [&](int i) { return sum(1, i); });
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) y[i] = sum(0, i);
  }
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

// FMT of the weights, R tiles of 16 rows a wave (GATED: R pairs of a gate's and an
// up projection's tile), 16 tokens at a time.
template <int FMT, int R, bool GATED, int SRC, int W>
__global__ __launch_bounds__(W * 64, GATED ? 2 : 4) void fp4_cols_kernel(ColsArgs a) {
  constexpr int TR = GATED ? 2 * R : R;
  __shared__ f32x4_t red[W][TR][64];
  __shared__ int lists[SRC == kInline ? W : 1][SRC == kInline ? kInlineMost : 1];
  const int t = (int)threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int* const list = lists[SRC == kInline ? wave : 0];
  const uint32_t slot = blockIdx.x / (uint32_t)a.row_blocks;
  const int rb = (int)(blockIdx.x - slot * (uint32_t)a.row_blocks);
  int64_t e = 0, first = 0, count;
  if constexpr (SRC == kDense) {
    first = (int64_t)slot * 16;
    count = a.tokens - first < 16 ? a.tokens - first : 16;
  } else if constexpr (SRC == kPlanned) {
    e = slot;
    first = a.off[slot];
    count = a.off[slot + 1] - first;
  } else {
    e = inline_expert<W>(a, (int)slot);
    if (e < 0) return;
    count = inline_rows(a, (int)slot, (int)e, list);
  }
  if (count <= 0) return;
  const float all = alpha_all(a.w, e);
  const int rows = GATED ? a.inner : a.w.rows;
  const int kpart = wave % a.wk, wr = W / a.wk;
  const int K = a.w.cols, steps = (K + kColsStep - 1) / kColsStep;
  // Row blocks begin at different steps: rows are a power of two of bytes apart
  // as often as not, and blocks at the same step then meet on few channels.
  const int turn = steps ? (int)((uint32_t)(rb * wr + wave / a.wk) % (uint32_t)steps) : 0;
  auto place = [&](int step) {
    const int p = step + turn;
    return p < steps ? p : p - steps;
  };
  // Buffers over the block's rows and over x: what lies past them, or past K, is
  // read as zeros, and zero times zero adds nothing.  The host keeps all
  // offsets under 2^31.
  constexpr int G = WeightFmt<FMT>::G;
  const int blk = rb * wr * 16 * R;      // first row of the workgroup
  __amdgpu_buffer_rsrc_t rc[GATED ? 2 : 1], rs[GATED ? 2 : 1];
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); h++) {
    const int n = blk + (h ? rows : 0), left = rows - blk;
    rc[h] = buffer_rsrc(code_row<FMT>(a.w, e, n), (int64_t)left * (K / 2));
    rs[h] = buffer_rsrc(scale_row<FMT>(a.w, e, n),
                        (int64_t)(a.w.tile_shift ? (left + 15) / 16 : left) * (K / G));
  }
  uint32_t coff[R], soff[R];
#pragma unroll
  for (int i = 0; i < R; i++) {
    const uint32_t n = (uint32_t)(wave / a.wk * 16 * R + 16 * i + r);
    coff[i] = n * (uint32_t)(K / 2) + 16 * g;
    soff[i] = (n >> a.w.tile_shift) * (uint32_t)(K / G);
  }
  struct Step {
    u32x4_t code[TR][2];
    StepScales<FMT> sc[TR];
  };
  auto load = [&](Step& f, int step) {
    constexpr int per = GATED ? 2 : 1;               // tile i: row tile i / per of buffer i % per
    const int k0 = place(step) * kColsStep, left = step < steps ? K - k0 : 0;
#pragma unroll
    for (int i = 0; i < TR; i++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int co = (int)(128 * h + 32 * g < left ? coff[i / per] + k0 / 2 + 64 * h : kBufferEnd);
        f.code[i][h] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rc[i % per], co, 0, 0));
      }
    if (left >= kColsStep) {                         // uniform
#pragma unroll
      for (int i = 0; i < TR; i++) f.sc[i].load(rs[i % per], (int)(soff[i / per] + k0 / G));
    } else {
#pragma unroll
      for (int i = 0; i < TR; i++) f.sc[i].load_tail(rs[i % per], (int)(soff[i / per] + k0 / G), left);
    }
  };
  const __amdgpu_buffer_rsrc_t rx =
      SRC == kDense ? buffer_rsrc(a.x + first * a.xs, ((count - 1) * a.xs + K) * 2)
                    : buffer_rsrc(a.x, a.x_bytes);

  for (int64_t c0 = 0; c0 < count; c0 += 16) {
    // columns past the last repeat it and are dropped
    int64_t row = c0 + r < count ? c0 + r : count - 1;
    if constexpr (SRC != kDense) {
      row = SRC == kPlanned ? a.order[first + row] : list[row];
      if (a.x_per_token) row = (int64_t)((uint32_t)row / (uint32_t)a.top_k);
    }
    const uint32_t xoff = (uint32_t)(row * a.xs * 2) + 16 * g;
    f32x4_t acc[TR] = {};
    auto multiply = [&](const Step& f, int half, const u32x4_t (&x)[4]) {
#pragma unroll
      for (int i = 0; i < TR; i++) {
        const u32x4_t code = turn_groups(f.code[i][half]);
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const u32x4_t op = decode8<FMT>(code[q], f.sc[i].at(half, q, g));
          acc[i] = mfma16_bf16(op, x[q], acc[i]);
        }
      }
    };
    auto load_x = [&](u32x4_t (&x)[4], int step, int half) {
      const int k0 = place(step) * kColsStep + 128 * half, left = step < steps ? K - k0 : 0;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int o = 32 * q < left ? (int)xoff + 2 * k0 + 64 * q : (int)kBufferEnd;
        x[q] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rx, o, 0, 0));
      }
    };
    // Loads come back in their order, so a step's second activations go out
    // before the next step's codes, which have the longest way.
    Step f0, f1;
    u32x4_t x0[4], x1[4];
    load_x(x0, kpart, 0);
    load(f0, kpart);
    auto one = [&](Step& f, Step& next, int step) {
      load_x(x1, step, 1);
      load(next, step + a.wk);
      multiply(f, 0, x0);
      load_x(x0, step + a.wk, 0);
      multiply(f, 1, x1);
    };
    for (int step = kpart; step < steps; step += 2 * a.wk) {
      one(f0, f1, step);
      one(f1, f0, step + a.wk);
    }
    // join the waves of a row block, one value of a lane each
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TR; i++) red[wave][i][lane] = acc[i];
    __syncthreads();
    for (int item = t; item < wr * R * 64; item += W * 64) {
      const int l = item & 63, tile = item / 64 % R, set = item / (64 * R);
      f32x4_t v[GATED ? 2 : 1];
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); h++) {
        const int at = GATED ? 2 * tile + h : tile;
        v[h] = red[set * a.wk][at][l];
        for (int w = 1; w < a.wk; w++) v[h] += red[set * a.wk + w][at][l];
      }
      const int n = blk + set * 16 * R + 16 * tile + 4 * (l >> 4);
      const int64_t c = c0 + (l & 15);
      if (c >= count || n >= rows) continue;
      int64_t orow = c;
      if constexpr (SRC == kDense) orow += first;
      else orow = SRC == kPlanned ? a.order[first + c] : list[c];
      put_rows<GATED>(a, e, rows, n, orow, all, v);
    }
  }
}

}  // namespace fp4q
