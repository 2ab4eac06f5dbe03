// linear_stream_kernels.h -- products of up to 16 activations at a time with
// FP4 weights, for matrices large enough that each wave has rows of its own:
// the mathematics of linear_kernels.h, bound by reading the codes.
//
// The operand layout of the matrix instructions puts 16 rows into 16
// neighbouring lanes; loads in that layout touch a cache line a lane and the
// L1's lookups limit them (64 tokens through 128 experts: 0.67 a cycle and CU,
// 3.3 TB/s).  Here codes, scales and activations go to LDS by direct loads in
// which neighbouring lanes read neighbouring bytes, and from there into the
// operand layout.
//
// A wave takes 32 rows (GATED: 16 of the gate's and the same 16 of the up
// projection's) in steps of 256 values, one cache line of codes a row, through
// two buffers of its own; a buffer is filled again as soon as its step is in
// registers.  The workgroup's activations lie in two shared buffers, a segment of
// K each, with one barrier a segment (a power of two of 512 wk at least).  A
// workgroup takes several row blocks one after another without a pause in the
// codes; where there are too few rows, `wk` waves share them and cut each
// segment's steps among them.
//
// 64 tokens through 128 experts of 4096 x 1024 (MXFP4): gate and up 120 us, down
// 71 us, 4.4 TB/s of codes and scales; with loads in the operand
// layout the whole call took 359 us, now 190.
#pragma once

#include "linear_kernels.h"

namespace fp4q {

constexpr int kStreamWaves = 4, kStreamThreads = kStreamWaves * 64;
constexpr int kStreamX = 16384;          // bytes of a segment of activations
constexpr int kStreamLeast = 9;          // log2 of the least segment, of which 16 columns fit

// A segment of K: as much as fits for `tokens` columns (16 at a time), at most all
// of it, and the columns that are taken at once, as many as fit.  An expert that a
// token names twice has more columns than there are tokens: they take more turns.
struct StreamSegment {
  int shift, span;
};
constexpr StreamSegment stream_segment(int64_t tokens, int cols) {
  const int64_t most = tokens < 16 ? tokens : 16;
  int shift = kStreamLeast;
  while ((most << (shift + 2)) <= kStreamX && (1 << shift) < cols) shift++;
  const int fit = kStreamX >> (shift + 1);
  return {shift, fit < 16 ? fit : 16};
}
constexpr bool stream_segments_fit() {
  for (int64_t tokens = 1; tokens <= 17; tokens++)
    for (int cols = 32; cols < 1 << 22; cols *= 2) {
      const StreamSegment s = stream_segment(tokens, cols + 32);
      if ((int64_t)s.span << (s.shift + 1) > kStreamX || s.span < (tokens < 16 ? tokens : 16)) return false;
    }
  return true;
}
static_assert(stream_segments_fit(), "the columns of a turn stay in their buffer");

// One step of a wave in LDS: [tile][row][128 bytes of codes], 16-byte piece p of
// row r at p ^ (r / 2 % 8), so that 16 rows' reads cover all banks; scales
// [tile][row][16 bytes].
struct StreamStep {
  uint8_t code[2][2048];
  uint8_t scale[2][256];
};

template <int FMT, bool GATED, int SRC>
__global__ __launch_bounds__(kStreamThreads, 2) void fp4_stream_kernel(ColsArgs a) {
  __shared__ __attribute__((aligned(16))) StreamStep step0[kStreamWaves], step1[kStreamWaves];
  __shared__ __attribute__((aligned(16))) uint8_t xs[2][kStreamX];
  __shared__ int lists[SRC == kInline ? kStreamWaves : 1][SRC == kInline ? kInlineMost : 1];
  constexpr int G = WeightFmt<FMT>::G;
  const int t = (int)threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int* const list = lists[SRC == kInline ? wave : 0];
  const uint32_t slot = blockIdx.x / (uint32_t)a.row_blocks;
  const int rb = (int)(blockIdx.x - slot * (uint32_t)a.row_blocks);
  int64_t e = 0, first = 0, count = 0;
  if constexpr (SRC == kDense) {
    first = (int64_t)slot * 16;
    count = a.tokens - first < 16 ? a.tokens - first : 16;
  } else if constexpr (SRC == kPlanned) {
    e = slot;
    first = a.off[slot];
    count = a.off[slot + 1] - first;
  } else {
    e = inline_expert<kStreamWaves>(a, (int)slot);   // its tokens follow below
    if (e < 0) return;
  }
  if (SRC != kInline && count <= 0) return;
  const float all = alpha_all(a.w, e);
  const int rows = GATED ? a.inner : a.w.rows, K = a.w.cols;
  constexpr int WAVE_ROWS = GATED ? 16 : 32;
  const int kpart = wave % a.wk, wr = kStreamWaves / a.wk, set = wave / a.wk;
  const int blk_rows = wr * WAVE_ROWS, blk = rb * a.blocks * blk_rows;
  const int blocks = min(a.blocks, (rows - blk + blk_rows - 1) / blk_rows);

  __amdgpu_buffer_rsrc_t rc[GATED ? 2 : 1], rs[GATED ? 2 : 1];
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); h++) {
    const int n = blk + (h ? rows : 0), left = rows - blk;
    rc[h] = buffer_rsrc(code_row<FMT>(a.w, e, n), (int64_t)left * (K / 2));
    rs[h] = buffer_rsrc(scale_row<FMT>(a.w, e, n),
                        (int64_t)(a.w.tile_shift ? (left + 15) / 16 : left) * (K / G));
  }
  // direct loads: codes, 8 rows of 8 pieces each; scales, 16 rows of 4 (MXFP4 2) dwords
  uint32_t coff[2][2], soff[2];
  const int cpiece = (lane & 7), crow = lane >> 3;
  constexpr int SD = FMT == 0 ? 4 : 2;
  const int srow = lane / SD, sdw = lane % SD;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t n = (uint32_t)(set * WAVE_ROWS + (GATED ? 0 : 16 * i));
#pragma unroll
    for (int h = 0; h < 2; h++) coff[i][h] = (n + 8 * h + crow) * (uint32_t)(K / 2);
    soff[i] = srow < 16 ? ((n + srow) >> a.w.tile_shift) * (uint32_t)(K / G) + 4 * sdw : kBufferEnd;
  }
  // Workgroups begin at different segments: rows are a power of two of bytes
  // apart as often as not, and blocks at the same step then meet on few channels.
  const int kseg = 1 << a.kseg_shift, segs = (K + kseg - 1) >> a.kseg_shift;
  const int per_shift = a.kseg_shift - 8, per = 1 << per_shift;          // steps of a segment
  const int first_seg = rb % segs;
  auto place = [&](int seg) {
    const int p = seg + first_seg;
    return p < segs ? p : p - segs;
  };
  // step `step` of row block b; steps past the last are the next block's
  const int block_codes = blk_rows * (K / 2), block_scales = (blk_rows >> a.w.tile_shift) * (K / G);
  auto fill = [&](StreamStep& s, int b, int step) {
    int seg = step >> per_shift;
    if (seg >= segs) {
      seg -= segs;
      b++;
    }
    const int k0 = b < blocks && seg < segs ? place(seg) * kseg + (step & (per - 1)) * kColsStep : K;
    const int co = b * block_codes + k0 / 2, so = b * block_scales + k0 / G;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const __amdgpu_buffer_rsrc_t c = rc[GATED ? i : 0], q = rs[GATED ? i : 0];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int piece = cpiece ^ (((8 * h + crow) >> 1) & 7);
        const bool in = k0 + 32 * piece < K;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(c, (lds_void_t*)(s.code[i] + 1024 * h), 16,
                                                 in ? coff[i][h] + co + 16 * piece : kBufferEnd, 0, 0, 0);
      }
      const bool in = k0 + 4 * G * sdw < K;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(q, (lds_void_t*)s.scale[i], 4,
                                               in ? soff[i] + so : kBufferEnd, 0, 0, 0);
    }
  };
  if constexpr (SRC == kInline) {
    // the first codes set out before the tokens are known
    fill(step0[wave], 0, kpart);
    fill(step1[wave], 0, kpart + a.wk);
    count = inline_rows(a, (int)slot, (int)e, list);
    if (count <= 0) {
      wait_vm<0>();
      return;
    }
  }
  const __amdgpu_buffer_rsrc_t rx =
      SRC == kDense ? buffer_rsrc(a.x + first * a.xs, ((count - 1) * a.xs + K) * 2)
                    : buffer_rsrc(a.x, a.x_bytes);

  for (int64_t c0 = 0; c0 < count; c0 += a.span) {
    const int cols = (int)(count - c0 < a.span ? count - c0 : a.span);
    // a wave's rows of x: wave, wave + 4, ...; 64 lanes take 512 values at once,
    // piece p of row c at p ^ c % 16
    uint32_t xoff[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      int64_t row = wave + 4 * i < cols ? c0 + wave + 4 * i : c0;
      if constexpr (SRC != kDense) {
        row = SRC == kPlanned ? a.order[first + row] : list[row];
        if (a.x_per_token) row = (int64_t)((uint32_t)row / (uint32_t)a.top_k);
      }
      xoff[i] = __builtin_amdgcn_readfirstlane((uint32_t)(row * a.xs * 2));
    }
    auto fill_x = [&](uint8_t* buf, int seg) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int c = wave + 4 * i;
        if (c >= cols) break;                        // uniform
        for (int p = 0; p < kseg; p += 512) {
          const int k = place(seg) * kseg + p + 8 * (lane ^ (c & 15));
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(buf + (c * kseg + p) * 2), 16,
                                                   k < K ? xoff[i] + 2 * k : kBufferEnd, 0, 0, 0);
        }
      }
    };
    const int xr = r < cols ? r : 0;                 // columns past the last are dropped
    f32x4_t acc[2] = {};
    // a step of block b from its buffer, whose next contents are step `next`'s; k: its
    // place in x
    auto multiply = [&](StreamStep& s, const uint8_t* x, int k, int b, int next) {
      wait_vm<6>();                                  // all but the other buffer's loads
      u32x4_t code[2][2];
      StepScales<FMT> sc[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
#pragma unroll
        for (int h = 0; h < 2; h++)
          code[i][h] = *(const u32x4_t*)(s.code[i] + r * 128 + 16 * ((4 * h + g) ^ (r >> 1)));
        if constexpr (FMT == 0) {
          const u32x4_t v = *(const u32x4_t*)(s.scale[i] + r * 16);
#pragma unroll
          for (int q = 0; q < 4; q++) sc[i].v[q] = v[q];
        } else {
          const u32x2_t v = *(const u32x2_t*)(s.scale[i] + r * 8);
          sc[i].v[0] = v[0];
          sc[i].v[1] = v[1];
        }
      }
      wait_lds();                                    // the buffer is free
      fill(s, b, next);
#pragma unroll
      for (int h = 0; h < 2; h++) {
        u32x4_t xv[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int piece = (k + 128 * h + 32 * q) / 8 + g;
          xv[q] = *(const u32x4_t*)(x + (xr * kseg + 8 * ((piece & ~15) | ((piece ^ xr) & 15))) * 2);
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const u32x4_t cd = turn_groups(code[i][h]);
#pragma unroll
          for (int q = 0; q < 4; q++)
            acc[i] = mfma16_bf16(decode8<FMT>(cd[q], sc[i].at(h, q, g)), xv[q], acc[i]);
        }
      }
    };
    if (c0 > 0) __syncthreads();                     // the buffers' readers of before are done
    fill_x(xs[0], 0);
    if (SRC != kInline || c0 > 0) {
      fill(step0[wave], 0, kpart);
      fill(step1[wave], 0, kpart + a.wk);
    } else {
      wait_vm<0>();                                  // codes and activations set out in another order
    }
    int side = 0;                                    // the segment's buffer
    for (int b = 0; b < blocks; b++) {
      acc[0] = acc[1] = f32x4_t{};
      for (int seg = 0; seg < segs; seg++) {
        const bool new_x = segs > 1 || b == 0;       // one segment stays for all blocks
        if (new_x) {
          // its activations are older than the last two steps' codes
          wait_vm<12>();
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          if (seg + 1 < segs) fill_x(xs[side ^ 1], seg + 1);
          else if (segs > 1 && b + 1 < blocks) fill_x(xs[side ^ 1], 0);
        }
        const uint8_t* x = xs[side];
        if (segs > 1) side ^= 1;
        for (int s = kpart; s < per; s += 2 * a.wk) {
          const int step = (seg << per_shift) + s;
          multiply(step0[wave], x, s * kColsStep, b, step + 2 * a.wk);
          multiply(step1[wave], x, (s + a.wk) * kColsStep, b, step + 3 * a.wk);
        }
      }
      constexpr int OUT = GATED ? 1 : 2;
      auto put = [&](int st, int tile, int l, const f32x4_t(&v)[GATED ? 2 : 1]) {
        const int n = blk + b * blk_rows + st * WAVE_ROWS + 16 * tile + 4 * (l >> 4), c = l & 15;
        if (c >= cols || n >= rows) return;
        int64_t orow = c0 + c;
        if constexpr (SRC == kDense) orow += first;
        else orow = SRC == kPlanned ? a.order[first + orow] : list[orow];
        put_rows<GATED>(a, e, rows, n, orow, all, v);
      };
      if (a.wk == 1) {                               // the wave's own rows
        if constexpr (GATED) {
          put(set, 0, lane, acc);
        } else {
          put(set, 0, lane, {acc[0]});
          put(set, 1, lane, {acc[1]});
        }
        continue;
      }
      // one block (then): join the waves of its rows
      f32x4_t(*red)[2][64] = (f32x4_t(*)[2][64])xs[0];
      __syncthreads();
      red[wave][0][lane] = acc[0];
      red[wave][1][lane] = acc[1];
      __syncthreads();
      for (int item = t; item < wr * OUT * 64; item += kStreamThreads) {
        const int l = item & 63, tile = item / 64 % OUT, st = item / (64 * OUT);
        f32x4_t v[GATED ? 2 : 1];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); h++) {
          v[h] = red[st * a.wk][GATED ? h : tile][l];
          for (int w = 1; w < a.wk; w++) v[h] += red[st * a.wk + w][GATED ? h : tile][l];
        }
        put(st, tile, l, v);
      }
    }
  }
  wait_vm<0>();                          // zeros on their way to LDS past the last step
}

// Scale bytes of a row's 128 values from k0 on, the same in the four lanes of a
// row: dwords of 4 scales.  One that would pass the row's end is read up to it
// and shifted, so that nothing behind a row is touched and nothing branches.
template <int FMT>
struct ChunkScales {
  static constexpr int N = FMT == 0 ? 2 : 1, SPAN = 4 * WeightFmt<FMT>::G;
  uint32_t v[N];
  int shift;                             // of the last dword in the row
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int k0, int K) {
    shift = 0;
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int left = K - k0 - i * SPAN;            // uniform
      const int missing = left >= SPAN || left <= 0 ? 0 : (SPAN - left) / WeightFmt<FMT>::G;
      const int at = (k0 + i * SPAN) / WeightFmt<FMT>::G - missing;
      shift = missing ? 8 * missing : shift;
      v[i] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)(left > 0 ? row + at : kBufferEnd), 0, 0);
    }
  }
  // of the values 32 q + 8 g ..
  __device__ __forceinline__ float at(int q, int g, int left) const {
    uint32_t w = v[FMT == 0 ? q / 2 : 0];
    if constexpr (FMT == 0) {            // an E4M3 scale's sign bit is ignored
      if (q < 2 ? left < 64 : left < 128) w >>= shift;         // uniform
      w = (w & 0x7F7F7F7Fu) >> (8 * (g >> 1));
      return q & 1 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 2) : __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    } else {
      // past the row's end any of its scales: the codes there are zeros
      return __uint_as_float((w >> ((shift + 8 * q) & 31) & 0xFFu) << 23);
    }
  }
};

// Up to 64 tokens at a time through one matrix: the activations of a segment of
// 512 values lie in LDS for the whole workgroup (two or three buffers, one
// barrier a segment), the codes of two chunks of 128 values in a wave's own part.
// A wave takes 32 rows; `wk` waves (1, 2 or 4) share rows and cut a segment's
// chunks among them.  Eight waves: one alone on its SIMD issues half of what two
// do.  Two more only fetch the activations: loads come back in a wave's order,
// and one that waited for activations would wait for all codes that it asked for
// before, from farther away.  48 tokens through 14336x4096 of MXFP4 take 15.0 us
// (codes, activations and outputs at the rate of a copy: 6.7), by fp4_cols_kernel 23.
// No unit is at its limit (vector 35% of the time, matrix 19%): waves wait for their
// loads, of which a CU has 32 KB of codes under way.
constexpr int kMidWaves = 8, kMidLoaders = 2, kMidThreads = (kMidWaves + kMidLoaders) * 64;
constexpr int kMidDepth = 2, kMidChunk = 128;
constexpr int kMidLeast = 128;           // cols: a dword of scales in every row

template <int FMT, int NT>
__global__ __launch_bounds__(kMidThreads, 3) void fp4_mid_kernel(ColsArgs a) {
  constexpr int TOKENS = 16 * NT, KSEG = 512, BUFFERS = NT <= 2 ? 3 : 2, G = WeightFmt<FMT>::G;
  __shared__ __attribute__((aligned(16))) uint8_t xs[BUFFERS][TOKENS * KSEG * 2];
  __shared__ __attribute__((aligned(16))) uint8_t cs[kMidDepth][kMidWaves][2][1024];
  const int t = (int)threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const uint32_t slot = blockIdx.x / (uint32_t)a.row_blocks;
  const int rb = (int)(blockIdx.x - slot * (uint32_t)a.row_blocks);
  const int64_t first = (int64_t)slot * TOKENS;
  const int cols = (int)(a.tokens - first < TOKENS ? a.tokens - first : TOKENS);
  const float all = alpha_all(a.w, 0);
  const int rows = a.w.rows, K = a.w.cols;
  const int kpart = wave % a.wk, wr = kMidWaves / a.wk, set = wave / a.wk;
  const int blk = rb * wr * 32, segs = (K + KSEG - 1) / KSEG;
  const int first_seg = rb % segs;       // blocks at the same step meet on few channels
  auto place = [&](int seg) {
    const int p = seg + first_seg;
    return p < segs ? p : p - segs;
  };
  const int rows_left = rows - blk;
  const __amdgpu_buffer_rsrc_t rc = buffer_rsrc(code_row<FMT>(a.w, 0, blk), (int64_t)rows_left * (K / 2));
  const __amdgpu_buffer_rsrc_t rs =
      buffer_rsrc(scale_row<FMT>(a.w, 0, blk),
                  (int64_t)(a.w.tile_shift ? (rows_left + 15) / 16 : rows_left) * (K / G));
  // direct loads of codes: lane -> row lane / 4, piece lane % 4 ^ row / 4 % 4 (16 rows'
  // reads cover all banks); scales by the 16 lanes of the rows
  uint32_t coff[2], soff[2];
  const int crow = lane >> 2, cpiece = (lane & 3) ^ (crow >> 2 & 3);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t n = (uint32_t)(set * 32 + 16 * i);
    coff[i] = (n + crow) * (uint32_t)(K / 2) + 16 * cpiece;
    soff[i] = lane < 16 ? ((n + r) >> a.w.tile_shift) * (uint32_t)(K / G) : kBufferEnd;
  }
  struct Chunk {
    ChunkScales<FMT> sc[2];
    int left;                            // values to the end of a row
  };
  // chunks of a wave: kpart, kpart + wk, ... of every segment's four, counted through;
  // as many loads past the end
  const int each = 4 / a.wk;             // of a segment
  const int rounds = (segs * each + kMidDepth - 1) / kMidDepth * kMidDepth / each;   // segments
  auto load = [&](Chunk& f, int d, int at) {
    const int seg = at / each;
    const int k0 = seg < segs ? place(seg) * KSEG + (at % each * a.wk + kpart) * kMidChunk : K;
    const int left = K - k0;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int co = (int)(32 * cpiece < left ? coff[i] + k0 / 2 : kBufferEnd);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void_t*)cs[d][wave][i], 16, co, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) f.sc[i].load(rs, soff[i], k0, K);
    f.left = left;
  };
  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x + first * a.xs, ((cols - 1) * a.xs + K) * 2);
  if (wave >= kMidWaves) {
    // tokens of a loader: every second; 64 lanes take a token's segment, piece p of
    // token c at p ^ c % 16
    constexpr int EACH = TOKENS / kMidLoaders;
    const int l0 = wave - kMidWaves;
    auto fill_x = [&](int seg) {
      const int k0 = seg < segs ? place(seg) * KSEG : K;
      uint8_t* const buf = xs[seg % BUFFERS];
#pragma unroll
      for (int i = 0; i < EACH; i++) {
        const int c = l0 + kMidLoaders * i;
        const int k = k0 + 8 * (lane ^ (c & 15));
        const bool in = (c < cols) & (k < K);
        const int o = (int)(in ? 2 * (c * (uint32_t)a.xs + k) : kBufferEnd);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(buf + c * KSEG * 2), 16, o, 0, 0, 0);
      }
    };
#pragma unroll
    for (int i = 0; i < BUFFERS - 1; i++) fill_x(i);
    for (int seg = 0; seg < rounds; seg++) {
      wait_vm<(BUFFERS - 2) * EACH>();             // all but the segments after it
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      fill_x(seg + BUFFERS - 1);                   // past the end: zeros
    }
    wait_vm<0>();
    __syncthreads();
    if (a.wk > 1) __syncthreads();
    return;
  }
  f32x4_t acc[2][NT] = {};
  auto multiply = [&](Chunk& f, int d, const uint8_t* x, int chunk, int next) {
    wait_vm<(2 + 2 * ChunkScales<FMT>::N) * (kMidDepth - 1)>();      // all but the later chunks
    u32x4_t v[4][NT], cd[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
      cd[i] = *(const u32x4_t*)(cs[d][wave][i] + 64 * r + 16 * (g ^ (r >> 2)));
    ChunkScales<FMT> sc[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      sc[i].shift = f.sc[i].shift;
#pragma unroll
      for (int q = 0; q < ChunkScales<FMT>::N; q++)
        sc[i].v[q] = (uint32_t)__shfl((int)f.sc[i].v[q], r, 64);
    }
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int piece = (chunk * kMidChunk + 32 * q) / 8 + g;
#pragma unroll
      for (int j = 0; j < NT; j++)
        v[q][j] = *(const u32x4_t*)(x + ((16 * j + r) * KSEG + 8 * (piece ^ r)) * 2);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 2; i++) cd[i] = turn_groups(cd[i]);
    const int left = f.left;
    __builtin_amdgcn_sched_barrier(0);   // the codes are in registers: their buffer is free
    load(f, d, next);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 4; q++) {
      u32x4_t op[2];
#pragma unroll
      for (int i = 0; i < 2; i++) op[i] = decode8<FMT>(cd[i][q], sc[i].at(q, g, left));
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < 2; i++) acc[i][j] = mfma16_bf16(op[i], v[q][j], acc[i][j]);
    }
  };
  // straight through in rounds of kMidDepth chunks, the last ones past the end: a
  // branch in between would have the compiler wait for all loads at once
  Chunk f[kMidDepth];
#pragma unroll
  for (int d = 0; d < kMidDepth; d++) {
    load(f[d], d, d);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int at = 0; at < rounds * each; at += kMidDepth)
    static_for<kMidDepth>([&](auto di) {
      constexpr int d = decltype(di)::value;
      const int step = at + d, seg = step / each;
      if (step % each == 0) {
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      multiply(f[d], d, xs[seg % BUFFERS], step % each * a.wk + kpart, step + kMidDepth);
      __builtin_amdgcn_sched_barrier(0);
    });
  wait_vm<0>();
  __syncthreads();                     // the last zeros have landed, and all is read
  if (a.wk > 1) {                      // the first wave of a set takes the others' sums
    f32x4_t(*red)[NT][2][64] = (f32x4_t(*)[NT][2][64])xs[0];
    if (kpart)
#pragma unroll
      for (int j = 0; j < NT; j++) {
        red[wave][j][0][lane] = acc[0][j];
        red[wave][j][1][lane] = acc[1][j];
      }
    __syncthreads();
    if (kpart) return;
    for (int w = 1; w < a.wk; w++)
#pragma unroll
      for (int j = 0; j < NT; j++) {
        acc[0][j] += red[wave + w][j][0][lane];
        acc[1][j] += red[wave + w][j][1][lane];
      }
  }
#pragma unroll
  for (int j = 0; j < NT; j++)
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int n = blk + set * 32 + 16 * i + 4 * g, c = 16 * j + r;
      if (c < cols && n < rows) put_rows<false>(a, 0, rows, n, first + c, all, {acc[i][j]});
    }
}

// The down projection of a few tokens (16 and 32 assignments at most), joined
// over their experts in the same launch: a workgroup takes 16 rows, its waves
// the steps of all assignments in turn, each the product of one expert's rows
// with one hidden row, which lands in its token's column of the sum with its
// weight.  An expert of several tokens is decoded for each of them.  Latency
// bounds it: 1 token, 6 experts of 1408 x 2048 8.4 us.
constexpr int kFewWaves = 8, kFewThreads = kFewWaves * 64, kFewMost = 32;

struct FewStep {
  uint8_t code[2048], scale[256], x[1024];
};

template <int FMT>
__global__ __launch_bounds__(kFewThreads, 2) void fp4_down_few_kernel(ColsArgs a, const float* weights) {
  __shared__ __attribute__((aligned(16))) FewStep step0[kFewWaves], step1[kFewWaves];
  __shared__ f32x4_t red[kFewWaves][64];
  constexpr int G = WeightFmt<FMT>::G, SD = FMT == 0 ? 4 : 2;
  const int t = (int)threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n = (int)(a.tokens * a.top_k), K = a.w.cols, rows = a.w.rows, blk = (int)blockIdx.x * 16;
  const int steps = (K + kColsStep - 1) / kColsStep, units = n * steps;
  int id = lane < n ? a.ids[lane] : -1;              // of assignment `lane`
  const float wt = lane < n ? weights[lane] : 0.0f;
  if (id < 0 || id >= a.experts) id = -1;
  auto expert = [&](int at) { return __builtin_amdgcn_readlane(id, at); };
  const int crow = lane >> 3, cpiece = lane & 7, srow = lane / SD, sdw = lane % SD;
  const int left = rows - blk;
  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, a.x_bytes);
  auto fill = [&](FewStep& s, int unit) {
    const int at = unit / steps, k0 = (unit - at * steps) * kColsStep;
    const int e = unit < units ? expert(at) : -1;
    const int64_t ee = e < 0 ? 0 : e;
    const __amdgpu_buffer_rsrc_t rc =
        buffer_rsrc(code_row<FMT>(a.w, ee, blk), e < 0 ? 0 : (int64_t)left * (K / 2));
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(
        scale_row<FMT>(a.w, ee, blk), e < 0 ? 0 : (int64_t)(a.w.tile_shift ? (left + 15) / 16 : left) * (K / G));
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int piece = cpiece ^ (((8 * h + crow) >> 1) & 7);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rc, (lds_void_t*)(s.code + 1024 * h), 16,
          k0 + 32 * piece < K ? (8 * h + crow) * (K / 2) + k0 / 2 + 16 * piece : (int)kBufferEnd, 0, 0, 0);
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (lds_void_t*)s.scale, 4,
        srow < 16 && k0 + 4 * G * sdw < K ? (srow >> a.w.tile_shift) * (K / G) + k0 / G + 4 * sdw
                                          : (int)kBufferEnd, 0, 0, 0);
    const int k = k0 + 8 * lane;         // 32 lanes have the step's values
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rx, (lds_void_t*)s.x, 16,
        e >= 0 && lane < 32 && k < K ? (int)((uint32_t)at * (uint32_t)K + k) * 2 : (int)kBufferEnd, 0, 0, 0);
  };
  f32x4_t total = {0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](FewStep& s, int unit) {
    wait_vm<4>();                        // all but the other buffer's loads
    u32x4_t code[2], x[8];
    StepScales<FMT> sc;
#pragma unroll
    for (int h = 0; h < 2; h++) code[h] = *(const u32x4_t*)(s.code + r * 128 + 16 * ((4 * h + g) ^ (r >> 1)));
    if constexpr (FMT == 0) {
      const u32x4_t v = *(const u32x4_t*)(s.scale + r * 16);
#pragma unroll
      for (int q = 0; q < 4; q++) sc.v[q] = v[q];
    } else {
      const u32x2_t v = *(const u32x2_t*)(s.scale + r * 8);
      sc.v[0] = v[0];
      sc.v[1] = v[1];
    }
#pragma unroll
    for (int q = 0; q < 8; q++) x[q] = *(const u32x4_t*)(s.x + 16 * (4 * q + g));
    wait_lds();                          // the buffer is free
    fill(s, unit + 2 * kFewWaves);
    const int at = unit / steps, e = unit < units ? expert(at) : -1;
    if (e < 0) return;                   // uniform
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const u32x4_t cd = turn_groups(code[h]);
#pragma unroll
      for (int q = 0; q < 4; q++)
        acc = mfma16_bf16(decode8<FMT>(cd[q], sc.at(h, q, g)), x[4 * h + q], acc);
    }
    const float w =
        __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(wt), at));
    if (r == at / a.top_k) {             // every column holds the product: its token's takes it
      const float all = alpha_all(a.w, e);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int row = blk + 4 * g + i;
        total[i] = __builtin_fmaf(w * alpha_row(a.w, e, row < rows ? row : rows - 1, all), acc[i], total[i]);
      }
    }
  };
  fill(step0[wave], wave);
  fill(step1[wave], wave + kFewWaves);
  for (int u = wave; u < units; u += 2 * kFewWaves) {
    multiply(step0[wave], u);
    multiply(step1[wave], u + kFewWaves);
  }
  wait_vm<0>();
  red[wave][lane] = total;
  __syncthreads();
  if (wave == 0 && r < a.tokens && 4 * g < left) {   // rows come in fours
    f32x4_t v = red[0][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; w++) v += red[w][lane];
    *(u32x2_t*)((uint16_t*)a.out + r * a.os + blk + 4 * g) = u32x2_t{bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3])};
  }
}

}  // namespace fp4q
