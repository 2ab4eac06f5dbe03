// linear_tiled_kernels.h -- products of many activations with FP4 weights
// (prompts), dense or through experts: the mathematics of linear_kernels.h in
// tiles of 128 tokens x 256 rows of weights.
//
// Four waves share the tile's activations through LDS and take 64 rows each,
// whose codes they decode straight into operand registers: every code of a
// tile is decoded once, and 128 tokens a decoded value keep the decode (2
// vector instructions a value of NVFP4, 1/2 of MXFP4) beside the matrix unit's
// work, 32x32x16 products with the weights as the first operand.
//
// K goes in stages of 128 values through two LDS buffers, filled by direct
// global-to-LDS loads.  A lane serves row lane % 32 and the 64 values number
// lane / 32 of a stage (32 bytes of codes in a row), in 8 groups of 8: the
// operands of a group are read and decoded between the products of the one
// before.  After a stage's last reads the wave waits for the next stage, the
// workgroup meets, and the loads of the stage after that go out: they have a
// whole stage to arrive.
//
// 8192 tokens through 14336x4096: NVFP4 831 to 950 us as the clock allows (1.16
// PFLOP/s), MXFP4 853; a library's product of the same size with weights in bf16
// 716.  Two workgroups share a CU, so two waves a SIMD, of 256 registers each: the
// sums take 128, and all but one form keep 2 to 12 values in scratch.  The matrix
// unit is busy 58% of the time and the vector unit, with the decode, 47%; waves wait
// 39%, at a stage's barrier and for its loads.  Experts' tiles are short (4096
// tokens, 6 of 64 experts, 2048 x 1408, NVFP4: gate and up 411 us, down 257, 600 and
// 480 TFLOP/s), so their first loads and last stores weigh more.
//
// LDS layout of a stage: 256 bytes a token, its 16-byte chunk c at position
// c ^ (token % 16), so that the reads of 16 tokens cover all banks.
#pragma once

#include "linear_kernels.h"

namespace fp4q {

constexpr int kTileTokens = 128, kTileWeights = 256, kTileK = 128;
constexpr int kTiledThreads = 256;
constexpr int kTileBytes = kTileTokens * kTileK * 2;           // of a stage in LDS

struct TiledArgs {
  WeightView w;
  const uint16_t* x;
  void* out;
  int64_t xs, os;
  int64_t tokens;
  const int32_t *off, *order;            // experts: [E + 1], [assignments]
  int top_k, experts;
  int inner;                             // gated: F
  int x_per_token;
  int64_t x_bytes;                       // experts: of x
  int out_f32, out_vec;                  // whole 16-byte stores fit
  uint32_t tiles_t, tiles_n;
};

__device__ __forceinline__ f32x16_t mfma32_bf16(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// A lane's codes of a stage: two row tiles, 64 values and their scales each.
template <int FMT>
struct StageCodes {
  u32x4_t c[2][2];
  uint32_t s[2];
};

// Expert and tile of 128 of its assignments: expert e's tiles start at
// off[e] / 128 + e, which leaves room for each one's last, partial tile without
// a sum over tiles; numbers between have none (count 0).
__device__ __forceinline__ void expert_tile(const TiledArgs& a, uint32_t t, int64_t& e,
                                            int64_t& first, int64_t& count) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0, n = (uint32_t)a.experts;
  while (n > 1) {
    const uint32_t step = (n + 63) / 64, at = step * lane;
    const bool below = at < n && (uint32_t)a.off[lo + at] / kTileTokens + lo + at <= t;
    const uint32_t skip = step * (uint32_t)(__popcll(__ballot(below)) - 1);
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int32_t o0 = a.off[lo], o1 = a.off[lo + 1];
  const int64_t tile = (int64_t)t - (o0 / kTileTokens + (int64_t)lo);
  e = lo;
  first = o0 + tile * kTileTokens;
  count = o1 - first < kTileTokens ? o1 - first : kTileTokens;
}

// FMT of the weights; GATED: wave w takes 32 rows of the gate and the same 32 of
// the up projection; EXPERTS: the tokens are an expert's assignments.
template <int FMT, bool GATED, bool EXPERTS>
__global__ __launch_bounds__(kTiledThreads, 2) void fp4_tiled_kernel(TiledArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kTileBytes], buf1[kTileBytes];
  const int lane = threadIdx.x & 63, r = lane & 31, hh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t e = 0, first, count;
  uint32_t tn;
  if constexpr (EXPERTS) {
    // an XCD (workgroup id % 8) takes four token tiles through all rows
    const uint32_t k = blockIdx.x / kXcds, xcd = blockIdx.x % kXcds;
    const uint32_t t = (k / (4 * a.tiles_n) * kXcds + xcd) * 4 + k % 4;
    tn = k / 4 % a.tiles_n;
    if (t >= a.tiles_t) return;
    expert_tile(a, t, e, first, count);
    if (count <= 0) return;
  } else {
    TileOrder to;
    if (!xcd_tile<8, 8>(blockIdx.x, a.tiles_t, a.tiles_n, to)) return;
    first = to.ty * kTileTokens;
    count = a.tokens - first < kTileTokens ? a.tokens - first : kTileTokens;
    tn = (uint32_t)to.tx;
  }
  const float all = alpha_all(a.w, e);
  const int rows = GATED ? a.inner : a.w.rows, K = a.w.cols;
  constexpr int WAVE_ROWS = GATED ? 32 : 64;
  const int n0 = (int)tn * (GATED ? kTileWeights / 2 : kTileWeights) + wave * WAVE_ROWS;

  // Buffers over the tile's rows of weights and over x: what lies past them, or
  // past K, is read as zeros, and zero times zero adds nothing.  The host keeps
  // all offsets under 2^31.
  constexpr int G = WeightFmt<FMT>::G;
  const int row0 = (int)tn * (GATED ? kTileWeights / 2 : kTileWeights);
  __amdgpu_buffer_rsrc_t rc[GATED ? 2 : 1], rs[GATED ? 2 : 1];
#pragma unroll
  for (int i = 0; i < (GATED ? 2 : 1); i++) {
    const int n = row0 + (i ? rows : 0), left = rows - row0;
    const int srows = a.w.tile_shift ? (left + 15) / 16 : left;
    rc[i] = buffer_rsrc(code_row<FMT>(a.w, e, n), (int64_t)left * (K / 2));
    rs[i] = buffer_rsrc(scale_row<FMT>(a.w, e, n), (int64_t)srows * (K / G));
  }
  uint32_t coff[2], soff[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int n = wave * WAVE_ROWS + (GATED ? 0 : 32 * i) + r;
    coff[i] = (uint32_t)n * (uint32_t)(K / 2) + 32 * hh;
    soff[i] = (uint32_t)(n >> a.w.tile_shift) * (uint32_t)(K / G) + 64 / G * hh;
  }
  const __amdgpu_buffer_rsrc_t rx =
      EXPERTS ? buffer_rsrc(a.x, a.x_bytes) : buffer_rsrc(a.x + first * a.xs, (count - 1) * a.xs * 2 + K * 2);
  // the wave's 8 direct loads: lane -> token lane / 16 of 4, position lane % 16
  uint32_t xoff[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int t = 32 * wave + 4 * i + (lane >> 4);
    int64_t row = t;
    if constexpr (EXPERTS) {
      row = a.order[first + (t < count ? t : 0)];
      if (a.x_per_token) row = (int64_t)((uint32_t)row / (uint32_t)a.top_k);
    }
    xoff[i] = t < count ? (uint32_t)(row * a.xs * 2) + 16 * ((lane & 15) ^ (t & 15)) : kBufferEnd;
  }

  auto fill = [&](uint8_t* buf, int ks) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int chunk = (lane & 15) ^ ((4 * i + (lane >> 4)) & 15);
      const bool in = ks * kTileK + 8 * chunk < K;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(buf + 1024 * (8 * wave + i)), 16,
                                               in ? xoff[i] + ks * (2 * kTileK) : kBufferEnd, 0, 0, 0);
    }
  };
  auto load_codes = [&](StageCodes<FMT>& c, int ks) {
    const int k0 = ks * kTileK;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      uint32_t b[2];
#pragma unroll
      for (int s = 0; s < 2; s++) {
        const bool in = k0 + 64 * hh + 32 * s < K;
        const int co = (int)(in ? coff[i] + k0 / 2 + 16 * s : kBufferEnd);
        const int so = (int)(in ? soff[i] + (k0 + 32 * s) / G : kBufferEnd);
        c.c[i][s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rc[GATED ? i : 0], co, 0, 0));
        if constexpr (FMT == 0) b[s] = __builtin_amdgcn_raw_buffer_load_b16(rs[GATED ? i : 0], so, 0, 0);
        else b[s] = __builtin_amdgcn_raw_buffer_load_b8(rs[GATED ? i : 0], so, 0, 0);
      }
      c.s[i] = b[0] | b[1] << (FMT == 0 ? 16 : 8);
    }
  };
  // operands of group g (32-value half g / 4, 8 values g % 4): token tile j, and
  // dword d of both row tiles
  auto read_x = [&](const uint8_t* buf, int g, int j) {
    return *(const u32x4_t*)(buf + (32 * j + r) * 256 + 16 * ((8 * hh + g) ^ (r & 15)));
  };
  auto decode = [&](const StageCodes<FMT>& c, auto gi, auto di, u32x4_t (&w)[2]) {
    constexpr int s = decltype(gi)::value / 4, q = decltype(gi)::value % 4, d = decltype(di)::value;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint32_t code = c.c[i][s][q];
      if constexpr (FMT == 0) {
        const float2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)(c.s[i] & 0x7F7F7F7Fu), 1.0f,
                                                                    s == 1);
        const float2_t f = fp4x2_to_f32<d>(code, 1.0f);
        w[i][d] = bf16x2_of(f[0] * v[q / 2], f[1] * v[q / 2]);
      } else {
        const float v = __uint_as_float((s == 0 ? c.s[i] & 0xFFu : c.s[i] >> 8) << 23);
        w[i][d] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, v, d));
      }
    }
  };

  f32x16_t acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = f32x16_t{};
  u32x4_t x[4], w0[2], w1[2];
  StageCodes<FMT> c0, c1;
  const int stages = (K + kTileK - 1) / kTileK;
  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // Stage ks from `cur`; its group 0 is in x, w0.  After the products of token
  // tile j its registers take the next group's, and a quarter of the next
  // group's weights is decoded.
  auto stage = [&](uint8_t* cur, const uint8_t* nxt, StageCodes<FMT>& cc, StageCodes<FMT>& cn, int ks) {
    static_for<8>([&](auto gi) {
      constexpr int g = decltype(gi)::value, gn = (g + 1) % 8;
      u32x4_t(&w)[2] = g % 2 ? w1 : w0;
      u32x4_t(&wn)[2] = g % 2 ? w0 : w1;
      static_for<4>([&](auto ji) {
        constexpr int j = decltype(ji)::value;
        acc[0][j] = mfma32_bf16(w[0], x[j], acc[0][j]);
        acc[1][j] = mfma32_bf16(w[1], x[j], acc[1][j]);
        if constexpr (g == 7 && j == 0) {
          // lgkmcnt(0), vmcnt(0): this stage's reads, the next stage's loads
          __builtin_amdgcn_s_waitcnt((7 << 4));
          barrier();
          fill(cur, ks + 2);
          load_codes(cc, ks + 2);
        }
        x[j] = read_x(g < 7 ? cur : nxt, gn, j);
        decode(g < 7 ? cc : cn, std::integral_constant<int, gn>{}, ji, wn);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };

  fill(buf0, 0);
  load_codes(c0, 0);
  fill(buf1, 1);
  load_codes(c1, 1);
  __builtin_amdgcn_s_waitcnt((7 << 4));
  barrier();
#pragma unroll
  for (int j = 0; j < 4; j++) x[j] = read_x(buf0, 0, j);
  static_for<4>([&](auto d) { decode(c0, std::integral_constant<int, 0>{}, d, w0); });
  for (int ks = 0; ks < stages; ks += 2) {           // a stage past the last adds zeros
    stage(buf0, buf1, c0, c1, ks);
    stage(buf1, buf0, c1, c0, ks + 1);
  }
  __builtin_amdgcn_s_waitcnt((7 << 4));  // zeros on their way to LDS past the last stage

  // a lane's 16 sums of a tile: rows 8 (v / 4) + 4 hh + v % 4, token lane % 32
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int64_t c = 32 * j + r;
    int64_t orow = first + (c < count ? c : 0);
    if constexpr (EXPERTS) orow = a.order[orow];
#pragma unroll
    for (int i = 0; i < (GATED ? 1 : 2); i++) {
      const int nb = n0 + 32 * i;
      float y[16];
      auto sum = [&](int h, int v) {     // of row tile i, or of projection h
        const int n = nb + 8 * (v / 4) + 4 * hh + v % 4, row = n < rows ? n : rows - 1;
        return acc[GATED ? h : i][j][v] * alpha_row(a.w, e, row + h * rows, all);
      };
      if constexpr (GATED) {
        silu_times(y, [&](int v) { return sum(0, v); }, [&](int v) { return sum(1, v); });
      } else {
#pragma unroll
        for (int v = 0; v < 16; v++) y[v] = sum(0, v);
      }
      if (a.out_f32) {
        if (c >= count) continue;
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int n = nb + 8 * q + 4 * hh;
          float* p = (float*)a.out + orow * a.os + n;
          if (a.out_vec && n + 3 < rows) {
            *(f32x4_t*)p = f32x4_t{y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
          } else {
#pragma unroll
            for (int v = 0; v < 4; v++)
              if (n + v < rows) p[v] = y[4 * q + v];
          }
        }
        continue;
      }
      uint16_t* const out = (uint16_t*)a.out + orow * a.os;
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        // halves of the wave hold rows 0..3 and 4..7 of each 8: swapped, a lane has 8 in a run
        const uint32_t a0 = bf16x2_of(y[4 * q], y[4 * q + 1]), a1 = bf16x2_of(y[4 * q + 2], y[4 * q + 3]);
        const uint32_t b0 = bf16x2_of(y[4 * q + 4], y[4 * q + 5]), b1 = bf16x2_of(y[4 * q + 6], y[4 * q + 7]);
        const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
        const u32x4_t v = {s0[0], s1[0], s0[1], s1[1]};
        const int n = nb + 8 * q + 8 * hh;
        if (c >= count) continue;
        if (a.out_vec && n + 7 < rows) {
          *(u32x4_t*)(out + n) = v;
        } else {
#pragma unroll
          for (int h = 0; h < 8; h++)
            if (n + h < rows) out[n + h] = (uint16_t)(v[h / 2] >> (16 * (h & 1)));
        }
      }
    }
  }
}

}  // namespace fp4q
