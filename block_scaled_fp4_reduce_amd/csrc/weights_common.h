// weights_common.h -- FP4 weights as operands of the bf16 matrix instructions.
//
// An NVFP4 value without its alpha is E2M1 x E4M3 (at most 6 significant
// bits, 2^-10 to 2688 in magnitude), an MXFP4 value E2M1 x 2^k: both are exact
// in bf16, so products with bf16 activations are exact in the matrix
// instructions' fp32 sums, and alpha is one factor of a row's sum.
//
// Decoding eight codes (a dword): MXFP4 4 conversions, which take the scale as
// their exponent; NVFP4 4 conversions to fp32, 8 products, 4 packs (no packed
// bf16 product exists, and fp16 operands would need the activations' range
// checked and moved).
#pragma once

#include "kv_common.h"

namespace fp4q {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

struct WeightView {
  const uint8_t *codes, *scales;
  const float* alpha;                    // NULL: MXFP4
  int64_t codes_e, scales_e, alpha_e;    // bytes, bytes and floats from one expert to the next
  int rows, cols;
  int tile_shift;                        // 4: a scale serves 16 rows
  int row_alpha;                         // floats from one row's alpha to the next (0 or 1)
};

// An offset past every buffer of activations, which the host keeps below it: reads
// as zeros.  Codes or scales of more bytes than that are read there instead, with
// activations that are zeros.
constexpr uint32_t kBufferEnd = 0x7FFFFF00u;

// FMT: FP4_FORMAT_NVFP4 (0) or FP4_FORMAT_MXFP4 (1).
template <int FMT>
struct WeightFmt {
  static constexpr int G = FMT == 0 ? 16 : 32;
};

// Row n of expert e.
template <int FMT>
__device__ __forceinline__ const uint8_t* code_row(const WeightView& w, int64_t e, int n) {
  return w.codes + e * w.codes_e + (int64_t)n * (w.cols / 2);
}
template <int FMT>
__device__ __forceinline__ const uint8_t* scale_row(const WeightView& w, int64_t e, int n) {
  return w.scales + e * w.scales_e + (int64_t)(n >> w.tile_shift) * (w.cols / WeightFmt<FMT>::G);
}
// An expert's alpha where it is one number, loaded early and by the scalar unit.
__device__ __forceinline__ float alpha_all(const WeightView& w, int64_t e) {
  return w.alpha && !w.row_alpha ? w.alpha[e * w.alpha_e] : 1.0f;
}
// A row's factor, all = alpha_all.
__device__ __forceinline__ float alpha_row(const WeightView& w, int64_t e, int n, float all) {
  return w.row_alpha ? w.alpha[e * w.alpha_e + n] : all;
}

// Eight codes (even element low) to a bf16 operand.
template <int FMT>
__device__ __forceinline__ u32x4_t decode8(uint32_t w, float s) {
  u32x4_t o;
  if constexpr (FMT == 0) {
    const float2_t a = fp4x2_to_f32<0>(w, 1.0f), b = fp4x2_to_f32<1>(w, 1.0f);
    const float2_t c = fp4x2_to_f32<2>(w, 1.0f), d = fp4x2_to_f32<3>(w, 1.0f);
    o[0] = bf16x2_of(a[0] * s, a[1] * s);
    o[1] = bf16x2_of(b[0] * s, b[1] * s);
    o[2] = bf16x2_of(c[0] * s, c[1] * s);
    o[3] = bf16x2_of(d[0] * s, d[1] * s);
  } else {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  }
  return o;
}

__device__ __forceinline__ f32x4_t mfma16_bf16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Wait until at most N of this wave's vector-memory operations are under way.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
}
// Wait for this wave's LDS operations.
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
  asm volatile("" ::: "memory");
}

// silu(g) u of N gates g(i) and values u(i).  Where e^-g leaves fp32 (g below
// -88.7) silu is g e^g, whose product with u need not be small: e^(g/2) twice, in a
// pass of its own that few waves take (a branch for each value keeps them from being
// computed side by side: 4096 tokens of 64 experts 661 us, so 625).
constexpr float kFarGate = -88.0f;
template <int N, typename G, typename U>
__device__ __forceinline__ void silu_times(float (&y)[N], G&& g, U&& u) {
  float least = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++) {
    const float v = g(i);
    least = fminf(least, v);
    y[i] = v / (1.0f + expf(-v)) * u(i);
  }
  if (least < kFarGate)
#pragma unroll
    for (int i = 0; i < N; i++) {
      const float v = g(i), h = expf(0.5f * v);
      if (v < kFarGate) y[i] = v * h * u(i) * h;
    }
}

}  // namespace fp4q
