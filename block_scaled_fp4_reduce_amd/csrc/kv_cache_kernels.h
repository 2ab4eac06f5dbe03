// kv_cache_kernels.h -- keys and values quantized into the pages of the FP4
// cache, and read back.
//
// Writing is the library's 1D quantizer on each head's values ("Four Over
// Six", Eq. 1-3 and the 4/6 choice; MXFP4 with UE8M0 scales) with the
// head's largest magnitude given, so the codes of a token are those of
// nvfp4_quantize with amax_in, or of mxfp4_quantize.  Reading is the decode
// of fp4_dequantize, rounded to bf16.
#pragma once

#include "kv_common.h"
#include "nvfp4_kernels.h"

namespace fp4q {

// Codes (two dwords) and scale byte of 16 values under NVFP4 with tensor
// constants ts.
template <bool F46>
__device__ __forceinline__ void kv_quant16(const float* y, const TensorScale& ts, uint32_t& w0,
                                           uint32_t& w1, uint32_t& scale) {
  const float m = block_amax16(y);
  uint32_t e6, e4;
  e4m3_pair(m * ts.k6, m * ts.k4, e6, e4);
  const float s6 = ts.alpha * e4m3_value(e6);
  w0 = w1 = 0;
  const float err6 = quant16_rtn(y, s6, s6 == 0.0f ? 0.0f : 1.0f / s6, w0, w1);
  scale = e6;
  if constexpr (F46) {
    const float s4 = ts.alpha * e4m3_value(e4);
    uint32_t u0 = 0, u1 = 0;
    const float err4 = quant16_rtn(y, s4, s4 == 0.0f ? 0.0f : 1.0f / s4, u0, u1);
    if (err4 < err6) {                   // ties keep M = 6
      w0 = u0;
      w1 = u1;
      scale = e4;
    }
  }
}

// Codes (two dwords per 16 values) and scale byte of 32 values under MXFP4.
__device__ __forceinline__ void kv_quant32(const float* y, uint32_t* w, uint32_t& scale) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i++) m = fmaxf(m, fabsf(y[i]));
  const int ef = (int)(__float_as_uint(m) >> 23);
  scale = (uint32_t)(ef > 2 ? ef - 2 : 0);
  const float s = __uint_as_float(scale << 23);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    w[i] = cvt_fp4x2<0>(0, y[8 * i], y[8 * i + 1], s);
    w[i] = cvt_fp4x2<1>(w[i], y[8 * i + 2], y[8 * i + 3], s);
    w[i] = cvt_fp4x2<2>(w[i], y[8 * i + 4], y[8 * i + 5], s);
    w[i] = cvt_fp4x2<3>(w[i], y[8 * i + 6], y[8 * i + 7], s);
  }
}

// MODE: 0 NVFP4, 1 NVFP4 with 4/6, 2 MXFP4.
template <int MODE>
constexpr int kv_group() { return MODE == 2 ? 32 : 16; }

// One lane per group of one head's key or value (the first half of the
// lanes of a token take its keys).
template <int MODE>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvView c, const uint16_t* k, int64_t ks,
                                                            const uint16_t* v, int64_t vs,
                                                            const int64_t* slots, int64_t tokens) {
  constexpr int G = kv_group<MODE>();
  const int gph = c.dim / G, per = c.heads * gph;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= tokens * 2 * per) return;
  const int64_t tok = i / (2 * per);
  int r = (int)(i - tok * (2 * per));
  const bool isv = r >= per;
  if (isv) r -= per;
  const int h = r / gph, g = r - h * gph;
  const int64_t slot = slots[tok], page = slot_page(c, slot);
  if (page < 0) return;
  const int P = 1 << c.page_shift, at = (int)(slot & (P - 1));
  const uint4* x = (const uint4*)(isv ? v + tok * vs : k + tok * ks) + (h * c.dim + g * G) / 8;
  float y[G];
#pragma unroll
  for (int j = 0; j < G / 8; j++) unpack8(x[j], y + 8 * j);
  uint32_t w[G / 8], scale;
  if constexpr (MODE == 2) kv_quant32(y, w, scale);
  else kv_quant16<MODE == 1>(y, tensor_scale((isv ? c.vam : c.kam)[h], MODE == 1), w[0], w[1], scale);
  const int64_t ph = page * c.heads + h;
  if (!isv) {
    uint32_t* o = (uint32_t*)(c.kc + (ph * P + at) * (c.dim / 2) + g * (G / 2));
#pragma unroll
    for (int j = 0; j < G / 8; j++) o[j] = w[j];
    c.ks[(ph * P + at) * gph + g] = (uint8_t)scale;
  } else {
    uint8_t* o = c.vc + (ph * (c.dim / 2) + g * (G / 2)) * P + at;
#pragma unroll
    for (int j = 0; j < G / 2; j++) o[(int64_t)j * P] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    c.vs[(ph * gph + g) * P + at] = (uint8_t)scale;
  }
}

// One lane per group, as above; slots without a page read as zeros.
template <int MODE>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvView c, const int64_t* slots,
                                                           int64_t tokens, uint16_t* k, int64_t ks,
                                                           uint16_t* v, int64_t vs) {
  constexpr int G = kv_group<MODE>();
  const int gph = c.dim / G, per = c.heads * gph;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= tokens * 2 * per) return;
  const int64_t tok = i / (2 * per);
  int r = (int)(i - tok * (2 * per));
  const bool isv = r >= per;
  if (isv) r -= per;
  const int h = r / gph, g = r - h * gph;
  const int64_t slot = slots[tok], page = slot_page(c, slot);
  const int P = 1 << c.page_shift, at = (int)(slot & (P - 1));
  uint32_t w[G / 8] = {};
  float s = 0.0f;
  if (page >= 0) {
    const int64_t ph = page * c.heads + h;
    uint32_t code;
    if (!isv) {
      const uint32_t* o = (const uint32_t*)(c.kc + (ph * P + at) * (c.dim / 2) + g * (G / 2));
#pragma unroll
      for (int j = 0; j < G / 8; j++) w[j] = o[j];
      code = c.ks[(ph * P + at) * gph + g];
    } else {
      const uint8_t* o = c.vc + (ph * (c.dim / 2) + g * (G / 2)) * P + at;
#pragma unroll
      for (int j = 0; j < G / 2; j++) w[j / 4] |= (uint32_t)o[(int64_t)j * P] << (8 * (j % 4));
      code = c.vs[(ph * gph + g) * P + at];
    }
    if constexpr (MODE == 2) s = __builtin_ldexpf(1.0f, (int)code - 127);
    else s = tensor_scale((isv ? c.vam : c.kam)[h], MODE == 1).alpha * e4m3_value(code & 0x7Fu);
  }
  uint4* o = (uint4*)(isv ? v + tok * vs : k + tok * ks) + (h * c.dim + g * G) / 8;
#pragma unroll
  for (int j = 0; j < G / 8; j++) {
    float y[8];
    const float2_t a = fp4x2_to_f32<0>(w[j], 1.0f), b = fp4x2_to_f32<1>(w[j], 1.0f);
    const float2_t d = fp4x2_to_f32<2>(w[j], 1.0f), e = fp4x2_to_f32<3>(w[j], 1.0f);
    y[0] = a.x * s; y[1] = a.y * s; y[2] = b.x * s; y[3] = b.y * s;
    y[4] = d.x * s; y[5] = d.y * s; y[6] = e.x * s; y[7] = e.y * s;
    o[j] = pack8(y);
  }
}

}  // namespace fp4q
