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
  // Up to 252, the scale of the largest finite values: with an infinity's 253 the
  // largest code reads as infinity, and in attention 0 times that is NaN for the
  // rows that give the token no weight.
  const int ef = (int)(__float_as_uint(m) >> 23);
  scale = (uint32_t)(ef > 2 ? min(ef - 2, 252) : 0);
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

// Both kernels: a workgroup takes TT consecutive tokens of one head.  Keys go
// straight through: a token's codes are one run, as its values are.  A
// value's tokens are a run for each pair of channels, so values are turned in
// LDS, and where 16 tokens in a row sit side by side in their page (a prompt
// stored or read in order) a lane moves all 16 bytes of a channel pair at
// once; otherwise byte by byte.  All loads go out before the first store.
//
// Memory bounds the long calls: 65536 tokens of 8 heads of 128 (NVFP4 4/6, 344
// MB) read in 71 to 73 us, 4.7 TB/s, where a large copy moves 4.85.  8192
// tokens written take 13 to 15 us (43 MB: 8.9 us at that rate; vector
// instructions issue in 47% of the dispatch's cycles, and a wave waits to issue
// for 46% of its time and for data for 34%) and 8.4 to 9.8 us read (27%, 30%
// and 49%).  One lane per group
// with byte loads and stores for the values took 169 us and 46 for the pair.
// A decoding step's 256 scattered tokens take 5.8 and 6.2 us, all latency.
//
// Slots of the tile, and which of its 16-token stretches sit side by side.
template <int TT>
struct KvSlots {
  int64_t slot[TT];
  uint32_t runs;                         // bit s: tokens 16 s .. 16 s + 15 are one aligned run
};

template <int TT>
__device__ __forceinline__ void load_slots(const KvView& c, const int64_t* slots, int64_t t0,
                                           int64_t tokens, KvSlots<TT>& sl) {
  if (threadIdx.x < 64) {
    const int i = (int)threadIdx.x;
    const bool in = i < TT && t0 + i < tokens;
    const int64_t s = in ? slots[t0 + i] : -1;
    const uint32_t lo = __shfl((uint32_t)s, i & 48, 64), hi = __shfl((uint32_t)(s >> 32), i & 48, 64);
    const int64_t head = (int64_t)((uint64_t)hi << 32 | lo);
    const uint64_t ok = __ballot(slot_page(c, s) >= 0 && (head & 15) == 0 && s == head + (i & 15));
    if (i < TT) sl.slot[i] = s;
    if (i == 0) {
      uint32_t runs = 0;
#pragma unroll
      for (int k = 0; k < TT / 16; k++)
        if (((ok >> (16 * k)) & 0xFFFFu) == 0xFFFFu) runs |= 1u << k;
      sl.runs = runs;
    }
  }
  __syncthreads();
}

template <int MODE, int D, int TT>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvView c, const uint16_t* k, int64_t ks,
                                                            const uint16_t* v, int64_t vs,
                                                            const int64_t* slots, int64_t tokens) {
  constexpr int G = kv_group<MODE>(), GPH = D / G, LD = TT + 4;
  __shared__ KvSlots<TT> sl;
  __shared__ __align__(16) uint8_t codes[D / 2 * LD], scales[GPH * LD];
  const int h = (int)(blockIdx.x % (uint32_t)c.heads);
  const int64_t t0 = (int64_t)(blockIdx.x / (uint32_t)c.heads) * TT;
  const int live = (int)(tokens - t0 < TT ? tokens - t0 : TT);
  // all inputs are on their way before the slots are looked at
  constexpr int ITEMS = (2 * TT * GPH + kThreads - 1) / kThreads;
  uint4 x[ITEMS][G / 8];
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    const int it = (int)threadIdx.x + i * kThreads;
    const bool isv = it < TT * GPH;      // values first, then keys
    const int r = isv ? it : it - TT * GPH, tok = r / GPH, g = r % GPH;
    if (it >= 2 * TT * GPH || tok >= live) continue;
    const uint4* from = (const uint4*)((isv ? v + (t0 + tok) * vs : k + (t0 + tok) * ks) + h * D + g * G);
#pragma unroll
    for (int e = 0; e < G / 8; e++) x[i][e] = from[e];
  }
  const float kam = MODE == 2 ? 0.0f : c.kam[h], vam = MODE == 2 ? 0.0f : c.vam[h];
  load_slots<TT>(c, slots, t0, tokens, sl);
  const int P = 1 << c.page_shift;
  const TensorScale kts = tensor_scale(kam, MODE == 1), vts = tensor_scale(vam, MODE == 1);
#pragma unroll
  for (int i = 0; i < ITEMS; i++) {
    const int it = (int)threadIdx.x + i * kThreads;
    const bool isv = it < TT * GPH;
    const int r = isv ? it : it - TT * GPH, tok = r / GPH, g = r % GPH;
    if (it >= 2 * TT * GPH || tok >= live) continue;
    const int64_t slot = sl.slot[tok], page = slot_page(c, slot);
    if (page < 0) continue;
    float y[G];
#pragma unroll
    for (int e = 0; e < G / 8; e++) unpack8(x[i][e], y + 8 * e);
    uint32_t w[G / 8], scale;
    if constexpr (MODE == 2) kv_quant32(y, w, scale);
    else kv_quant16<MODE == 1>(y, isv ? vts : kts, w[0], w[1], scale);
    if (isv) {
#pragma unroll
      for (int e = 0; e < G / 2; e++)
        codes[(g * (G / 2) + e) * LD + tok] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
      scales[g * LD + tok] = (uint8_t)scale;
    } else {
      const int64_t at = (page * c.heads + h) * P + (slot & (P - 1));
      uint32_t* o = (uint32_t*)(c.kc + at * (D / 2) + g * (G / 2));
      if constexpr (MODE == 2) *(uint4*)o = make_uint4(w[0], w[1], w[2], w[3]);
      else *(uint2*)o = make_uint2(w[0], w[1]);
      c.ks[at * GPH + g] = (uint8_t)scale;
    }
  }
  __syncthreads();
  for (int it = (int)threadIdx.x; it < (D / 2 + GPH) * (TT / 16); it += kThreads) {
    const int seg = it % (TT / 16), row = it / (TT / 16);
    const bool sc = row >= D / 2;
    const uint8_t* from = (sc ? scales + (row - D / 2) * LD : codes + row * LD) + seg * 16;
    // [page][head][row][P]
    auto to = [&](int64_t slot, int64_t page) {
      const int64_t ph = page * c.heads + h;
      return (sc ? c.vs + (ph * GPH + row - D / 2) * P : c.vc + (ph * (D / 2) + row) * P) +
             (slot & (P - 1));
    };
    if (sl.runs >> seg & 1) {
      const uint32_t* f = (const uint32_t*)from;
      const int64_t slot = sl.slot[seg * 16];
      *(uint4*)to(slot, slot >> c.page_shift) = make_uint4(f[0], f[1], f[2], f[3]);
    } else {
      for (int e = 0; e < 16 && seg * 16 + e < live; e++) {
        const int64_t slot = sl.slot[seg * 16 + e], page = slot_page(c, slot);
        if (page >= 0) *to(slot, page) = from[e];
      }
    }
  }
}

// Eight bf16 values of a code dword times its scale.
__device__ __forceinline__ uint4 kv_decode8(uint32_t w, float s) {
  const float2_t a = fp4x2_to_f32<0>(w, 1.0f), b = fp4x2_to_f32<1>(w, 1.0f);
  const float2_t d = fp4x2_to_f32<2>(w, 1.0f), e = fp4x2_to_f32<3>(w, 1.0f);
  return make_uint4(bf16x2_of(a.x * s, a.y * s), bf16x2_of(b.x * s, b.y * s),
                    bf16x2_of(d.x * s, d.y * s), bf16x2_of(e.x * s, e.y * s));
}
template <int MODE>
__device__ __forceinline__ float kv_scale(uint32_t code, float alpha) {
  if constexpr (MODE == 2) return __builtin_ldexpf(1.0f, (int)code - 127);
  else return alpha * e4m3_value(code & 0x7Fu);
}

// Slots without a page read as zeros.
template <int MODE, int D, int TT>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvView c, const int64_t* slots,
                                                           int64_t tokens, uint16_t* k, int64_t ks,
                                                           uint16_t* v, int64_t vs) {
  constexpr int G = kv_group<MODE>(), GPH = D / G, LD = D / 2 + 1;
  __shared__ KvSlots<TT> sl;
  __shared__ uint32_t turned[TT * LD];   // [token][channel pair] bf16
  const int h = (int)(blockIdx.x % (uint32_t)c.heads);
  const int64_t t0 = (int64_t)(blockIdx.x / (uint32_t)c.heads) * TT;
  load_slots<TT>(c, slots, t0, tokens, sl);
  const int P = 1 << c.page_shift, live = (int)(tokens - t0 < TT ? tokens - t0 : TT);
  const float ka = MODE == 2 ? 1.0f : tensor_scale(c.kam[h], MODE == 1).alpha;
  const float va = MODE == 2 ? 1.0f : tensor_scale(c.vam[h], MODE == 1).alpha;
  // every load of the codes goes out before the first store
  constexpr int VI = (D / 2 * (TT / 16) + kThreads - 1) / kThreads, KI = TT * (D / 8) / kThreads;
  constexpr int KITEMS = KI ? KI : 1;
  uint32_t vw[VI][4], vsc[VI][4], kw[KITEMS], ksc[KITEMS];
#pragma unroll
  for (int i = 0; i < VI; i++) {
    const int it = (int)threadIdx.x + i * kThreads;
    const int seg = it % (TT / 16), row = it / (TT / 16), g = 2 * row / G;
#pragma unroll
    for (int e = 0; e < 4; e++) vw[i][e] = vsc[i][e] = 0;
    if (it >= D / 2 * (TT / 16)) continue;
    if (sl.runs >> seg & 1) {
      const int64_t slot = sl.slot[seg * 16], ph = (slot >> c.page_shift) * c.heads + h;
      const uint4 a = *(const uint4*)(c.vc + (ph * (D / 2) + row) * P + (slot & (P - 1)));
      const uint4 b = *(const uint4*)(c.vs + (ph * GPH + g) * P + (slot & (P - 1)));
      vw[i][0] = a.x; vw[i][1] = a.y; vw[i][2] = a.z; vw[i][3] = a.w;
      vsc[i][0] = b.x; vsc[i][1] = b.y; vsc[i][2] = b.z; vsc[i][3] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 16; e++) {
        const int64_t slot = sl.slot[seg * 16 + e], page = slot_page(c, slot);
        if (page < 0) continue;
        const int64_t ph = page * c.heads + h;
        vw[i][e / 4] |= (uint32_t)c.vc[(ph * (D / 2) + row) * P + (slot & (P - 1))] << (8 * (e % 4));
        vsc[i][e / 4] |= (uint32_t)c.vs[(ph * GPH + g) * P + (slot & (P - 1))] << (8 * (e % 4));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < KITEMS; i++) {
    const int it = (int)threadIdx.x + i * kThreads, tok = it / (D / 8), ch = it % (D / 8) * 8;
    kw[i] = ksc[i] = 0;
    if (tok >= live) continue;
    const int64_t slot = sl.slot[tok], page = slot_page(c, slot);
    if (page >= 0) {
      const int64_t at = (page * c.heads + h) * P + (slot & (P - 1));
      kw[i] = *(const uint32_t*)(c.kc + at * (D / 2) + ch / 2);
      ksc[i] = c.ks[at * GPH + ch / G];
    }
  }
#pragma unroll
  for (int i = 0; i < VI; i++) {
    const int it = (int)threadIdx.x + i * kThreads, seg = it % (TT / 16), row = it / (TT / 16);
    if (it >= D / 2 * (TT / 16)) continue;
    static_for<16>([&](auto ee) {
      constexpr int e = decltype(ee)::value;
      const float2_t x = fp4x2_to_f32<e % 4>(vw[i][e / 4], 1.0f);
      const float f = kv_scale<MODE>((vsc[i][e / 4] >> (8 * (e % 4))) & 255u, va);
      turned[(seg * 16 + e) * LD + row] = bf16x2_of(x.x * f, x.y * f);
    });
  }
#pragma unroll
  for (int i = 0; i < KITEMS; i++) {
    const int it = (int)threadIdx.x + i * kThreads, tok = it / (D / 8), ch = it % (D / 8) * 8;
    if (tok >= live) continue;
    *(uint4*)(k + (t0 + tok) * ks + h * D + ch) = kv_decode8(kw[i], kv_scale<MODE>(ksc[i], ka));
  }
  __syncthreads();
#pragma unroll
  for (int it = (int)threadIdx.x; it < TT * (D / 8); it += kThreads) {
    const int tok = it / (D / 8), ch = it % (D / 8) * 8;
    if (tok >= live) continue;
    const uint32_t* f = turned + tok * LD + ch / 2;
    *(uint4*)(v + (t0 + tok) * vs + h * D + ch) = make_uint4(f[0], f[1], f[2], f[3]);
  }
}

}  // namespace fp4q
