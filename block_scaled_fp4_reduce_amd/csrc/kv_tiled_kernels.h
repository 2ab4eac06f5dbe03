// kv_tiled_kernels.h -- attention over the paged FP4 cache for many query
// rows per kv head (prompts, chunks): the mathematics of
// kv_attention_kernels.h, with the decoded keys and values of 32 tokens
// shared through LDS.
//
// A workgroup of 4 waves takes 128 rows, 32 a wave (one column tile of the
// 32x32x16 products).  Decoding a value costs about 1.3 vector instructions
// and a row's softmax about 4 per key (12 with capped scores), so 128 rows per
// decoded value keep the decode at a third of the vector work.  That work and
// the matrix products take about as long as each other, so they are woven
// together: the next tile is decoded into LDS between the products of the
// scores, and the second half of the tile's exponentials is taken between the
// products of the first half's values (double buffers, one barrier per tile).
// Tiles of 32 keys keep the registers of a wave at 168, so that three run on
// a SIMD.  Vector instructions bound it: counted at D = 128, MXFP4, capped,
// they issue in 73% of the cycles and the matrix unit runs in 36%.  With parts
// of a cached context (chunks, below) they issue in 53% and the matrix unit
// runs in 34%: a sequence's tiles are cut into equal whole numbers of parts, so
// the longest item has 80 key tiles where the mean has 63.
//
// Measured, D = 128, 32 query and 8 kv heads: a prompt of 8192 tokens, window
// 4096, capped, MXFP4: 481 to 490 us (850 TFLOP/s of the products); 4 sequences
// with up to 512 new tokens over 6144, NVFP4 4/6: 136 to 139 us with the join
// (730 TFLOP/s).  When they were measured side by side (522 and 158 us then), tiles
// of 64 keys and two waves a SIMD took the same on the prompt and 169 us on the
// chunks.
//
// LDS layout: 16-byte chunks, column after column, so that a wave's operand
// reads are contiguous.  Keys: chunk (channels 8 x .. 8 x + 7, key).  Values:
// chunk (tokens 8 y .. 8 y + 7, channel), even channels before odd ones.  The
// padding of a column (16 and 64 bytes) spreads the decoding lanes' stores
// over all banks.
#pragma once

#include "kv_attention_kernels.h"

namespace fp4q {

constexpr int kTileRows = 128;           // query rows of a workgroup
constexpr int kTileKeys = 32;            // keys of a tile

typedef float f32x16_t __attribute__((ext_vector_type(16)));

template <int MODE>
__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (MODE == 2)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// The codes of a thread's part of a tile: D/8 channels of one key, and TOK
// tokens of one channel pair.
template <int MODE, int D>
struct TileCodes {
  static constexpr int G = MODE == 2 ? 32 : 16;
  static constexpr int B = D / 16, W = D / 64;       // bytes and dwords of either
  static constexpr int TOK = B, TG = kTileKeys / TOK;
  static constexpr int VU = D == 64 ? 1 : W / 2;     // pieces of 8 tokens (D = 64: half of one)
  static constexpr int UNITS = W + VU;
  uint32_t k[W], ks, v[W], vs[W];
  int kpage, vpage;
};

template <int MODE, int D, bool WIDE>
__device__ __forceinline__ void load_tile(const AttnArgs& a, int h, uint32_t base, int kpage,
                                          int vpage, TileCodes<MODE, D>& f) {
  using C = TileCodes<MODE, D>;
  constexpr int G = C::G, SB = D / 8 >= G ? D / 8 / G : 1;
  const int t = (int)threadIdx.x, shift = a.c.page_shift, part = t & 7;
  const uint32_t P = 1u << shift;
  f.kpage = kpage;
  f.vpage = vpage;
  // page and token of it (the same for the wave when WIDE), and the lane's offset
  const int64_t pk = head_page(a, h, kpage);
  const int64_t at = pk + ((WIDE ? base : base + (t >> 3)) & (P - 1));
  const uint32_t row = WIDE ? t >> 3 : 0;
  const auto k = KvLoad<C::B, WIDE>::at(a.c.kc + at * (D / 2), row * (D / 2) + part * C::B, 0);
  f.ks = KvLoad<SB, WIDE>::at(a.c.ks + at * (D / G), row * (D / G) + part * (D / 8) / G, 0)[0];
  const int64_t pv = WIDE ? pk : head_page(a, h, vpage);
  const uint32_t tok = (t % C::TG) * C::TOK, av = (WIDE ? base : base + tok) & (P - 1);
  const uint32_t i = t / C::TG, off = WIDE ? tok : 0;
  const auto v = KvLoad<C::B, WIDE>::at(a.c.vc + pv * (D / 2) + av, (i << shift) + off, 0);
  const auto s = KvLoad<C::B, WIDE>::at(a.c.vs + pv * (D / G) + av,
                                        ((2 * i / G) << shift) + off, 0);
#pragma unroll
  for (int e = 0; e < C::W; e++) {
    f.k[e] = k[e];
    f.v[e] = v[e];
    f.vs[e] = s[e];
  }
}

template <int D>
struct TileLds {
  static constexpr int KS = kTileKeys * 16 + 16, VS = D * 16 + 64;      // bytes of a column
  static constexpr int K = D / 8 * KS, V = kTileKeys / 8 * VS;
  uint8_t k[2][K], v[2][V];
  int ok[2][2];                          // narrow pages: that of each 16 tokens is in the cache
};

// The bits of the scales that count.  Values of tokens outside [lo, hi)
// or without a page count as zeros: their scales become zero.
template <int MODE, int D>
__device__ __forceinline__ void clean_scales(TileCodes<MODE, D>& f, uint32_t base, uint32_t lo, uint32_t hi) {
  using C = TileCodes<MODE, D>;
  f.ks &= kScaleBits<MODE>;
#pragma unroll
  for (int w = 0; w < C::W; w++) f.vs[w] &= kScaleBits<MODE>;
  if (base >= lo && base + kTileKeys <= hi && __all(f.vpage >= 0)) return;
  const int tok = ((int)threadIdx.x % C::TG) * C::TOK;
#pragma unroll
  for (int w = 0; w < C::W; w++) {
    uint32_t keep = 0;
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const uint32_t j = base + tok + 4 * w + r;
      if (f.vpage >= 0 && j >= lo && j < hi) keep |= 255u << (8 * r);
    }
    f.vs[w] &= keep;
  }
}

// Unit U of a tile's decode into LDS: a code dword of the keys, then pieces of
// the values.
template <int U, int MODE, int D>
__device__ __forceinline__ void store_unit(const TileCodes<MODE, D>& f, TileLds<D>& lds, int buf) {
  using C = TileCodes<MODE, D>;
  using L = TileLds<D>;
  const int t = (int)threadIdx.x;
  if constexpr (U < C::W) {
    *(u32x4_t*)(lds.k[buf] + ((t & 7) * C::W + U) * L::KS + (t >> 3) * 16) =
        key_operand<MODE, U * 8 / C::G>(f.k[U], f.ks);
  } else {
    constexpr int y = U - C::W, lo = D == 64 ? 0 : 2 * y, hi = D == 64 ? 0 : 2 * y + 1;
    const int tok = (t % C::TG) * C::TOK + 8 * y;
    u32x4_t even, odd;
    value_operands<MODE>(f.v[lo], f.v[hi], f.vs[lo], f.vs[hi], even, odd);
    uint8_t* o = lds.v[buf] + (tok / 8) * L::VS + (t / C::TG) * 16 + (tok % 8) * 2;
    if constexpr (D == 64) {             // 4 tokens
      *(u32x2_t*)o = u32x2_t{even[0], even[1]};
      *(u32x2_t*)(o + D / 2 * 16) = u32x2_t{odd[0], odd[1]};
    } else {
      *(u32x4_t*)o = even;
      *(u32x4_t*)(o + D / 2 * 16) = odd;
    }
  }
}

__device__ __forceinline__ float half_max(float v) {
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Waves a SIMD, which are also the workgroups a CU.  LONG: capped scores above
// kShortCap, in a kernel of its own, because their form takes registers that
// the other calls' waves do not leave; it runs one wave less.
constexpr int tile_waves(int dim, bool wide, bool lng) {
  return dim == 64 ? 4 - lng : (dim == 128 ? 2 + (wide && !lng) : 1);
}

template <int MODE, int D, bool WIDE, bool LONG>
__global__ __launch_bounds__(kThreads, tile_waves(D, WIDE, LONG)) void kv_tiled_kernel(AttnArgs a) {
  constexpr float kOff = MODE == 2 ? 0.0f : 12.0f, kLag = MODE == 2 ? 8.0f : 3.0f;
  constexpr int QS = D / 16, NT = D / 32;
  using L = TileLds<D>;
  __shared__ __align__(16) L lds;
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c = lane & 31, hh = lane >> 5;
  // from the last place on: late rows see the most keys, so they start first
  const uint32_t place = blockIdx.x / (uint32_t)a.c.heads;
  const int h = (int)(blockIdx.x - place * (uint32_t)a.c.heads);
  Work rt;
  if (!find_work<D, kTileRows>(a, h, gridDim.x / (uint32_t)a.c.heads - 1 - place, rt)) return;
  const int split = (int)rt.split;
  const uint32_t group = (uint32_t)a.group;
  auto hi_of = [&](uint32_t row) {
    const int64_t x = (int64_t)rt.len - rt.n + row / group + 1;
    return (int)(x < 0 ? 0 : x);
  };
  auto lo_of = [&](int hi) { return a.window > 0 && hi > a.window ? hi - a.window : 0; };
  auto end_of = [&](uint32_t row) { return row < rt.rows ? row : rt.rows - 1; };
  const int tlo = lo_of(hi_of(rt.row0)), thi = hi_of(end_of(rt.row0 + kTileRows - 1));
  const uint32_t base0 = (uint32_t)tlo & ~(uint32_t)(kTileKeys - 1);
  const uint32_t blocks =
      a.c.pages > 0 && thi > tlo ? ((uint32_t)thi - base0 + kTileKeys - 1) / kTileKeys : 0;
  const uint32_t per = (blocks + rt.parts - 1) / rt.parts;
  const uint32_t first = split * per;
  const uint32_t end = first + per < blocks ? first + per : blocks;
  if (a.splits > 1) {
    const bool empty = first >= blocks;
    note_parts(a, rt, h, kTileRows, empty, kThreads);
    if (empty) return;
  }
  const uint32_t w0 = rt.row0 + 32 * wave;
  const int whmin = hi_of(end_of(w0)), wlmax = lo_of(hi_of(end_of(w0 + 31)));
  const bool live = w0 + c < rt.rows;
  const uint32_t row = end_of(w0 + c);   // columns past the last row repeat it, unstored
  const int64_t tok = rt.tok0 + row / group;
  const int head = (int)(h * group + row % group);
  const int hi = hi_of(row), lo = lo_of(hi);

  // queries: step s, slot j is channel 16 s + 8 hh + j
  u32x4_t q[QS];
  const ScoreScale sc = score_scale(
      a, load_query<MODE, QS, 16>(a, h, a.q + tok * a.qs + (int64_t)head * D + 8 * hh, q, half_max));

  float m = -__builtin_inff(), l = 0.0f;
  f32x16_t o[NT];
#pragma unroll
  for (int T = 0; T < NT; T++)
#pragma unroll
    for (int r = 0; r < 16; r++) o[T][r] = 0.0f;
  // row c of a key tile is the key that puts 8 consecutive ones into a lane's weights
  const int krow = (c & 16) | ((c & 4) << 1) | ((c & 8) >> 1) | (c & 3);

  constexpr int kAhead = 2;              // operands are read this many products early
  auto key_at = [&](int buf, int i) {
    return *(const u32x4_t*)(lds.k[buf] + (2 * i + hh) * L::KS + krow * 16);
  };
  auto value_at = [&](int buf, int i) {
    return *(const u32x4_t*)(lds.v[buf] + (2 * (i / NT) + hh) * L::VS + (32 * (i % NT) + c) * 16);
  };
  const bool alive = w0 < rt.rows;       // a wave without rows only decodes
  using C = TileCodes<MODE, D>;
  C f;

  // one tile: its scores while the next is decoded, its weights, its values
  auto tile = [&](int buf, uint32_t base, int here) {
    f32x16_t s;
    u32x4_t ring[kAhead];
    static_for<kAhead>([&](auto ii) { ring[decltype(ii)::value] = key_at(buf, decltype(ii)::value); });
#pragma unroll
    for (int r = 0; r < 16; r++) s[r] = 0.0f;
    __builtin_amdgcn_sched_barrier(0);
    // a wave at its products goes before one at its softmax: the matrix unit
    // is refilled at once (chunks 145.5 -> 140 us)
    __builtin_amdgcn_s_setprio(1);
    static_for<QS>([&](auto ii) {
      constexpr int i = decltype(ii)::value, u0 = i * C::UNITS / QS, u1 = (i + 1) * C::UNITS / QS;
      s = mfma32<MODE>(ring[i % kAhead], q[i], s);
      if constexpr (i + kAhead < QS) ring[i % kAhead] = key_at(buf, i + kAhead);
      static_for<u1 - u0>([&](auto kk) { store_unit<u0 + decltype(kk)::value>(f, lds, buf ^ 1); });
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_setprio(0);
    int ok0 = here >= 0, ok1 = ok0;      // of the tile's two runs of 16 tokens
    if constexpr (!WIDE) {
      const int2 v = *(const int2*)lds.ok[buf];
      ok0 = v.x;
      ok1 = v.y;
    }
    static_for<kAhead>([&](auto ii) { ring[decltype(ii)::value] = value_at(buf, decltype(ii)::value); });
    if (LONG || a.cap > 0.0f) cap_scores<LONG>(sc, s);
    if (base < (uint32_t)wlmax || base + kTileKeys > (uint32_t)whmin || !(ok0 & ok1)) {
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int key = (int)base + 16 * (r >> 3) + 8 * hh + (r & 7);
        s[r] = !(r < 8 ? ok0 : ok1) || key < lo || key >= hi ? -__builtin_inff() : s[r];
      }
    }
    float mx = s[0];
#pragma unroll
    for (int r = 1; r < 16; r++) mx = fmaxf(mx, s[r]);
    mx = fmaxf(m, __builtin_fmaf(half_max(mx), sc.f, sc.off));
    if (__any(mx > m + kLag)) {
      const float fac = mx > m ? __builtin_amdgcn_exp2f(m - mx) : 1.0f;
      l *= fac;
#pragma unroll
      for (int T = 0; T < NT; T++)
#pragma unroll
        for (int r = 0; r < 16; r++) o[T][r] *= fac;
      m = mx;
    }
    float ref = (m == -__builtin_inff() ? 0.0f : m) - kOff - sc.off;
    if (fabsf(ref) > kFarMax) {
      far_scores(sc, m, s);
      ref = -kOff;
    }
    // weights two at a time (pair j); a pair's arguments, exponentials and sum
    // are taken in three successive places
    u32x4_t p[2];
    float x0, x1, e0 = 0.0f, e1 = 0.0f;
    auto args = [&](auto jj) {
      constexpr int r = 2 * decltype(jj)::value;
      x0 = __builtin_fmaf(s[r], sc.f, -ref);
      x1 = __builtin_fmaf(s[r + 1], sc.f, -ref);
    };
    auto pack = [&](auto jj) {
      constexpr int j = decltype(jj)::value;
      l += e0;
      l += e1;
      uint32_t w;
      if constexpr (MODE == 2) w = bf16x2_of(e0, e1);
      else w = bits_of(f16x2_t{(_Float16)e0, (_Float16)e1});
      p[j >> 2][j & 3] = w;
    };
    auto weight = [&](auto jj) {
      constexpr int j = decltype(jj)::value;
      if constexpr (j % 4 > 0) pack(std::integral_constant<int, j - 1>{});
      e0 = __builtin_amdgcn_exp2f(x0);
      e1 = __builtin_amdgcn_exp2f(x1);
      if constexpr (j % 4 < 3) args(std::integral_constant<int, j + 1>{});
    };
    args(std::integral_constant<int, 0>{});
    static_for<4>(weight);
    pack(std::integral_constant<int, 3>{});
    args(std::integral_constant<int, 4>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    static_for<2 * NT>([&](auto ii) {
      constexpr int i = decltype(ii)::value, j0 = i * 4 / NT, j1 = (i + 1) * 4 / NT;
      o[i % NT] = mfma32<MODE>(ring[i % kAhead], p[i / NT], o[i % NT]);
      if constexpr (i + kAhead < 2 * NT) ring[i % kAhead] = value_at(buf, i + kAhead);
      if constexpr (i < NT) {
        static_for<j1 - j0>([&](auto kk) { weight(std::integral_constant<int, 4 + j0 + decltype(kk)::value>{}); });
        if constexpr (i == NT - 1) pack(std::integral_constant<int, 7>{});
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_setprio(0);
  };

  // Tiles past the end are decoded too (from page 0 where there is none), which
  // keeps the loop free of cases; nothing uses them.
  if (first < end) {
    const uint32_t count = end - first;
    const PageRow pages(a, rt.b);
    auto base_of = [&](uint32_t i) { return base0 + (first + i) * kTileKeys; };
    auto key_page = [&](uint32_t i) {
      return pages.at(base_of(i) + (WIDE ? 0 : threadIdx.x >> 3));
    };
    auto value_page = [&](uint32_t i) {
      return pages.at(base_of(i) + threadIdx.x % C::TG * C::TOK);
    };
    auto load = [&](uint32_t i, int kp, int vp) {
      load_tile<MODE, D, WIDE>(a, h, base_of(i), kp, vp, f);
    };
    auto ready = [&](uint32_t i) {       // what the decode of tile i needs once
      clean_scales(f, base_of(i), tlo, thi);
      if constexpr (!WIDE)
        if (lane == 0) lds.ok[i & 1][wave >> 1] = f.kpage >= 0;  // 8 keys a wave
    };
    auto store_all = [&](int buf) {
      static_for<C::UNITS>([&](auto u) { store_unit<decltype(u)::value>(f, lds, buf); });
    };
    int kp = key_page(0), vp = WIDE ? kp : value_page(0);
    load(0, kp, vp);
    const int first_page = kp;
    kp = key_page(1), vp = WIDE ? kp : value_page(1);
    ready(0);
    store_all(0);
    load(1, kp, vp);
    int here = first_page;
    for (uint32_t i = 0; i < count; i++) {
      const int buf = (int)i & 1, next = f.kpage;
      kp = key_page(i + 2);
      vp = WIDE ? kp : value_page(i + 2);
      __syncthreads();                   // tile i is decoded, the other buffer free
      ready(i + 1);
      if (alive) tile(buf, base_of(i), here);
      else store_all(buf ^ 1);
      here = next;
      load(i + 2, kp, vp);
    }
  }

  l = half_sum(l);
  if (!live) return;
  const float va = MODE == 2 ? 1.0f : a.c.vam[h] / (6.0f * (MODE == 1 ? 256.0f : 448.0f));
  const float inv = l == 0.0f ? 0.0f : va / l;
  const int64_t at = ((int64_t)split * a.tokens + tok) * a.hq + head;
#pragma unroll
  for (int T = 0; T < NT / 2; T++)
#pragma unroll
    for (int rg = 0; rg < 4; rg++) {
      const int ch = 2 * (32 * T + 8 * rg + 4 * hh);
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        x[2 * e] = o[T][4 * rg + e];
        x[2 * e + 1] = o[T + NT / 2][4 * rg + e];
      }
      if (a.splits > 1) {
        float4* y = (float4*)(a.po + at * D + ch);
        y[0] = make_float4(x[0], x[1], x[2], x[3]);
        y[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] *= inv;
        *(uint4*)(a.out + tok * a.os + (int64_t)head * D + ch) = pack8(x);
      }
    }
  if (hh == 0) {
    if (a.splits > 1) {
      *(float2*)(a.pm + at * 2) = make_float2(m, l);
    } else if (a.lse) {
      a.lse[tok * a.hq + head] =
          l == 0.0f ? -__builtin_inff() : __builtin_fmaf(m - kOff, kLn2, logf(l));
    }
  }
}

}  // namespace fp4q
