// kv_tiled_kernels.h -- attention over the paged FP4 cache for many query
// rows per kv head (prompts, chunks): the mathematics of
// kv_attention_kernels.h, with the decoded keys and values of 64 tokens
// shared through LDS.
//
// A workgroup of 4 waves takes 128 rows, 32 a wave (one column tile of the
// 32x32x16 products).  Decoding a value costs about 1.3 vector instructions
// and a row's softmax about 4 per key, so 128 rows per decoded value keep
// the decode under a tenth of the softmax.  LDS holds two tiles; while one is
// computed the next is decoded from registers into the other and the codes
// after that are on their way from memory, with one barrier per 64 keys.
//
// LDS layout: 16-byte chunks, column after column, so that a wave's operand
// reads are contiguous.  Keys: chunk (channels 8 x .. 8 x + 7, key).  Values:
// chunk (tokens 8 y .. 8 y + 7, channel), even channels before odd ones.  The
// padding of a column (16 and 32 bytes) spreads the decoding lanes' stores
// over all banks.
#pragma once

#include "kv_attention_kernels.h"

namespace fp4q {

constexpr int kTileRows = 128;           // query rows of a workgroup

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

// The codes of a thread's part of 64 tokens: D/4 channels of one key, and
// TOK tokens of ROWS channel pairs.
template <int MODE, int D>
struct TileCodes {
  static constexpr int G = MODE == 2 ? 32 : 16;
  static constexpr int KW = D / 32;                  // dwords of the key
  static constexpr int TOK = D == 64 ? 8 : 16, TG = 64 / TOK;
  static constexpr int ROWS = D / 2 * TG / kThreads;
  static constexpr int VW = TOK / 4;                 // dwords of a channel pair
  uint32_t k[KW], ks;
  uint32_t v[ROWS][VW], vs[ROWS][VW];
  int kpage, vpage;
};

template <int MODE, int D, bool WIDE>
__device__ __forceinline__ KvPages tile_pages(const AttnArgs& a, uint32_t b, int64_t base) {
  using C = TileCodes<MODE, D>;
  const int t = (int)threadIdx.x;
  KvPages p;
  p.k = page_id(a, b, WIDE ? base : base + (t >> 2));
  p.v = WIDE ? p.k : page_id(a, b, base + (t % C::TG) * C::TOK);
  return p;
}

template <int MODE, int D, bool WIDE>
__device__ __forceinline__ void load_tile(const AttnArgs& a, int h, int64_t base, KvPages pg,
                                          TileCodes<MODE, D>& f) {
  using C = TileCodes<MODE, D>;
  constexpr int G = C::G, KB = C::KW * 4 > 16 ? 16 : C::KW * 4, VB = C::VW * 4;
  constexpr int SB = D / 4 >= G ? D / 4 / G : 1;
  const int t = (int)threadIdx.x, P = 1 << a.c.page_shift, part = t & 3;
  f.kpage = pg.k;
  f.vpage = pg.v;
  const int64_t pk = (int64_t)(pg.k < 0 ? 0 : pg.k) * a.c.heads + h;
  const int64_t pv = (int64_t)(pg.v < 0 ? 0 : pg.v) * a.c.heads + h;
  // token of the page (the same for the wave when WIDE), and the lane's offset from it
  const int64_t at = pk * P + (int)((WIDE ? base : base + (t >> 2)) & (P - 1));
  const uint32_t row = WIDE ? t >> 2 : 0;
  const uint8_t* kc = a.c.kc + at * (D / 2);
#pragma unroll
  for (int i = 0; i < C::KW; i += KB / 4) {
    const auto w = KvLoad<KB, WIDE>::at(kc, row * (D / 2) + part * (D / 8) + i * 4, 0);
#pragma unroll
    for (int e = 0; e < KB / 4; e++) f.k[i + e] = w[e];
  }
  f.ks = KvLoad<SB, WIDE>::at(a.c.ks + at * (D / G), row * (D / G) + part * (D / 4) / G, 0)[0];
  const int tok = (t % C::TG) * C::TOK, av = (int)((WIDE ? base : base + tok) & (P - 1));
  const uint8_t* vc = a.c.vc + pv * (D / 2) * P + av;
  const uint8_t* vs = a.c.vs + pv * (D / G) * P + av;
#pragma unroll
  for (int r = 0; r < C::ROWS; r++) {
    const uint32_t i = t / C::TG + r * (kThreads / C::TG), off = WIDE ? tok : 0;
    const auto w = KvLoad<VB, WIDE>::at(vc, (i << a.c.page_shift) + off, 0);
    const auto s = KvLoad<VB, WIDE>::at(vs, ((2 * i / G) << a.c.page_shift) + off, 0);
#pragma unroll
    for (int e = 0; e < C::VW; e++) {
      f.v[r][e] = w[e];
      f.vs[r][e] = s[e];
    }
  }
}

template <int D>
struct TileLds {
  static constexpr int KS = 64 * 16 + 16, VS = D * 16 + 32;      // bytes of a column
  static constexpr int K = D / 8 * KS, V = 8 * VS;
  uint8_t k[2][K], v[2][V];
  int ok[2][4];                          // the page of each 16 tokens is in the cache
};

// Decode into LDS; tokens outside [lo, hi) or without a page become zeros.
template <int MODE, int D>
__device__ __forceinline__ void store_tile(const TileCodes<MODE, D>& f, int64_t base, int lo, int hi,
                                           TileLds<D>& lds, int buf) {
  using C = TileCodes<MODE, D>;
  using L = TileLds<D>;
  const int t = (int)threadIdx.x, part = t & 3, key = t >> 2;
  static_for<C::KW>([&](auto dd) {
    constexpr int d = decltype(dd)::value;
    const u32x4_t w = key_operand<MODE, d * 8 / C::G>(f.k[d], f.ks);
    *(u32x4_t*)(lds.k[buf] + (part * C::KW + d) * L::KS + key * 16) = w;
  });
  if ((t & 63) == 0) lds.ok[buf][t >> 6] = f.kpage >= 0;
  const int tok = (t % C::TG) * C::TOK;
  uint32_t keep[C::VW];
#pragma unroll
  for (int w = 0; w < C::VW; w++) keep[w] = ~0u;
  if (base < lo || base + 64 > hi || !__all(f.vpage >= 0)) {
#pragma unroll
    for (int w = 0; w < C::VW; w++) {
      keep[w] = 0;
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int j = (int)base + tok + 4 * w + r;
        if (f.vpage >= 0 && j >= lo && j < hi) keep[w] |= 255u << (8 * r);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < C::ROWS; r++) {
    const int i = t / C::TG + r * (kThreads / C::TG);
#pragma unroll
    for (int y = 0; y < C::TOK / 8; y++) {
      u32x4_t even, odd;
      value_operands<MODE>(f.v[r][2 * y], f.v[r][2 * y + 1], f.vs[r][2 * y] & keep[2 * y],
                           f.vs[r][2 * y + 1] & keep[2 * y + 1], even, odd);
      uint8_t* o = lds.v[buf] + (tok / 8 + y) * L::VS + i * 16;
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

template <int MODE, int D, bool WIDE>
__global__ __launch_bounds__(kThreads, D < 256 ? 2 : 1) void kv_tiled_kernel(AttnArgs a) {
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
  if (!find_work<kTileRows>(a, gridDim.x / (uint32_t)a.c.heads - 1 - place, rt)) return;
  const int split = (int)rt.split;
  const uint32_t group = (uint32_t)a.group;
  auto hi_of = [&](uint32_t row) {
    const int64_t x = (int64_t)rt.len - rt.n + row / group + 1;
    return (int)(x < 0 ? 0 : x);
  };
  auto lo_of = [&](int hi) { return a.window > 0 && hi > a.window ? hi - a.window : 0; };
  auto end_of = [&](uint32_t row) { return row < rt.rows ? row : rt.rows - 1; };
  const int tlo = lo_of(hi_of(rt.row0)), thi = hi_of(end_of(rt.row0 + kTileRows - 1));
  const int64_t base0 = tlo & ~(kAttnKeys - 1);
  const uint32_t blocks =
      a.c.pages > 0 && thi > tlo ? ((uint32_t)(thi - base0) + kAttnKeys - 1) / kAttnKeys : 0;
  const uint32_t per = (blocks + rt.parts - 1) / rt.parts;
  const uint32_t first = split * per;
  const uint32_t end = first + per < blocks ? first + per : blocks;
  if (a.splits > 1) {
    const bool empty = first >= blocks;
    note_parts(a, rt, h, kTileRows, empty, kThreads);
    if (empty) return;
  }
  const uint32_t w0 = rt.row0 + 32 * wave;
  const bool alive = w0 < rt.rows;
  const int whmin = hi_of(end_of(w0)), whmax = alive ? hi_of(end_of(w0 + 31)) : 0;
  const int wlmin = lo_of(whmin), wlmax = lo_of(whmax);
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

  auto compute = [&](int buf, int64_t base) {
    // operands are read kAhead products early; the two key tiles alternate, so
    // that a product never waits for the one before it
    constexpr int kAhead = 4;
    f32x16_t s[2];
#pragma unroll
    for (int kt = 0; kt < 2; kt++)
#pragma unroll
      for (int r = 0; r < 16; r++) s[kt][r] = 0.0f;
    auto key_at = [&](int i) {
      return *(const u32x4_t*)(lds.k[buf] + (i & ~1) * L::KS + hh * L::KS + (32 * (i & 1) + krow) * 16);
    };
    u32x4_t ring[kAhead];
    static_for<kAhead>([&](auto ii) { ring[decltype(ii)::value] = key_at(decltype(ii)::value); });
    __builtin_amdgcn_sched_barrier(0);
    static_for<2 * QS>([&](auto ii) {
      constexpr int i = decltype(ii)::value;
      s[i & 1] = mfma32<MODE>(ring[i % kAhead], q[i >> 1], s[i & 1]);
      if constexpr (i + kAhead < 2 * QS) ring[i % kAhead] = key_at(i + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    });
    auto value_at = [&](int i) {
      return *(const u32x4_t*)(lds.v[buf] + (2 * (i / NT) + hh) * L::VS + (32 * (i % NT) + c) * 16);
    };
    static_for<kAhead>([&](auto ii) { ring[decltype(ii)::value] = value_at(decltype(ii)::value); });
    if (a.cap > 0.0f) {
#pragma unroll
      for (int kt = 0; kt < 2; kt++)
#pragma unroll
        for (int r = 0; r < 16; r++) s[kt][r] = capped(s[kt][r], sc.in);
    }
    const int4 ok = *(const int4*)lds.ok[buf];
    if (base < wlmax || base + 64 > whmin || !(ok.x & ok.y & ok.z & ok.w)) {
      const int oks[4] = {ok.x, ok.y, ok.z, ok.w};
#pragma unroll
      for (int kt = 0; kt < 2; kt++)
#pragma unroll
        for (int r = 0; r < 16; r++) {
          const int key = (int)base + 32 * kt + 16 * (r >> 3) + 8 * hh + (r & 7);
          s[kt][r] = !oks[2 * kt + (r >> 3)] || key < lo || key >= hi ? -__builtin_inff() : s[kt][r];
        }
    }
    float mx = s[0][0];
#pragma unroll
    for (int kt = 0; kt < 2; kt++)
#pragma unroll
      for (int r = 0; r < 16; r++) mx = fmaxf(mx, s[kt][r]);
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
    const float ref = (m == -__builtin_inff() ? 0.0f : m) - kOff - sc.off;
    u32x4_t p[4];
#pragma unroll
    for (int kt = 0; kt < 2; kt++)
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][r], sc.f, -ref));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][r + 1], sc.f, -ref));
        l += e0;
        l += e1;
        uint32_t w;
        if constexpr (MODE == 2) w = bf16x2_of(e0, e1);
        else w = bits_of(f16x2_t{(_Float16)e0, (_Float16)e1});
        p[2 * kt + (r >> 3)][(r & 7) >> 1] = w;
      }
    __builtin_amdgcn_sched_barrier(0);
    static_for<4 * NT>([&](auto ii) {
      constexpr int i = decltype(ii)::value;
      o[i % NT] = mfma32<MODE>(ring[i % kAhead], p[i / NT], o[i % NT]);
      if constexpr (i + kAhead < 4 * NT) ring[i % kAhead] = value_at(i + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  if (first < end) {
    auto base_of = [&](uint32_t i) { return base0 + (int64_t)i * kAttnKeys; };
    TileCodes<MODE, D> f;
    KvPages pg = tile_pages<MODE, D, WIDE>(a, rt.b, base_of(first));
    load_tile<MODE, D, WIDE>(a, h, base_of(first), pg, f);
    pg = tile_pages<MODE, D, WIDE>(a, rt.b, base_of(first + 1));
    store_tile<MODE, D>(f, base_of(first), tlo, thi, lds, 0);
    if (first + 1 < end) load_tile<MODE, D, WIDE>(a, h, base_of(first + 1), pg, f);
    pg = tile_pages<MODE, D, WIDE>(a, rt.b, base_of(first + 2));
    for (uint32_t i = first; i < end; i++) {
      const int buf = (int)(i - first) & 1;
      __syncthreads();                   // tile i is decoded; the other buffer is free
      if (i + 1 < end) {
        store_tile<MODE, D>(f, base_of(i + 1), tlo, thi, lds, buf ^ 1);
        if (i + 2 < end) {
          const KvPages next = tile_pages<MODE, D, WIDE>(a, rt.b, base_of(i + 3));
          load_tile<MODE, D, WIDE>(a, h, base_of(i + 2), pg, f);
          pg = next;
        }
      }
      const int64_t base = base_of(i);
      if (base < whmax && base + kAttnKeys > wlmin) compute(buf, base);
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
