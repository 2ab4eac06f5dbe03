// kv_attention_kernels.h -- attention of new tokens over the paged FP4 cache.
//
// Token i of a sequence's n new ones stands at position pos = len - n + i
// and sees the cached tokens j <= pos (with a window W also j > pos - W):
//   s_j = scale q . K_j,  s_j <- cap tanh(s_j / cap) with a cap,
//   p = softmax(s),  out = sum p_j V_j,  lse = log sum exp(s_j)
// K and V are the decoded values of the cache.  A token that sees nothing
// gets out = 0 and lse = -inf.
//
// One pass over the keys with a running maximum m and sum l (in powers of
// two: s is scaled by log2 e), so a row's weights are exp2(s_j - m) and its
// output the weighted sum over l.  The query rows of one kv head (tokens x
// the heads that share it) form the columns of both matrix products,
//   S^T = K Q^T   (rows: keys)      O^T = V^T P^T   (rows: channels)
// so a lane owns one query column throughout: its maximum, sum and rescaling
// are lane scalars, and the weights leave the first product in the lane
// that feeds them to the second.
//
// Operands.  NVFP4 values are E2M1 x E4M3 (at most 6 significant bits, from
// 2^-10 to 2688), exact in fp16; the head's alpha and the scale of the
// scores go to one factor per column.  Queries become fp16 after a power of
// two per row that puts their largest magnitude at 2^14, exact down to 2^-28
// of it.  MXFP4 values are E2M1 x 2^k, exact in bf16, as the queries are.
// The weights are rounded to the operand's type, to half a step of 2^-10
// (fp16) or 2^-7 (bf16) of each: the sum over the row uses the unrounded
// ones, and the accumulators are fp32.  fp16 weights carry a factor 2^12,
// so that only those under 2^-26 of the largest lose bits.
#pragma once

#include "kv_common.h"

namespace fp4q {

struct AttnArgs {
  KvView c;
  const uint16_t* q;
  const int32_t *pt, *lens, *cu;
  uint16_t* out;
  float* lse;                            // [tokens][hq] or NULL
  float *po, *pm;                        // partials [splits][tokens][hq][D], [..][2] (max, sum)
  int64_t qs, os;                        // elements between tokens
  int64_t tokens, seqs, width;
  int hq, group, window, splits;
  float scale, cap;                      // cap 0: none
};

constexpr int kAttnKeys = 64;            // keys per step of a wave
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// MODE: 0 NVFP4, 1 NVFP4 with 4/6, 2 MXFP4.
template <int MODE>
__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (MODE == 2)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <int BYTE>
__device__ __forceinline__ f16x2_t fp4x2_f16(uint32_t w) {
  return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, BYTE));
}
template <int BYTE>
__device__ __forceinline__ uint32_t fp4x2_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, BYTE));
}
// E4M3 scale bytes 2 HI and 2 HI + 1 of w as fp16 (exact; the sign bit of a scale is not read).
template <bool HI>
__device__ __forceinline__ f16x2_t e4m3x2_f16(uint32_t w) {
  return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HI));
}
__device__ __forceinline__ uint32_t bits_of(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }

// Codes of four tokens x two channels (one byte a token: channel 2i low,
// 2i + 1 high) to a channel's tokens in pairs: bytes 0 and 2 of `even` and
// `odd` hold (token 0, 1) and (token 2, 3).
__device__ __forceinline__ void channel_pairs(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t t = w >> 4, u = w >> 8;
  even = (w & 0x000F000Fu) | (t & ~0x000F000Fu);
  odd = (t & 0x000F000Fu) | (u & ~0x000F000Fu);
}

// Reductions over the four lanes that share a column (lane, lane ^ 16, ^ 32, ^ 48).
__device__ __forceinline__ float col_max(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float col_sum(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A tile of query rows: rows row0 .. row0 + M - 1 of sequence b, row r being
// token r / group with head r % group of the kv head's own.
struct RowTile {
  int64_t b, tok0;                       // the sequence's first token
  int64_t row0, rows;                    // rows of the whole sequence
  int64_t len, n;
};

__device__ __forceinline__ int64_t cu_at(const AttnArgs& a, int64_t b) {
  const int64_t v = a.cu[b];
  return v < 0 ? 0 : (v > a.tokens ? a.tokens : v);
}

// Tile `t` of the grid.  Sequence b's tiles start at floor(cu[b] group / M) + b,
// which leaves room for every sequence's ceil(n group / M) whatever the n, so
// the grid needs no sizes from the device; ids between have no rows.  The
// search takes 64 boundaries at a time, one a lane.
__device__ __forceinline__ bool row_tile(const AttnArgs& a, int64_t t, int M, RowTile& r) {
  int64_t first = t;
  if (a.cu) {
    int64_t lo = 0, n = a.seqs;          // the answer is in [lo, lo + n)
    while (n > 1) {
      const int64_t step = (n + 63) / 64;
      const int64_t at = lo + step * (int64_t)(threadIdx.x & 63);
      const bool below = at < lo + n && cu_at(a, at) * a.group / M + at <= t;
      const int64_t k = __popcll(__ballot(below)) - 1;   // monotone: a prefix of the lanes
      const int64_t end = lo + n;
      lo += step * (k < 0 ? 0 : k);
      n = end - lo < step ? end - lo : step;
    }
    r.b = lo;
    r.tok0 = cu_at(a, lo);
    const int64_t next = cu_at(a, lo + 1);
    r.n = next > r.tok0 ? next - r.tok0 : 0;
    first = r.tok0 * a.group / M + lo;
  } else {
    const int64_t per = (a.group + M - 1) / M;
    r.b = t / per;
    first = r.b * per;
    if (r.b >= a.seqs) return false;
    r.tok0 = r.b;
    r.n = 1;
  }
  r.rows = r.n * a.group;
  r.row0 = (t - first) * M;
  if (r.row0 < 0 || r.row0 >= r.rows) return false;
  r.len = a.lens[r.b];
  const int64_t most = a.width << a.c.page_shift;
  if (r.len > most) r.len = most;
  return true;
}

// One wave's share of 64 cached tokens: lane (c = lane & 15, g = lane >> 4)
// holds of keys 16 (c / 4) + 4 t + c % 4, t = 0..3, the channels D/4 g ..
// D/4 g + D/4 - 1, and of values the tokens 16 g .. 16 g + 15 of channel
// pairs 16 T + c.  The row order of the keys is what makes a lane's weights
// of the first product those of 16 consecutive tokens.
template <int MODE, int D>
struct KvFragment {
  static constexpr int G = MODE == 2 ? 32 : 16;
  static constexpr int KD = D / 32;                  // dwords of a key; pieces of the values
  uint32_t k[4][KD], ks[4];
  u32x4_t v[KD], vs[KD];
};

struct KvPages {
  int k, v;                              // page ids, -1 outside the cache or the table
};

__device__ __forceinline__ int page_id(const AttnArgs& a, int64_t b, int64_t key) {
  const int64_t i = key >> a.c.page_shift;
  if (i >= a.width) return -1;
  const int p = a.pt[b * a.width + i];
  return p >= 0 && p < a.c.pages ? p : -1;
}

__device__ __forceinline__ KvPages load_pages(const AttnArgs& a, int64_t b, int64_t base) {
  const int lane = (int)threadIdx.x & 63;
  KvPages p;
  p.k = page_id(a, b, base + 16 * ((lane & 15) >> 2));
  p.v = page_id(a, b, base + 16 * (lane >> 4));
  return p;
}

template <int MODE, int D>
__device__ __forceinline__ void load_kv(const AttnArgs& a, int h, int64_t base, KvPages pg,
                                        KvFragment<MODE, D>& f) {
  constexpr int G = KvFragment<MODE, D>::G, KD = D / 32;
  const int lane = (int)threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int P = 1 << a.c.page_shift;
  const int64_t pk = (int64_t)(pg.k < 0 ? 0 : pg.k) * a.c.heads + h;
  const int64_t pv = (int64_t)(pg.v < 0 ? 0 : pg.v) * a.c.heads + h;
  const int ak = (int)((base + 16 * (c >> 2)) & (P - 1)) + (c & 3);
  const int av = (int)((base + 16 * g) & (P - 1));
  const uint8_t* kc = a.c.kc + (pk * P + ak) * (D / 2) + g * (D / 8);
  constexpr int SB = D / 4 >= G ? D / 4 / G : 1;     // scale bytes of a lane's channels
  const uint8_t* ks = a.c.ks + (pk * P + ak) * (D / G) + g * (D / 4) / G;
#pragma unroll
  for (int t = 0; t < 4; t++) {
    if constexpr (KD == 2) {
      const u32x2_t w = *(const u32x2_t*)(kc + t * 4 * (D / 2));
      f.k[t][0] = w[0];
      f.k[t][1] = w[1];
    } else {
#pragma unroll
      for (int i = 0; i < KD; i += 4) {
        const u32x4_t w = *(const u32x4_t*)(kc + t * 4 * (D / 2) + i * 4);
#pragma unroll
        for (int e = 0; e < 4; e++) f.k[t][i + e] = w[e];
      }
    }
    const uint8_t* s = ks + t * 4 * (D / G);
    if constexpr (SB == 4) f.ks[t] = *(const uint32_t*)s;
    else if constexpr (SB == 2) f.ks[t] = *(const uint16_t*)s;
    else f.ks[t] = *s;
  }
  const uint8_t* vc = a.c.vc + (pv * (D / 2) + c) * P + av;
  const uint8_t* vs = a.c.vs + pv * (D / G) * P + av;
#pragma unroll
  for (int T = 0; T < KD; T++) {
    f.v[T] = *(const u32x4_t*)(vc + (int64_t)T * 16 * P);
    const int sg = MODE == 2 ? T : 2 * T + (c >> 3);
    f.vs[T] = *(const u32x4_t*)(vs + (int64_t)sg * P);
  }
}

// A operand of key rows: 8 channels of code dword `w` and the lane's scale.
// IDX: position of the dword's scale among the lane's scale bytes.
template <int MODE, int IDX>
__device__ __forceinline__ u32x4_t key_operand(uint32_t w, uint32_t ks) {
  u32x4_t r;
  if constexpr (MODE == 2) {
    const float s = __uint_as_float(((ks >> (8 * IDX)) & 255u) << 23);
    r[0] = fp4x2_bf16<0>(w, s);
    r[1] = fp4x2_bf16<1>(w, s);
    r[2] = fp4x2_bf16<2>(w, s);
    r[3] = fp4x2_bf16<3>(w, s);
  } else {
    const f16x2_t p = e4m3x2_f16<(IDX >= 2)>(ks);
    const f16x2_t s = {p[IDX & 1], p[IDX & 1]};
    r[0] = bits_of(fp4x2_f16<0>(w) * s);
    r[1] = bits_of(fp4x2_f16<1>(w) * s);
    r[2] = bits_of(fp4x2_f16<2>(w) * s);
    r[3] = bits_of(fp4x2_f16<3>(w) * s);
  }
  return r;
}

// A operands of the even and odd channels of a piece of the values: the
// tokens of dwords w0, w1 with their scale bytes s0, s1.
template <int MODE>
__device__ __forceinline__ void value_operands(uint32_t w0, uint32_t w1, uint32_t s0, uint32_t s1,
                                               u32x4_t& even, u32x4_t& odd) {
  if constexpr (MODE == 2) {
    uint32_t x[8];
    auto four = [&](uint32_t w, uint32_t s, uint32_t* o) {
      o[0] = fp4x2_bf16<0>(w, __uint_as_float((s & 255u) << 23));
      o[1] = fp4x2_bf16<1>(w, __uint_as_float(((s >> 8) & 255u) << 23));
      o[2] = fp4x2_bf16<2>(w, __uint_as_float(((s >> 16) & 255u) << 23));
      o[3] = fp4x2_bf16<3>(w, __uint_as_float((s >> 24) << 23));
    };
    four(w0, s0, x);
    four(w1, s1, x + 4);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      even[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100u);
      odd[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
    }
  } else {
    uint32_t e0, o0, e1, o1;
    channel_pairs(w0, e0, o0);
    channel_pairs(w1, e1, o1);
    const f16x2_t a0 = e4m3x2_f16<false>(s0), a1 = e4m3x2_f16<true>(s0);
    const f16x2_t a2 = e4m3x2_f16<false>(s1), a3 = e4m3x2_f16<true>(s1);
    even[0] = bits_of(fp4x2_f16<0>(e0) * a0);
    even[1] = bits_of(fp4x2_f16<2>(e0) * a1);
    even[2] = bits_of(fp4x2_f16<0>(e1) * a2);
    even[3] = bits_of(fp4x2_f16<2>(e1) * a3);
    odd[0] = bits_of(fp4x2_f16<0>(o0) * a0);
    odd[1] = bits_of(fp4x2_f16<2>(o0) * a1);
    odd[2] = bits_of(fp4x2_f16<0>(o1) * a2);
    odd[3] = bits_of(fp4x2_f16<2>(o1) * a3);
  }
}

// Queries of one column as B operands: step s, slot j is channel D/4 g + 8 s + j.
// Returns the factor that turns the products into scores in powers of two.
template <int MODE, int D>
__device__ __forceinline__ float load_query(const AttnArgs& a, int h, const uint16_t* q, bool live,
                                            u32x4_t (&o)[D / 32]) {
  const int g = ((int)threadIdx.x & 63) >> 4;
  const float k = fabsf(a.scale) * kLog2e;
  if (a.scale == 0.0f) live = false;                 // every score is 0
  float y[D / 4];
#pragma unroll
  for (int s = 0; s < D / 32; s++) {
    const uint4 w = live ? *(const uint4*)(q + g * (D / 4) + s * 8) : make_uint4(0, 0, 0, 0);
    unpack8(w, y + 8 * s);
  }
  if (a.scale < 0.0f) {
#pragma unroll
    for (int i = 0; i < D / 4; i++) y[i] = -y[i];
  }
  if constexpr (MODE == 2) {
#pragma unroll
    for (int s = 0; s < D / 32; s++) {
      const uint4 w = pack8(y + 8 * s);
      o[s] = u32x4_t{w.x, w.y, w.z, w.w};
    }
    return fmaxf(k, 0x1p-126f);
  } else {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 4; i++) m = fmaxf(m, fabsf(y[i]));
    m = col_max(m);
    int shift = 141 - (int)(__float_as_uint(m) >> 23);           // 2^14 <= m 2^shift < 2^15
    shift = shift > 127 ? 127 : shift;
#pragma unroll
    for (int s = 0; s < D / 32; s++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float x0 = __builtin_ldexpf(y[8 * s + 2 * i], shift);
        const float x1 = __builtin_ldexpf(y[8 * s + 2 * i + 1], shift);
        o[s][i] = bits_of(f16x2_t{(_Float16)x0, (_Float16)x1});
      }
    const float alpha = a.c.kam[h] / (6.0f * (MODE == 1 ? 256.0f : 448.0f));
    return fmaxf(__builtin_ldexpf(k * alpha, -shift), 0x1p-126f);
  }
}

// c tanh(s / c) of a score in powers of two: tanh y = 1 - 2 / (exp(2 y) + 1).
__device__ __forceinline__ float capped(float s, float in, float out) {
  const float e = __builtin_amdgcn_exp2f(s * in);    // in = 2 / c (s is in powers of two)
  return out - 2.0f * out * __builtin_amdgcn_rcpf(e + 1.0f);
}

// NT columns of 16 query rows, WAVES waves that take the blocks of 64 keys of
// the workgroup's part of the context in turn and join their sums at the end.
template <int MODE, int D, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D < 256 && NT == 1 ? 2 : 1) void kv_attention_kernel(AttnArgs a) {
  constexpr int KD = D / 32, M = 16 * NT;
  constexpr float kOff = MODE == 2 ? 0.0f : 12.0f;   // weights carry 2^kOff
  __shared__ float so[WAVES][16][D + 4];
  __shared__ float sm[WAVES][16][2];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  uint32_t id = blockIdx.x;
  const int h = (int)(id % (uint32_t)a.c.heads);
  id /= (uint32_t)a.c.heads;
  const int split = (int)(id % (uint32_t)a.splits);
  RowTile rt;
  if (!row_tile(a, id / (uint32_t)a.splits, M, rt)) return;
  // reach of the tile's rows: [lo, hi) of each column, and of all together
  const int64_t last = rt.row0 + M < rt.rows ? rt.row0 + M - 1 : rt.rows - 1;
  auto hi_of = [&](int64_t row) {
    const int64_t x = rt.len - rt.n + row / a.group + 1;
    return (int)(x < 0 ? 0 : x);
  };
  auto lo_of = [&](int hi) { return a.window > 0 && hi > a.window ? hi - a.window : 0; };
  const int hmin = hi_of(rt.row0), hmax = hi_of(last);
  const int lmin = lo_of(hmin), lmax = lo_of(hmax);
  int hi[NT], lo[NT];
  int64_t tok[NT];
  int head[NT];
  u32x4_t q[NT][KD];
  float qf[NT], m[NT], l[NT];
  f32x4_t o[NT][KD][2];
#pragma unroll
  for (int i = 0; i < NT; i++) {
    const int64_t row = rt.row0 + 16 * i + c;
    const bool live = row < rt.rows;
    tok[i] = live ? rt.tok0 + row / a.group : -1;
    head[i] = h * a.group + (int)(row % a.group);
    hi[i] = live ? hi_of(row) : 0;
    lo[i] = lo_of(hi[i]);
    qf[i] = load_query<MODE, D>(a, h, a.q + tok[i] * a.qs + (int64_t)head[i] * D, live, q[i]);
    m[i] = -__builtin_inff();
    l[i] = 0.0f;
#pragma unroll
    for (int T = 0; T < KD; T++) o[i][T][0] = o[i][T][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int64_t base0 = lmin & ~(kAttnKeys - 1);
  const int64_t blocks = a.c.pages > 0 && hmax > lmin ? (hmax - base0 + kAttnKeys - 1) / kAttnKeys : 0;
  const int64_t per = (blocks + a.splits - 1) / a.splits;
  const int64_t end = (split + 1) * per < blocks ? (split + 1) * per : blocks;
  int64_t blk = split * per + wave;

  const float cap_in = a.cap > 0.0f ? 2.0f / a.cap : 0.0f, cap_out = a.cap * kLog2e;
  auto step = [&](const KvFragment<MODE, D>& f, int64_t base, KvPages pg) {
    f32x4_t s[NT][4];
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
      for (int t = 0; t < 4; t++) s[i][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    static_for<4>([&](auto tt) {
      constexpr int t = decltype(tt)::value;
      static_for<KD>([&](auto ss) {
        constexpr int st = decltype(ss)::value;
        const u32x4_t k = key_operand<MODE, st * 8 / KvFragment<MODE, D>::G>(f.k[t][st], f.ks[t]);
#pragma unroll
        for (int i = 0; i < NT; i++) s[i][t] = mfma16<MODE>(k, q[i][st], s[i][t]);
      });
    });
    const bool whole = base >= lmax && base + kAttnKeys <= hmin && __all(pg.v >= 0);
    uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};         // bytes of the tokens that count
    if (!whole) {
#pragma unroll
      for (int t = 0; t < 4; t++) {
        keep[t] = 0;
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int key = (int)base + 16 * g + 4 * t + r;
          if (pg.v >= 0 && key >= lmin && key < hmax) keep[t] |= 255u << (8 * r);
#pragma unroll
          for (int i = 0; i < NT; i++)
            if (pg.v < 0 || key < lo[i] || key >= hi[i]) s[i][t][r] = -__builtin_inff();
        }
      }
    }
    u32x4_t p[NT][2];
#pragma unroll
    for (int i = 0; i < NT; i++) {
      float f1 = qf[i];
      if (a.cap > 0.0f) {
#pragma unroll
        for (int t = 0; t < 4; t++)
#pragma unroll
          for (int r = 0; r < 4; r++) {
            const float x = capped(s[i][t][r] * qf[i], cap_in, cap_out);
            s[i][t][r] = s[i][t][r] == -__builtin_inff() && !whole ? s[i][t][r] : x;
          }
        f1 = 1.0f;
      }
      float mx = s[i][0][0];
#pragma unroll
      for (int t = 0; t < 4; t++)
#pragma unroll
        for (int r = 0; r < 4; r++) mx = fmaxf(mx, s[i][t][r]);
      mx = fmaxf(m[i], col_max(mx) * f1);
      if (__any(mx > m[i])) {
        const float fac = mx > m[i] ? __builtin_amdgcn_exp2f(m[i] - mx) : 1.0f;
        l[i] *= fac;
#pragma unroll
        for (int T = 0; T < KD; T++)
#pragma unroll
          for (int r = 0; r < 4; r++) {
            o[i][T][0][r] *= fac;
            o[i][T][1][r] *= fac;
          }
        m[i] = mx;
      }
      const float ref = (m[i] == -__builtin_inff() ? 0.0f : m[i]) - kOff;
#pragma unroll
      for (int t = 0; t < 4; t++) {
        float e[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
          e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][t][r], f1, -ref));
          l[i] += e[r];
        }
        if constexpr (MODE == 2) {
          p[i][t >> 1][2 * (t & 1)] = bf16x2_of(e[0], e[1]);
          p[i][t >> 1][2 * (t & 1) + 1] = bf16x2_of(e[2], e[3]);
        } else {
          p[i][t >> 1][2 * (t & 1)] = bits_of(f16x2_t{(_Float16)e[0], (_Float16)e[1]});
          p[i][t >> 1][2 * (t & 1) + 1] = bits_of(f16x2_t{(_Float16)e[2], (_Float16)e[3]});
        }
      }
    }
#pragma unroll
    for (int T = 0; T < KD; T++)
#pragma unroll
      for (int u = 0; u < 2; u++) {
        u32x4_t even, odd;
        value_operands<MODE>(f.v[T][2 * u], f.v[T][2 * u + 1], f.vs[T][2 * u] & keep[2 * u],
                             f.vs[T][2 * u + 1] & keep[2 * u + 1], even, odd);
#pragma unroll
        for (int i = 0; i < NT; i++) {
          o[i][T][0] = mfma16<MODE>(even, p[i][u], o[i][T][0]);
          o[i][T][1] = mfma16<MODE>(odd, p[i][u], o[i][T][1]);
        }
      }
  };

  // two fragments in turn: the next block's loads are under way while this one is used
  if (blk < end) {
    KvFragment<MODE, D> f0, f1;
    auto base_of = [&](int64_t i) { return base0 + i * kAttnKeys; };
    KvPages p0 = load_pages(a, rt.b, base_of(blk)), p1 = load_pages(a, rt.b, base_of(blk + WAVES));
    load_kv<MODE, D>(a, h, base_of(blk), p0, f0);
    while (true) {
      const bool more = blk + WAVES < end;
      KvPages p2 = p1;
      if (more) {
        load_kv<MODE, D>(a, h, base_of(blk + WAVES), p1, f1);
        p2 = load_pages(a, rt.b, base_of(blk + 2 * WAVES));
      }
      step(f0, base_of(blk), p0);
      blk += WAVES;
      if (!more) break;
      const bool again = blk + WAVES < end;
      KvPages p3 = p2;
      if (again) {
        load_kv<MODE, D>(a, h, base_of(blk + WAVES), p2, f0);
        p3 = load_pages(a, rt.b, base_of(blk + 2 * WAVES));
      }
      step(f1, base_of(blk), p1);
      blk += WAVES;
      if (!again) break;
      p0 = p2;
      p1 = p3;
    }
  }

  // join the waves: 16 rows at a time through LDS
#pragma unroll
  for (int i = 0; i < NT; i++) {
    const float sum = col_sum(l[i]);
    if (i) __syncthreads();
    if (g == 0) {
      sm[wave][c][0] = m[i];
      sm[wave][c][1] = sum;
    }
    __syncthreads();
    float mm = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < WAVES; w++) mm = fmaxf(mm, sm[w][c][0]);
    const float fac = m[i] == mm ? 1.0f : __builtin_amdgcn_exp2f(m[i] - mm);
#pragma unroll
    for (int T = 0; T < KD; T++)
#pragma unroll
      for (int r = 0; r < 4; r++) {
        so[wave][c][32 * T + 8 * g + 2 * r] = o[i][T][0][r] * fac;
        so[wave][c][32 * T + 8 * g + 2 * r + 1] = o[i][T][1][r] * fac;
      }
    __syncthreads();
    constexpr int PER = 16 * D / (64 * WAVES) < D / 4 ? 16 * D / (64 * WAVES) : D / 4;
    constexpr int LANES = D / PER;                    // lanes per row
    const int row = (int)threadIdx.x / LANES, part = (int)threadIdx.x % LANES;
    for (int rr = row; rr < 16; rr += 64 * WAVES / LANES) {
      const int64_t full = rt.row0 + 16 * i + rr;
      if (full >= rt.rows) break;
      float mw[WAVES], ll = 0.0f, top = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < WAVES; w++) top = fmaxf(top, mw[w] = sm[w][rr][0]);
#pragma unroll
      for (int w = 0; w < WAVES; w++)
        ll += sm[w][rr][1] * (mw[w] == top ? 1.0f : __builtin_amdgcn_exp2f(mw[w] - top));
      const int64_t tk = rt.tok0 + full / a.group;
      const int hd = h * a.group + (int)(full % a.group);
      const float va = MODE == 2 ? 1.0f : a.c.vam[h] / (6.0f * (MODE == 1 ? 256.0f : 448.0f));
      const float inv = ll == 0.0f ? 0.0f : va / ll;
      const int64_t at = ((int64_t)split * a.tokens + tk) * a.hq + hd;
#pragma unroll
      for (int e = 0; e < PER; e += 4) {
        const int ch = part * 4 + e * LANES;          // 16 bytes a lane, lanes side by side
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WAVES; w++)
#pragma unroll
          for (int z = 0; z < 4; z++) x[z] += so[w][rr][ch + z];
        if (a.splits > 1) {
          *(float4*)(a.po + at * D + ch) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
          *(uint2*)(a.out + tk * a.os + (int64_t)hd * D + ch) =
              make_uint2(bf16x2_of(x[0] * inv, x[1] * inv), bf16x2_of(x[2] * inv, x[3] * inv));
        }
      }
      if (part == 0) {
        if (a.splits > 1) {
          *(float2*)(a.pm + at * 2) = make_float2(top, ll);
        } else if (a.lse) {
          a.lse[tk * a.hq + hd] = ll == 0.0f ? -__builtin_inff()
                                             : __builtin_fmaf(top - kOff, kLn2, logf(ll));
        }
      }
    }
  }
}

// Joins the parts of the context: D/4 lanes (16 bytes each) times `parts`
// (a power of two) for a query row, the parts taking the splits in turn.
template <int MODE, int D>
__global__ __launch_bounds__(kThreads) void kv_attention_join_kernel(AttnArgs a, int parts) {
  constexpr float kOff = MODE == 2 ? 0.0f : 12.0f;
  constexpr int L = D / 4;
  __shared__ float4 sx[kThreads];
  __shared__ float2 sm[kThreads];
  const int t = (int)threadIdx.x, lane = t % L, part = t / L % parts;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / (L * parts)) + t / (L * parts);
  const int64_t rows = a.tokens * a.hq;
  const bool live = row < rows;
  float top = -__builtin_inff(), l = 0.0f, x[4] = {};
  auto add = [&](float m1, float l1, float4 y) {
    const float mm = fmaxf(top, m1);
    const float f0 = top == mm ? 1.0f : __builtin_amdgcn_exp2f(top - mm);
    const float f1 = m1 == mm ? 1.0f : __builtin_amdgcn_exp2f(m1 - mm);
    l = l * f0 + l1 * f1;
    x[0] = x[0] * f0 + y.x * f1;
    x[1] = x[1] * f0 + y.y * f1;
    x[2] = x[2] * f0 + y.z * f1;
    x[3] = x[3] * f0 + y.w * f1;
    top = mm;
  };
  if (live) {
#pragma unroll 4
    for (int s = part; s < a.splits; s += parts) {
      const float2 ml = *(const float2*)(a.pm + (s * rows + row) * 2);
      const float4 y = *(const float4*)(a.po + (s * rows + row) * D + lane * 4);
      add(ml.x, ml.y, y);
    }
  }
  if (parts > 1) {
    for (int half = parts / 2; half > 0; half >>= 1) {
      __syncthreads();
      sx[t] = make_float4(x[0], x[1], x[2], x[3]);
      sm[t] = make_float2(top, l);
      __syncthreads();
      if (part < half) add(sm[t + half * L].x, sm[t + half * L].y, sx[t + half * L]);
    }
  }
  if (!live || part) return;
  const int64_t tok = row / a.hq;
  const int head = (int)(row - tok * a.hq), h = head / a.group;
  const float va = MODE == 2 ? 1.0f : a.c.vam[h] / (6.0f * (MODE == 1 ? 256.0f : 448.0f));
  const float inv = l == 0.0f ? 0.0f : va / l;
  *(uint2*)(a.out + tok * a.os + (int64_t)head * D + lane * 4) =
      make_uint2(bf16x2_of(x[0] * inv, x[1] * inv), bf16x2_of(x[2] * inv, x[3] * inv));
  if (a.lse && lane == 0)
    a.lse[row] = l == 0.0f ? -__builtin_inff() : __builtin_fmaf(top - kOff, kLn2, logf(l));
}

}  // namespace fp4q
